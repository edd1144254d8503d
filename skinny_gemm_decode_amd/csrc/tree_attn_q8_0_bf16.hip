// Attention over a q8_0 cache, bf16 rows.
#include "tree_attn_instances.h"

namespace skg {

SKG_TREE_ATTN_DECL(tree_attn_q8_0_bf16) { return tree_attn_by_dim<__bf16, KV_Q8_0>(a, D, form, grid, stream); }

}  // namespace skg
