// Attention over a bf16 cache, bf16 rows.
#include "tree_attn_instances.h"

namespace skg {

SKG_TREE_ATTN_DECL(tree_attn_bf16_bf16) { return tree_attn_by_dim<__bf16, KV_BF16>(a, D, form, grid, stream); }

}  // namespace skg
