// Attention over a q8_0 cache, float32 rows.
#include "tree_attn_instances.h"

namespace skg {

SKG_TREE_ATTN_DECL(tree_attn_q8_0_f32) { return tree_attn_by_dim<float, KV_Q8_0>(a, D, form, grid, stream); }

}  // namespace skg
