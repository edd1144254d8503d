// Attention over a bf16 cache, float32 rows.
#include "tree_attn_instances.h"

namespace skg {

SKG_TREE_ATTN_DECL(tree_attn_bf16_f32) { return tree_attn_by_dim<float, KV_BF16>(a, D, form, grid, stream); }

}  // namespace skg
