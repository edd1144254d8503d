// The attention kernel's instances, one source file per cache format and row
// type: D = 64, 128, 256 and one or two row tiles a wave.
#pragma once

#include "tree_attn.h"

namespace skg {

#define SKG_TREE_ATTN_DECL(name) hipError_t name(const TreeArgs& a, int D, int rt, unsigned grid, hipStream_t stream)
SKG_TREE_ATTN_DECL(tree_attn_bf16_f32);
SKG_TREE_ATTN_DECL(tree_attn_bf16_bf16);
SKG_TREE_ATTN_DECL(tree_attn_q8_0_f32);
SKG_TREE_ATTN_DECL(tree_attn_q8_0_bf16);
SKG_TREE_ATTN_DECL(tree_attn_q4_0_f32);
SKG_TREE_ATTN_DECL(tree_attn_q4_0_bf16);

template <class T, int KIND, int D, int RT>
hipError_t tree_attn_go(const TreeArgs& a, unsigned grid, hipStream_t stream) {
  constexpr int NT = sizeof(T) == 2 ? 1 : KIND == KV_BF16 ? 3 : 2;
  hipLaunchKernelGGL((tree_attn_kernel<T, KIND, D, NT, RT>), dim3(grid), dim3(kAttnThreads), 0, stream, a);
  return hipGetLastError();
}
template <class T, int KIND>
hipError_t tree_attn_by_dim(const TreeArgs& a, int D, int rt, unsigned grid, hipStream_t s) {
  if (D == 64) return rt == 1 ? tree_attn_go<T, KIND, 64, 1>(a, grid, s) : tree_attn_go<T, KIND, 64, 2>(a, grid, s);
  if (D == 128) return rt == 1 ? tree_attn_go<T, KIND, 128, 1>(a, grid, s) : tree_attn_go<T, KIND, 128, 2>(a, grid, s);
  return rt == 1 ? tree_attn_go<T, KIND, 256, 1>(a, grid, s) : tree_attn_go<T, KIND, 256, 2>(a, grid, s);
}

}  // namespace skg
