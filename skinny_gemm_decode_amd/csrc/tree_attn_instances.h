// The attention kernels' instances, one source file per cache format and row
// type, D = 64, 128 and 256.
#pragma once

#include "tree_attn.h"

namespace skg {

// Waves share the keys of 16 or 32 rows (32: D <= 128), or 64, 128 or 256 rows
// (128: D <= 128; 256: also bf16 rows).
enum AttnForm { kKeys1, kKeys2, kRows64, kRows128, kRows256 };

#define SKG_TREE_ATTN_DECL(name) hipError_t name(const TreeArgs& a, int D, AttnForm form, dim3 grid, hipStream_t stream)
SKG_TREE_ATTN_DECL(tree_attn_bf16_f32);
SKG_TREE_ATTN_DECL(tree_attn_bf16_bf16);
SKG_TREE_ATTN_DECL(tree_attn_q8_0_f32);
SKG_TREE_ATTN_DECL(tree_attn_q8_0_bf16);
SKG_TREE_ATTN_DECL(tree_attn_q4_0_f32);
SKG_TREE_ATTN_DECL(tree_attn_q4_0_bf16);

template <class T, int KIND, int D>
hipError_t tree_attn_go(const TreeArgs& a, AttnForm form, dim3 grid, hipStream_t stream) {
  constexpr int NT = sizeof(T) == 2 ? 1 : KIND == KV_BF16 ? 3 : 2;
  if constexpr (NT == 1 && D <= 128) {
    if (form == kRows256) {
      hipLaunchKernelGGL((tree_attn_rows_kernel<T, KIND, D, NT, 2, 8>), grid, dim3(512), 0, stream, a);
      return hipGetLastError();
    }
  }
  if constexpr (D <= 128) {
    if (form == kKeys2) {
      hipLaunchKernelGGL((tree_attn_kernel<T, KIND, D, NT, 2>), grid, dim3(256), 0, stream, a);
      return hipGetLastError();
    }
  }
  if constexpr (D <= 128) {
    if (form == kRows128) {
      hipLaunchKernelGGL((tree_attn_rows_kernel<T, KIND, D, NT, 1, 8>), grid, dim3(512), 0, stream, a);
      return hipGetLastError();
    }
  }
  if (form == kRows64)
    hipLaunchKernelGGL((tree_attn_rows_kernel<T, KIND, D, NT, 1, 4>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((tree_attn_kernel<T, KIND, D, NT, 1>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}
template <class T, int KIND>
hipError_t tree_attn_by_dim(const TreeArgs& a, int D, AttnForm form, dim3 grid, hipStream_t s) {
  return D == 64 ? tree_attn_go<T, KIND, 64>(a, form, grid, s)
                 : D == 128 ? tree_attn_go<T, KIND, 128>(a, form, grid, s) : tree_attn_go<T, KIND, 256>(a, form, grid, s);
}

}  // namespace skg
