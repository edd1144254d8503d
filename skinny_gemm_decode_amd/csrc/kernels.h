// Host-side launchers of the library's kernels (internal).
#pragma once

#include <atomic>
#include <vector>

#include "common.h"
#include "kv_layout.h"

namespace skg {

hipError_t launch_pack(int wk, int64_t N, int64_t K, const void* src, void* dst, hipStream_t stream);
hipError_t launch_quantize_q8_1(int64_t M, int64_t K, const float* x, void* xq, hipStream_t stream);
// RMSNorm (+ Q8_1 of its output): K <= kNormMaxK, K % 32 == 0, M <= kNormMaxM.
constexpr int64_t kNormMaxK = 16384;
constexpr int64_t kNormMaxM = int64_t(1) << 24;
hipError_t launch_rmsnorm_q8_1(int64_t M, int64_t K, const float* x, const float* g, float eps, float* xn,
                               void* xq, hipStream_t stream);
hipError_t launch_block_dots(int fmt, const void* W, const Layout& L, int64_t n0, int64_t nr, const void* xq,
                             int32_t* out, hipStream_t stream);
hipError_t launch_stream_read(const void* buf, size_t bytes, uint32_t* out, int grid, hipStream_t stream);
hipError_t launch_empty(int64_t grid, int block, hipStream_t stream);
// Prefill kernel in use: 0 = one role per wave, 1 = producer/consumer waves.
extern std::atomic<int> g_gemm_variant;
extern const int kGemmDefaultVariant;

hipError_t launch_gemm_i8(int64_t M, int64_t K, int64_t N, const void* W, const Layout& L, const void* xq, float* y,
                          hipStream_t stream);
hipError_t launch_gemm_tiled(int64_t M, int64_t K, int64_t N, const void* W, const Layout& L, const void* x,
                             float* y, hipStream_t stream);

// Rotation, cache and attention.  Counts, strides (elements) and pointers are
// checked by the ABI.
hipError_t launch_qk_norm_rope(skg_dtype dt, int64_t T, int hq, int hk, int D, const void* q, int64_t ldq,
                               const void* k, int64_t ldk, const skg_rope* rope, void* qo, int64_t ldqo, void* ko,
                               int64_t ldko, hipStream_t stream);
hipError_t launch_kv_store(const KvView& c, int kind, int D, skg_dtype dt, int64_t T, const void* k, int64_t ldk,
                           const void* v, int64_t ldv, const int64_t* slots, hipStream_t stream);
hipError_t launch_kv_load(const KvView& c, int kind, int D, skg_dtype dt, int64_t T, const int64_t* slots, void* k,
                          int64_t ldk, void* v, int64_t ldv, hipStream_t stream);
hipError_t launch_qkv_rope_store(const KvView& c, int kind, int D, skg_dtype dt, int64_t T, int hq, const void* q,
                                 int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                 const skg_rope* rope, const int64_t* slots, void* qo, int64_t ldqo,
                                 hipStream_t stream);
struct TreeArgs;
size_t tree_attn_workspace(int kind, int D, int heads, skg_dtype dt, int64_t T, int64_t n_seqs, int hq, int max_draft,
                           int64_t max_kv);
hipError_t launch_tree_attn(const TreeArgs& a, int kind, int D, skg_dtype dt, int heads, void* ws,
                            hipStream_t stream);

}  // namespace skg
