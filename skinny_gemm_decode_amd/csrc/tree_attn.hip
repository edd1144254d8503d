// Attention of drafted tokens over a paged cache.
//
// One wave per (token, query head) walks the keys once with the running
// maximum m and sum l of the softmax: for a new score s,
//   m' = max(m, s),  l = l e^(m - m') + e^(s - m'),  o = o e^(m - m') + e^(s - m') v.
// Each lane holds D / 64 elements of the row.
#include "tree_attn.h"
#include "kernels.h"

namespace skg {

namespace {

// Element e of token t of a chunk.
template <int KIND, int D>
__device__ inline float cache_value(const uint8_t* chunk, uint32_t shift, uint32_t t, int e) {
  const uint8_t* row = chunk + kv_codes_at(KIND, D, t);
  if constexpr (KIND == KV_BF16) return bf16_lo(reinterpret_cast<const uint16_t*>(row)[e]);
  constexpr int NB = D / 32;
  const int b = e / 32, c = (e % 32) / 2, i = e & 1;
  const float d = h2f(reinterpret_cast<const uint16_t*>(chunk + kv_scales_at(KIND, D, shift, t))[b]);
  if constexpr (KIND == KV_Q8_0) return d * (float(row[2 * NB * c + 2 * b + i]) - 128.f);
  return d * (float((row[NB * c + b] >> (4 * i)) & 15) - 8.f);
}

template <class T, int KIND, int D>
__global__ __launch_bounds__(64) void tree_attn_kernel(TreeArgs a) {
  constexpr int E = D / 64;
  const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z, lane = threadIdx.x;
  const int64_t per = a.T / a.n_seqs;
  const int64_t t0 = a.cu ? a.cu[b] : b * per, t1 = a.cu ? a.cu[b + 1] : (b + 1) * per;
  const KvSpan sp = kv_span(a.ctx[b], int32_t(t0), int32_t(t1), a.T, a.max_draft, a.max_kv);
  if (i >= sp.n) return;
  const int64_t tok = sp.t0 + i;
  const uint64_t mask = a.mask ? a.mask[tok] : ~uint64_t(0) >> (63 - i);
  const T* q = reinterpret_cast<const T*>(a.q + tok * a.ldq) + h * D;
  float x[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = float(q[lane * E + e]) * a.scale;
    o[e] = 0.f;
  }
  const uint32_t head = h / a.group, in_page = (1u << a.cache.shift) - 1;
  for (int j = 0; j < sp.keys; ++j) {
    if (j >= sp.ctx && !((mask >> (j - sp.ctx)) & 1)) continue;
    const int32_t page = a.table[b * a.width + (j >> a.cache.shift)];
    if (!kv_page_in(a.cache, page)) continue;
    const uint64_t at = kv_chunk_at(a.cache, page, head);
    const uint32_t t = uint32_t(j) & in_page;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(x[e], cache_value<KIND, D>(a.cache.k + at, a.cache.shift, t, lane * E + e), s);
    s = wave_sum(s);
    const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * f + p * cache_value<KIND, D>(a.cache.v + at, a.cache.shift, t, lane * E + e);
  }
  __shared__ float out[D];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    o[e] = l == 0.f ? 0.f : o[e] / l;
    out[lane * E + e] = o[e];
    if (a.o) reinterpret_cast<T*>(a.o + tok * a.ldo)[h * D + lane * E + e] = T(o[e]);
  }
  __syncthreads();
  if (a.oq && lane < D / 32) {
    float v[QK];
#pragma unroll
    for (int e = 0; e < QK; ++e) v[e] = out[lane * QK + e];
    const Q8_1Block blk = quantize_block_q8_1(v);
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.oq + ((tok * a.hq + h) * (D / QK) + lane) * 36);
    dst[0] = blk.d16 | (blk.s16 << 16);
#pragma unroll
    for (int k = 0; k < 8; ++k) dst[1 + k] = blk.q[k];
  }
}

template <class T, int KIND, int D>
hipError_t go(const TreeArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((tree_attn_kernel<T, KIND, D>), dim3(unsigned(a.hq), unsigned(a.max_draft), unsigned(a.n_seqs)),
                     dim3(64), 0, stream, a);
  return hipGetLastError();
}
template <class T, int KIND>
hipError_t by_dim(int D, const TreeArgs& a, hipStream_t s) {
  return D == 64 ? go<T, KIND, 64>(a, s) : D == 128 ? go<T, KIND, 128>(a, s) : go<T, KIND, 256>(a, s);
}
template <class T>
hipError_t by_kind(int kind, int D, const TreeArgs& a, hipStream_t s) {
  return kind == KV_BF16 ? by_dim<T, KV_BF16>(D, a, s)
                         : kind == KV_Q8_0 ? by_dim<T, KV_Q8_0>(D, a, s) : by_dim<T, KV_Q4_0>(D, a, s);
}

}  // namespace

size_t tree_attn_workspace(int, int, int, int64_t, int64_t, int, int, int64_t) { return 0; }

hipError_t launch_tree_attn(const TreeArgs& a, int kind, int D, skg_dtype dt, int, void*, hipStream_t stream) {
  return dt == SKG_F32 ? by_kind<float>(kind, D, a, stream) : by_kind<__bf16>(kind, D, a, stream);
}

}  // namespace skg
