// How an attention call is split, and the join of its splits' partial results.
#include "tree_attn.h"
#include "tree_attn_instances.h"

namespace skg {

namespace {

// Joins the splits of a row: with M* the largest M, o = sum 2^(M - M*) o_s and
// l likewise.  A row's D / 8 threads of 8 elements are repeated over `par`
// lanes of splits, which meet in LDS.
template <class T, int D>
__global__ __launch_bounds__(256) void tree_attn_join_kernel(TreeArgs a, float unit, int par) {
  constexpr int EPT = 8, kRow = D / EPT;   // threads of a row
  constexpr int kSlots = 256 / kRow;       // rows times split lanes of a workgroup
  __shared__ __attribute__((aligned(16))) float buf[kSlots][D];
  __shared__ float ml[kSlots][2];
  const int slot = threadIdx.x / kRow, e = (threadIdx.x % kRow) * EPT;
  const int lane = slot % par, nrow = kSlots / par;
  // rows (i, head) of sequence blockIdx.y
  const KvSpan sp = span_of(a, blockIdx.y);
  const int r = int(blockIdx.x) * nrow + slot / par;
  const bool is = r < sp.n * a.hq;
  if (int(blockIdx.x) * nrow >= sp.n * a.hq) return;  // uniform
  const int64_t tok = sp.t0 + (is ? r / a.hq : 0);
  const int hd = is ? r % a.hq : 0;
  const int per = steps_per_split(sp.keys, a.splits);
  const int steps = sp.keys / kStep + (sp.keys % kStep != 0);
  int n = (steps + per - 1) / per;
  n = n < 1 ? 1 : n;
  const int64_t at = (tok * a.hq + hd) * a.splits;
  const float* po = a.ws + at * D + e;
  const float* pm = a.ws + a.T * a.hq * int64_t(a.splits) * D + 2 * at;
  float M = kNoMax, l = 0.f, y[EPT];
#pragma unroll
  for (int j = 0; j < EPT; ++j) y[j] = 0.f;
  if (is)
    for (int s = lane; s < n; s += par) {
      const float ms = pm[2 * s], ls = pm[2 * s + 1];
      const f32x4 o0 = *reinterpret_cast<const f32x4*>(po + int64_t(s) * D);
      const f32x4 o1 = *reinterpret_cast<const f32x4*>(po + int64_t(s) * D + 4);
      const float m = fmaxf(M, ms), f = exp2_fast(M - m), g = exp2_fast(ms - m);
      M = m;
      l = fmaf(l, f, ls * g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = fmaf(y[j], f, o0[j] * g);
        y[4 + j] = fmaf(y[4 + j], f, o1[j] * g);
      }
    }
  if (par > 1) {  // uniform
#pragma unroll
    for (int j = 0; j < EPT; j += 4) *reinterpret_cast<f32x4*>(&buf[slot][e + j]) = f32x4{y[j], y[j + 1], y[j + 2], y[j + 3]};
    if (e == 0) {
      ml[slot][0] = M;
      ml[slot][1] = l;
    }
    __syncthreads();
    const int first = slot - lane;
    M = kNoMax;
    for (int s = 0; s < par; ++s) M = fmaxf(M, ml[first + s][0]);
    l = 0.f;
#pragma unroll
    for (int j = 0; j < EPT; ++j) y[j] = 0.f;
    for (int s = 0; s < par; ++s) {
      const float f = exp2_fast(ml[first + s][0] - M);
      l = fmaf(ml[first + s][1], f, l);
#pragma unroll
      for (int j = 0; j < EPT; ++j) y[j] = fmaf(buf[first + s][e + j], f, y[j]);
    }
  }
  const float inv = unit / l;
#pragma unroll
  for (int j = 0; j < EPT; ++j) y[j] = l == 0.f ? 0.f : y[j] * inv;
  put_out<T, EPT>(a, tok, int64_t(hd) * D + e, y, is && lane == 0);
}

template <class T, int D>
hipError_t join(const TreeArgs& a, float unit, hipStream_t stream) {
  constexpr int kSlots = 256 / (D / 8);
  int par = 1;
  while (par < a.splits && par < kSlots) par *= 2;
  const int nrow = kSlots / par;
  const int64_t rows = int64_t(a.max_draft) * a.hq;
  hipLaunchKernelGGL((tree_attn_join_kernel<T, D>), dim3(unsigned((rows + nrow - 1) / nrow), unsigned(a.n_seqs)),
                     dim3(256), 0, stream, a, unit, par);
  return hipGetLastError();
}
template <class T>
hipError_t join_dim(const TreeArgs& a, int D, float unit, hipStream_t s) {
  return D == 64 ? join<T, 64>(a, unit, s) : D == 128 ? join<T, 128>(a, unit, s) : join<T, 256>(a, unit, s);
}

struct Plan {
  int rt, row_groups, splits;
};

// Two row tiles of 16 a wave where there are more rows than one tile has: the
// keys' conversion then serves both.  The keys are split until there are two
// workgroups for each of 256 CUs, but none into less than two steps a wave.
Plan plan(int heads, int64_t n_seqs, int hq, int max_draft, int64_t max_kv) {
  Plan p;
  const int64_t rows = int64_t(max_draft) * (hq / heads);
  p.rt = rows <= 16 ? 1 : 2;
  p.row_groups = int((rows + 16 * p.rt - 1) / (16 * p.rt));
  const int64_t units = n_seqs * heads * p.row_groups, steps = (max_kv + kStep - 1) / kStep;
  int64_t s = (512 + units - 1) / units;
  const int64_t most = (steps + kMinSteps - 1) / kMinSteps;
  s = s < most ? s : most;
  p.splits = int(s < 1 ? 1 : s);
  return p;
}

}  // namespace

size_t tree_attn_workspace(int, int D, int heads, int64_t T, int64_t n_seqs, int hq, int max_draft, int64_t max_kv) {
  const Plan p = plan(heads, n_seqs, hq, max_draft, max_kv);
  return p.splits == 1 ? 0 : size_t(T) * size_t(hq) * size_t(p.splits) * size_t(D + 2) * sizeof(float);
}

hipError_t launch_tree_attn(const TreeArgs& args, int kind, int D, skg_dtype dt, int heads, void* ws,
                            hipStream_t stream) {
  TreeArgs a = args;
  const Plan p = plan(heads, a.n_seqs, a.hq, a.max_draft, a.max_kv);
  a.splits = p.splits;
  a.row_groups = p.row_groups;
  a.ws = static_cast<float*>(ws);
  a.blocks = int64_t(a.hq) * D / QK;
  const int64_t grid = int64_t(heads) * p.splits * p.row_groups * a.n_seqs;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  const bool f32 = dt == SKG_F32;
  hipError_t e;
  switch (kind) {
    case KV_BF16: e = f32 ? tree_attn_bf16_f32(a, D, p.rt, unsigned(grid), stream) : tree_attn_bf16_bf16(a, D, p.rt, unsigned(grid), stream); break;
    case KV_Q8_0: e = f32 ? tree_attn_q8_0_f32(a, D, p.rt, unsigned(grid), stream) : tree_attn_q8_0_bf16(a, D, p.rt, unsigned(grid), stream); break;
    default: e = f32 ? tree_attn_q4_0_f32(a, D, p.rt, unsigned(grid), stream) : tree_attn_q4_0_bf16(a, D, p.rt, unsigned(grid), stream); break;
  }
  if (e != hipSuccess || p.splits == 1) return e;
  const float unit = kind == KV_BF16 ? 1.f : kVScale;
  return f32 ? join_dim<float>(a, D, unit, stream) : join_dim<__bf16>(a, D, unit, stream);
}

}  // namespace skg
