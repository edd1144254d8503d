// How an attention call is split, its launch, and the join of the splits.
#include "tree_attn.h"
#include "tree_attn_instances.h"

namespace skg {

namespace {

// Joins the splits of a row: with M* the largest M, o = sum 2^(M - M*) o_s, and
// l likewise.  SUBS groups of 16 lanes take the splits in turn and meet by
// shuffles and, with more than a wave's four, in LDS; the order is fixed.  It
// is a launch of its own because the partial results then come through all
// CUs: the last workgroup to arrive joining them (write-through stores and a
// counter) took 3.3 us where this takes 3.9 with its launch at 16 splits of 8
// rows, but 8 where this takes 5 at 64, and needed a workspace kept at zero.
template <class T, int D, int SUBS, bool WEIGH>
__global__ __launch_bounds__(256) void tree_attn_join_kernel(TreeArgs a, float unit) {
  constexpr int B = D / 32, kDeep = 4;
  __shared__ __attribute__((aligned(16))) float buf[SUBS > 4 ? 4 : 1][D];
  __shared__ float ml[4][2];
  const int wave = threadIdx.x >> 6, je = 2 * (threadIdx.x & 15);
  const int sub = SUBS > 4 ? threadIdx.x >> 4 : (threadIdx.x >> 4) & 3;
  const int h = SUBS > 4 ? blockIdx.x : 4 * blockIdx.x + wave, i = blockIdx.y;
  Unit unit_of;
  if (!find_unit<WEIGH>(a, blockIdx.z, unit_of, true)) return;
  const KvSpan sp = unit_of.sp;
  const int splits = unit_of.splits, before = unit_of.base;
  if (i >= sp.n || splits <= 1 || h >= a.hq) return;  // uniform over a wave, with SUBS > 4 over the workgroup
  const int row = i * a.group + h % a.group, head = h / a.group;
  const int rg = row / a.tile, local = row - rg * a.tile;
  const int64_t step = int64_t(a.row_groups) * a.cache.heads;
  const int64_t at = ((before * step + int64_t(rg) * a.cache.heads + head) * a.tile + local);
  const float* po = a.sums + at * D + je;
  const float* pm = a.ml + 2 * at;
  const int64_t so = step * a.tile * D, sm = step * a.tile * 2;
  float M = kNoMax, l = 0.f, y[2 * B];
#pragma unroll
  for (int j = 0; j < 2 * B; ++j) y[j] = 0.f;
#pragma unroll 1
  for (int s0 = sub; s0 < splits; s0 += kDeep * SUBS) {
    f32x2 m[kDeep], o[kDeep][B];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int s = s0 + k * SUBS < splits ? s0 + k * SUBS : s0;
      m[k] = *reinterpret_cast<const f32x2*>(pm + s * sm);
#pragma unroll
      for (int j = 0; j < B; ++j) o[k][j] = *reinterpret_cast<const f32x2*>(po + s * so + 32 * j);
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kDeep; ++k) top = fmaxf(top, m[k].x);
    const float f = exp2_fast(M - top);
    M = top;
    l *= f;
#pragma unroll
    for (int j = 0; j < 2 * B; ++j) y[j] *= f;
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const float e = s0 + k * SUBS < splits ? exp2_fast(m[k].x - M) : 0.f;
      l = fmaf(m[k].y, e, l);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        y[2 * j] = fmaf(o[k][j].x, e, y[2 * j]);
        y[2 * j + 1] = fmaf(o[k][j].y, e, y[2 * j + 1]);
      }
    }
  }
  {  // the wave's four groups of lanes
    const float top = row_max(M), e = exp2_fast(M - top);
    M = top;
    l = row_sum(l * e);
#pragma unroll
    for (int j = 0; j < 2 * B; ++j) y[j] = row_sum(y[j] * e);
  }
  if constexpr (SUBS > 4) {
    if ((threadIdx.x & 63) < 16) {
#pragma unroll
      for (int j = 0; j < B; ++j) *reinterpret_cast<f32x2*>(&buf[wave][32 * j + je]) = f32x2{y[2 * j], y[2 * j + 1]};
      ml[wave][0] = M;
      ml[wave][1] = l;
    }
    __syncthreads();
    M = kNoMax;
#pragma unroll
    for (int k = 0; k < 4; ++k) M = fmaxf(M, ml[k][0]);
    l = 0.f;
#pragma unroll
    for (int j = 0; j < 2 * B; ++j) y[j] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float e = exp2_fast(ml[k][0] - M);
      l = fmaf(ml[k][1], e, l);
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const f32x2 o = *reinterpret_cast<const f32x2*>(&buf[k][32 * j + je]);
        y[2 * j] = fmaf(o.x, e, y[2 * j]);
        y[2 * j + 1] = fmaf(o.y, e, y[2 * j + 1]);
      }
    }
  }
  finish<T, B>(a, sp.t0 + i, int64_t(h) * D, y, l, unit, sub == 0);
}

template <class T, int D>
hipError_t join(const TreeArgs& a, float unit, bool wide, hipStream_t stream) {
  auto launch = [&](auto kernel, int heads) {  // heads of a workgroup
    hipLaunchKernelGGL(kernel, dim3(unsigned((a.hq + heads - 1) / heads), unsigned(a.max_draft), unsigned(a.n_seqs)),
                       dim3(256), 0, stream, a, unit);
    return hipGetLastError();
  };
  if (a.tile > 64)
    return wide ? launch(tree_attn_join_kernel<T, D, 16, true>, 1) : launch(tree_attn_join_kernel<T, D, 4, true>, 4);
  return wide ? launch(tree_attn_join_kernel<T, D, 16, false>, 1) : launch(tree_attn_join_kernel<T, D, 4, false>, 4);
}
template <class T>
hipError_t join_dim(const TreeArgs& a, int D, float unit, bool wide, hipStream_t s) {
  return D == 64 ? join<T, 64>(a, unit, wide, s) : D == 128 ? join<T, 128>(a, unit, wide, s) : join<T, 256>(a, unit, wide, s);
}

struct Plan {
  AttnForm form;
  int row_groups, want;
  int64_t slots;  // splits at most
  bool wide;      // the join: 16 lanes groups a row, not four
  size_t ml, bytes;
};

// Up to 32 rows of a head: the waves share the keys.  More: they share the
// rows, so that the cache is read once for 64, 128 or (one term a product,
// two row tiles a wave) 256 of them; at D = 256 a row tile fills a wave's
// registers, and only four waves have room.  Trees of 61 tokens of four heads
// over bf16 42.9 us with 256 rows a workgroup, 49.1 with 128, 72.8 with four
// tiles a wave (q8_0 63 and 74).
AttnForm form_of(int D, skg_dtype dt, int64_t rows) {
  if (rows <= 16) return kKeys1;
  if (rows <= 32 && D <= 128) return kKeys2;
  if (rows <= 64 || D > 128) return kRows64;
  if (rows <= 128 || dt == SKG_F32) return kRows128;
  return kRows256;
}
constexpr int kTileOf[] = {16, 32, 64, 128, 256};

// Workgroups of a form that a CU holds at once.
template <int KIND, int D, int NT>
int per_cu(AttnForm f) {
  if (f == kKeys1) return AttnShape<KIND, D, NT, 1, 4, false>::kPerCu;
  if constexpr (D <= 128)
    if (f == kKeys2) return AttnShape<KIND, D, NT, 2, 4, false>::kPerCu;
  return f == kRows64 ? AttnShape<KIND, D, NT, 1, 4, true>::kPerCu : 1;
}
template <int KIND, int D>
int per_cu(AttnForm f, skg_dtype dt) {
  return dt == SKG_F32 ? per_cu<KIND, D, KIND == KV_BF16 ? 3 : 2>(f) : per_cu<KIND, D, 1>(f);
}
template <int KIND>
int per_cu(AttnForm f, int D, skg_dtype dt) {
  return D == 64 ? per_cu<KIND, 64>(f, dt) : D == 128 ? per_cu<KIND, 128>(f, dt) : per_cu<KIND, 256>(f, dt);
}

// Splits: as many workgroups as 256 CUs hold, counted over all heads, row
// groups and sequences (at D = 256, where a CU holds one, twice as many took
// 38 us for 60000 keys, this 28.8).  Where there are half that many without
// splitting, twice as many, so that long sequences do not stand alone at the
// end: 64 q8_0 sequences of up to 2000 keys 37.7 us, with as many as the CUs
// hold 39.9, with four times as many 45.4; bf16 47.1, 53.2 and 48.7.  A single
// sequence splits evenly, and where its steps are 8 KB one workgroup's copies
// keep a CU busy (q8_0 of 128 elements: 131071 keys 51.9 us with one, 54.6 with
// two; sixteen ragged sequences 36.1 and 32.9; a single one in steps of half
// that 49.3 and 42.7).  More than 256 sequences are not split.
Plan plan(int kind, int D, int heads, skg_dtype dt, int64_t T, int64_t n_seqs, int hq, int max_draft, int64_t max_kv) {
  Plan p;
  const int64_t rows = int64_t(max_draft) * (hq / heads);
  p.form = form_of(D, dt, rows);
  const int tile = kTileOf[p.form];
  p.row_groups = int((rows + tile - 1) / tile);
  const int64_t lanes = int64_t(heads) * p.row_groups;  // workgroups of a split
  const int64_t steps = (max_kv + kStep - 1) / kStep, each = (steps + kMinSteps - 1) / kMinSteps;
  int64_t want = 0;
  if (n_seqs <= kMaxSplitSeqs && each > 1) {
    const int fits = kind == KV_BF16   ? per_cu<KV_BF16>(p.form, D, dt)
                     : kind == KV_Q8_0 ? per_cu<KV_Q8_0>(p.form, D, dt)
                                       : per_cu<KV_Q4_0>(p.form, D, dt);
    const int64_t full = 256 * (n_seqs == 1 && kv_row_bytes(kind, D) >= 128 ? 1 : fits);
    const int64_t fill = lanes * n_seqs <= full / 2 ? full : 2 * full;
    want = fill / lanes - n_seqs / 2;
    want = want < 1 ? 1 : want;
  }
  p.want = int(want);
  p.slots = want ? (want + n_seqs < n_seqs * each ? want + n_seqs : n_seqs * each) : n_seqs;
  const int64_t most = want < each ? want : each;  // splits of a sequence
  p.wide = most > 4 && T * hq < 2048;
  p.ml = p.bytes = 0;
  if (want) {
    const size_t part = size_t(p.slots) * size_t(lanes) * size_t(tile);
    p.ml = (part * 2 * 4 + 255) & ~size_t(255);
    p.bytes = p.ml + part * size_t(D) * 4;
  }
  return p;
}

}  // namespace

size_t tree_attn_workspace(int kind, int D, int heads, skg_dtype dt, int64_t T, int64_t n_seqs, int hq, int max_draft,
                           int64_t max_kv) {
  return plan(kind, D, heads, dt, T, n_seqs, hq, max_draft, max_kv).bytes;
}

hipError_t launch_tree_attn(const TreeArgs& args, int kind, int D, skg_dtype dt, int heads, void* ws,
                            hipStream_t stream) {
  TreeArgs a = args;
  const Plan p = plan(kind, D, heads, dt, a.T, a.n_seqs, a.hq, a.max_draft, a.max_kv);
  a.want = p.want;
  a.cost_shift = kv_cost_shift(a.max_kv, a.n_seqs);
  a.row_groups = p.row_groups;
  a.tile = kTileOf[p.form];
  a.per_seq = int(a.T / a.n_seqs);
  a.blocks = int64_t(a.hq) * D / QK;
  a.ml = static_cast<float*>(ws);
  a.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.ml);
  const dim3 grid{unsigned(heads), unsigned(p.slots), unsigned(p.row_groups)};
  const bool f32 = dt == SKG_F32;
  hipError_t e;
  switch (kind) {
    case KV_BF16: e = f32 ? tree_attn_bf16_f32(a, D, p.form, grid, stream) : tree_attn_bf16_bf16(a, D, p.form, grid, stream); break;
    case KV_Q8_0: e = f32 ? tree_attn_q8_0_f32(a, D, p.form, grid, stream) : tree_attn_q8_0_bf16(a, D, p.form, grid, stream); break;
    default: e = f32 ? tree_attn_q4_0_f32(a, D, p.form, grid, stream) : tree_attn_q4_0_bf16(a, D, p.form, grid, stream); break;
  }
  if (e != hipSuccess || !p.want) return e;
  const float unit = kind == KV_BF16 ? 1.f : kVScale;
  return f32 ? join_dim<float>(a, D, unit, p.wide, stream) : join_dim<__bf16>(a, D, unit, p.wide, stream);
}

}  // namespace skg
