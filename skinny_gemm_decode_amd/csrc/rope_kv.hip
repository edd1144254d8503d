// Per-head normalisation and rotation of queries and keys, and the cache's
// encoder and decoder.
//
// Rotation.  Position p turns the pair (a, b) of frequency f_i by th = p f_i:
//   (a cos th - b sin th, a sin th + b cos th),
// either adjacent elements or elements half a rotated part apart.  At far
// positions th is many turns, and its binary32 form would have lost the angle
// (p = 10^6: 2^-4 of a radian), so th is formed exactly in binary64 (a 24-bit
// frequency times a 31-bit position), reduced there to within pi/4 and only
// then evaluated in binary32.  A workgroup computes its token's rot / 2 angles
// once, one per thread, and its rows read them from LDS.
//
// A row is D / 2 units of 16 bytes, two per lane: unit l and the unit half the
// rotated part further, so both styles of pairing stay within a lane and need
// no exchange (lanes past the rotated part hold two adjacent units).  The sum
// of squares meets over the row's 4..32 lanes.
//
// Cache rows.  The encoder and the decoder give a lane 16 bytes of the row in
// each of two adjacent blocks: the row's accesses are whole, a block's maximum
// is two or three DPP steps, and the codes of a column's two blocks are
// adjacent in the cache row.
#include "kv_common.h"
#include "kernels.h"

namespace skg {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kManyGroups = 1024;  // four workgroups a CU
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;  // of a launch, which has less than 2^32 threads

template <int CTRL>
__device__ inline int dpp_u(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}

// Largest value / smallest integer over aligned groups of L lanes (4 or 8), in all of them.
template <int L>
__device__ inline float group_max(float v) {
  v = fmaxf(v, dpp_f<SKG_DPP_QUAD_XOR1>(v));
  v = fmaxf(v, dpp_f<SKG_DPP_QUAD_XOR2>(v));
  return L == 8 ? fmaxf(v, dpp_f<SKG_DPP_ROW_HALF_MIRROR>(v)) : v;
}
template <int L>
__device__ inline int group_min(int v) {
  v = min(v, dpp_u<SKG_DPP_QUAD_XOR1>(v));
  v = min(v, dpp_u<SKG_DPP_QUAD_XOR2>(v));
  return L == 8 ? min(v, dpp_u<SKG_DPP_ROW_HALF_MIRROR>(v)) : v;
}
// Sum over aligned groups of L lanes (a power of two, 4..32), in all of them.
template <int L>
__device__ inline float group_sum(float v) {
  v += dpp_f<SKG_DPP_QUAD_XOR1>(v);
  v += dpp_f<SKG_DPP_QUAD_XOR2>(v);
  if constexpr (L >= 8) v += dpp_f<SKG_DPP_ROW_HALF_MIRROR>(v);
  if constexpr (L >= 16) v += dpp_f<SKG_DPP_ROW_MIRROR>(v);
  if constexpr (L >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// cos and sin of pos * f.  n = nearest multiple of pi/2; what is left of the
// angle is within pi/4, where the Taylor polynomials below are exact to 2^-28.
__device__ inline f32x2 cos_sin(int32_t pos, float f) {
  const double th = double(pos) * double(f);
  const double n = rint(th * 0.63661977236758134308);
  const double r64 = fma(-n, 6.123233995736766e-17, fma(-n, 1.5707963267948966, th));
  const float r = float(r64), z = r * r;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(r * z, s, r);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  // quadrant: n mod 4, from the low bits of the exact integer n
  const int64_t q = int64_t(n) & 3;
  const float cq = (q & 1) ? s : c, sq = (q & 1) ? c : s;
  return f32x2{(q == 1 || q == 2) ? -cq : cq, (q >= 2) ? -sq : sq};
}

struct RopeArgs {
  int rot, interleaved, norm;
  float eps;
  const int32_t* pos;
  const float* inv_freq;
  const float* gq;
  const float* gk;
};

// The rows of a tensor: token stride in bytes, heads adjacent.
struct Rows {
  uint8_t* p;
  int64_t ld;
};

template <class T, int D>
struct RowShape {
  static constexpr int kVec = Elem<T>::kVec;
  static constexpr int kUnits = D / kVec;
  static constexpr int kLanes = kUnits / 2;          // lanes of a row
  static constexpr int kRows = kThreads / kLanes;    // rows of a pass
};

// The two units of lane l: half the rotated part apart within it, adjacent past it.
template <class T, int D>
__device__ inline void units_of(int l, int rot, int& ua, int& ub) {
  const int half = rot / (2 * Elem<T>::kVec);
  ua = l < half ? l : 2 * l;
  ub = l < half ? l + half : 2 * l + 1;
}

// One row in its lanes' registers: normalised (norm) and turned.  Every lane
// of the row executes it.
template <class T, int D>
__device__ inline void norm_rope(float (&a)[Elem<T>::kVec], float (&b)[Elem<T>::kVec], int l, int ua, int ub,
                                 const RopeArgs& r, const float* g, const f32x2* cs) {
  constexpr int V = Elem<T>::kVec;
  if (r.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
    ss = group_sum<RowShape<T, D>::kLanes>(ss);
    const float rs = 1.0f / sqrtf(ss / float(D) + r.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      a[i] *= rs;
      b[i] *= rs;
    }
    if (g) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const f32x4 ga = *reinterpret_cast<const f32x4*>(g + ua * V + i);
        const f32x4 gb = *reinterpret_cast<const f32x4*>(g + ub * V + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[i + j] *= ga[j];
          b[i + j] *= gb[j];
        }
      }
    }
  }
  if (l < r.rot / (2 * V)) {
    if (r.interleaved) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const f32x2 ca = cs[(ua * V + i) / 2], cb = cs[(ub * V + i) / 2];
        const float a0 = a[i], b0 = b[i];
        a[i] = a0 * ca.x - a[i + 1] * ca.y;
        a[i + 1] = a0 * ca.y + a[i + 1] * ca.x;
        b[i] = b0 * cb.x - b[i + 1] * cb.y;
        b[i + 1] = b0 * cb.y + b[i + 1] * cb.x;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const f32x2 c = cs[ua * V + i];
        const float a0 = a[i];
        a[i] = a0 * c.x - b[i] * c.y;
        b[i] = a0 * c.y + b[i] * c.x;
      }
    }
  }
}

// The angles of token `tok` into cs[0 .. rot / 2).
__device__ inline void fill_angles(const RopeArgs& r, int64_t tok, f32x2* cs) {
  const int t = threadIdx.x;
  if (t < r.rot / 2) cs[t] = cos_sin(r.pos[tok], r.inv_freq[t]);
}

// P rows per thread, all loaded before the first is used.  Two of them where
// there are workgroups enough all the same: 32 + 8 heads of 128 bf16 elements
// of 8191 tokens 43.7 us with one, 33.6 with two or four, 31.7 with two and
// stores past the caches (168 MB: 5.3 TB/s); 64 heads of 512 binary32 tokens
// 7.3, 7.4, 7.8 and 6.4 us.  A small call keeps one, for its latency (one token's
// 64 heads 2.1 us, with two 2.5), and its rows in the caches for their reader.
template <class T, int D, int P>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(Rows q, Rows k, Rows qo, Rows ko, int hq, int hk,
                                                                int chunks, RopeArgs r) {
  using S = RowShape<T, D>;
  __shared__ f32x2 cs[D / 2];
  const int64_t tok = blockIdx.x / unsigned(chunks);
  const int first = int(blockIdx.x % unsigned(chunks)) * S::kRows * P + threadIdx.x / S::kLanes;
  const int l = threadIdx.x % S::kLanes;
  int ua, ub;
  units_of<T, D>(l, r.rot, ua, ub);
  u32x4 xa[P], xb[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int row = first + p * S::kRows;
    if (row < hq + hk) {
      const bool isq = row < hq;
      const u32x4* src = reinterpret_cast<const u32x4*>((isq ? q.p : k.p) + tok * (isq ? q.ld : k.ld)) +
                         (isq ? row : row - hq) * S::kUnits;
      xa[p] = src[ua];
      xb[p] = src[ub];
    }
  }
  fill_angles(r, tok, cs);
  __syncthreads();
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int row = first + p * S::kRows;
    if (row < hq + hk) {
      const bool isq = row < hq;
      float a[S::kVec], b[S::kVec];
      Elem<T>::unpack(xa[p], a);
      Elem<T>::unpack(xb[p], b);
      norm_rope<T, D>(a, b, l, ua, ub, r, isq ? r.gq : r.gk, cs);
      u32x4* dst = reinterpret_cast<u32x4*>((isq ? qo.p : ko.p) + tok * (isq ? qo.ld : ko.ld)) +
                   (isq ? row : row - hq) * S::kUnits;
      if constexpr (P > 1) {
        __builtin_nontemporal_store(Elem<T>::pack(a), dst + ua);
        __builtin_nontemporal_store(Elem<T>::pack(b), dst + ub);
      } else {
        dst[ua] = Elem<T>::pack(a);
        dst[ub] = Elem<T>::pack(b);
      }
    }
  }
}

// ---- cache rows -------------------------------------------------------------

// Lane (j, bp) of a row has V elements, V j .. V j + V - 1, of each of blocks
// 2 bp and 2 bp + 1: 16 bytes of a row in memory.
template <int V, int D>
struct UnitShape {
  static constexpr int kBlock = 32 / V;              // lanes of a block
  static constexpr int kLanes = kBlock * (D / 64);   // of a row
  static constexpr int kRows = kThreads / kLanes;    // rows of a workgroup
};

__device__ inline int round_code(float x, float id, int lo, int hi) {
#pragma clang fp contract(off)
  return int(fminf(fmaxf(roundf(x * id), float(lo)), float(hi)));
}
__device__ inline uint32_t scale16(float d) {
  return __half_as_ushort(__float2half_rn(fminf(fmaxf(d, -65504.f), 65504.f)));
}

// One block, V elements from each of 32 / V lanes: the codes and the scale.
// q8_0 codes are offset by 128, q4_0's by 8.
template <int KIND, int V>
__device__ inline void encode_block(const float (&x)[V], int j, uint32_t (&q)[V], uint32_t& s) {
#pragma clang fp contract(off)
  float amax = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < V; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = group_max<32 / V>(amax);
  float d;
  if constexpr (KIND == KV_Q8_0) {
    d = amax / 127.0f;
  } else {
    // the first element of magnitude amax: its index and, in bit 0, its sign
    int at = 4096;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) at = fabsf(x[i]) == amax ? 2 * (V * j + i) + int(__float_as_uint(x[i]) >> 31) : at;
    d = ((group_min<32 / V>(at) & 1) ? -amax : amax) / -8.0f;
  }
  const float id = q8_1_id(d);
#pragma unroll
  for (int i = 0; i < V; ++i)
    q[i] = uint32_t(KIND == KV_Q8_0 ? round_code(x[i], id, -127, 127) + 128 : round_code(x[i], id, -8, 7) + 8);
  s = scale16(d);
}

// A cache row from its lanes (see UnitShape).  chunk: the (page, head)'s.
template <int KIND, int D, int V>
__device__ inline void put_units(uint8_t* chunk, uint32_t shift, uint32_t tok, int j, int bp, const float (&x)[V],
                                 const float (&y)[V], bool store) {
  uint8_t* row = chunk + kv_codes_at(KIND, D, tok);
  if constexpr (KIND == KV_BF16) {
    if (store) {
      uint32_t* w = reinterpret_cast<uint32_t*>(row) + 32 * bp + V / 2 * j;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        w[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
        w[16 + i] = bf16_pair(y[2 * i], y[2 * i + 1]);
      }
    }
  } else {
    constexpr int NB = D / 32;
    uint32_t a[V], b[V], s0, s1;
    encode_block<KIND, V>(x, j, a, s0);
    encode_block<KIND, V>(y, j, b, s1);
    if (store) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const int c = (V * j + i) / 2;
        if constexpr (KIND == KV_Q8_0)
          *reinterpret_cast<uint32_t*>(row + 2 * NB * c + 4 * bp) = a[i] | (a[i + 1] << 8) | (b[i] << 16) | (b[i + 1] << 24);
        else
          *reinterpret_cast<uint16_t*>(row + NB * c + 2 * bp) = uint16_t(a[i] | (a[i + 1] << 4) | (b[i] << 8) | (b[i + 1] << 12));
      }
      if (j == 0)
        *reinterpret_cast<uint32_t*>(chunk + kv_scales_at(KIND, D, shift, tok) + 4 * bp) = s0 | (s1 << 16);
    }
  }
}

template <class T, int KIND, int D>
__device__ inline void get_units(const uint8_t* chunk, uint32_t shift, uint32_t tok, int j, int bp,
                                 float (&x)[Elem<T>::kVec], float (&y)[Elem<T>::kVec]) {
  constexpr int V = Elem<T>::kVec;
  const uint8_t* row = chunk + kv_codes_at(KIND, D, tok);
  if constexpr (KIND == KV_BF16) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + 32 * bp + V / 2 * j;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
      y[2 * i] = bf16_lo(w[16 + i]);
      y[2 * i + 1] = bf16_hi(w[16 + i]);
    }
  } else {
    constexpr int NB = D / 32;
    const uint32_t s = *reinterpret_cast<const uint32_t*>(chunk + kv_scales_at(KIND, D, shift, tok) + 4 * bp);
    const float d0 = h2f(s & 0xFFFFu), d1 = h2f(s >> 16);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const int c = V / 2 * j + i;
      if constexpr (KIND == KV_Q8_0) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(row + 2 * NB * c + 4 * bp);
        x[2 * i] = d0 * (cvt_ubyte<0>(w) - 128.f);
        x[2 * i + 1] = d0 * (cvt_ubyte<1>(w) - 128.f);
        y[2 * i] = d1 * (cvt_ubyte<2>(w) - 128.f);
        y[2 * i + 1] = d1 * (cvt_ubyte<3>(w) - 128.f);
      } else {
        const uint32_t w = *reinterpret_cast<const uint16_t*>(row + NB * c + 2 * bp);
        x[2 * i] = d0 * (float(w & 15u) - 8.f);
        x[2 * i + 1] = d0 * (float((w >> 4) & 15u) - 8.f);
        y[2 * i] = d1 * (float((w >> 8) & 15u) - 8.f);
        y[2 * i + 1] = d1 * (float(w >> 12) - 8.f);
      }
    }
  }
}

// Keys (blockIdx.y == 0) or values into the cache.  Bound by the rounding's
// instructions, about 40 an element pair: 512 tokens of 32 heads of 128 from
// binary32 to q4_0 (43 MB with their load) 12.2 us for store and load; with an
// element pair a lane, whose share of reductions and addresses is twice as
// large, 13.6.
template <class T, int KIND, int D>
__global__ __launch_bounds__(kThreads) void kv_store_kernel(KvView cache, Rows k, Rows v, const int64_t* slots,
                                                            uint32_t rows) {
  constexpr int V = Elem<T>::kVec;
  using S = UnitShape<V, D>;
  const Rows in = blockIdx.y ? v : k;
  uint8_t* buf = blockIdx.y ? cache.v : cache.k;
  const int lane = threadIdx.x % S::kLanes, j = lane % S::kBlock, bp = lane / S::kBlock;
  const uint32_t r = blockIdx.x * S::kRows + threadIdx.x / S::kLanes;
  if (r >= rows) return;
  const uint32_t tok = r / cache.heads, head = r - tok * cache.heads;
  const u32x4* src = reinterpret_cast<const u32x4*>(in.p + tok * in.ld + (int64_t(head) * D + 64 * bp) * int(sizeof(T))) + j;
  float x[V], y[V];
  Elem<T>::unpack(src[0], x);
  Elem<T>::unpack(src[S::kBlock], y);
  const int64_t slot = slots[tok];
  const bool in_cache = kv_slot_in(cache, slot);
  const int64_t s = in_cache ? slot : 0;
  put_units<KIND, D, V>(buf + kv_chunk_at(cache, s >> cache.shift, head), cache.shift,
                        uint32_t(s & ((int64_t(1) << cache.shift) - 1)), j, bp, x, y, in_cache);
}

// The cache's keys (blockIdx.y == 0) or values as rows.  Bound by the bytes
// written: 16383 rows of 4 heads of 256 from q8_0 to bf16 (103 MB) with the
// store of 1000 of them 24.0 us, where the encoder's lanes (an element pair of
// two blocks, 4-byte stores) took 34.2 and stores past the caches 27.
template <class T, int KIND, int D>
__global__ __launch_bounds__(kThreads) void kv_load_kernel(KvView cache, Rows k, Rows v, const int64_t* slots,
                                                           uint32_t rows) {
  using S = UnitShape<Elem<T>::kVec, D>;
  const Rows out = blockIdx.y ? v : k;
  const uint8_t* buf = blockIdx.y ? cache.v : cache.k;
  const int lane = threadIdx.x % S::kLanes, j = lane % S::kBlock, bp = lane / S::kBlock;
  const uint32_t r = blockIdx.x * S::kRows + threadIdx.x / S::kLanes;
  if (r >= rows) return;
  float x[Elem<T>::kVec] = {}, y[Elem<T>::kVec] = {};
  const uint32_t tok = r / cache.heads, head = r - tok * cache.heads;
  const int64_t s = slots[tok];
  if (kv_slot_in(cache, s))
    get_units<T, KIND, D>(buf + kv_chunk_at(cache, s >> cache.shift, head), cache.shift,
                          uint32_t(s & ((int64_t(1) << cache.shift) - 1)), j, bp, x, y);
  u32x4* dst = reinterpret_cast<u32x4*>(out.p + tok * out.ld + (int64_t(head) * D + 64 * bp) * int(sizeof(T))) + j;
  dst[0] = Elem<T>::pack(x);
  dst[S::kBlock] = Elem<T>::pack(y);
}

// Rotation and store in one launch.  Workgroups 0 .. rope_chunks - 1 of a
// token take its query and key rows; a key row passes through LDS (binary32)
// from the rotation's lanes to the encoder's.  The others take value rows.  For
// the one launch that it saves a decode step: one token of 32, 32 and 32 heads
// of 128 into q8_0 in 2.2 to 3.2 us, bound by its latencies.
template <class T, int KIND, int D>
__global__ __launch_bounds__(kThreads) void qkv_rope_store_kernel(KvView cache, Rows q, Rows k, Rows v, Rows qo,
                                                                  int hq, int rope_chunks, int chunks,
                                                                  const int64_t* slots, RopeArgs r) {
  using S = RowShape<T, D>;
  constexpr int V = S::kVec;
  __shared__ f32x2 cs[D / 2];
  __shared__ __attribute__((aligned(16))) float rows_f32[S::kRows * D];
  const int64_t tok = blockIdx.x / unsigned(chunks);
  const int chunk = int(blockIdx.x % unsigned(chunks));
  const int hk = int(cache.heads);
  const int64_t slot = slots[tok];
  const bool in_cache = kv_slot_in(cache, slot);
  const int64_t s = in_cache ? slot : 0;
  const int64_t page = s >> cache.shift;
  const uint32_t at = uint32_t(s & ((int64_t(1) << cache.shift) - 1));
  if (chunk >= rope_chunks) {  // uniform over the workgroup
    using E = UnitShape<V, D>;
    const int lane = threadIdx.x % E::kLanes, j = lane % E::kBlock, bp = lane / E::kBlock;
    const int head = (chunk - rope_chunks) * E::kRows + threadIdx.x / E::kLanes;
    if (head >= hk) return;
    const u32x4* src = reinterpret_cast<const u32x4*>(v.p + tok * v.ld + (int64_t(head) * D + 64 * bp) * int(sizeof(T))) + j;
    float x[V], y[V];
    Elem<T>::unpack(src[0], x);
    Elem<T>::unpack(src[E::kBlock], y);
    put_units<KIND, D, V>(cache.v + kv_chunk_at(cache, page, head), cache.shift, at, j, bp, x, y, in_cache);
    return;
  }
  const int first = chunk * S::kRows, row = first + threadIdx.x / S::kLanes, l = threadIdx.x % S::kLanes;
  const bool isq = row < hq, is = row < hq + hk;
  int ua, ub;
  units_of<T, D>(l, r.rot, ua, ub);
  u32x4 xa{}, xb{};
  if (is) {
    const u32x4* src = reinterpret_cast<const u32x4*>((isq ? q.p : k.p) + tok * (isq ? q.ld : k.ld)) +
                       (isq ? row : row - hq) * S::kUnits;
    xa = src[ua];
    xb = src[ub];
  }
  fill_angles(r, tok, cs);
  __syncthreads();
  float a[S::kVec], b[S::kVec];
  Elem<T>::unpack(xa, a);
  Elem<T>::unpack(xb, b);
  if (is) norm_rope<T, D>(a, b, l, ua, ub, r, isq ? r.gq : r.gk, cs);
  if (isq) {
    u32x4* dst = reinterpret_cast<u32x4*>(qo.p + tok * qo.ld) + row * S::kUnits;
    dst[ua] = Elem<T>::pack(a);
    dst[ub] = Elem<T>::pack(b);
  } else if (is) {
    float* dst = rows_f32 + (row - first) * D;
#pragma unroll
    for (int i = 0; i < S::kVec; i += 4) {
      *reinterpret_cast<f32x4*>(dst + ua * S::kVec + i) = f32x4{a[i], a[i + 1], a[i + 2], a[i + 3]};
      *reinterpret_cast<f32x4*>(dst + ub * S::kVec + i) = f32x4{b[i], b[i + 1], b[i + 2], b[i + 3]};
    }
  }
  if (first + S::kRows <= hq) return;  // no key row here (uniform)
  __syncthreads();
  using E = UnitShape<4, D>;
  const int lane = threadIdx.x % E::kLanes, j = lane % E::kBlock, bp = lane / E::kBlock;
  for (int i = threadIdx.x / E::kLanes; i < S::kRows; i += E::kRows) {
    const int head = first + i - hq;
    if (head < 0 || head >= hk) continue;
    const u32x4* src = reinterpret_cast<const u32x4*>(rows_f32 + i * D + 64 * bp) + j;
    float x[4], y[4];
    Elem<float>::unpack(src[0], x);
    Elem<float>::unpack(src[E::kBlock], y);
    put_units<KIND, D, 4>(cache.k + kv_chunk_at(cache, page, head), cache.shift, at, j, bp, x, y, in_cache);
  }
}

// The arguments of a launch that begins at token t.
RopeArgs rope_args(const skg_rope* r, int64_t t) {
  return RopeArgs{r->rot, r->interleaved, r->norm, r->eps, r->pos ? r->pos + t : nullptr, r->inv_freq, r->gq, r->gk};
}

Rows rows_of(const void* p, int64_t ld, skg_dtype dt, int64_t t) {
  const int64_t bytes = ld * (dt == SKG_F32 ? 4 : 2);
  return Rows{p ? static_cast<uint8_t*>(const_cast<void*>(p)) + t * bytes : nullptr, bytes};
}

// f(t, n) for tokens t .. t + n - 1, in as few launches as they fit: `groups`
// workgroups for `tokens` of them.
template <class F>
hipError_t by_tokens(int64_t T, int64_t tokens, int64_t groups, F&& f) {
  const int64_t most = kMaxGroups / groups * tokens;
  for (int64_t t = 0; t < T; t += most) {
    f(t, T - t < most ? T - t : most);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Calls f with the type, cache kind and head size as template arguments.
template <class F>
hipError_t by_type(skg_dtype dt, F&& f) {
  return dt == SKG_F32 ? f(float{}) : f(__bf16{});
}
template <class F>
hipError_t by_dim(int D, F&& f) {
  return D == 64 ? f(std::integral_constant<int, 64>{})
                 : D == 128 ? f(std::integral_constant<int, 128>{}) : f(std::integral_constant<int, 256>{});
}
template <class F>
hipError_t by_kind(int kind, F&& f) {
  return kind == KV_BF16 ? f(std::integral_constant<int, KV_BF16>{})
                         : kind == KV_Q8_0 ? f(std::integral_constant<int, KV_Q8_0>{})
                                           : f(std::integral_constant<int, KV_Q4_0>{});
}

}  // namespace

hipError_t launch_qk_norm_rope(skg_dtype dt, int64_t T, int hq, int hk, int D, const void* q, int64_t ldq,
                               const void* k, int64_t ldk, const skg_rope* rope, void* qo, int64_t ldqo, void* ko,
                               int64_t ldko, hipStream_t stream) {
  return by_type(dt, [&](auto t) {
    return by_dim(D, [&](auto d) {
      using E = decltype(t);
      constexpr int N = RowShape<E, d()>::kRows;
      auto launch = [&](auto kernel, int rows) {  // rows of a workgroup
        const int64_t chunks = (hq + hk + rows - 1) / rows;
        return by_tokens(T, 1, chunks, [&](int64_t t, int64_t n) {
          hipLaunchKernelGGL(kernel, dim3(unsigned(n * chunks)), dim3(kThreads), 0, stream, rows_of(q, ldq, dt, t),
                             rows_of(k, ldk, dt, t), rows_of(qo, ldqo, dt, t), rows_of(ko, ldko, dt, t), hq, hk,
                             int(chunks), rope_args(rope, t));
        });
      };
      if (T * ((hq + hk + N - 1) / N) >= kManyGroups) return launch(qk_norm_rope_kernel<E, d(), 2>, 2 * N);
      return launch(qk_norm_rope_kernel<E, d(), 1>, N);
    });
  });
}

hipError_t launch_kv_store(const KvView& c, int kind, int D, skg_dtype dt, int64_t T, const void* k, int64_t ldk,
                           const void* v, int64_t ldv, const int64_t* slots, hipStream_t stream) {
  return by_type(dt, [&](auto t) {
    return by_dim(D, [&](auto d) {
      return by_kind(kind, [&](auto kd) {
        constexpr int N = UnitShape<Elem<decltype(t)>::kVec, d()>::kRows;
        return by_tokens(T, N, c.heads, [&](int64_t t0, int64_t n) {  // N tokens fill as many workgroups as they have heads
          const int64_t rows = n * c.heads;
          hipLaunchKernelGGL((kv_store_kernel<decltype(t), kd(), d()>), dim3(unsigned((rows + N - 1) / N), 2),
                             dim3(kThreads), 0, stream, c, rows_of(k, ldk, dt, t0), rows_of(v, ldv, dt, t0), slots + t0,
                             uint32_t(rows));
        });
      });
    });
  });
}

hipError_t launch_kv_load(const KvView& c, int kind, int D, skg_dtype dt, int64_t T, const int64_t* slots, void* k,
                          int64_t ldk, void* v, int64_t ldv, hipStream_t stream) {
  return by_type(dt, [&](auto t) {
    return by_dim(D, [&](auto d) {
      return by_kind(kind, [&](auto kd) {
        constexpr int N = UnitShape<Elem<decltype(t)>::kVec, d()>::kRows;
        return by_tokens(T, N, c.heads, [&](int64_t t0, int64_t n) {  // N tokens fill as many workgroups as they have heads
          const int64_t rows = n * c.heads;
          hipLaunchKernelGGL((kv_load_kernel<decltype(t), kd(), d()>), dim3(unsigned((rows + N - 1) / N), 2),
                             dim3(kThreads), 0, stream, c, rows_of(k, ldk, dt, t0), rows_of(v, ldv, dt, t0), slots + t0,
                             uint32_t(rows));
        });
      });
    });
  });
}

hipError_t launch_qkv_rope_store(const KvView& c, int kind, int D, skg_dtype dt, int64_t T, int hq, const void* q,
                                 int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                 const skg_rope* rope, const int64_t* slots, void* qo, int64_t ldqo,
                                 hipStream_t stream) {
  return by_type(dt, [&](auto t) {
    return by_dim(D, [&](auto d) {
      return by_kind(kind, [&](auto kd) {
        using E = decltype(t);
        constexpr int N = RowShape<E, d()>::kRows, M = UnitShape<Elem<E>::kVec, d()>::kRows;
        const int64_t rope_chunks = (hq + int(c.heads) + N - 1) / N, chunks = rope_chunks + (c.heads + M - 1) / M;
        return by_tokens(T, 1, chunks, [&](int64_t t0, int64_t n) {
          hipLaunchKernelGGL((qkv_rope_store_kernel<E, kd(), d()>), dim3(unsigned(n * chunks)), dim3(kThreads), 0,
                             stream, c, rows_of(q, ldq, dt, t0), rows_of(k, ldk, dt, t0), rows_of(v, ldv, dt, t0),
                             rows_of(qo, ldqo, dt, t0), hq, int(rope_chunks), int(chunks), slots + t0,
                             rope_args(rope, t0));
        });
      });
    });
  });
}

}  // namespace skg
