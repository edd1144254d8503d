// Attention of drafted tokens over a paged cache: arguments and the kernel
// (instantiated per cache format and row type by tree_attn_*.hip).
//
// The rows of a cache head are its drafted tokens' query heads, r = i * group
// + h, in tiles of 16.  A wave walks its keys 32 at a time, once, with the
// running maximum and sum of the softmax:
//   S^T = K Q^T   : A = 16 keys, B = 16 rows, per 32-element block of a head;
//                   the block's product is scaled by the key's scale of that
//                   block in binary32, so the codes stay exact in fp16;
//   p   = 2^(s - M)
//   O^T = V^T P^T : A = 16 elements of one block, B = the 16 rows' p times the
//                   keys' scales of that block.
// Transposed so, a lane holds one row (lane & 15) throughout: M and l are
// lane-local, and p goes from the first product's result to the second's
// operand without leaving its lane (the order of keys within an operand is
// free as long as V uses the same one).  The cache's byte order makes both
// A operands whole bytes of the lane's loads: for K eight consecutive elements
// of a block, for V one element of eight keys.
//
// Precision.  Codes are exact in fp16 (times 2^-9, see f16 conversions below).
// For float32 rows q and p are sums of fp16 (or, for a bf16 cache, bf16)
// terms: two of 11 bits, three of 8.  p 2^x times a scale could leave fp16's
// range, so M carries a power of two as well: M = m - sigma with sigma such
// that the largest scale seen times p's largest 2^4 lands on 2^15; o and l
// share it and it drops out of o / l.  M moves only when a score passes it by
// 4 or a larger scale comes (rare), which a wave finds out with one ballot.
// What is below fp16's smallest step is lost: at most 2^-33 of the largest
// scale's value a key (2^-25 against a p of 1 at 2^11 times a scale that may
// be three bits below its bound).
#pragma once

#include "kv_common.h"
#include "kernels.h"

namespace skg {

struct TreeArgs {
  KvView cache;
  const uint8_t* q;
  int64_t ldq;  // bytes
  uint8_t* o;   // or null
  int64_t ldo;  // bytes
  uint8_t* oq;  // or null
  const int32_t* cu;  // or null: T / n_seqs each
  const int32_t* ctx;
  const int32_t* table;
  int64_t width;
  int64_t max_kv;
  const uint64_t* mask;  // or null: a chain
  float scale;
  int64_t T;
  int n_seqs;
  int hq;
  int group;  // query heads of a cache head
  int max_draft;
  int64_t blocks;  // Q8_1 blocks of a token's row
  // how the work is split
  int splits;      // workgroups along the keys; > 1: partial results in ws
  int row_groups;  // workgroups along the rows
  float* ws;       // [T * hq][splits][D] sums, then [T * hq][splits][2] (M, l)
};

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kStep = 32;                 // keys of a wave's step
constexpr int kMinSteps = 2 * kAttnWaves; // steps of a split at least

// Steps of each split of a sequence of `keys` keys (the same in the kernel
// that writes the partial results and in the one that joins them).
__host__ __device__ inline int steps_per_split(int keys, int splits) {
  const int steps = keys / kStep + (keys % kStep != 0);
  const int per = (steps + splits - 1) / splits;
  return per < kMinSteps ? kMinSteps : per;
}

__device__ inline KvSpan span_of(const TreeArgs& a, int b) {
  const int64_t per = a.T / a.n_seqs;
  const int32_t t0 = a.cu ? a.cu[b] : int32_t(b * per), t1 = a.cu ? a.cu[b + 1] : int32_t((b + 1) * per);
  return kv_span(a.ctx[b], t0, t1, a.T, a.max_draft, a.max_kv);
}

constexpr int kLazy = 4;          // a score may pass M by this much (a power of two) before M moves
constexpr float kNoMax = -1e37f;  // M of a row that has seen nothing

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <bool F16>
__device__ inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ inline uint32_t f16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, f16x2{static_cast<_Float16>(a), static_cast<_Float16>(b)});
}
__device__ inline float f16_lo(uint32_t u) { return float(__builtin_bit_cast(f16x2, u).x); }
__device__ inline float f16_hi(uint32_t u) { return float(__builtin_bit_cast(f16x2, u).y); }

// NT terms of the pair (a, b): t[0] the rounded values, t[1] what is left, ...
template <bool F16, int NT>
__device__ inline void split_pair(float a, float b, uint32_t (&t)[NT]) {
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if constexpr (F16) {
      t[i] = f16_pair(a, b);
      a = __builtin_fmaf(f16_lo(t[i]), -1.0f, a);
      b = __builtin_fmaf(f16_hi(t[i]), -1.0f, b);
    } else {
      t[i] = bf16_pair(a, b);
      a -= bf16_lo(t[i]);
      b -= bf16_hi(t[i]);
    }
  }
}

// The terms of (p0 s0, p1 s1), s the low or high fp16 of w0 and w1: the rounded
// products, and with NT = 2 what each leaves.  Written as fused operations
// whose operands are widened fp16 values, which the compiler turns into one
// mixed-precision instruction a term; a plain product is formed in binary32
// and converted (2.5 times the instructions).
template <int NT>
__device__ inline void scaled_pair(float p0, float p1, uint32_t w0, uint32_t w1, int high, uint32_t (&t)[NT]) {
  const f16x2 a = __builtin_bit_cast(f16x2, w0), b = __builtin_bit_cast(f16x2, w1);
  const _Float16 s0 = high ? a.y : a.x, s1 = high ? b.y : b.x;
  const _Float16 h0 = static_cast<_Float16>(__builtin_fmaf(p0, float(s0), 0.f));
  const _Float16 h1 = static_cast<_Float16>(__builtin_fmaf(p1, float(s1), 0.f));
  t[0] = __builtin_bit_cast(uint32_t, f16x2{h0, h1});
  if constexpr (NT > 1) {
    const _Float16 l0 = static_cast<_Float16>(__builtin_fmaf(p0, float(s0), -float(h0)));
    const _Float16 l1 = static_cast<_Float16>(__builtin_fmaf(p1, float(s1), -float(h1)));
    t[1] = __builtin_bit_cast(uint32_t, f16x2{l0, l1});
  }
}

// Codes as fp16.  Two unsigned bytes in 16-bit halves are the fp16 subnormals
// n 2^-24, which the matrix instructions take as they are: K's operand is that
// (a high nibble is 16 n, against q / 16), and the zero of the codes is taken
// off by the product's initial value, -zero 2^-24 sum q of the block, which is
// constant for a row.  For V the same would leave differences of long sums, so
// one packed fma makes (n - zero) 2^-9 of them, exactly (mul = 2^15, or 2^11
// for a high nibble).
__device__ inline uint32_t f16_codes(uint32_t x, float mul, float zero) {
  const f16x2 m = {static_cast<_Float16>(mul), static_cast<_Float16>(mul)};
  const f16x2 z = {static_cast<_Float16>(-zero), static_cast<_Float16>(-zero)};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, x), m, z));
}
__device__ inline uint32_t q8_pair(uint32_t x) { return f16_codes(x, 32768.f, 0.25f); }
__device__ inline uint32_t q4_low(uint32_t x) { return f16_codes(x & 0x000F000Fu, 32768.f, 0.015625f); }
__device__ inline uint32_t q4_high(uint32_t x) { return f16_codes(x & 0x00F000F0u, 2048.f, 0.015625f); }
constexpr float kVScale = 512.f;          // 2^9
constexpr float kKScale = 16777216.f;     // 2^24
// -zero 2^-24 in both halves: of q8_0, of q4_0's low and high nibbles
constexpr uint32_t kZero8 = 0x80808080u, kZero4Low = 0x80088008u, kZero4High = 0x80808080u;

// Byte y0 of w0 and byte y1 of w1, each in a 16-bit half.
__device__ inline uint32_t two_bytes(uint32_t w0, int y0, uint32_t w1, int y1) {
  return __builtin_amdgcn_perm(w1, w0, 0x0C000C00u | uint32_t((4 + y1) << 16) | uint32_t(y0));
}
// The low (hi = 0) or high 16 bits of w0 and w1.
__device__ inline uint32_t two_halves(uint32_t w0, uint32_t w1, int hi) {
  return __builtin_amdgcn_perm(w1, w0, hi ? 0x07060302u : 0x05040100u);
}

template <int KIND, int D>
struct AttnShape {
  static constexpr bool kF16 = KIND != KV_BF16;
  static constexpr int NB = D / 32;
  // 32-bit words of a lane: K of one 16-key tile (four of the sixteen pair
  // columns), V of one key (one column), scales of four keys
  static constexpr int KW = KIND == KV_BF16 ? 4 * NB : KIND == KV_Q8_0 ? 2 * NB : NB;
  static constexpr int VW = KIND == KV_BF16 ? NB : KIND == KV_Q8_0 ? NB / 2 : (NB + 3) / 4;
  static constexpr int SW = 2 * NB;

  // A wave's LDS slot for a step of 32 keys: K codes, V codes [2][16][row],
  // then the scales of K and V, [32][NB] fp16, each in whole 256 bytes.
  static constexpr int kRow = int(kv_row_bytes(KIND, D));
  static constexpr int kRC = kRow / 16;                        // 16-byte units of a row
  static constexpr int kTile = 16 * kRow;
  static constexpr int kScales = !kF16 ? 0 : NB <= 4 ? 256 : 512;
  static constexpr int kSlot = 4 * kTile + 2 * kScales;
  static constexpr int kKOff = 0, kVOff = 2 * kTile, kSkOff = 4 * kTile, kSvOff = kSkOff + kScales;
  // slots of a wave: what lets two workgroups share a CU's 160 KB
  static constexpr int kFit = 80 * 1024 / (kAttnWaves * kSlot);
  static constexpr int kSlots = kFit < 1 ? 1 : kFit > 4 ? 4 : kFit;
  // transfers of K (or V) of a step
  static constexpr int kCopies = kRow / 32 + kScales / 256;
  static_assert(kCopies * (2 * kSlots + 1) <= 63, "vmcnt");
};

// LDS position of a tile's 16-byte unit j of row c: the units of eight and of
// sixteen consecutive rows at one j lie on different banks.
template <int RC>
__device__ inline int k_swizzle(int c) {
  return RC >= 16 ? c : RC == 8 ? (c & 7) ^ (c >> 3) : RC == 4 ? ((c >> 1) & 3) ^ (c >> 3) : 0;
}
// LDS row of V's key c (and back): the rows 4g + i of the four g differ modulo 4.
__device__ inline int v_row(int c) { return c ^ (c >> 2); }

__device__ inline void dma4(const void* src, uint32_t dst) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(__builtin_amdgcn_readfirstlane(dst)),
               "v"(src)
               : "memory", "m0");
#pragma clang diagnostic pop
}
template <int N>
__device__ inline void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Waits for a step's K (or V) while `ahead` later steps, and for V the K of
// one more, are on their way.  C copies for each of K and V.
template <int C, int SLOTS, bool K>
__device__ inline void wait_ahead(int ahead, bool more) {
  if (more) {
    wait_copies<2 * C * (SLOTS - 1) + C>();
  } else if (ahead == SLOTS - 1) {
    wait_copies<2 * C * (SLOTS - 1) + (K ? C : 0)>();
  } else if constexpr (SLOTS > 1) {
    wait_ahead<C, SLOTS - 1, K>(ahead, false);
  }
}
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Copies K (V = false) or V of the step's two 16-key tiles and their scales
// into the slot at LDS address dst.  A page outside the cache is replaced by
// page 0 (every key of it is masked).
struct StepAt {
  uint64_t codes[2], scales[2];  // offsets of the tiles in the buffers of K and V
};
template <int KIND, int D>
__device__ inline StepAt step_at(const KvView& c, uint32_t head, int key, int32_t p0, int32_t p1) {
  StepAt s;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int32_t page = t ? p1 : p0;
    const uint64_t chunk = kv_chunk_at(c, kv_page_in(c, page) ? page : 0, head);
    const uint32_t tok = uint32_t(key + 16 * t) & ((1u << c.shift) - 1);
    s.codes[t] = chunk + kv_codes_at(KIND, D, tok);
    s.scales[t] = chunk + kv_scales_at(KIND, D, c.shift, tok);
  }
  return s;
}
template <int KIND, int D, bool V>
__device__ inline void copy_step(const KvView& c, const StepAt& from, uint32_t dst) {
  using S = AttnShape<KIND, D>;
  const int lane = threadIdx.x & 63;
  const uint8_t* buf = V ? c.v : c.k;
  const uint32_t codes = dst + (V ? S::kVOff : S::kKOff);
  if constexpr (S::kRow >= 64) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < S::kRow / 64; ++j) {
        const int row = j * (64 / S::kRC) + lane / S::kRC, unit = lane % S::kRC;
        const uint32_t off = V ? v_row(row) * S::kRow + 16 * unit : row * S::kRow + 16 * (unit ^ k_swizzle<S::kRC>(row));
        dma16_sv(buf + from.codes[t], off, codes + t * S::kTile + 1024 * j);
      }
  } else {  // both tiles in one transfer
    static_assert(S::kRow >= 64 || S::kRow == 32, "row");
    const int row = (lane & 31) / 2, unit = lane & 1;
    const uint8_t* src = buf + (lane < 32 ? from.codes[0] : from.codes[1]);
    dma16(src + (V ? v_row(row) : row) * S::kRow + 16 * unit, codes);
  }
  if constexpr (S::kF16) {
    // 16 NB words over both tiles (NB = 2: the upper lanes repeat the lower)
#pragma unroll
    for (int j = 0; j < S::kScales / 256; ++j) {
      const int w = (64 * j + lane) % (16 * S::NB), t = w / (8 * S::NB);
      dma4(buf + (t ? from.scales[1] : from.scales[0]) + 4 * (w - t * 8 * S::NB), dst + (V ? S::kSvOff : S::kSkOff) + 256 * j);
    }
  }
}

template <int N>
__device__ inline void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 t = *reinterpret_cast<const u32x4*>(p + 4 * i);
      w[i] = t.x, w[i + 1] = t.y, w[i + 2] = t.z, w[i + 3] = t.w;
    }
  } else if constexpr (N == 2) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    w[0] = t.x, w[1] = t.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// What a lane holds of a step, lane (c, g) = (lane & 15, lane >> 4).
template <int KIND, int D>
struct StepRegs {
  using S = AttnShape<KIND, D>;
  uint32_t k[2][S::KW];   // key c of each tile, its elements 8g .. 8g + 7 of every block
  uint32_t v[8][S::VW];   // keys 4g + i (tile 0), 4g + i - 4 (tile 1), column c
  uint32_t sk[2][S::SW];  // scales of keys 4g .. 4g + 3 of each tile
  uint32_t sv[2][S::SW];
  int key;                // first key
  bool there[2];          // whether a tile's page is in the cache
};

template <int KIND, int D>
__device__ inline void read_k(StepRegs<KIND, D>& r, const uint8_t* slot) {
  using S = AttnShape<KIND, D>;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const uint8_t* row = slot + S::kKOff + t * S::kTile + c * S::kRow;
    const int z = k_swizzle<S::kRC>(c);
    if constexpr (KIND == KV_BF16) {  // block b's elements 8g .. 8g + 7 are unit 4b + g
#pragma unroll
      for (int b = 0; b < S::NB; ++b) load_words<4>(row + 16 * ((4 * b + g) ^ z), &r.k[t][4 * b]);
    } else if constexpr (S::KW >= 4) {
#pragma unroll
      for (int j = 0; j < S::KW / 4; ++j) load_words<4>(row + 16 * ((g * (S::KW / 4) + j) ^ z), &r.k[t][4 * j]);
    } else {
      load_words<S::KW>(row + 4 * S::KW * g, r.k[t]);
    }
    if constexpr (S::kF16) load_words<S::SW>(slot + S::kSkOff + (16 * t + 4 * g) * 2 * S::NB, r.sk[t]);
  }
}
template <int KIND, int D>
__device__ inline void read_v(StepRegs<KIND, D>& r, const uint8_t* slot) {
  using S = AttnShape<KIND, D>;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* p = slot + S::kVOff + t * S::kTile + v_row(4 * g + i) * S::kRow + S::kRC * c;
      if constexpr (S::kRC == 2) r.v[4 * t + i][0] = *reinterpret_cast<const uint16_t*>(p);
      else load_words<S::VW>(p, r.v[4 * t + i]);
    }
    if constexpr (S::kF16) load_words<S::SW>(slot + S::kSvOff + (16 * t + 4 * g) * 2 * S::NB, r.sv[t]);
  }
}

// K operand of block b of tile t: elements 8g .. 8g + 7 of the block (for q4_0
// in the order 0 2 1 3 4 6 5 7, see q_order).
template <int KIND, int D>
__device__ inline u32x4 k_operand(const StepRegs<KIND, D>& r, int t, int b) {
  constexpr int NB = D / 32;
  u32x4 a;
  if constexpr (KIND == KV_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = r.k[t][4 * b + i];
  } else if constexpr (KIND == KV_Q8_0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = r.k[t][i * (NB / 2) + (b >> 1)];
      a[i] = two_bytes(w, 2 * (b & 1), w, 2 * (b & 1) + 1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {  // bytes i NB + b and (i + 1) NB + b
      const int y0 = i * NB + b, y1 = (i + 1) * NB + b;
      const uint32_t x = two_bytes(r.k[t][y0 >> 2], y0 & 3, r.k[t][y1 >> 2], y1 & 3);
      a[i] = x & 0x000F000Fu;
      a[i + 1] = x & 0x00F000F0u;
    }
  }
  return a;
}

// V operand: column element n of the lane's eight keys.  Quantised: n = 2 b + e;
// bf16: element (D / 16) c + n.
template <int KIND, int D>
__device__ inline u32x4 v_operand(const StepRegs<KIND, D>& r, int n) {
  u32x4 a;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (KIND == KV_BF16) {
      a[i] = two_halves(r.v[2 * i][n >> 1], r.v[2 * i + 1][n >> 1], n & 1);
    } else if constexpr (KIND == KV_Q8_0) {
      a[i] = q8_pair(two_bytes(r.v[2 * i][n >> 2], n & 3, r.v[2 * i + 1][n >> 2], n & 3));
    } else {
      const uint32_t x = two_bytes(r.v[2 * i][n >> 3], (n >> 1) & 3, r.v[2 * i + 1][n >> 3], (n >> 1) & 3);
      a[i] = (n & 1) ? q4_high(x) : q4_low(x);
    }
  }
  return a;
}

// Element of the result that lane (., g) holds at [n][i].
template <int KIND, int D>
__device__ inline int o_element(int g, int n, int i) {
  return KIND == KV_BF16 ? (D / 16) * (4 * g + i) + n : 32 * (n >> 1) + 2 * (4 * g + i) + (n & 1);
}

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ inline float pow2(int e) { return __builtin_bit_cast(float, uint32_t(127 + e) << 23); }
// Largest of the four lanes of a row.
__device__ inline float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ inline float row_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// A wave's rows: RT tiles of 16, lane & 15 each.
template <int KIND, int D, int NT, int RT>
struct WaveRows {
  uint32_t q[RT][D / 32][NT][4];
  f32x4 zero[RT][KIND == KV_BF16 ? 1 : D / 32];  // of the codes, times the row's q
  f32x4 o[RT][D / 16];
  float rs[RT];  // scores are acc * rs
  float M[RT], l[RT];
  int be;        // quantised: M's sigma allows for scales up to 2^be
  uint64_t mask[RT];
};

template <int KIND, int D, int NT, int RT>
__device__ inline void raise(WaveRows<KIND, D, NT, RT>& w, int rt, float m) {
  const float f = exp2_fast(w.M[rt] - m);
  w.M[rt] = m;
  w.l[rt] *= f;
#pragma unroll
  for (int n = 0; n < D / 16; ++n) w.o[rt][n] *= f;
}

// Scores of the row with the lane's eight keys.
template <int KIND, int D, int NT, int RT>
__device__ inline void do_scores(WaveRows<KIND, D, NT, RT>& w, StepRegs<KIND, D>& r, float (&s)[RT][8]) {
  using S = AttnShape<KIND, D>;
  constexpr int NB = S::NB;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    f32x4 acc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const u32x4 a = k_operand<KIND, D>(r, t, b);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        f32x4 x = KIND == KV_BF16 ? acc[rt] : w.zero[rt][b];
#pragma unroll
        for (int i = NT - 1; i >= 0; --i)
          x = mfma<S::kF16>(a, u32x4{w.q[rt][b][i][0], w.q[rt][b][i][1], w.q[rt][b][i][2], w.q[rt][b][i][3]}, x);
        if constexpr (KIND == KV_BF16) {
          acc[rt] = x;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // scale of key 4g + i, block b
            const uint32_t sw = r.sk[t][(i * NB + b) >> 1];
            acc[rt][i] = __builtin_fmaf((b & 1) ? f16_hi(sw) : f16_lo(sw), x[i], acc[rt][i]);
          }
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[rt][4 * t + i] = acc[rt][i] * w.rs[rt];
  }

}

// The softmax's step and the sums with V.  EDGE: keys that are not there, or
// that not every row sees.
template <int KIND, int D, int NT, int RT, bool EDGE>
__device__ inline void do_values(WaveRows<KIND, D, NT, RT>& w, StepRegs<KIND, D>& r, float (&s)[RT][8], int ctx,
                                 int keys, const uint8_t* slot) {
  using S = AttnShape<KIND, D>;
  constexpr int NB = S::NB;
  const int lane = threadIdx.x & 63, g = lane >> 4;
  // keys that the row does not see
  uint32_t seen[RT];  // bit i: the lane's key i
  if constexpr (EDGE) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      seen[rt] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = r.key + 16 * (i >> 2) + 4 * g + (i & 3), j = key - ctx;
        const bool in = r.there[i >> 2] && key < keys && (j < 0 || ((w.mask[rt] >> (j & 63)) & 1));
        seen[rt] |= uint32_t(in) << i;
        s[rt][i] = in ? s[rt][i] : -INFINITY;
      }
    }
  }

  // the largest scale of a value that is seen, and the scores, against M
  if constexpr (S::kF16) {
    uint32_t big = 0;
    if constexpr (EDGE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bool any = false;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) any |= (seen[rt] >> i) & 1;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t sw = r.sv[i >> 2][((i & 3) * NB + b) >> 1];
          const uint32_t h = ((b & 1) ? sw >> 16 : sw) & 0x7FFFu;
          big = any && h < 0x7C00u && h > big ? h : big;
        }
      }
    } else {  // every row sees all: the scales spread over the lanes
      const uint32_t* sv = reinterpret_cast<const uint32_t*>(slot + S::kSvOff);
#pragma unroll
      for (int j = 0; j < S::kScales / 256; ++j) {
        const uint32_t x = sv[64 * j + lane] & 0x7FFF7FFFu;
        big = max(big, max(x & 0xFFFFu, x >> 16));
      }
    }
    const float top = h2f(big);
    if (__ballot(!(top <= pow2(w.be)))) {
      // the next power of two and two bits of room; at most 2^18 (fp16's largest)
      float t = row_max(top);
      if constexpr (!EDGE) {
        t = fmaxf(t, dpp_f<SKG_DPP_QUAD_XOR1>(t));
        t = fmaxf(t, dpp_f<SKG_DPP_QUAD_XOR2>(t));
        t = fmaxf(t, dpp_f<SKG_DPP_ROW_HALF_MIRROR>(t));
        t = fmaxf(t, dpp_f<SKG_DPP_ROW_MIRROR>(t));
      }
      t = t < 65504.f ? t : 65504.f;
      const int be = max(w.be, int(__builtin_bit_cast(uint32_t, t) >> 23) - 127 + 3);
      const float up = float(be - w.be);
      w.be = be;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) raise<KIND, D, NT, RT>(w, rt, w.M[rt] + up);
    }
  }
  // sigma = 15 - kLazy - be: M = m - sigma, p <= 2^kLazy 2^sigma
  float room = float(kLazy);
  if constexpr (S::kF16) room = float(15 - w.be);
  bool over = false;
  float mx[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    mx[rt] = s[rt][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mx[rt] = fmaxf(mx[rt], s[rt][i]);
    over |= mx[rt] > w.M[rt] + room;
  }
  if (__ballot(over)) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float m = row_max(mx[rt]) - (room - float(kLazy));
      raise<KIND, D, NT, RT>(w, rt, fmaxf(m, w.M[rt]));
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[rt][i] = exp2_fast(s[rt][i] - w.M[rt]);
      w.l[rt] += s[rt][i];
    }

  if constexpr (KIND == KV_BF16) {
    if constexpr (EDGE) {
      // a value that is not there may be anything: zero; one that some rows
      // see may be infinite or NaN, which must not reach the others as 0 * v
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = r.key + 16 * (i >> 2) + 4 * g + (i & 3);
        const bool in = r.there[i >> 2] && key < keys;
#pragma unroll
        for (int j = 0; j < S::VW; ++j) {
          const uint32_t x = in ? r.v[i][j] : 0;
          r.v[i][j] = x;
          bad |= uint32_t((x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u);
        }
      }
      if (__ballot(bad != 0)) {
        // The sums take zeros in their place; where a row sees one, which the
        // product of "is not finite" and "is seen" counts, its sum becomes NaN.
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          const u32x4 x = v_operand<KIND, D>(r, n);
          u32x4 odd;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            odd[i] = ((x[i] & 0x7F80u) == 0x7F80u ? 0x3F80u : 0u) | ((x[i] & 0x7F800000u) == 0x7F800000u ? 0x3F800000u : 0u);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            u32x4 see;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              see[i] = ((seen[rt] >> (2 * i)) & 1 ? 0x3F80u : 0u) | ((seen[rt] >> (2 * i + 1)) & 1 ? 0x3F800000u : 0u);
            const f32x4 count = mfma<false>(odd, see, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int i = 0; i < 4; ++i) w.o[rt][n][i] = count[i] > 0.f ? __builtin_nanf("") : w.o[rt][n][i];
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < S::VW; ++j) {
            const uint32_t x = r.v[i][j];
            r.v[i][j] = ((x & 0x7F80u) == 0x7F80u ? 0u : x & 0xFFFFu) | ((x & 0x7F800000u) == 0x7F800000u ? 0u : x & 0xFFFF0000u);
          }
      }
    }
    uint32_t pt[RT][4][NT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) split_pair<false, NT>(s[rt][2 * i], s[rt][2 * i + 1], pt[rt][i]);
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      const u32x4 a = v_operand<KIND, D>(r, n);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = NT - 1; i >= 0; --i)
          w.o[rt][n] = mfma<false>(a, u32x4{pt[rt][0][i], pt[rt][1][i], pt[rt][2][i], pt[rt][3][i]}, w.o[rt][n]);
    }
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const u32x4 a0 = v_operand<KIND, D>(r, 2 * b), a1 = v_operand<KIND, D>(r, 2 * b + 1);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        uint32_t pt[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t sw[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int k = 2 * i + j;
            sw[j] = r.sv[k >> 2][((k & 3) * NB + b) >> 1];
            if constexpr (EDGE) sw[j] = ((seen[rt] >> k) & 1) ? sw[j] : 0u;  // an unseen key's scale may be NaN
          }
          scaled_pair<NT>(s[rt][2 * i], s[rt][2 * i + 1], sw[0], sw[1], b & 1, pt[i]);
        }
#pragma unroll
        for (int i = NT - 1; i >= 0; --i) {
          const u32x4 p{pt[0][i], pt[1][i], pt[2][i], pt[3][i]};
          w.o[rt][2 * b] = mfma<true>(a0, p, w.o[rt][2 * b]);
          w.o[rt][2 * b + 1] = mfma<true>(a1, p, w.o[rt][2 * b + 1]);
        }
      }
    }
  }
}

// Queries of the wave's rows [first, first + 16 RT) of a sequence's n * group
// into operand registers.  A row is scaled by a power of two into fp16's range.
template <class T, int KIND, int D, int NT, int RT>
__device__ inline void load_rows(WaveRows<KIND, D, NT, RT>& w, const TreeArgs& a, const KvSpan& sp, int head, int first) {
  constexpr bool F16 = KIND != KV_BF16;
  constexpr int NB = D / 32;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int rows = sp.n * a.group;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = first + 16 * rt + c;
    const bool is = row < rows;
    const int i = is ? row / a.group : 0, h = is ? row % a.group : 0;
    const uint8_t* src = a.q + int64_t(sp.t0 + i) * a.ldq + (int64_t(head * a.group + h) * D + 8 * g) * int(sizeof(T));
    float x[NB][8];
    float amax = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      constexpr int V = Elem<T>::kVec;
#pragma unroll
      for (int u = 0; u < 8 / V; ++u) {
        float y[V];
        u32x4 raw{0, 0, 0, 0};
        if (is) raw = *reinterpret_cast<const u32x4*>(src + (32 * b + u * V) * int(sizeof(T)));
        Elem<T>::unpack(raw, y);
#pragma unroll
        for (int j = 0; j < V; ++j) x[b][u * V + j] = y[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[b][j]));
    }
    float to = 1.f;
    w.rs[rt] = a.scale * 1.44269504f;
    if constexpr (F16) {
      amax = row_max(amax);
      int e = int((__builtin_bit_cast(uint32_t, amax) >> 23) & 255);  // |q| < 2^(e - 126)
      e = e < 40 ? 40 : (e > 220 ? 220 : e);
      to = __builtin_bit_cast(float, uint32_t(127 + 14 - (e - 126)) << 23);
      w.rs[rt] *= kKScale * __builtin_bit_cast(float, uint32_t(127 - 14 + (e - 126)) << 23);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // q4_0's operand order: 0 2 1 3 4 6 5 7
        const int i0 = KIND == KV_Q4_0 ? 4 * (j >> 1) + (j & 1) : 2 * j, i1 = KIND == KV_Q4_0 ? i0 + 2 : 2 * j + 1;
        uint32_t t[NT];
        const float f = KIND == KV_Q4_0 && (j & 1) ? to * 0.0625f : to;  // against high nibbles
        split_pair<F16, NT>(x[b][i0] * f, x[b][i1] * f, t);
#pragma unroll
        for (int k = 0; k < NT; ++k) w.q[rt][b][k][j] = t[k];
      }
    if constexpr (F16) {
      const u32x4 z = KIND == KV_Q8_0 ? u32x4{kZero8, kZero8, kZero8, kZero8}
                                      : u32x4{kZero4Low, kZero4High, kZero4Low, kZero4High};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        w.zero[rt][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = NT - 1; k >= 0; --k)
          w.zero[rt][b] = mfma<true>(z, u32x4{w.q[rt][b][k][0], w.q[rt][b][k][1], w.q[rt][b][k][2], w.q[rt][b][k][3]}, w.zero[rt][b]);
      }
    }
    w.mask[rt] = !is ? 0 : a.mask ? a.mask[sp.t0 + i] : ~uint64_t(0) >> (63 - i);
    w.M[rt] = kNoMax;
    w.l[rt] = 0.f;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) w.o[rt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  w.be = -40;
}

// EPT consecutive elements of a token's row, from `at`, in float32, bf16 or as Q8_1 (lanes of a
// 32-element block adjacent).  Every lane executes it; `is` stores.
template <class T, int EPT>
__device__ inline void put_out(const TreeArgs& a, int64_t tok, int64_t at, const float (&y)[EPT], bool is) {
  if (a.o && is) {
    uint8_t* dst = a.o + tok * a.ldo + at * int(sizeof(T));
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < EPT; i += 4) reinterpret_cast<f32x4*>(dst)[i / 4] = f32x4{y[i], y[i + 1], y[i + 2], y[i + 3]};
    } else {
      uint32_t u[EPT / 2];
#pragma unroll
      for (int i = 0; i < EPT / 2; ++i) u[i] = bf16_pair(y[2 * i], y[2 * i + 1]);
      if constexpr (EPT == 8) *reinterpret_cast<u32x4*>(dst) = u32x4{u[0], u[1], u[2], u[3]};
      else *reinterpret_cast<uint2*>(dst) = uint2{u[0], u[1]};
    }
  }
  if constexpr (sizeof(T) == 4) {
    if (a.oq) {
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < EPT; ++i) am = fmaxf(am, fabsf(y[i]));
      am = fmaxf(am, dpp_f<SKG_DPP_QUAD_XOR1>(am));
      am = fmaxf(am, dpp_f<SKG_DPP_QUAD_XOR2>(am));
      if constexpr (EPT == 4) am = fmaxf(am, dpp_f<SKG_DPP_ROW_HALF_MIRROR>(am));
      const float d = q8_1_d(am), id = q8_1_id(d);
      int sum = 0;
      uint32_t word[EPT / 4];
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int q = q8_1_code(y[i], id);
        sum += q;
        word[i / 4] = (i % 4 ? word[i / 4] : 0u) | (uint32_t(q) & 0xFFu) << (8 * (i % 4));
      }
      sum += __builtin_amdgcn_update_dpp(0, sum, SKG_DPP_QUAD_XOR1, 0xF, 0xF, false);
      sum += __builtin_amdgcn_update_dpp(0, sum, SKG_DPP_QUAD_XOR2, 0xF, 0xF, false);
      if constexpr (EPT == 4) sum += __builtin_amdgcn_update_dpp(0, sum, SKG_DPP_ROW_HALF_MIRROR, 0xF, 0xF, false);
      if (is) {
        const int lane = int(at % QK) / EPT;
        uint32_t* dst = reinterpret_cast<uint32_t*>(a.oq) + (tok * a.blocks + at / QK) * 9;
        if (lane == 0) dst[0] = q8_1_d16(d) | (q8_1_s16(d, sum) << 16);
#pragma unroll
        for (int i = 0; i < EPT / 4; ++i) dst[1 + lane * (EPT / 4) + i] = word[i];
      }
    }
  }
}

template <class T, int KIND, int D, int NT, int RT>
__global__ __launch_bounds__(kAttnThreads, (RT * D <= 256 && AttnShape<KIND, D>::kFit >= 1) ? 2 : 1) void tree_attn_kernel(TreeArgs a) {
  using S = AttnShape<KIND, D>;
  constexpr int C = D < 128 ? D : 128;                       // elements joined at a time
  constexpr int EPT = 16 * C / kAttnThreads;                 // of a thread
  constexpr int kRing = kAttnWaves * S::kSlots * S::kSlot, kJoin = kAttnWaves * 16 * (C + 4) * 4;
  // the ring, and after the last step the waves' sums
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing > kJoin ? kRing : kJoin];
  __shared__ float ml[kAttnWaves][RT][16][2];
  // heads fastest, then splits, rows and sequences
  unsigned id = blockIdx.x;
  const int head = int(id % a.cache.heads);
  id /= a.cache.heads;
  const int split = int(id % unsigned(a.splits));
  id /= unsigned(a.splits);
  const int rg = int(id % unsigned(a.row_groups)), seq = int(id / unsigned(a.row_groups));

  const KvSpan sp = span_of(a, seq);
  const int first = rg * 16 * RT, rows = sp.n * a.group;
  if (first >= rows) return;
  const int per = steps_per_split(sp.keys, a.splits);
  const int begin = split * per, steps = sp.keys / kStep + (sp.keys % kStep != 0);
  if (begin >= steps && split > 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int left = (begin + per < steps ? begin + per : steps) - begin - wave;
  const int n = left > 0 ? (left + kAttnWaves - 1) / kAttnWaves : 0;  // this wave's steps

  // pages of the wave's next 32 steps, two tiles each, over its lanes
  const int32_t* table = a.table + int64_t(seq) * a.width;
  auto key_of = [&](int i) SKG_INL { return (begin + wave + i * kAttnWaves) * kStep; };
  auto pages_of = [&](int i0) SKG_INL -> int32_t {
    const int i = i0 + (lane >> 1), key = key_of(i) + 16 * (lane & 1);
    return i < n && key < sp.keys ? table[key >> a.cache.shift] : -1;
  };
  int32_t pages = pages_of(0);
  uint8_t* ring = lds + wave * (S::kSlots * S::kSlot);
  const uint32_t ring_at = lds_addr(ring);
  auto page = [&](int i, int t) SKG_INL { return __builtin_amdgcn_readlane(pages, 2 * (i & 31) + t); };
  auto at_of = [&](int i) SKG_INL { return step_at<KIND, D>(a.cache, head, key_of(i), page(i, 0), page(i, 1)); };

  WaveRows<KIND, D, NT, RT> w;
  load_rows<T, KIND, D, NT, RT>(w, a, sp, head, first);

  auto there_of = [&](int i) SKG_INL -> uint32_t {
    return uint32_t(kv_page_in(a.cache, page(i, 0))) | uint32_t(kv_page_in(a.cache, page(i, 1))) << 1;
  };
  uint32_t there = 0;
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i)
    if (i < n) {
      there |= there_of(i) << (2 * i);
      const StepAt from = at_of(i);
      copy_step<KIND, D, false>(a.cache, from, ring_at + i * S::kSlot);
      copy_step<KIND, D, true>(a.cache, from, ring_at + i * S::kSlot);
    }
  int slot = 0;
  uint32_t flags = there;  // the copied steps' pages in the cache, two bits each, oldest first
  for (int i = 0; i < n; ++i) {
    const int ahead = n - 1 - i < S::kSlots - 1 ? n - 1 - i : S::kSlots - 1;  // later steps on their way
    const bool more = i + S::kSlots < n;
    uint8_t* at = ring + slot * S::kSlot;
    StepRegs<KIND, D> r;
    r.key = key_of(i);
    r.there[0] = flags & 1;
    r.there[1] = flags & 2;
    flags >>= 2;
    float s[RT][8];
    StepAt next;
    wait_ahead<S::kCopies, S::kSlots, true>(ahead, false);
    read_k<KIND, D>(r, at);
    do_scores<KIND, D, NT, RT>(w, r, s);
    if (more) {
      if (((i + S::kSlots) & 31) == 0) pages = pages_of(i + S::kSlots);
      flags |= there_of(i + S::kSlots) << (2 * (S::kSlots - 1));
      wait_lds();
      next = at_of(i + S::kSlots);
      copy_step<KIND, D, false>(a.cache, next, ring_at + slot * S::kSlot);
    }
    wait_ahead<S::kCopies, S::kSlots, false>(ahead, more);
    read_v<KIND, D>(r, at);
    if (r.key + kStep <= sp.ctx && r.there[0] && r.there[1])
      do_values<KIND, D, NT, RT, false>(w, r, s, sp.ctx, sp.keys, at);
    else
      do_values<KIND, D, NT, RT, true>(w, r, s, sp.ctx, sp.keys, at);
    if (more) {
      wait_lds();
      copy_step<KIND, D, true>(a.cache, next, ring_at + slot * S::kSlot);
    }
    slot = slot + 1 == S::kSlots ? 0 : slot + 1;
  }

  // join the waves
  float(*obuf)[16][C + 4] = reinterpret_cast<float(*)[16][C + 4]>(lds);
  const int c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float l = row_sum(w.l[rt]);
    if (g == 0) {
      ml[wave][rt][c][0] = w.M[rt];
      ml[wave][rt][c][1] = l;
    }
  }
  const int jr = threadIdx.x / (C / EPT), je = (threadIdx.x % (C / EPT)) * EPT;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int h = 0; h < D / C; ++h) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = o_element<KIND, D>(g, n, i);
          if (e / C == h) obuf[wave][c][e % C] = w.o[rt][n][i];
        }
      __syncthreads();
      float M = kNoMax, l = 0.f, f[kAttnWaves], y[EPT];
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k) M = fmaxf(M, ml[k][rt][jr][0]);
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k) {
        f[k] = exp2_fast(ml[k][rt][jr][0] - M);
        l = fmaf(f[k], ml[k][rt][jr][1], l);
      }
#pragma unroll
      for (int i = 0; i < EPT; ++i) y[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kAttnWaves; ++k)
#pragma unroll
        for (int i = 0; i < EPT; i += 4) {
          const f32x4 o = *reinterpret_cast<const f32x4*>(&obuf[k][jr][je + i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i + j] = fmaf(f[k], o[j], y[i + j]);
        }
      const int row = first + 16 * rt + jr;
      const bool is = row < rows;
      const int i = is ? row / a.group : 0, hd = head * a.group + (is ? row % a.group : 0);
      const int64_t tok = sp.t0 + i;
      if (a.splits == 1) {
        const float inv = l == 0.f ? 0.f : (KIND == KV_BF16 ? 1.f : kVScale) / l;
#pragma unroll
        for (int j = 0; j < EPT; ++j) y[j] = l == 0.f ? 0.f : y[j] * inv;
        put_out<T, EPT>(a, tok, int64_t(hd) * D + h * C + je, y, is);
      } else if (is) {
        const int64_t at = (tok * a.hq + hd) * a.splits + split;
        float* dst = a.ws + at * D + h * C + je;
#pragma unroll
        for (int j = 0; j < EPT; j += 4) *reinterpret_cast<f32x4*>(dst + j) = f32x4{y[j], y[j + 1], y[j + 2], y[j + 3]};
        if (h == 0 && je == 0) {
          float* m = a.ws + a.T * a.hq * int64_t(a.splits) * D + 2 * at;
          m[0] = M;
          m[1] = l;
        }
      }
    }
}

}  // namespace skg
