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

// Two unsigned bytes in 16-bit halves are fp16 subnormals n 2^-24; one packed
// fma makes them (n - zero) 2^-9, exactly.  mul = 2^15 (2^11 for a high nibble,
// which arrives as 16 n).
__device__ inline uint32_t f16_codes(uint32_t x, float mul, float zero) {
  const f16x2 m = {static_cast<_Float16>(mul), static_cast<_Float16>(mul)};
  const f16x2 z = {static_cast<_Float16>(-zero), static_cast<_Float16>(-zero)};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, x), m, z));
}
__device__ inline uint32_t q8_pair(uint32_t x) { return f16_codes(x, 32768.f, 0.25f); }
__device__ inline uint32_t q4_low(uint32_t x) { return f16_codes(x & 0x000F000Fu, 32768.f, 0.015625f); }
__device__ inline uint32_t q4_high(uint32_t x) { return f16_codes(x & 0x00F000F0u, 2048.f, 0.015625f); }
constexpr float kCodeScale = 512.f;  // 2^9

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
  // columns), V of one key (one column)
  static constexpr int KW = KIND == KV_BF16 ? 4 * NB : KIND == KV_Q8_0 ? 2 * NB : NB;
  static constexpr int VW = KIND == KV_BF16 ? NB : KIND == KV_Q8_0 ? NB / 2 : (NB + 3) / 4;
  static constexpr int SW = KIND == KV_BF16 ? 1 : 2 * NB;  // scales of four keys
};

// What a lane has loaded of a step: lane (c, g) = (lane & 15, lane >> 4).
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

template <int N>
__device__ inline void load_words(const uint8_t* p, uint32_t (&w)[N]) {
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

template <int KIND, int D>
__device__ inline void load_step(StepRegs<KIND, D>& r, const KvView& c, uint32_t head, int key, int32_t p0,
                                 int32_t p1) {
  using S = AttnShape<KIND, D>;
  const uint32_t lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  r.key = key;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int32_t page = t ? p1 : p0;
    r.there[t] = kv_page_in(c, page);
    const uint64_t at = kv_chunk_at(c, r.there[t] ? page : 0, head);
    const uint32_t tok = uint32_t(key + 16 * t) & ((1u << c.shift) - 1);
    const uint8_t* kc = c.k + at + kv_codes_at(KIND, D, tok);
    const uint8_t* vc = c.v + at + kv_codes_at(KIND, D, tok);
    if constexpr (KIND == KV_BF16) {
      // block b's elements 8g .. 8g + 7 are 16 bytes in place
      uint32_t w[4];
#pragma unroll
      for (int b = 0; b < S::NB; ++b) {
        load_words(kc + col * (2 * D) + 64 * b + 16 * g, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.k[t][4 * b + i] = w[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words(vc + (4 * g + i) * (2 * D) + 4 * S::NB * col, r.v[4 * t + i]);
    } else {
      const uint32_t row = kv_row_bytes(KIND, D);
      load_words(kc + col * row + 4 * S::KW * g, r.k[t]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = vc + (4 * g + i) * row + (row / 16) * col;
        if constexpr (KIND == KV_Q4_0 && D == 64)
          r.v[4 * t + i][0] = *reinterpret_cast<const uint16_t*>(p);
        else
          load_words(p, r.v[4 * t + i]);
      }
      const uint32_t s = kv_scales_at(KIND, D, c.shift, tok + 4 * g);
      load_words(c.k + at + s, r.sk[t]);
      load_words(c.v + at + s, r.sv[t]);
    }
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
      a[i] = q8_pair(two_bytes(w, 2 * (b & 1), w, 2 * (b & 1) + 1));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {  // bytes i NB + b and (i + 1) NB + b
      const int y0 = i * NB + b, y1 = (i + 1) * NB + b;
      const uint32_t x = two_bytes(r.k[t][y0 >> 2], y0 & 3, r.k[t][y1 >> 2], y1 & 3);
      a[i] = q4_low(x);
      a[i + 1] = q4_high(x);
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

template <int KIND, int D, int NT, int RT, bool EDGE>
__device__ inline void do_step(WaveRows<KIND, D, NT, RT>& w, StepRegs<KIND, D>& r, int ctx, int keys) {
  using S = AttnShape<KIND, D>;
  constexpr int NB = S::NB;
  const int lane = threadIdx.x & 63, g = lane >> 4;

  // scores of the row with the lane's eight keys
  float s[RT][8];
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
        f32x4 x = KIND == KV_BF16 ? acc[rt] : f32x4{0.f, 0.f, 0.f, 0.f};
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
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < S::SW; ++i) {
          const uint32_t h = max(r.sv[t][i] & 0x7FFFu, (r.sv[t][i] >> 16) & 0x7FFFu);
          big = max(big, h);
        }
    }
    const float top = h2f(big);
    if (__ballot(!(top <= pow2(w.be)))) {
      // the next power of two and two bits of room; at most 2^18 (fp16's largest)
      float t = row_max(top);
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
      // a value that no row sees may be anything: zero; one that some rows see
      // may be infinite or NaN, which must not reach the others through 0 * v
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
        // row by row, with the values that the row does not see at zero
        for (int row = 0; row < 16; ++row) {
          for (int rt = 0; rt < RT; ++rt) {
            uint32_t pt[4][NT];
            uint32_t vis = 0;
#pragma unroll
            for (int k = 0; k < RT; ++k)
              if (k == rt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) split_pair<false, NT>(s[k][2 * i], s[k][2 * i + 1], pt[i]);
                vis = __shfl(seen[k], (lane & 48) | row, 64);
              }
            StepRegs<KIND, D> z = r;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int j = 0; j < S::VW; ++j) z.v[i][j] = ((vis >> i) & 1) ? r.v[i][j] : 0;
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              const u32x4 a = v_operand<KIND, D>(z, n);
              f32x4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int i = NT - 1; i >= 0; --i) x = mfma<false>(a, u32x4{pt[0][i], pt[1][i], pt[2][i], pt[3][i]}, x);
#pragma unroll
              for (int k = 0; k < RT; ++k)
                if (k == rt && (lane & 15) == row) w.o[k][n] += x;
            }
          }
        }
        return;
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
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t sw = r.sv[i >> 2][((i & 3) * NB + b) >> 1];
          y[i] = __builtin_fmaf((b & 1) ? f16_hi(sw) : f16_lo(sw), s[rt][i], 0.f);
          if constexpr (EDGE) y[i] = ((seen[rt] >> i) & 1) ? y[i] : 0.f;  // an unseen key's scale may be NaN
        }
        uint32_t pt[4][NT];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_pair<true, NT>(y[2 * i], y[2 * i + 1], pt[i]);
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
      w.rs[rt] *= kCodeScale * __builtin_bit_cast(float, uint32_t(127 - 14 + (e - 126)) << 23);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // q4_0's operand order: 0 2 1 3 4 6 5 7
        const int i0 = KIND == KV_Q4_0 ? 4 * (j >> 1) + (j & 1) : 2 * j, i1 = KIND == KV_Q4_0 ? i0 + 2 : 2 * j + 1;
        uint32_t t[NT];
        split_pair<F16, NT>(x[b][i0] * to, x[b][i1] * to, t);
#pragma unroll
        for (int k = 0; k < NT; ++k) w.q[rt][b][k][j] = t[k];
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
__global__ __launch_bounds__(kAttnThreads, (RT == 1 && D <= 128) ? 2 : 1) void tree_attn_kernel(TreeArgs a) {
  constexpr int C = D < 128 ? D : 128;                       // elements joined at a time
  constexpr int EPT = 16 * C / kAttnThreads;                 // of a thread
  __shared__ __attribute__((aligned(16))) float obuf[kAttnWaves][16][C + 4];
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
  const int begin = split * per, steps = (sp.keys + kStep - 1) / kStep;
  if (a.splits > 1 && begin >= steps && split > 0) return;
  const int end = begin + per < steps ? begin + per : steps;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  WaveRows<KIND, D, NT, RT> w;
  load_rows<T, KIND, D, NT, RT>(w, a, sp, head, first);

  const int32_t* table = a.table + int64_t(seq) * a.width;
  auto page = [&](int step, int t) SKG_INL -> int32_t {
    const int key = step * kStep + 16 * t;
    return step < end && key < sp.keys ? __builtin_amdgcn_readfirstlane(table[key >> a.cache.shift]) : -1;
  };
  for (int step = begin + wave; step < end; step += kAttnWaves) {
    StepRegs<KIND, D> r;
    load_step<KIND, D>(r, a.cache, head, step * kStep, page(step, 0), page(step, 1));
    if (step * kStep + kStep <= sp.ctx && r.there[0] && r.there[1])
      do_step<KIND, D, NT, RT, false>(w, r, sp.ctx, sp.keys);
    else
      do_step<KIND, D, NT, RT, true>(w, r, sp.ctx, sp.keys);
  }

  // join the waves
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
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
        const float inv = l == 0.f ? 0.f : (KIND == KV_BF16 ? 1.f : kCodeScale) / l;
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
