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

#include <type_traits>

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
  const int32_t* cu;  // or null: per_seq tokens each
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
  // set by the launch
  int64_t blocks;    // Q8_1 blocks of a token's row
  int per_seq;       // T / n_seqs
  int want;          // splits to make of all sequences' keys together; 0: each sequence is one
  int cost_shift;    // unit of a sequence's cost (2^cost_shift steps), so that the sum fits 31 bits
  int row_groups;    // workgroups along a sequence's rows
  int tile;          // rows of a workgroup
  float* sums;       // partial results: [split][row group][head][tile][D]
  float* ml;         // their M and l: [split][row group][head][tile][2]
};

constexpr int kMaxSplitSeqs = 256;  // sequences that a launch may split

__device__ inline KvSpan span_of(const TreeArgs& a, int b) {
  const int32_t t0 = a.cu ? a.cu[b] : b * a.per_seq, t1 = a.cu ? a.cu[b + 1] : (b + 1) * a.per_seq;
  return kv_span(a.ctx[b], t0, t1, a.T, a.max_draft, a.max_kv);
}

// Sum over the lanes up to each (within 16 lanes, then over the rows of 16).
__device__ inline int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 to rows 1 and 3
  return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 to rows 2 and 3
}
__device__ inline int lane_of(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Splits are of equal cost over all sequences: per = the cost of all of them
// over the splits that are wanted, so a long sequence gets many and a short one
// gets one, and a workgroup finds its own from the lengths, one lane a sequence.
// A step costs 1; where eight waves share its rows (WEIGH) 5 if more than half
// of them are there and else 3 (trees of 61, 61, 6 and 23 drafted tokens over
// bf16, steps of 1.34 and 0.8 us: 47.9 us without that, 41.5 with it; six of up
// to 30 of float32 rows over q8_0 48.3 and 42.2).
struct Splits {  // of 64 sequences, one a lane
  KvSpan sp;
  int n, incl;  // splits of the sequence; of it and all before it
};
__device__ __forceinline__ Splits lane_span(const TreeArgs& a, int b) {
  Splits s{KvSpan{0, 0, 0, 0}, 0, 0};
  if (b < a.n_seqs) s.sp = span_of(a, b);
  return s;
}
constexpr int kDear = kMaxWeight, kCheap = 3;
__device__ inline bool dear(const TreeArgs& a, const KvSpan& sp) { return 2 * sp.n * a.group > a.tile; }
template <bool WEIGH>
__device__ inline int cost_of(const TreeArgs& a, const KvSpan& sp) {
  return sp.n == 0 ? 0 : kv_cost(kv_steps(sp.keys), !WEIGH ? 1 : dear(a, sp) ? kDear : kCheap, a.cost_shift);
}
// Cost of a split.
template <bool WEIGH>
__device__ __forceinline__ int split_cost(const TreeArgs& a, const Splits& first) {
  int total = cost_of<WEIGH>(a, first.sp);
  if (a.n_seqs > 1) {
#pragma unroll 1
    for (int b = 64; b < a.n_seqs; b += 64) total += cost_of<WEIGH>(a, lane_span(a, b + (threadIdx.x & 63)).sp);
    total = lane_of(wave_scan(total), 63);
  }
  total = __builtin_amdgcn_readfirstlane(total);
  return total / a.want + (total % a.want != 0);
}
// Steps of a split of a sequence.
template <bool WEIGH>
__device__ __forceinline__ int split_steps(const TreeArgs& a, const KvSpan& sp, int cost) {
  return !WEIGH          ? kv_split_steps(cost, 1, a.cost_shift)
         : dear(a, sp) ? kv_split_steps(cost, kDear, a.cost_shift)
                       : kv_split_steps(cost, kCheap, a.cost_shift);
}
template <bool WEIGH>
__device__ __forceinline__ void count_splits(const TreeArgs& a, Splits& s, int cost, int before) {
  s.n = s.sp.n == 0 ? 0 : kv_splits(kv_steps(s.sp.keys), split_steps<WEIGH>(a, s.sp, cost));
  const int incl = a.n_seqs > 1 ? wave_scan(s.n) : s.n;
  s.incl = before + incl;
}

// What a workgroup does: steps [begin, end) of a sequence, one of `splits`, of
// which the first is split `base` of all.
struct Unit {
  KvSpan sp;
  int seq, begin, end, splits, base;
};
// Split u of all (by_seq: the splits of sequence u); false if there is none.
template <bool WEIGH>
__device__ __forceinline__ bool find_unit(const TreeArgs& a, int u, Unit& w, bool by_seq = false) {
  if (a.want == 0) {
    w.seq = u;
    w.sp = span_of(a, u);
    w.begin = 0;
    w.end = kv_steps(w.sp.keys);
    w.splits = 1;
    w.base = 0;
    return true;
  }
  const int lane = threadIdx.x & 63;
  Splits s = lane_span(a, lane);
  const int cost = split_cost<WEIGH>(a, s);
  int before = 0;  // splits of the sequences of earlier rounds
#pragma unroll 1
  for (int b0 = 0; b0 < a.n_seqs; b0 += 64) {
    if (b0) s = lane_span(a, b0 + lane);
    count_splits<WEIGH>(a, s, cost, before);
    const uint64_t hit = __ballot(by_seq ? b0 + lane == u : s.incl > u && s.n > 0);
    if (hit) {
      const int b = __builtin_ctzll(hit);
      w.seq = b0 + b;
      w.splits = lane_of(s.n, b);
      w.base = lane_of(s.incl, b) - w.splits;
      w.sp = KvSpan{lane_of(s.sp.t0, b), lane_of(s.sp.ctx, b), lane_of(s.sp.n, b), lane_of(s.sp.keys, b)};
      const int per = split_steps<WEIGH>(a, w.sp, cost);
      w.begin = (u - w.base) * per;
      const int all = kv_steps(w.sp.keys);
      w.end = w.begin + per < all ? w.begin + per : all;
      return true;
    }
    before = lane_of(s.incl, 63);
  }
  return false;
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
    asm("" : "+v"(t[0]));  // read back from the pair, not computed once more
    const f16x2 h = __builtin_bit_cast(f16x2, t[0]);
    const _Float16 l0 = static_cast<_Float16>(__builtin_fmaf(p0, float(s0), -float(h.x)));
    const _Float16 l1 = static_cast<_Float16>(__builtin_fmaf(p1, float(s1), -float(h.y)));
    t[1] = __builtin_bit_cast(uint32_t, f16x2{l0, l1});
  }
}

// Codes as fp16.  Two unsigned bytes in 16-bit halves are the fp16 subnormals
// n 2^-24, which the matrix instructions take as they are: K's operand is that,
// and the zero of the codes is taken off by the product's initial value, -zero
// 2^-24 sum q of the block, which is constant for a row.  The instructions
// line a subnormal's products up as if its highest bit were set, so its leading
// zeros are lost to the sum: q4_0's nibbles are both taken as 16 n (the low one
// as n had left scores of 2^-18 instead of 2^-22).  For V the same would leave differences of long sums, so
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
constexpr float kKScale8 = 16777216.f, kKScale4 = 1048576.f;  // 2^24, 2^20
constexpr uint32_t kZero = 0x80808080u;  // two -128 2^-24

// Byte y0 of w0 and byte y1 of w1, each in a 16-bit half.
__device__ inline uint32_t two_bytes(uint32_t w0, int y0, uint32_t w1, int y1) {
  return __builtin_amdgcn_perm(w1, w0, 0x0C000C00u | uint32_t((4 + y1) << 16) | uint32_t(y0));
}

// NT terms of q and p; RT tiles of 16 rows a wave; W waves, which share the keys
// of a split between them (each its own steps) or, with ROWS, the rows (all the
// same steps, from one ring).
template <int KIND, int D, int NT, int RT, int W, bool ROWS>
struct AttnShape {
  static constexpr bool kF16 = KIND != KV_BF16;
  static constexpr int NB = D / 32;
  // 32-bit words of a lane: K of one 16-key tile (four of the sixteen pair
  // columns), V of one key (one column), scales of four keys
  static constexpr int KW = KIND == KV_BF16 ? 4 * NB : KIND == KV_Q8_0 ? 2 * NB : NB;
  static constexpr int VW = KIND == KV_BF16 ? NB : KIND == KV_Q8_0 ? NB / 2 : (NB + 3) / 4;
  static constexpr int SW = 2 * NB;

  // q: in registers, or in LDS where all waves have the same rows and their
  // sums leave no room
  static constexpr bool kQLds = !ROWS && (RT > 1 || D > 128);
  static constexpr int kQBytes = kQLds ? RT * NB * NT * 1024 : 0;
  // K's codes as subnormals, which need the row's zeros in registers; with
  // several tiles the conversion serves all of them
  static constexpr bool kSubnormal = kF16 && !kQLds && RT == 1;

  // An LDS slot for a step of 32 keys: K codes, V codes [2][16][row], then the
  // scales of K and V, [32][NB] fp16, each in whole 256 bytes.
  static constexpr int kRow = int(kv_row_bytes(KIND, D));
  static constexpr int kRC = kRow / 16;  // 16-byte units of a row
  static constexpr int kTile = 16 * kRow;
  static constexpr int kScales = !kF16 ? 0 : NB <= 4 ? 256 : 512;
  static constexpr int kSlot = 4 * kTile + 2 * kScales;
  static constexpr int kKOff = 0, kVOff = 2 * kTile, kSkOff = 4 * kTile, kSvOff = kSkOff + kScales;
  // Workgroups of a CU: two of four waves, where they fit its 160 KB and 256
  // registers a lane.  (A spilled register costs far more than its traffic
  // here: waiting for its reload waits for every copy on its way.)
  static constexpr int kRings = ROWS ? 1 : W;
  static constexpr int kPerCu = W == 4 && kRings * kSlot + kQBytes <= 80 * 1024 && D <= 128 && !(RT == 2 && kF16) ? 2 : 1;
  static constexpr int kFit = (160 / kPerCu * 1024 - kQBytes - (kQLds ? 256 : 0)) / (kRings * kSlot);
  static constexpr int kSlots = kFit < 1 ? 1 : kFit > 4 ? 4 : kFit;
  // transfers of a wave: of K (or V) of a step, or of its part of both
  static constexpr int kCopies = kRow / 32 + kScales / 256;
  static constexpr int kPart = (2 * kRow / 32 + W - 1) / W + kScales / 256;
  static_assert(ROWS ? kPart * kSlots <= 63 && kSlots >= 2 : 2 * kCopies * kSlots <= 63, "vmcnt");

  // LDS: the ring and q; after the last step the waves' sums, M and l
  static constexpr int C = D < 128 ? D : 128;  // elements joined at a time
  static constexpr int kRing = kRings * kSlots * kSlot;
  static constexpr int kJoin = W * 16 * (C + 4) * 4;
  static constexpr int kMl = ROWS ? 0 : W * RT * 16 * 2 * 4;
  static constexpr int kLds = kRing + kQBytes > kJoin + kMl ? kRing + kQBytes : kJoin + kMl;
  static_assert(kLds <= 160 * 1024, "LDS");
};

// LDS position of a tile's 16-byte unit j of row c: the units of eight and of
// sixteen consecutive rows at one j lie on different banks.
template <int RC>
__device__ inline int k_swizzle(int c) {
  return RC >= 16 ? c : RC == 8 ? (c & 7) ^ (c >> 3) : RC == 4 ? ((c >> 1) & 3) ^ (c >> 3) : 0;
}
// LDS row of V's key c (and back): the rows 4g + i of the four g differ modulo 4.
__device__ inline int v_row(int c) { return c ^ (c >> 2); }
// Offset in a tile of the 16-byte unit that a transfer puts at unit u of row c:
// for K, and V in bf16, swizzled units; for V's codes permuted rows.
template <class S, bool V>
__device__ inline uint32_t tile_unit(int c, int u) {
  if (V && S::kF16) return v_row(c) * S::kRow + 16 * u;
  return c * S::kRow + 16 * (u ^ k_swizzle<S::kRC>(c));
}

// Transfers as dma16_sv: 4 bytes a lane, and 16 with the streaming hint.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ inline void dma4(const void* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(__builtin_amdgcn_readfirstlane(dst)),
               "v"(src)
               : "memory", "m0");
}
__device__ inline void dma16_sv_stream(const void* base, uint32_t off, uint32_t dst) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint64_t sb = uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(b)))) |
                      (uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(b >> 32)))) << 32);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(__builtin_amdgcn_readfirstlane(dst)),
               "v"(off), "s"(sb)
               : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N>
__device__ inline void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Waits for a step while `ahead` later ones are on their way: C copies for each
// of K and V.
template <int C, int SLOTS>
__device__ inline void wait_ahead(int ahead) {
  if (ahead == SLOTS - 1) {
    wait_copies<2 * C * (SLOTS - 1)>();
  } else if constexpr (SLOTS > 1) {
    wait_ahead<C, SLOTS - 1>(ahead);
  }
}
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A page outside the cache is replaced by page 0 (every key of it is masked).
__device__ inline uint64_t pick(bool first, uint64_t a, uint64_t b) { return first ? a : b; }
struct StepAt {
  uint64_t codes[2], scales[2];  // offsets of the tiles in the buffers of K and V
};
// The same for 32 steps at once, two lanes a step (its tiles).
struct StepsAt {
  uint64_t codes, scales;  // of the lane's tile
  uint64_t there;          // bit: whether the lane's tile is in the cache
};
// page: the lane's; key: its tile's first key.
template <int KIND, int D>
__device__ inline StepsAt steps_at(const KvView& c, uint32_t head, int key, int32_t page) {
  StepsAt s;
  const bool in = kv_page_in(c, page);
  s.there = __ballot(in);
  const uint64_t chunk = kv_chunk_at(c, in ? page : 0, head);
  const uint32_t tok = uint32_t(key) & ((1u << c.shift) - 1);
  s.codes = chunk + kv_codes_at(KIND, D, tok);
  s.scales = chunk + kv_scales_at(KIND, D, c.shift, tok);
  return s;
}
__device__ inline uint64_t lane64_of(uint64_t v, int lane) {
  return uint64_t(uint32_t(lane_of(int(v), lane))) | uint64_t(uint32_t(lane_of(int(v >> 32), lane))) << 32;
}
// Step i's, i counted from a multiple of 32.
template <bool SCALES>
__device__ inline StepAt step_at(const StepsAt& s, int i) {
  StepAt r{};
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    r.codes[t] = lane64_of(s.codes, 2 * (i & 31) + t);
    if constexpr (SCALES) r.scales[t] = lane64_of(s.scales, 2 * (i & 31) + t);
  }
  return r;
}
__device__ inline uint32_t there_of(const StepsAt& s, int i) { return uint32_t(s.there >> (2 * (i & 31))) & 3u; }

// Copies K (V = false) or V of the step's two 16-key tiles and their scales
// into the slot at LDS address dst.
template <class S, int KIND, int D, bool V>
__device__ inline void copy_step(const KvView& c, const StepAt& from, uint32_t dst) {
  const int lane = threadIdx.x & 63;
  const uint8_t* buf = V ? c.v : c.k;
  const uint32_t codes = dst + (V ? S::kVOff : S::kKOff);
  if constexpr (S::kRow >= 64) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < S::kRow / 64; ++j) {
        const int row = j * (64 / S::kRC) + lane / S::kRC, unit = lane % S::kRC;
        const uint32_t off = tile_unit<S, V>(row, unit);
        dma16_sv_stream(buf + from.codes[t], off, codes + t * S::kTile + 1024 * j);
      }
  } else {  // both tiles in one transfer
    static_assert(S::kRow >= 64 || S::kRow == 32, "row");
    const int row = (lane & 31) / 2, unit = lane & 1;
    const uint8_t* src = buf + pick(lane < 32, from.codes[0], from.codes[1]);
    dma16_stream(src + (V ? v_row(row) : row) * S::kRow + 16 * unit, codes);
  }
  if constexpr (S::kF16) {
    // 16 NB words over both tiles (NB = 2: the upper lanes repeat the lower)
#pragma unroll
    for (int j = 0; j < S::kScales / 256; ++j) {
      const int w = (64 * j + lane) % (16 * S::NB), t = w / (8 * S::NB);
      dma4(buf + pick(t != 0, from.scales[1], from.scales[0]) + 4 * (w - t * 8 * S::NB), dst + (V ? S::kSvOff : S::kSkOff) + 256 * j);
    }
  }
}

// One wave's part of a step's copies, every wave as many: W shares of the 1 KB
// transfers of K and V (where there are fewer, some are made twice), and the
// scales of K by even and of V by odd waves.
template <class S, int KIND, int D, int W>
__device__ inline void copy_part(const KvView& c, const StepAt& from, uint32_t dst, int wave) {
  const int lane = threadIdx.x & 63;
  constexpr int kAll = 2 * S::kRow / 32, kEach = (kAll + W - 1) / W;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int x = (wave * kEach + j) % kAll;  // [V][transfer]
    const bool v = x >= kAll / 2;
    const uint8_t* buf = v ? c.v : c.k;
    if constexpr (S::kRow >= 64) {
      const int y = v ? x - kAll / 2 : x, t = y / (S::kRow / 64), i = y % (S::kRow / 64);
      const int row = i * (64 / S::kRC) + lane / S::kRC, unit = lane % S::kRC;
      const uint32_t off = v ? tile_unit<S, true>(row, unit) : tile_unit<S, false>(row, unit);
      dma16_sv(buf + (t ? from.codes[1] : from.codes[0]), off, dst + (v ? S::kVOff : S::kKOff) + t * S::kTile + 1024 * i);
    } else {
      const int row = (lane & 31) / 2, unit = lane & 1;
      const uint8_t* src = buf + pick(lane < 32, from.codes[0], from.codes[1]);
      dma16(src + (v ? v_row(row) : row) * S::kRow + 16 * unit, dst + (v ? S::kVOff : S::kKOff));
    }
  }
  if constexpr (S::kF16) {
    const bool v = wave & 1;
    const uint8_t* buf = v ? c.v : c.k;
#pragma unroll
    for (int j = 0; j < S::kScales / 256; ++j) {
      const int w = (64 * j + lane) % (16 * S::NB), t = w / (8 * S::NB);
      dma4(buf + pick(t != 0, from.scales[1], from.scales[0]) + 4 * (w - t * 8 * S::NB), dst + (v ? S::kSvOff : S::kSkOff) + 256 * j);
    }
  }
}
// Waits until at most `steps` steps' parts of C copies are on their way.
template <int C, int MOST>
__device__ inline void wait_parts(int steps) {
  if (steps >= MOST) wait_copies<C * MOST>();
  else if constexpr (MOST > 0) wait_parts<C, MOST - 1>(steps);
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
template <class S>
struct StepRegs {
  uint32_t k[2][S::KW];   // key c of each tile, its elements 8g .. 8g + 7 of every block
  // codes: keys 4g + i (tile 0), 4g + i - 4 (tile 1), column c; bf16: words
  // 4n .. 4n + 3 are element 16n + c of those keys in pairs
  uint32_t v[8][S::VW];
  uint32_t sk[2][S::SW];  // scales of keys 4g .. 4g + 3 of each tile
  uint32_t sv[2][S::SW];
  uint32_t all[2];        // the step's scales of V, spread over the lanes
  int key;                // first key
  bool there[2];          // whether a tile's page is in the cache
};

template <class S, int KIND>
__device__ inline void read_k(StepRegs<S>& r, const uint8_t* slot) {
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
// Word w of StepRegs::v.
template <class S>
__device__ inline uint32_t& v_word(StepRegs<S>& r, int w) { return r.v[w / S::VW][w % S::VW]; }

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <class S, int KIND>
__device__ inline void read_v(StepRegs<S>& r, const uint8_t* slot) {
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  if constexpr (KIND == KV_BF16) {
    // Transposing reads: the 16 lanes of g give the addresses of four elements
    // of keys 4g .. 4g + 3 each, and get one element of all four.
    const int row = 4 * g + (c >> 2);
    const uint32_t at = lds_addr(slot) + S::kVOff + row * S::kRow + 8 * (c & 1);
    const int z = k_swizzle<S::kRC>(row) ^ ((c >> 1) & 1);
#pragma unroll
    for (int n = 0; n < 2 * S::NB; ++n)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t from = at + 16 * ((2 * n) ^ z) + t * S::kTile;
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)from);
        const uint2 y = __builtin_bit_cast(uint2, x);
        v_word(r, 4 * n + 2 * t) = y.x;
        v_word(r, 4 * n + 2 * t + 1) = y.y;
      }
    return;
  }
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
#pragma unroll
  for (int j = 0; j < S::kScales / 256; ++j) r.all[j] = reinterpret_cast<const uint32_t*>(slot + S::kSvOff)[64 * j + lane];
}

// K operand of block b of tile t: elements 8g .. 8g + 7 of the block (for q4_0
// in the order 0 2 1 3 4 6 5 7, which convert_rows gives q too).
template <class S, int KIND, int NB>
__device__ inline u32x4 k_operand(const StepRegs<S>& r, int t, int b) {
  u32x4 a;
  if constexpr (KIND == KV_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = r.k[t][4 * b + i];
  } else if constexpr (KIND == KV_Q8_0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = r.k[t][i * (NB / 2) + (b >> 1)];
      const uint32_t x = two_bytes(w, 2 * (b & 1), w, 2 * (b & 1) + 1);
      a[i] = S::kSubnormal ? x : q8_pair(x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {  // bytes i NB + b and (i + 1) NB + b
      const int y0 = i * NB + b, y1 = (i + 1) * NB + b;
      const uint32_t x = two_bytes(r.k[t][y0 >> 2], y0 & 3, r.k[t][y1 >> 2], y1 & 3);
      a[i] = S::kSubnormal ? (x << 4) & 0x00F000F0u : q4_low(x);
      a[i + 1] = S::kSubnormal ? x & 0x00F000F0u : q4_high(x);
    }
  }
  return a;
}

// V operand: an element of the lane's eight keys.  Quantised: n = 2 b + e of
// column c; bf16: element 16 n + c.
template <class S, int KIND>
__device__ inline u32x4 v_operand(StepRegs<S>& r, int n) {
  u32x4 a;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (KIND == KV_BF16) {
      a[i] = v_word(r, 4 * n + i);
    } else if constexpr (KIND == KV_Q8_0) {
      a[i] = q8_pair(two_bytes(r.v[2 * i][n >> 2], n & 3, r.v[2 * i + 1][n >> 2], n & 3));
    } else {
      const uint32_t x = two_bytes(r.v[2 * i][n >> 3], (n >> 1) & 3, r.v[2 * i + 1][n >> 3], (n >> 1) & 3);
      a[i] = (n & 1) ? q4_high(x) : q4_low(x);
    }
  }
  return a;
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
template <class S, int D, int NT, int RT>
struct WaveRows {
  uint32_t q[S::kQLds ? 1 : RT][D / 32][NT][4];
  f32x4 zero[S::kSubnormal ? D / 32 : 1];  // of the codes, times the row's q
  const uint8_t* q_lds;                    // [RT][NB][NT] operands of 64 lanes, 16 bytes each
  f32x4 o[RT][D / 16];
  float rs[RT];  // scores are acc * rs, rs >= 0
  float M[RT], l[RT];
  int be;        // quantised: M's sigma allows for scales up to 2^be
  uint64_t mask[RT];
};

template <class W, int D>
__device__ inline void raise(W& w, int rt, float m) {
  const float f = exp2_fast(w.M[rt] - m);
  w.M[rt] = m;
  w.l[rt] *= f;
#pragma unroll
  for (int n = 0; n < D / 16; ++n) w.o[rt][n] *= f;
}

// Products of the row's q with the lane's eight keys, scaled by the keys' scales.
template <class S, int KIND, int D, int NT, int RT>
__device__ inline void do_scores(WaveRows<S, D, NT, RT>& w, StepRegs<S>& r, float (&s)[RT][8]) {
  constexpr int NB = S::NB;
  f32x4 acc[2][RT];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[t][rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    u32x4 a[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) a[t] = k_operand<S, KIND, NB>(r, t, b);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      u32x4 q[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if constexpr (S::kQLds)
          q[i] = *reinterpret_cast<const u32x4*>(w.q_lds + ((rt * NB + b) * NT + i) * 1024);
        else
          q[i] = u32x4{w.q[rt][b][i][0], w.q[rt][b][i][1], w.q[rt][b][i][2], w.q[rt][b][i][3]};
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (!S::kF16) x = acc[t][rt];
        else if constexpr (S::kSubnormal) x = w.zero[b];
#pragma unroll
        for (int i = NT - 1; i >= 0; --i) x = mfma<S::kF16>(a[t], q[i], x);
        if constexpr (!S::kF16) {
          acc[t][rt] = x;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // scale of key 4g + i, block b
            const uint32_t sw = r.sk[t][(i * NB + b) >> 1];
            acc[t][rt][i] = __builtin_fmaf((b & 1) ? f16_hi(sw) : f16_lo(sw), x[i], acc[t][rt][i]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[rt][i] = acc[i >> 2][rt][i & 3];
}

// The softmax's step and the sums with V.  EDGE: keys that are not there, or
// that not every row sees.
template <class S, int KIND, int D, int NT, int RT, bool EDGE>
__device__ inline void do_values(WaveRows<S, D, NT, RT>& w, StepRegs<S>& r, float (&s)[RT][8], int ctx, int keys) {
  constexpr int NB = S::NB;
  const int lane = threadIdx.x & 63, g = lane >> 4;
  uint32_t seen[RT];  // bit i: whether the row sees the lane's key i
  if constexpr (EDGE) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      seen[rt] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = r.key + 16 * (i >> 2) + 4 * g + (i & 3), j = key - ctx;
        const bool in = r.there[i >> 2] && key < keys && (j < 0 || ((w.mask[rt] >> (j & 63)) & 1));
        seen[rt] |= uint32_t(in) << i;
      }
    }
  }

  // the largest scale of a value that is seen against M's sigma
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
#pragma unroll
      for (int j = 0; j < S::kScales / 256; ++j) {
        const uint32_t x = r.all[j] & 0x7FFF7FFFu;
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
      for (int rt = 0; rt < RT; ++rt) raise<WaveRows<S, D, NT, RT>, D>(w, rt, w.M[rt] + up);
    }
  }
  // sigma = 15 - kLazy - be: M = m - sigma, p <= 2^kLazy 2^sigma
  float room = float(kLazy);
  if constexpr (S::kF16) room = float(15 - w.be);
  bool over = false;
  float mx[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (EDGE) m = ((seen[rt] >> i) & 1) ? fmaxf(m, s[rt][i]) : m;
      else m = i ? fmaxf(m, s[rt][i]) : s[rt][i];
    }
    mx[rt] = EDGE && !seen[rt] ? -INFINITY : m * w.rs[rt];
    over |= mx[rt] > w.M[rt] + room;
  }
  if (__ballot(over)) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float m = row_max(mx[rt]) - (room - float(kLazy));
      raise<WaveRows<S, D, NT, RT>, D>(w, rt, fmaxf(m, w.M[rt]));
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = exp2_fast(__builtin_fmaf(s[rt][i], w.rs[rt], -w.M[rt]));
      s[rt][i] = EDGE && !((seen[rt] >> i) & 1) ? 0.f : p;
      w.l[rt] += s[rt][i];
    }

  if constexpr (KIND == KV_BF16) {
    if constexpr (EDGE) {
      // a value that is not there may be anything: zero; one that some rows
      // see may be infinite or NaN, which must not reach the others as 0 * v
      uint32_t bad = 0, in[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = r.key + 16 * (i >> 1) + 4 * g + 2 * (i & 1);
        in[i] = !r.there[i >> 1] || key >= keys ? 0u : key + 1 < keys ? ~0u : 0xFFFFu;
      }
#pragma unroll
      for (int j = 0; j < D / 4; ++j) {
        const uint32_t x = v_word(r, j) & in[j & 3];
        v_word(r, j) = x;
        bad |= uint32_t((x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u);
      }
      if (__ballot(bad != 0)) {
        // The sums take zeros in their place; where a row sees one, which the
        // product of "is not finite" and "is seen" counts, its sum becomes NaN.
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          const u32x4 x = v_operand<S, KIND>(r, n);
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
        for (int j = 0; j < D / 4; ++j) {
          const uint32_t x = v_word(r, j);
          v_word(r, j) = ((x & 0x7F80u) == 0x7F80u ? 0u : x & 0xFFFFu) | ((x & 0x7F800000u) == 0x7F800000u ? 0u : x & 0xFFFF0000u);
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
      const u32x4 a = v_operand<S, KIND>(r, n);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = NT - 1; i >= 0; --i)
          w.o[rt][n] = mfma<false>(a, u32x4{pt[rt][0][i], pt[rt][1][i], pt[rt][2][i], pt[rt][3][i]}, w.o[rt][n]);
    }
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const u32x4 a0 = v_operand<S, KIND>(r, 2 * b), a1 = v_operand<S, KIND>(r, 2 * b + 1);
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

// Row `row` of a sequence: its token (from the first) and its query head.
__device__ inline void row_of(const TreeArgs& a, int row, bool is, int& i, int& h) {
  i = is ? int(unsigned(row) / unsigned(a.group)) : 0;
  h = is ? row - i * a.group : 0;
}

// The raw q of row tile `first` .. + 15: lane (c, g) takes elements 8g .. 8g + 7
// of every block of row c (zeros past the sequence's rows).
template <class T, int D>
struct RawRows {
  u32x4 x[D / 32][8 / Elem<T>::kVec];
};
template <class T, int D>
__device__ inline void fetch_rows(RawRows<T, D>& r, const TreeArgs& a, const KvSpan& sp, int head, int first) {
  const int lane = threadIdx.x & 63, row = first + (lane & 15), g = lane >> 4;
  const bool is = row < sp.n * a.group;
  int i, h;
  row_of(a, row, is, i, h);
  const uint8_t* src = a.q + int64_t(sp.t0 + i) * a.ldq + (int64_t(head * a.group + h) * D + 8 * g) * int(sizeof(T));
#pragma unroll
  for (int b = 0; b < D / 32; ++b)
#pragma unroll
    for (int u = 0; u < 8 / Elem<T>::kVec; ++u) {
      r.x[b][u] = u32x4{0, 0, 0, 0};
      if (is) r.x[b][u] = *reinterpret_cast<const u32x4*>(src + (32 * b + u * Elem<T>::kVec) * int(sizeof(T)));
    }
}

// Operand terms of a tile's rows, scaled by a power of two into fp16's range;
// put(b, k, words) stores them.  Returns the scores' factor (>= 0: a negative
// scale turns q).
template <class T, class S, int KIND, int D, int NT, class Put>
__device__ inline float convert_rows(const RawRows<T, D>& raw, float scale, Put&& put) {
  constexpr int NB = D / 32, V = Elem<T>::kVec;
  float x[NB][8];
  float amax = 0.f;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int u = 0; u < 8 / V; ++u) {
      float y[V];
      Elem<T>::unpack(raw.x[b][u], y);
#pragma unroll
      for (int j = 0; j < V; ++j) x[b][u * V + j] = y[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[b][j]));
  }
  float to = scale < 0.f ? -1.f : 1.f;
  float rs = fabsf(scale) * 1.44269504f;
  if constexpr (S::kF16) {
    amax = row_max(amax);
    int e = int((__builtin_bit_cast(uint32_t, amax) >> 23) & 255);  // |q| < 2^(e - 126)
    e = e < 40 ? 40 : (e > 220 ? 220 : e);
    to *= pow2(14 - (e - 126));
    rs *= (!S::kSubnormal ? kVScale : KIND == KV_Q8_0 ? kKScale8 : kKScale4) * pow2(e - 126 - 14);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    uint32_t w[NT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // q4_0's operand order: 0 2 1 3 4 6 5 7
      const int i0 = KIND == KV_Q4_0 ? 4 * (j >> 1) + (j & 1) : 2 * j, i1 = KIND == KV_Q4_0 ? i0 + 2 : 2 * j + 1;
      uint32_t t[NT];
      split_pair<S::kF16, NT>(x[b][i0] * to, x[b][i1] * to, t);
#pragma unroll
      for (int k = 0; k < NT; ++k) w[k][j] = t[k];
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) put(b, k, w[k]);
  }
  return rs;
}

// Sixteen lanes hold a row's elements in the joins: lane t of them has 32 k + 2 t
// and the next of each 32-element block k, so that every store of theirs is
// contiguous and a Q8_1 block lies in one 16-lane row.
//
// The blocks from element `at` of a token's row, in float32, bf16 or as Q8_1.
// Every lane executes it; `is` stores.
template <class T, int BLOCKS>
__device__ inline void put_out(const TreeArgs& a, int64_t tok, int64_t at, const float (&y)[2 * BLOCKS], bool is) {
  const int t = threadIdx.x & 15;
  if (a.o && is) {
    uint8_t* dst = a.o + tok * a.ldo + (at + 2 * t) * int(sizeof(T));
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) Elem<T>::put_pair(dst + 32 * k * sizeof(T), y[2 * k], y[2 * k + 1]);
  }
  if constexpr (sizeof(T) == 4) {
    if (a.oq) {
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        float am = fmaxf(fabsf(y[2 * k]), fabsf(y[2 * k + 1]));
        am = fmaxf(am, dpp_f<SKG_DPP_QUAD_XOR1>(am));
        am = fmaxf(am, dpp_f<SKG_DPP_QUAD_XOR2>(am));
        am = fmaxf(am, dpp_f<SKG_DPP_ROW_HALF_MIRROR>(am));
        am = fmaxf(am, dpp_f<SKG_DPP_ROW_MIRROR>(am));
        const float d = q8_1_d(am), id = q8_1_id(d);
        const int q0 = q8_1_code(y[2 * k], id), q1 = q8_1_code(y[2 * k + 1], id);
        int sum = q0 + q1;
        sum += __builtin_amdgcn_update_dpp(0, sum, SKG_DPP_QUAD_XOR1, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, SKG_DPP_QUAD_XOR2, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, SKG_DPP_ROW_HALF_MIRROR, 0xF, 0xF, false);
        sum += __builtin_amdgcn_update_dpp(0, sum, SKG_DPP_ROW_MIRROR, 0xF, 0xF, false);
        if (is) {
          uint8_t* dst = a.oq + (tok * a.blocks + at / QK + k) * 36;
          reinterpret_cast<uint16_t*>(dst + 4)[t] = uint16_t((q0 & 0xFF) | (q1 & 0xFF) << 8);
          if (t == 0) *reinterpret_cast<uint32_t*>(dst) = q8_1_d16(d) | (q8_1_s16(d, sum) << 16);
        }
      }
    }
  }
}

// o = y / l (nothing seen: 0) to the outputs.
template <class T, int BLOCKS>
__device__ inline void finish(const TreeArgs& a, int64_t tok, int64_t at, float (&y)[2 * BLOCKS], float l, float unit, bool is) {
  const float inv = unit / l;
#pragma unroll
  for (int j = 0; j < 2 * BLOCKS; ++j) y[j] = l == 0.f ? 0.f : y[j] * inv;
  put_out<T, BLOCKS>(a, tok, at, y, is);
}

// The products' initial values: minus the zero of the codes times the row's q.
template <class S, int KIND, int NB, int NT, class W>
__device__ inline void fill_zero(W& w) {
  const u32x4 z{kZero, kZero, kZero, kZero};
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    w.zero[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = NT - 1; k >= 0; --k)
      w.zero[b] = mfma<true>(z, u32x4{w.q[0][b][k][0], w.q[0][b][k][1], w.q[0][b][k][2], w.q[0][b][k][3]}, w.zero[b]);
  }
}

// A wave's sums of a row tile, elements h C .. h C + C - 1, to LDS [16][C + 4].
template <class S, int KIND, int D>
__device__ inline void put_tile(const f32x4 (&o)[D / 16], float (*obuf)[S::C + 4], int c, int g, int h) {
  constexpr int C = S::C;
  if constexpr (KIND == KV_BF16) {  // element 16 n + 4 g + i at [n][i]
#pragma unroll
    for (int m = 0; m < C / 16; ++m) *reinterpret_cast<f32x4*>(&obuf[c][16 * m + 4 * g]) = o[h * (C / 16) + m];
  } else {  // element 32 b + 8 g + 2 i + e at [2b + e][i]
#pragma unroll
    for (int b = 0; b < C / 32; ++b)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const int n = 2 * (h * (C / 32) + b);
        *reinterpret_cast<f32x4*>(&obuf[c][32 * b + 8 * g + 2 * i]) = f32x4{o[n][i], o[n + 1][i], o[n][i + 1], o[n + 1][i + 1]};
      }
  }
}

// Up to 16 RT rows a workgroup: its waves take every fourth step each and join
// their sums at the end.  Over a long q8_0 cache it is bound by the bytes (one
// token of 64 heads over 131071 keys of 8, 285 MB in 48 us and 4 for the join;
// the loop alone reads at 6.9 TB/s); q4_0, half the bytes for the same
// instructions, by those (16 sequences to 8000 keys, 71 MB in 26 us: 410 a step
// and wave); short caches by the loads that follow each other, lengths, table,
// keys, about 1 us each (37 keys 6.1 us).
template <class T, int KIND, int D, int NT, int RT>
__global__ __launch_bounds__(256, (AttnShape<KIND, D, NT, RT, 4, false>::kPerCu)) void tree_attn_kernel(TreeArgs a) {
  using S = AttnShape<KIND, D, NT, RT, 4, false>;
  constexpr int kWaves = 4;
  constexpr int C = S::C, NB = S::NB;
  constexpr int B = C / 32, EPT = 2 * B;  // blocks and elements of a thread in the joins
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  __shared__ float rs_lds[S::kQLds ? RT * 16 : 1];
  const int head = blockIdx.x, rg = blockIdx.z;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int c = lane & 15, g = lane >> 4;

  Unit unit;
  if (!find_unit<false>(a, blockIdx.y, unit)) return;
  const KvSpan sp = unit.sp;
  const int first = rg * 16 * RT, rows = sp.n * a.group;
  if (first >= rows) return;
  const int left = unit.end - unit.begin - wave;
  const int n = left > 0 ? (left + kWaves - 1) / kWaves : 0;  // this wave's steps

  WaveRows<S, D, NT, RT> w;
  // q first, then the pages, whose use waits for both
  RawRows<T, D> raw;
  const bool mine = !S::kQLds || wave < RT;
  if (mine) fetch_rows<T, D>(raw, a, sp, head, first + (S::kQLds ? 16 * wave : 0));
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = first + 16 * rt + c;
    const bool is = row < rows;
    int i, h;
    row_of(a, row, is, i, h);
    w.mask[rt] = !is ? 0 : a.mask ? a.mask[sp.t0 + i] : ~uint64_t(0) >> (63 - i);
  }
  // where the wave's next 32 steps lie, two tiles each, over its lanes
  const int32_t* table = a.table + int64_t(unit.seq) * a.width;
  auto key_of = [&](int i) SKG_INL { return int(unsigned(unit.begin + wave + i * kWaves) * kStep); };
  auto where_from = [&](int i0) SKG_INL {
    const int i = i0 + (lane >> 1), key = key_of(i) + 16 * (lane & 1);
    return steps_at<KIND, D>(a.cache, head, key, i < n && key < sp.keys ? table[key >> a.cache.shift] : -1);
  };
  StepsAt where = where_from(0);
  uint8_t* ring = lds + wave * (S::kSlots * S::kSlot);
  const uint32_t ring_at = lds_addr(ring);
  uint32_t flags = 0;  // the copied steps' tiles in the cache, two bits each, oldest first
  auto copy_both = [&](int i) SKG_INL {
    flags |= there_of(where, i) << (2 * i);
    const StepAt from = step_at<S::kF16>(where, i);
    copy_step<S, KIND, D, false>(a.cache, from, ring_at + i * S::kSlot);
    copy_step<S, KIND, D, true>(a.cache, from, ring_at + i * S::kSlot);
  };
  // one step's copies, and q's conversion before the others: their issue
  // waits for room in the memory pipeline
  if (n > 0) copy_both(0);

  w.q_lds = lds + S::kRing + 16 * lane;
  if (mine) {
    const float rs = convert_rows<T, S, KIND, D, NT>(raw, a.scale, [&](int b, int k, const uint32_t(&x)[4]) SKG_INL {
      if constexpr (S::kQLds) {
        *reinterpret_cast<u32x4*>(lds + S::kRing + 16 * lane + ((wave * NB + b) * NT + k) * 1024) = u32x4{x[0], x[1], x[2], x[3]};
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w.q[0][b][k][j] = x[j];
      }
    });
    if constexpr (S::kQLds) rs_lds[16 * wave + c] = rs;
    else w.rs[0] = rs;
  }
#pragma unroll 1
  for (int i = 1; i < S::kSlots && i < n; ++i) copy_both(i);
  if constexpr (S::kSubnormal) fill_zero<S, KIND, NB, NT>(w);
  if constexpr (S::kQLds) {
    __syncthreads();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) w.rs[rt] = rs_lds[16 * rt + c];
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    w.M[rt] = kNoMax;
    w.l[rt] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) w.o[rt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  w.be = -40;

  // A SIMD serves its oldest wave first, so of two workgroups of a CU the first
  // ran ahead and left the other alone, at one wave a SIMD, for the last third.
  // The further a wave is, the lower its priority.
  __builtin_amdgcn_s_setprio(3);
  const int n1 = n / 4 - 1, n2 = n / 2 - 1, n3 = 3 * n / 4 - 1;
  int slot = 0;
  auto step = [&](int i, auto edge) SKG_INL {
    const int ahead = n - 1 - i < S::kSlots - 1 ? n - 1 - i : S::kSlots - 1;  // later steps on their way
    const int later = i + S::kSlots;
    const bool more = later < n;
    uint8_t* at = ring + slot * S::kSlot;
    StepRegs<S> r;
    r.key = key_of(i);
    r.there[0] = flags & 1;
    r.there[1] = flags & 2;
    flags >>= 2;
    float s[RT][8];
    wait_ahead<S::kCopies, S::kSlots>(ahead);
    read_k<S, KIND>(r, at);
    read_v<S, KIND>(r, at);
    do_scores<S, KIND, D, NT, RT>(w, r, s);
    if (more) {
      if ((later & 31) == 0) where = where_from(later);
      flags |= there_of(where, later) << (2 * (S::kSlots - 1));
      const StepAt next = step_at<S::kF16>(where, later);
      wait_lds();  // its slot is this step's, read by now
      copy_step<S, KIND, D, false>(a.cache, next, ring_at + slot * S::kSlot);
      copy_step<S, KIND, D, true>(a.cache, next, ring_at + slot * S::kSlot);
    }
    do_values<S, KIND, D, NT, RT, edge()>(w, r, s, sp.ctx, sp.keys);
    slot = slot + 1 == S::kSlots ? 0 : slot + 1;
    if (i == n1) __builtin_amdgcn_s_setprio(2);
    if (i == n2) __builtin_amdgcn_s_setprio(1);
    if (i == n3) __builtin_amdgcn_s_setprio(0);
  };
  // steps that every row sees whole, then (from the first that is not) the rest
  int i = 0;
#pragma unroll 1
  for (; i < n && (flags & 3) == 3 && key_of(i) + kStep <= sp.ctx; ++i) step(i, std::false_type{});
#pragma unroll 1
  for (; i < n; ++i) step(i, std::true_type{});

  // Join the waves: lane t of the sixteen of row jr sums elements 32 k + 2 t and
  // the next.
  float(*obuf)[16][C + 4] = reinterpret_cast<float(*)[16][C + 4]>(lds);
  float(*ml)[RT][16][2] = reinterpret_cast<float(*)[RT][16][2]>(lds + S::kJoin);
  const int jr = threadIdx.x >> 4, je = 2 * (threadIdx.x & 15);
  const bool whole = unit.splits == 1;
  constexpr float kUnit = KIND == KV_BF16 ? 1.f : kVScale;
  // this split's partial results
  const int64_t at = (int64_t(blockIdx.y) * gridDim.z + rg) * gridDim.x + head;
  float* sums = a.sums + at * (16 * RT * D);
  float* sums_ml = a.ml + at * (16 * RT * 2);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float l = row_sum(w.l[rt]);
#pragma unroll
    for (int h = 0; h < D / C; ++h) {
      __syncthreads();
      if (g == 0 && h == 0) {
        ml[wave][rt][c][0] = w.M[rt];
        ml[wave][rt][c][1] = l;
      }
      put_tile<S, KIND, D>(w.o[rt], obuf[wave], c, g, h);
      __syncthreads();
      float M = kNoMax, lsum = 0.f, f[kWaves], y[EPT];
#pragma unroll
      for (int k = 0; k < kWaves; ++k) M = fmaxf(M, ml[k][rt][jr][0]);
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        f[k] = exp2_fast(ml[k][rt][jr][0] - M);
        lsum = fmaf(f[k], ml[k][rt][jr][1], lsum);
      }
#pragma unroll
      for (int i = 0; i < EPT; ++i) y[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k)
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const f32x2 o = *reinterpret_cast<const f32x2*>(&obuf[k][jr][32 * i + je]);
          y[2 * i] = fmaf(f[k], o.x, y[2 * i]);
          y[2 * i + 1] = fmaf(f[k], o.y, y[2 * i + 1]);
        }
      const int row = first + 16 * rt + jr;
      const bool is = row < rows;
      if (whole) {
        int i, hd;
        row_of(a, row, is, i, hd);
        finish<T, B>(a, sp.t0 + i, int64_t(head * a.group + hd) * D + h * C, y, lsum, kUnit, is);
      } else if (is) {
        float* dst = sums + (16 * rt + jr) * D + h * C + je;
#pragma unroll
        for (int j = 0; j < B; ++j) *reinterpret_cast<f32x2*>(dst + 32 * j) = f32x2{y[2 * j], y[2 * j + 1]};
        if (h == 0 && je == 0) *reinterpret_cast<f32x2*>(sums_ml + 2 * (16 * rt + jr)) = f32x2{M, lsum};
      }
    }
  }
}

// Up to 16 RT W rows a workgroup: every wave its own, all waves the same steps
// from a ring that they fill together, so the cache is read once for all of
// them.  One barrier a step: past it the step's copies (each wave waits for its
// own before it) are there and the slot of the step before is free.  256 rows
// over bf16 take 1.34 us a step: 0.43 of LDS reads (a wave's 32 rows read the
// step's 16 KB), 0.43 of matrix and about 0.5 of vector instructions, which
// waves in step hardly overlap (trees of 61, 61, 6 and 23: 12.3 GFLOP in 33 us
// and 8 for the join).
template <class T, int KIND, int D, int NT, int RT, int W>
__global__ __launch_bounds__(64 * W, (W == 8 ? 2 : AttnShape<KIND, D, NT, RT, W, true>::kPerCu)) void tree_attn_rows_kernel(TreeArgs a) {
  using S = AttnShape<KIND, D, NT, RT, W, true>;
  constexpr int C = S::C, NB = S::NB, B = C / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::kLds];
  const int head = blockIdx.x, rg = blockIdx.z;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int c = lane & 15, g = lane >> 4;

  Unit unit;
  if (!find_unit<W == 8>(a, blockIdx.y, unit)) return;
  const KvSpan sp = unit.sp;
  const int rows = sp.n * a.group, group_first = rg * 16 * RT * W;
  if (group_first >= rows) return;
  const int first = group_first + 16 * RT * wave;
  const int n = unit.end - unit.begin;

  WaveRows<S, D, NT, RT> w;
  RawRows<T, D> raw[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    fetch_rows<T, D>(raw[rt], a, sp, head, first + 16 * rt);
    const int row = first + 16 * rt + c;
    const bool is = row < rows;
    int i, h;
    row_of(a, row, is, i, h);
    w.mask[rt] = !is ? 0 : a.mask ? a.mask[sp.t0 + i] : ~uint64_t(0) >> (63 - i);
  }
  const int32_t* table = a.table + int64_t(unit.seq) * a.width;
  auto key_of = [&](int i) SKG_INL { return int(unsigned(unit.begin + i) * kStep); };
  auto where_from = [&](int i0) SKG_INL {
    const int i = i0 + (lane >> 1), key = key_of(i) + 16 * (lane & 1);
    return steps_at<KIND, D>(a.cache, head, key, i < n && key < sp.keys ? table[key >> a.cache.shift] : -1);
  };
  StepsAt where = where_from(0);
  const uint32_t ring_at = lds_addr(lds);
  uint32_t flags = 0;  // the copied steps' tiles in the cache, two bits each, oldest first
  auto copy = [&](int i, int slot, int at) SKG_INL {
    flags |= there_of(where, i) << (2 * at);
    copy_part<S, KIND, D, W>(a.cache, step_at<S::kF16>(where, i), ring_at + slot * S::kSlot, wave);
  };
#pragma unroll 1
  for (int i = 0; i < S::kSlots - 1 && i < n; ++i) copy(i, i, i);

#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    w.rs[rt] = convert_rows<T, S, KIND, D, NT>(raw[rt], a.scale, [&](int b, int k, const uint32_t(&x)[4]) SKG_INL {
#pragma unroll
      for (int j = 0; j < 4; ++j) w.q[rt][b][k][j] = x[j];
    });
    w.M[rt] = kNoMax;
    w.l[rt] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) w.o[rt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  w.be = -40;
  if constexpr (S::kSubnormal) fill_zero<S, KIND, NB, NT>(w);

  int slot = 0;
  auto step = [&](int i, auto edge) SKG_INL {
    wait_parts<S::kPart, S::kSlots - 2>(n - 1 - i);
    wait_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const uint8_t* at = lds + slot * S::kSlot;
    StepRegs<S> r;
    r.key = key_of(i);
    r.there[0] = flags & 1;
    r.there[1] = flags & 2;
    flags >>= 2;
    const int later = i + S::kSlots - 1;
    if (later < n) {
      if ((later & 31) == 0) where = where_from(later);
      copy(later, slot == 0 ? S::kSlots - 1 : slot - 1, S::kSlots - 2);
    }
    if (first < rows) {  // a wave without rows copies only
      float s[RT][8];
      read_k<S, KIND>(r, at);
      do_scores<S, KIND, D, NT, RT>(w, r, s);
      read_v<S, KIND>(r, at);
      do_values<S, KIND, D, NT, RT, edge()>(w, r, s, sp.ctx, sp.keys);
    }
    slot = slot + 1 == S::kSlots ? 0 : slot + 1;
  };
  int i = 0;
#pragma unroll 1
  for (; i < n && (flags & 3) == 3 && key_of(i) + kStep <= sp.ctx; ++i) step(i, std::false_type{});
#pragma unroll 1
  for (; i < n; ++i) step(i, std::true_type{});

  // each wave's rows through its part of LDS, four rows of 16 lanes at a time
  __syncthreads();
  float(*obuf)[C + 4] = reinterpret_cast<float(*)[C + 4]>(lds) + 16 * wave;
  const bool whole = unit.splits == 1;
  constexpr float kUnit = KIND == KV_BF16 ? 1.f : kVScale;
  const int64_t at = (int64_t(blockIdx.y) * gridDim.z + rg) * gridDim.x + head;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const float l = row_sum(w.l[rt]);
#pragma unroll
    for (int h = 0; h < D / C; ++h) {
      wait_lds();
      put_tile<S, KIND, D>(w.o[rt], obuf, c, g, h);
      wait_lds();
#pragma unroll 1
      for (int i4 = 0; i4 < 4; ++i4) {
        const int jr = 4 * i4 + g, je = 2 * c;  // row, elements 32 j + je
        float y[2 * B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
          const f32x2 o = *reinterpret_cast<const f32x2*>(&obuf[jr][32 * j + je]);
          y[2 * j] = o.x;
          y[2 * j + 1] = o.y;
        }
        const float M = __shfl(w.M[rt], jr, 64), lsum = __shfl(l, jr, 64);
        const int local = 16 * (RT * wave + rt) + jr, row = group_first + local;
        const bool is = row < rows;
        if (whole) {
          int i, hd;
          row_of(a, row, is, i, hd);
          finish<T, B>(a, sp.t0 + i, int64_t(head * a.group + hd) * D + h * C, y, lsum, kUnit, is);
        } else if (is) {
          float* dst = a.sums + (at * a.tile + local) * D + h * C + je;
#pragma unroll
          for (int j = 0; j < B; ++j) *reinterpret_cast<f32x2*>(dst + 32 * j) = f32x2{y[2 * j], y[2 * j + 1]};
          if (h == 0 && je == 0) *reinterpret_cast<f32x2*>(a.ml + 2 * (at * a.tile + local)) = f32x2{M, lsum};
        }
      }
    }
  }
}

}  // namespace skg
