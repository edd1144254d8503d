// Where a paged cache keeps what: plain C++, so that the bounds of every slot
// and page are checked on the host by the tests as well.
//
// A buffer is [pages][heads][chunk]; a chunk is the codes of a page's tokens
// of one head and then their scales (the layout that skg.h documents).  Page
// sizes are powers of two of at least 16 tokens, so an aligned run of 16 keys
// lies on one page and a slot splits by a shift.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define SKG_HD __host__ __device__
#else
#define SKG_HD
#endif

namespace skg {

enum KvKind { KV_BF16 = 0, KV_Q8_0 = 1, KV_Q4_0 = 2 };

constexpr int64_t kKvMaxPage = int64_t(1) << 20;

// Bytes of one token's codes of one head; of its scales.
SKG_HD constexpr uint32_t kv_row_bytes(int kind, int D) {
  return kind == KV_BF16 ? 2u * unsigned(D) : kind == KV_Q8_0 ? unsigned(D) : unsigned(D) / 2;
}
SKG_HD constexpr uint32_t kv_scale_bytes(int kind, int D) { return kind == KV_BF16 ? 0u : unsigned(D) / 16; }

struct KvView {
  uint8_t* k;
  uint8_t* v;
  int64_t pages;
  uint32_t heads;
  uint32_t shift;  // log2 of the page size
  uint32_t chunk;  // bytes of a page's codes and scales of one head (< 2^30)
};

// Whether slot s is in the cache (a negative or too large one is not), and
// whether a page of a block table is.
SKG_HD inline bool kv_slot_in(const KvView& c, int64_t s) { return s >= 0 && (s >> c.shift) < c.pages; }
SKG_HD inline bool kv_page_in(const KvView& c, int32_t page) { return page >= 0 && int64_t(page) < c.pages; }

// Byte offset of (page, head)'s chunk.
SKG_HD inline uint64_t kv_chunk_at(const KvView& c, int64_t page, uint32_t head) {
  return (uint64_t(page) * c.heads + head) * c.chunk;
}
// Within a chunk: offset of token t's codes, and of its scales.
SKG_HD inline uint32_t kv_codes_at(int kind, int D, uint32_t t) { return t * kv_row_bytes(kind, D); }
SKG_HD inline uint32_t kv_scales_at(int kind, int D, uint32_t shift, uint32_t t) {
  return (kv_row_bytes(kind, D) << shift) + t * kv_scale_bytes(kind, D);
}

// Keys that a sequence really has: its context and drafted tokens, cut at
// what the table and the caller's bound allow.  n is its drafted tokens (at
// most max_draft of them).
struct KvSpan {
  int32_t t0;    // first token's row
  int32_t ctx;   // keys every token sees
  int32_t n;     // drafted tokens
  int32_t keys;  // keys that are there
};
SKG_HD inline KvSpan kv_span(int32_t ctx, int32_t t0, int32_t t1, int64_t T, int max_draft, int64_t max_kv) {
  KvSpan s;
  const int64_t a = t0 < 0 ? 0 : (t0 > T ? T : t0), b = t1 < 0 ? 0 : (t1 > T ? T : t1);
  const int64_t n = b > a ? (b - a < max_draft ? b - a : max_draft) : 0;
  int64_t c = ctx < 0 ? 0 : ctx;
  if (c > max_kv) c = max_kv;
  int64_t keys = int64_t(c) + n;
  if (ctx > max_kv || keys > max_kv) keys = max_kv;
  s.t0 = int32_t(a);
  s.ctx = int32_t(c);
  s.n = int32_t(n);
  s.keys = int32_t(keys);
  return s;
}

// How attention's keys are split, in steps of 32: splits of equal cost over
// `want` of them, a sequence's cost being steps * each (its weight, 1 to 5) in
// units of 2^shift, so that the sum over all sequences fits 31 bits.  A
// sequence with tokens has at least one split, so all of them have at most
// want + n_seqs: the workspace's size rests on that.
constexpr int kStep = 32;
constexpr int kMinSteps = 8;  // of a split at least, where a sequence is split
constexpr int kMaxWeight = 5;

SKG_HD inline int kv_cost_shift(int64_t max_kv, int n_seqs) {
  int shift = 0;
  while (((((max_kv + kStep - 1) / kStep * kMaxWeight) >> shift) + 1) > INT32_MAX / n_seqs) ++shift;
  return shift;
}
SKG_HD inline int kv_steps(int32_t keys) { return keys / kStep + (keys % kStep != 0); }
SKG_HD inline int kv_cost(int steps, int each, int shift) {
  return int((uint32_t(steps) * uint32_t(each) + (1u << shift) - 1) >> shift);
}
// Steps of a split that costs `cost`.  A sequence has at most 2^26, so a split
// of 2^29 / kMaxWeight always holds one whole.
SKG_HD inline int kv_split_steps(int cost, int each, int shift) {
  const uint32_t most = (1u << 29) >> shift, c = (uint32_t(cost) < most ? uint32_t(cost) : most) << shift;
  const int per = int((c + uint32_t(each) - 1) / uint32_t(each));
  return per < kMinSteps ? kMinSteps : per;
}
SKG_HD inline int kv_splits(int steps, int per) {
  const int n = int((uint32_t(steps) + uint32_t(per) - 1) / uint32_t(per));
  return n < 1 ? 1 : n;
}

}  // namespace skg
