// C ABI of the rotation, cache and attention entry points: host-side
// validation before any HIP call, then the launch.
#include <climits>
#include <cmath>

#include "api_common.h"
#include "kernels.h"
#include "tree_attn.h"

using namespace skg;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;

int elem_bytes(skg_dtype dt) { return dt == SKG_F32 ? 4 : 2; }

skg_status check_dtype(skg_dtype dt) {
  if (dt != SKG_F32 && dt != SKG_BF16) return fail(SKG_E_INVALID_ARG, "unknown dtype %d", int(dt));
  return SKG_OK;
}
skg_status check_dim(int D) {
  if (D != 64 && D != 128 && D != 256) return fail(SKG_E_SHAPE, "head_dim must be 64, 128 or 256 (got %d)", D);
  return SKG_OK;
}
skg_status check_tokens(int64_t T) {
  if (T < 1 || T > kMaxTokens) return fail(SKG_E_SHAPE, "T must be in [1, 2^24] (got %lld)", (long long)T);
  return SKG_OK;
}

skg_status kv_size(int fmt, int heads, int D, int page, int64_t pages, size_t* bytes) {
  if (fmt != SKG_KV_BF16 && fmt != SKG_KV_Q8_0 && fmt != SKG_KV_Q4_0)
    return fail(SKG_E_INVALID_ARG, "unknown cache fmt %d", fmt);
  if (heads < 1 || heads > 65535) return fail(SKG_E_SHAPE, "cache heads must be in [1, 65535] (got %d)", heads);
  if (skg_status st = check_dim(D); st != SKG_OK) return st;
  if (page < 16 || page > kKvMaxPage || (page & (page - 1)))
    return fail(SKG_E_SHAPE, "page_size must be a power of two in [16, 2^20] (got %d)", page);
  if (pages < 1 || pages > INT32_MAX) return fail(SKG_E_SHAPE, "pages must be in [1, 2^31 - 1] (got %lld)", (long long)pages);
  const size_t chunk = size_t(page) * (kv_row_bytes(fmt, D) + kv_scale_bytes(fmt, D));
  size_t all = 0;
  if (__builtin_mul_overflow(chunk * size_t(heads), size_t(pages), &all) || all > (size_t(1) << 62))
    return fail(SKG_E_SHAPE, "cache of %lld pages is too large", (long long)pages);
  *bytes = all;
  return SKG_OK;
}

skg_status check_cache(const skg_kv_cache* c, KvView* v, size_t* bytes, bool buffers = true) {
  if (!c) return fail(SKG_E_INVALID_ARG, "null cache");
  if (skg_status st = kv_size(c->fmt, c->heads, c->head_dim, c->page_size, c->pages, bytes); st != SKG_OK) return st;
  if (buffers) {
    if (!c->k || !c->v) return fail(SKG_E_INVALID_ARG, "null cache buffer");
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return fail(SKG_E_ALIGN, "cache buffers must be 16-byte aligned");
  }
  v->k = static_cast<uint8_t*>(c->k);
  v->v = static_cast<uint8_t*>(c->v);
  v->pages = c->pages;
  v->heads = uint32_t(c->heads);
  v->shift = uint32_t(__builtin_ctz(unsigned(c->page_size)));
  v->chunk = uint32_t(c->page_size) * (kv_row_bytes(c->fmt, c->head_dim) + kv_scale_bytes(c->fmt, c->head_dim));
  return SKG_OK;
}

// T rows of `width` elements, ld elements apart.
struct Span {
  const char* name;
  const void* p;
  int64_t ld, width;
};

skg_status check_rows(const Span& s, int64_t T, skg_dtype dt) {
  const int es = elem_bytes(dt);
  if (!s.p) return fail(SKG_E_INVALID_ARG, "null %s", s.name);
  if (T > 1 && s.ld < s.width)
    return fail(SKG_E_SHAPE, "stride of %s is %lld elements, its rows have %lld", s.name, (long long)s.ld,
                (long long)s.width);
  if (s.ld < 0 || s.ld > (int64_t(1) << 32) || (s.ld * es) % 16)
    return fail(SKG_E_SHAPE, "stride of %s must be a multiple of 16 bytes and at most 2^32 elements (got %lld)",
                s.name, (long long)s.ld);
  if (!aligned(s.p, 16)) return fail(SKG_E_ALIGN, "%s must be 16-byte aligned", s.name);
  return SKG_OK;
}

// Whether any element of a is one of b.  Rows of one stride interleave
// without meeting where their columns differ (q and k of a fused buffer);
// other strides are compared by their whole extent.
bool overlap(const Span& a, const Span& b, int64_t T, skg_dtype dt) {
  const int64_t es = elem_bytes(dt);
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t ea = pa + uintptr_t(((T - 1) * a.ld + a.width) * es), eb = pb + uintptr_t(((T - 1) * b.ld + b.width) * es);
  if (ea <= pb || eb <= pa) return false;
  if (a.ld != b.ld || T == 1) return true;
  const int64_t period = a.ld * es;
  const int64_t d = int64_t((pb >= pa ? pb - pa : pa - pb) % uintptr_t(period));
  const int64_t first = pb >= pa ? a.width * es : b.width * es, second = pb >= pa ? b.width * es : a.width * es;
  return d < first || d + second > period;
}

bool meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}

bool overlap_bytes(const Span& a, int64_t T, skg_dtype dt, const void* p, size_t n) {
  return meet(a.p, size_t((T - 1) * a.ld + a.width) * size_t(elem_bytes(dt)), p, n);
}

skg_status check_rope(const skg_rope* r, int D) {
  if (!r) return fail(SKG_E_INVALID_ARG, "null rope");
  if (r->rot < 0 || r->rot > D || r->rot % 16)
    return fail(SKG_E_SHAPE, "rot must be a multiple of 16 in [0, %d] (got %d)", D, r->rot);
  if (r->rot && (!r->pos || !r->inv_freq)) return fail(SKG_E_INVALID_ARG, "null pos or inv_freq");
  if (r->rot && (!aligned(r->pos, 4) || !aligned(r->inv_freq, 4)))
    return fail(SKG_E_ALIGN, "pos and inv_freq must be 4-byte aligned");
  if (r->norm) {
    if (!(r->eps >= 0.f) || !std::isfinite(r->eps)) return fail(SKG_E_INVALID_ARG, "eps must be finite and >= 0");
    if (!aligned(r->gq, 16) || !aligned(r->gk, 16)) return fail(SKG_E_ALIGN, "gq and gk must be 16-byte aligned");
  }
  return SKG_OK;
}

// In place is the same rows; anything else that meets is refused.
skg_status check_in_out(const Span& in, const Span& out, int64_t T, skg_dtype dt, bool in_place) {
  if (in_place && in.p == out.p && (in.ld == out.ld || T == 1)) return SKG_OK;
  if (overlap(in, out, T, dt)) return fail(SKG_E_INVALID_ARG, "%s and %s overlap", in.name, out.name);
  return SKG_OK;
}

#define SKG_TRY(expr)                                      \
  do {                                                     \
    if (skg_status st_ = (expr); st_ != SKG_OK) return st_; \
  } while (0)

skg_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(SKG_E_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

size_t skg_kv_bytes(skg_kv_fmt fmt, int heads, int head_dim, int page_size, int64_t pages) {
  size_t bytes = 0;
  return kv_size(fmt, heads, head_dim, page_size, pages, &bytes) == SKG_OK ? (ok(), bytes) : 0;
}

skg_status skg_qk_norm_rope(skg_dtype dtype, int64_t T, int hq, int hk, int head_dim, const void* q, int64_t ldq,
                            const void* k, int64_t ldk, const skg_rope* rope, void* qo, int64_t ldqo, void* ko,
                            int64_t ldko, hipStream_t stream) {
  SKG_TRY(check_dtype(dtype));
  SKG_TRY(check_tokens(T));
  SKG_TRY(check_dim(head_dim));
  if (hq < 0 || hk < 0 || int64_t(hq) + hk < 1 || int64_t(hq) + hk > 65535)
    return fail(SKG_E_SHAPE, "hq + hk must be in [1, 65535] (got %d, %d)", hq, hk);
  SKG_TRY(check_rope(rope, head_dim));
  const int64_t wq = int64_t(hq) * head_dim, wk = int64_t(hk) * head_dim;
  const Span sq{"q", q, ldq, wq}, sk{"k", k, ldk, wk}, sqo{"qo", qo, ldqo, wq}, sko{"ko", ko, ldko, wk};
  if (hq) {
    SKG_TRY(check_rows(sq, T, dtype));
    SKG_TRY(check_rows(sqo, T, dtype));
    SKG_TRY(check_in_out(sq, sqo, T, dtype, true));
  }
  if (hk) {
    SKG_TRY(check_rows(sk, T, dtype));
    SKG_TRY(check_rows(sko, T, dtype));
    SKG_TRY(check_in_out(sk, sko, T, dtype, true));
  }
  if (hq && hk) {
    SKG_TRY(check_in_out(sq, sko, T, dtype, false));
    SKG_TRY(check_in_out(sk, sqo, T, dtype, false));
    SKG_TRY(check_in_out(sqo, sko, T, dtype, false));
  }
  SKG_TRY(check_device());
  return launched(launch_qk_norm_rope(dtype, T, hq, hk, head_dim, q, ldq, k, ldk, rope, qo, ldqo, ko, ldko, stream),
                  "qk_norm_rope");
}

skg_status skg_kv_store(const skg_kv_cache* cache, skg_dtype dtype, int64_t T, const void* k, int64_t ldk,
                        const void* v, int64_t ldv, const int64_t* slots, hipStream_t stream) {
  KvView c;
  size_t bytes = 0;
  SKG_TRY(check_dtype(dtype));
  SKG_TRY(check_cache(cache, &c, &bytes));
  SKG_TRY(check_tokens(T));
  const int64_t w = int64_t(cache->heads) * cache->head_dim;
  const Span sk{"k", k, ldk, w}, sv{"v", v, ldv, w};
  for (const Span* s : {&sk, &sv}) {
    SKG_TRY(check_rows(*s, T, dtype));
    if (overlap_bytes(*s, T, dtype, cache->k, bytes) || overlap_bytes(*s, T, dtype, cache->v, bytes))
      return fail(SKG_E_INVALID_ARG, "%s overlaps the cache", s->name);
  }
  if (!slots) return fail(SKG_E_INVALID_ARG, "null slots");
  if (!aligned(slots, 8)) return fail(SKG_E_ALIGN, "slots must be 8-byte aligned");
  SKG_TRY(check_device());
  return launched(launch_kv_store(c, cache->fmt, cache->head_dim, dtype, T, k, ldk, v, ldv, slots, stream), "kv_store");
}

skg_status skg_kv_load(const skg_kv_cache* cache, skg_dtype dtype, int64_t T, const int64_t* slots, void* k,
                       int64_t ldk, void* v, int64_t ldv, hipStream_t stream) {
  KvView c;
  size_t bytes = 0;
  SKG_TRY(check_dtype(dtype));
  SKG_TRY(check_cache(cache, &c, &bytes));
  SKG_TRY(check_tokens(T));
  const int64_t w = int64_t(cache->heads) * cache->head_dim;
  const Span sk{"k", k, ldk, w}, sv{"v", v, ldv, w};
  for (const Span* s : {&sk, &sv}) {
    SKG_TRY(check_rows(*s, T, dtype));
    if (overlap_bytes(*s, T, dtype, cache->k, bytes) || overlap_bytes(*s, T, dtype, cache->v, bytes))
      return fail(SKG_E_INVALID_ARG, "%s overlaps the cache", s->name);
  }
  SKG_TRY(check_in_out(sk, sv, T, dtype, false));
  if (!slots) return fail(SKG_E_INVALID_ARG, "null slots");
  if (!aligned(slots, 8)) return fail(SKG_E_ALIGN, "slots must be 8-byte aligned");
  SKG_TRY(check_device());
  return launched(launch_kv_load(c, cache->fmt, cache->head_dim, dtype, T, slots, k, ldk, v, ldv, stream), "kv_load");
}

skg_status skg_qkv_rope_store(const skg_kv_cache* cache, skg_dtype dtype, int64_t T, int hq, const void* q,
                              int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                              const skg_rope* rope, const int64_t* slots, void* qo, int64_t ldqo,
                              hipStream_t stream) {
  KvView c;
  size_t bytes = 0;
  SKG_TRY(check_dtype(dtype));
  SKG_TRY(check_cache(cache, &c, &bytes));
  SKG_TRY(check_tokens(T));
  if (hq < 1 || int64_t(hq) + cache->heads > 65535)
    return fail(SKG_E_SHAPE, "hq must be >= 1 and hq + heads at most 65535 (got %d)", hq);
  SKG_TRY(check_rope(rope, cache->head_dim));
  const int64_t wq = int64_t(hq) * cache->head_dim, w = int64_t(cache->heads) * cache->head_dim;
  const Span sq{"q", q, ldq, wq}, sk{"k", k, ldk, w}, sv{"v", v, ldv, w}, sqo{"qo", qo, ldqo, wq};
  for (const Span* s : {&sq, &sk, &sv, &sqo}) {
    SKG_TRY(check_rows(*s, T, dtype));
    if (overlap_bytes(*s, T, dtype, cache->k, bytes) || overlap_bytes(*s, T, dtype, cache->v, bytes))
      return fail(SKG_E_INVALID_ARG, "%s overlaps the cache", s->name);
  }
  SKG_TRY(check_in_out(sq, sqo, T, dtype, true));
  SKG_TRY(check_in_out(sk, sqo, T, dtype, false));
  SKG_TRY(check_in_out(sv, sqo, T, dtype, false));
  if (!slots) return fail(SKG_E_INVALID_ARG, "null slots");
  if (!aligned(slots, 8)) return fail(SKG_E_ALIGN, "slots must be 8-byte aligned");
  SKG_TRY(check_device());
  return launched(launch_qkv_rope_store(c, cache->fmt, cache->head_dim, dtype, T, hq, q, ldq, k, ldk, v, ldv, rope,
                                        slots, qo, ldqo, stream),
                  "qkv_rope_store");
}

namespace {

// The counts of an attention call; max_kv is set to the bound that applies.
skg_status check_attn(const skg_kv_cache* cache, int64_t T, int64_t n_seqs, int hq, int max_draft, int64_t width,
                      int64_t* max_kv) {
  SKG_TRY(check_tokens(T));
  if (n_seqs < 1 || n_seqs > 65535) return fail(SKG_E_SHAPE, "n_seqs must be in [1, 65535] (got %lld)", (long long)n_seqs);
  if (hq < 1 || hq % cache->heads || hq / cache->heads > 256)
    return fail(SKG_E_SHAPE, "hq must be 1 to 256 times the cache's %d heads (got %d)", cache->heads, hq);
  if (max_draft < 1 || max_draft > 64) return fail(SKG_E_SHAPE, "max_draft must be in [1, 64] (got %d)", max_draft);
  if (width < 1 || width > (int64_t(1) << 26)) return fail(SKG_E_SHAPE, "width must be in [1, 2^26] (got %lld)", (long long)width);
  const int64_t most = int64_t(INT32_MAX) - 64, room = width * cache->page_size;
  if (*max_kv < 0 || *max_kv > most) return fail(SKG_E_SHAPE, "max_kv must be in [0, 2^31 - 65] (got %lld)", (long long)*max_kv);
  if (*max_kv == 0 || *max_kv > room) *max_kv = room < most ? room : most;
  return SKG_OK;
}

}  // namespace

size_t skg_tree_attn_workspace(const skg_kv_cache* cache, skg_dtype dtype, int64_t T, int64_t n_seqs, int hq, int max_draft,
                               int64_t width, int64_t max_kv) {
  KvView c;
  size_t bytes = 0;
  if (check_dtype(dtype) != SKG_OK || check_cache(cache, &c, &bytes, false) != SKG_OK) return 0;
  if (check_attn(cache, T, n_seqs, hq, max_draft, width, &max_kv) != SKG_OK) return 0;
  ok();
  return tree_attn_workspace(cache->fmt, cache->head_dim, cache->heads, dtype, T, n_seqs, hq, max_draft, max_kv);
}

skg_status skg_tree_attn(const skg_kv_cache* cache, skg_dtype dtype, int64_t T, int64_t n_seqs, int hq,
                         int max_draft, const void* q, int64_t ldq, const int32_t* cu, const int32_t* ctx,
                         const int32_t* table, int64_t width, int64_t max_kv, const uint64_t* mask, float scale,
                         void* o, int64_t ldo, void* oq, void* ws, size_t ws_bytes, hipStream_t stream) {
  TreeArgs a;
  size_t bytes = 0;
  SKG_TRY(check_dtype(dtype));
  SKG_TRY(check_cache(cache, &a.cache, &bytes));
  SKG_TRY(check_attn(cache, T, n_seqs, hq, max_draft, width, &max_kv));
  if (!cu && T % n_seqs)
    return fail(SKG_E_SHAPE, "without cu, T must be a multiple of n_seqs (got %lld, %lld)", (long long)T, (long long)n_seqs);
  if (!std::isfinite(scale)) return fail(SKG_E_INVALID_ARG, "scale must be finite");
  if (!ctx || !table) return fail(SKG_E_INVALID_ARG, "null ctx or table");
  if (!aligned(cu, 4) || !aligned(ctx, 4) || !aligned(table, 4) || !aligned(mask, 8))
    return fail(SKG_E_ALIGN, "cu, ctx and table must be 4-byte, mask 8-byte aligned");
  if (!o && !oq) return fail(SKG_E_INVALID_ARG, "o and oq are both null");
  if (oq && dtype != SKG_F32) return fail(SKG_E_UNSUPPORTED, "Q8_1 output needs SKG_F32");
  const int64_t w = int64_t(hq) * cache->head_dim;
  const Span sq{"q", q, ldq, w}, so{"o", o, ldo, w};
  SKG_TRY(check_rows(sq, T, dtype));
  if (o) {
    SKG_TRY(check_rows(so, T, dtype));
    SKG_TRY(check_in_out(sq, so, T, dtype, false));
    if (overlap_bytes(so, T, dtype, cache->k, bytes) || overlap_bytes(so, T, dtype, cache->v, bytes))
      return fail(SKG_E_INVALID_ARG, "o overlaps the cache");
  }
  if (oq) {
    const size_t nq = size_t(T) * size_t(w / QK) * 36;
    if (!aligned(oq, 4)) return fail(SKG_E_ALIGN, "oq must be 4-byte aligned");
    if (overlap_bytes(sq, T, dtype, oq, nq) || (o && overlap_bytes(so, T, dtype, oq, nq)))
      return fail(SKG_E_INVALID_ARG, "oq overlaps q or o");
    if (meet(oq, nq, cache->k, bytes) || meet(oq, nq, cache->v, bytes))
      return fail(SKG_E_INVALID_ARG, "oq overlaps the cache");
  }
  const size_t need = tree_attn_workspace(cache->fmt, cache->head_dim, cache->heads, dtype, T, n_seqs, hq, max_draft, max_kv);
  if (need) {
    if (!ws || ws_bytes < need)
      return fail(SKG_E_INVALID_ARG, "workspace of %zu bytes needed (got %zu)", need, ws ? ws_bytes : size_t(0));
    if (!aligned(ws, 256)) return fail(SKG_E_ALIGN, "ws must be 256-byte aligned");
    if (meet(ws, need, cache->k, bytes) || meet(ws, need, cache->v, bytes) || overlap_bytes(sq, T, dtype, ws, need) ||
        (o && overlap_bytes(so, T, dtype, ws, need)) || (oq && meet(ws, need, oq, size_t(T) * size_t(w / QK) * 36)))
      return fail(SKG_E_INVALID_ARG, "ws overlaps another argument");
  }
  SKG_TRY(check_device());
  const int es = elem_bytes(dtype);
  a.q = static_cast<const uint8_t*>(q);
  a.ldq = ldq * es;
  a.o = static_cast<uint8_t*>(o);
  a.ldo = ldo * es;
  a.oq = static_cast<uint8_t*>(oq);
  a.cu = cu;
  a.ctx = ctx;
  a.table = table;
  a.width = width;
  a.max_kv = max_kv;
  a.mask = mask;
  a.scale = scale;
  a.T = T;
  a.n_seqs = int(n_seqs);
  a.hq = hq;
  a.group = hq / cache->heads;
  a.max_draft = max_draft;
  return launched(launch_tree_attn(a, cache->fmt, cache->head_dim, dtype, cache->heads, ws, stream), "tree_attn");
}

}  // extern "C"
