"""Attention of drafted tokens against the float64 oracle (GPU)."""

import numpy as np
import pytest

import oracle
from tests._gpu import dev, host, note
from tests.test_gpu_rope_kv import kinds, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skg():
    import skinny_gemm_decode_amd as m
    return m


@pytest.fixture(scope="module")
def torch():
    import torch as t
    return t


def tree(rng, n):
    """Ancestor bits of a random tree of n nodes."""
    bits = []
    for i in range(n):
        p = int(rng.integers(max(-1, i - 5), i)) if i else -1
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    return bits


class Problem:
    """Sequences with contexts ctx and drafted counts n over a shuffled paged
    cache whose unused bytes are all ones (NaN scales, NaN bf16) and whose
    unused table entries name pages outside it."""

    def __init__(self, skg, torch, fmt, ctx, n, hq, hk, D, page, bf16=False, masks="tree", seed=0, extra=(0, 0), qs=1.0):
        rng = np.random.default_rng(seed + sum(ctx) + hq)
        self.skg, self.torch, self.fmt, self.bf16 = skg, torch, fmt, bf16
        self.ctx, self.n, self.hq, self.hk, self.D, self.page = ctx, n, hq, hk, D, page
        B = len(ctx)
        need = [-(-(c + t) // page) for c, t in zip(ctx, n)]
        self.width = max(max(need), 1) + 1
        pages = sum(need) + 2
        order = rng.permutation(pages)
        self.table = np.full((B, self.width), -1, np.int32)
        self.table[:, 1::2] = 2**31 - 1
        at = 0
        for b, u in enumerate(need):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.kp, self.vp = (oracle.Pages(fmt, pages, hk, page, D) for _ in range(2))
        for b in range(B):
            for j in range(ctx[b] + n[b]):
                s = int(self.table[b, j // page]) * page + j % page
                self.kp.put(s, values(rng, (hk, D)))
                self.vp.put(s, values(rng, (hk, D)))
        lead, tail = extra
        T = lead + sum(n) + tail
        self.cu = np.cumsum([lead] + list(n)).astype(np.int32)
        self.q = qs * values(rng, (T, hq, D), bf16)
        if bf16:
            self.q = oracle.formats.bf16_bits_to_f64(oracle.attention.bf16_rne(self.q.astype(np.float32))).astype(np.float32)
        self.q = self.q.astype(np.float32)
        self.T, self.masks = T, None
        if masks is not None:
            bits = [0] * lead
            for t in n:
                bits += tree(rng, t) if masks == "tree" else [0] * t if masks == "none" else [int(rng.integers(0, 2**63)) for _ in range(t)]
            self.masks = np.array(bits + [0] * tail, dtype=np.uint64)
        self.cache = skg.KvCache(kinds(skg)[fmt], hk, D, page, dev(self.kp.raw), dev(self.vp.raw))

    def sees(self, b, max_draft=64, max_kv=None):
        n, c = min(self.n[b], max_draft), self.ctx[b]
        s = np.zeros((n, c + n), bool)
        s[:, :c] = True
        for i in range(n):
            m = (1 << (i + 1)) - 1 if self.masks is None else int(self.masks[self.cu[b] + i])
            for j in range(n):
                s[i, c + j] = (m >> j) & 1
        if max_kv:
            s[:, max_kv:] = False
        return s

    def reference(self, max_draft=64, max_kv=None, drop=()):
        """(o, tolerance, computed rows); drop: (sequence, page index) that are not there."""
        o, tol, done = np.zeros((self.T, self.hq, self.D)), np.zeros((self.T, self.hq, self.D)), np.zeros(self.T, bool)
        for b, (c, t) in enumerate(zip(self.ctx, self.n)):
            t = min(t, max_draft)
            j = np.arange(c + t)
            s = self.sees(b, max_draft, max_kv)
            slots = self.table[b, j // self.page].astype(np.int64) * self.page + j % self.page
            for db, dp in drop:
                if db == b:
                    s[:, j // self.page == dp] = False
                    slots[j // self.page == dp] = 0
            r = slice(self.cu[b], self.cu[b] + t)
            scale = 1 / np.sqrt(self.D)
            v = self.vp.get(slots)
            o[r], a, e = oracle.tree_attn_ref(self.q[r], self.kp.get(slots), v, s, scale)
            vmax = np.max(np.abs(v), where=np.isfinite(v), initial=0.0)
            tol[r] = oracle.tree_attn_tolerance(o[r], a, e, self.D, self.bf16, self.fmt == "bf16", len(slots), vmax)
            done[r] = True
        return o, tol, done

    def args(self):
        t = self.torch
        q = dev(self.q).to(t.bfloat16 if self.bf16 else t.float32)
        m = None if self.masks is None else dev(self.masks.view(np.int64))
        return dict(q=q, table=dev(self.table), ctx=dev(np.array(self.ctx, np.int32)), cu=dev(self.cu), mask=m)

    def run(self, **kw):
        a = self.args()
        o = self.torch.full(a["q"].shape, 77.0, device="cuda", dtype=a["q"].dtype)
        kw.setdefault("max_draft", max(max(self.n), 1))
        self.skg.tree_attn(self.cache, a["q"], a["table"], a["ctx"], cu=a["cu"], mask=a["mask"], o=o, **kw)
        return host(o.float())

    def check(self, max_draft=None, max_kv=0, drop=()):
        got = self.run(max_draft=max_draft or max(max(self.n), 1), max_kv=max_kv)
        o, tol, done = self.reference(max_draft or 64, max_kv, drop)
        assert np.all(got[~done] == 77.0), "rows of no sequence were written"
        err = np.abs(got - o)[done]
        assert np.all(err <= tol[done]), float(np.max(err / tol[done]))
        norm = np.linalg.norm(o)
        if norm and not self.bf16:  # roundings are independent: far closer together than the bound of each
            assert np.linalg.norm(err) <= 1e-5 * norm, np.linalg.norm(err) / norm
        return got


CASES = [
    # ctx, n, hq, hk, D, page
    ([0], [1], 1, 1, 64, 16),
    ([1], [1], 4, 4, 128, 16),
    ([37], [1], 32, 32, 128, 16),
    ([15, 16, 17, 31, 32, 33], [1, 1, 2, 1, 3, 1], 8, 2, 128, 16),
    ([700, 3, 0, 129], [8, 5, 0, 1], 8, 8, 128, 32),
    ([250], [64], 16, 2, 128, 64),
    ([90, 400], [33, 64], 5, 1, 64, 16),
    ([333, 10], [7, 2], 6, 3, 256, 64),
    ([500], [3], 20, 1, 128, 1024),
    ([63, 64, 65], [1, 1, 1], 14, 2, 64, 128),
    ([1500], [1], 40, 8, 128, 256),
    # many rows a cache head: the waves share rows (64, 128, 256 and past it), with splits and without
    ([700], [16], 12, 3, 128, 16),
    ([40, 900, 0], [3, 31, 2], 12, 3, 64, 32),
    ([2000, 5], [64, 40], 16, 4, 128, 64),
    ([100], [57], 10, 2, 256, 16),
    ([300], [9], 16, 1, 64, 16),
]


@pytest.mark.parametrize("fmt", oracle.KV_FMTS)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_tree_attn(skg, torch, fmt, bf16, case):
    ctx, n, hq, hk, D, page = CASES[case]
    note(f"tree_attn {fmt} bf16={bf16} {CASES[case]}")
    Problem(skg, torch, fmt, ctx, n, hq, hk, D, page, bf16, seed=case, extra=(1, 2)).check()


@pytest.mark.parametrize("fmt", oracle.KV_FMTS)
@pytest.mark.parametrize("masks", [None, "none", "random"])
def test_masks(skg, torch, fmt, masks):
    """A chain, masks that leave nothing but the context (or nothing at all: a
    row of zeros), and arbitrary bits, also past the drafted tokens."""
    note(f"tree_attn masks {fmt} {masks}")
    p = Problem(skg, torch, fmt, [40, 0, 7], [9, 4, 20], 8, 4, 128, 16, masks=masks)
    got = p.check()
    if masks == "none":
        assert np.all(got[p.cu[1]:p.cu[2]] == 0)


@pytest.mark.parametrize("fmt", oracle.KV_FMTS)
def test_bounds_of_lengths(skg, torch, fmt):
    """Tokens past max_draft, keys past max_kv and pages outside the cache are
    not there."""
    note(f"tree_attn bounds {fmt}")
    p = Problem(skg, torch, fmt, [100, 20], [9, 3], 4, 2, 64, 16)
    p.check(max_draft=4)
    p.check(max_kv=50)
    p.check(max_kv=104)
    p.table[0, 1] = -1
    p.table[0, 4] = p.kp.raw.shape[0]
    p.table[1, 0] = -(2**31)
    got = p.check(drop=[(0, 1), (0, 4), (1, 0)])
    p.table[:] = -1
    assert np.all(p.run()[p.cu[0]:p.cu[-1]] == 0)
    assert got.shape == p.q.shape


def test_lengths_that_disagree_stay_in_bounds(skg, torch):
    """cu past T, falling cu and contexts below 0 or past the table: clamped, so
    the second sequence takes what it can (over keys that nobody stored) and
    no other row is written."""
    p = Problem(skg, torch, "q8_0", [30, 30], [3, 3], 4, 2, 64, 16)
    note("tree_attn wild lengths")
    p.cu = np.array([4, 2, 900], np.int32)
    p.ctx = [-7, 2**31 - 1]
    got = p.run(max_draft=3)
    assert np.all(got[:2] == 77.0) and np.all(got[5:] == 77.0) and not np.any(got[2:5] == 77.0)


@pytest.mark.parametrize("fmt", oracle.KV_FMTS)
def test_non_finite_values_that_a_row_does_not_see(skg, torch, fmt):
    """NaN and infinities in one branch's drafted token do not reach the others."""
    p = Problem(skg, torch, fmt, [20], [6], 4, 2, 128, 16, masks=None)
    p.masks = np.array([1, 2, 4, 8 | 1, 16, 32], dtype=np.uint64)
    slot = int(p.table[0, 22 // 16]) * 16 + 22 % 16  # drafted token 2
    for pages in (p.kp, p.vp):
        if fmt == "bf16":
            w = pages.codes[slot // 16, :, slot % 16].view(np.uint16)
            w[:, :40], w[:, 40:60], w[:, 60:] = 0x7FC0, 0x7F80, 0xFF80
        else:
            pages.scales[slot // 16, :, slot % 16].view(np.uint16)[:] = 0x7E00
    p.cache = skg.KvCache(kinds(skg)[fmt], 2, 128, 16, dev(p.kp.raw), dev(p.vp.raw))
    note(f"tree_attn non-finite {fmt}")
    got = p.run()
    o, tol, _ = p.reference()
    at = [0, 1, 3, 4, 5]
    r = p.cu[0] + np.array(at)
    assert np.all(np.abs(got[r] - o[r]) <= tol[r])
    assert np.all(np.isnan(got[p.cu[0] + 2]))


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("size", [1e-6, 3e4])
def test_ranges_of_values(skg, torch, fmt, size):
    """Scales of the values from near fp16's smallest to near its largest, and
    tokens of very different magnitude in one sequence."""
    rng = np.random.default_rng(4)
    p = Problem(skg, torch, fmt, [200], [2], 4, 2, 64, 32)
    for j in range(202):
        s = int(p.table[0, j // 32]) * 32 + j % 32
        p.vp.put(s, values(rng, (2, 64)) * np.float32(size * 10.0 ** rng.uniform(0, 2)))
    p.cache = skg.KvCache(kinds(skg)[fmt], 2, 64, 32, dev(p.kp.raw), dev(p.vp.raw))
    note(f"tree_attn ranges {fmt} {size}")
    p.check()


def test_large_scores(skg, torch):
    """Scores of hundreds: one key takes all."""
    for fmt in oracle.KV_FMTS:
        note(f"tree_attn large scores {fmt}")
        p = Problem(skg, torch, fmt, [300], [2], 4, 2, 128, 16, qs=60.0)
        got = p.run()
        o, tol, done = p.reference()
        assert np.all(np.abs(got - o)[done] <= tol[done])


def test_equal_counts_without_cu_and_defaults(skg, torch):
    p = Problem(skg, torch, "q8_0", [50, 60], [4, 4], 8, 2, 128, 16, masks=None)
    a = p.args()
    note("tree_attn without cu")
    o = skg.tree_attn(p.cache, a["q"], a["table"], a["ctx"])
    ref, tol, _ = p.reference()
    assert np.all(np.abs(host(o) - ref) <= tol)


def test_strided_rows(skg, torch):
    p = Problem(skg, torch, "q4_0", [90], [5], 8, 2, 128, 16)
    a = p.args()
    note("tree_attn strided rows")
    buf = torch.full((5, 12, 128), float("nan"), device="cuda")
    buf[:, 2:10] = a["q"]
    out = torch.full((5, 9, 128), 5.0, device="cuda")
    skg.tree_attn(p.cache, buf[:, 2:10], a["table"], a["ctx"], cu=a["cu"], mask=a["mask"], o=out[:, :8])
    want = p.run()
    assert np.array_equal(host(out[:, :8]), want) and np.all(host(out[:, 8]) == 5.0)


@pytest.mark.parametrize("ctx", [[70], [2500, 20, 0]])
def test_q8_1_output(skg, torch, ctx):
    """The blocks are the standalone quantiser's of the float32 output; rows
    outside the sequences keep theirs."""
    p = Problem(skg, torch, "q8_0", ctx, [5] * len(ctx), 8, 4, 128, 32, extra=(1, 1))
    a = p.args()
    note(f"tree_attn Q8_1 {ctx}")
    kw = dict(cu=a["cu"], mask=a["mask"], max_draft=5)
    oq = torch.full((p.T, 8 * 128 // 32, 36), 0xEE, dtype=torch.uint8, device="cuda")
    o = torch.zeros_like(a["q"])
    skg.tree_attn(p.cache, a["q"], a["table"], a["ctx"], o=o, oq=oq, **kw)
    want = skg.quantize_act_q8_1(o.view(p.T, -1))
    inside = slice(1, p.T - 1)
    assert torch.equal(oq[inside], want[inside]) and bool((oq[[0, p.T - 1]] == 0xEE).all())
    none, only = skg.tree_attn(p.cache, a["q"], a["table"], a["ctx"], o=False, oq=True, **kw)
    assert none is None and torch.equal(only[inside], oq[inside])


def test_repeats_and_streams_give_identical_bits(skg, torch):
    p = Problem(skg, torch, "q8_0", [3000], [8], 32, 8, 128, 64, extra=(0, 0))
    a = p.args()
    kw = dict(cu=a["cu"], mask=a["mask"], max_draft=8)
    note("tree_attn repeats")
    want = skg.tree_attn(p.cache, a["q"], a["table"], a["ctx"], **kw)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    outs = [skg.tree_attn(p.cache, a["q"], a["table"], a["ctx"], stream=s[i % 3], **kw) for i in range(12)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_captured_and_replayed(skg, torch):
    """One captured step (rotation, store, attention) replayed as the context
    grows on the device, against eager calls on a second cache; two graphs,
    each with its workspace."""
    hq, hk, D, page, pages = 8, 2, 128, 16, 64
    rng = np.random.default_rng(11)
    width, steps = 40, 5
    table = dev(rng.permutation(pages)[:width].astype(np.int32)[None])
    f = dev((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32))
    caches = [skg.kv_cache(skg.KV_Q8_0, hk, D, page, pages) for _ in range(3)]
    for c in caches:
        c.k.zero_(), c.v.zero_()
    T = 4
    x = torch.zeros((T, hq + 2 * hk, D), device="cuda")
    ctx, pos, slots = (torch.zeros(n, dtype=d, device="cuda") for n, d in ((1, torch.int32), (T, torch.int32), (T, torch.int64)))
    mask = dev(np.array([1, 3, 5, 11], np.int64))

    def step(c):
        q = skg.qkv_rope_store(c, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], slots, pos, f)
        return skg.tree_attn(c, q, table, ctx, mask=mask)

    note("captured step")
    step(caches[0]), step(caches[1]), step(caches[2])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in caches[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c))
        graphs.append(g)
    n = 0
    for i in range(steps):
        note(f"replay {i} at context {n}")
        x.copy_(torch.from_numpy(values(np.random.default_rng(100 + i), (T, hq + 2 * hk, D))).cuda())
        at = np.arange(n, n + T)
        ctx.fill_(n)
        pos.copy_(dev(np.array([n, n + 1, n + 1, n + 2], np.int32)))
        slots.copy_(dev(host(table)[0].astype(np.int64)[at // page] * page + at % page))
        want = step(caches[2])
        for g, o in zip(graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
        assert torch.equal(caches[0].k, caches[2].k) and torch.equal(caches[1].v, caches[2].v)
        n += [1, 130, 7, 300, 0][i]


def test_decode_layer_chain(skg, torch):
    """QKV product, rotation and store, attention and the output product run
    together, as a decode step does, against the oracle of the whole."""
    from synth import inputs as si
    M, H, D = 3, 4, 64
    K = H * D
    rng = si.rng_for(1, 9, 77)
    W = [si.q8_0_weights(rng, K, K) for _ in range(4)]
    x = si.activations_f32(rng, M, K)
    packed = skg.pack_weights_multi(skg.Q8_0_F32, [K] * 3, K, [dev(w) for w in W[:3]])
    wo = skg.pack_weights(skg.Q8_0_Q8_1, K, K, dev(W[3]))
    cache = skg.kv_cache(skg.KV_BF16, H, D, 16, 4)
    f = (10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)
    note("decode layer chain")
    q, k, v = (t.view(M, H, D) for t in skg.gemv_multi(skg.Q8_0_F32, M, K, [K] * 3, packed, dev(x)))
    table, ctx = dev(np.array([[2, 0]], np.int32)), dev(np.zeros(1, np.int32))
    slots, pos = dev(np.arange(32, 32 + M).astype(np.int64)), dev(np.arange(M, dtype=np.int32))
    qr = skg.qkv_rope_store(cache, q, k, v, slots, pos, dev(f), interleaved=True)
    o, oq = skg.tree_attn(cache, qr, table, ctx, oq=True)
    y = host(skg.gemv(skg.Q8_0_Q8_1, M, K, K, wo, oq))
    # the oracle takes each stage's stored values, as the other parity tests do
    hq, hk, hv = (host(t) for t in (q, k, v))
    pos_h = np.arange(M)
    rq, rk = (oracle.rope_ref(t, pos_h, f, True) for t in (hq, hk))
    kk = oracle.formats.bf16_bits_to_f64(oracle.attention.bf16_rne(rk.astype(np.float32)))
    vv = oracle.formats.bf16_bits_to_f64(oracle.attention.bf16_rne(hv))
    ref, a, e = oracle.tree_attn_ref(rq, kk, vv, np.tril(np.ones((M, M), bool)), 1 / np.sqrt(D))
    # the key may be rounded to the other bf16 neighbour: 2^-8 of a score
    tol = a * np.expm1(2 * e * 2.0**-7) + 2.0**-14 * a
    assert np.all(np.abs(host(o) - ref) <= tol)
    yr, b = oracle.gemv_q8_0_q8_1_ref(W[3], host(oq).reshape(M, -1, 36))
    assert oracle.check_close(y, yr, oracle.tolerance(b))[0]


@pytest.mark.parametrize("fmt", oracle.KV_FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3, 24, 61])
def test_float32_rows_keep_float32_scores(skg, torch, fmt, D, n):
    """Random rows of 64 query heads that see two keys (n = 1) or their own and
    those before: what the bounds over all roundings above leave, their root
    mean square does not.  A score's: q in two terms of 11 bits is off by 2^-23
    relative to each of D products of about 2 / sqrt(D), 2^-22 altogether; a
    block's sum of codes times q is about 128 * 2 * sqrt(32) steps of amax / 127
    = 2.2 / 127, 25 of values, rounded to 2^-24 in each of four additions of
    D / 32 blocks, over sqrt(D): 2^-21.4; for the bf16 cache less.  It reaches
    o as p (1 - p) |v - v'| <= 0.35 of that, below 2^-22.5 with the 2^-23.5 of
    p and v.  A quarter of that margin is left to spare."""
    note(f"tree_attn precision {fmt} D={D} n={n}")
    p = Problem(skg, torch, fmt, [1 if n == 1 else 3], [n], 64, 64 if n == 1 else 8, D, 16, masks=None, qs=2.0, seed=5)
    o, want = p.run().astype(np.float64), p.reference()[0]
    assert np.sqrt(np.mean((o - want) ** 2)) <= 2.0**-20


@pytest.mark.parametrize("fmt", oracle.KV_FMTS)
def test_pages_past_32_bit_offsets(skg, torch, fmt):
    """A cache buffer over 4 GiB: keys on its last pages, against the same keys
    in a small cache (the order of pages is not seen)."""
    H, D, page, n = 32, 128, 64, 200
    per = skg.kv_bytes(kinds(skg)[fmt], H, D, page, 1)
    pages = (1 << 32) // per + 9
    note(f"tree_attn and store past 4 GiB {fmt}: {pages} pages")
    rng = np.random.default_rng(8)
    k, v, q = (dev(values(rng, (m, H, D))) for m in (n, n, 3))
    out = []
    for total, table in ((pages, [pages - 1, pages - 3, pages - 2, pages - 5]), (4, [0, 2, 1, 3])):
        c = skg.kv_cache(kinds(skg)[fmt], H, D, page, total)
        t = torch.tensor([table], dtype=torch.int32, device="cuda")
        j = torch.arange(n, device="cuda")
        slots = t[0].long()[j // page] * page + j % page
        skg.kv_store(c, k, v, slots)
        out.append((skg.tree_attn(c, q, t, dev(np.array([n - 3], np.int32))), *skg.kv_load(c, slots)))
        del c
    for a, b in zip(*out):
        assert np.array_equal(host(a), host(b))
    assert np.all(np.isfinite(host(out[0][0]))) and np.abs(host(out[0][0])).max() > 0


@pytest.mark.parametrize("fmt,bf16,hq,hk,B,draft", [("q8_0", False, 2, 2, 70, 1), ("q4_0", True, 4, 1, 130, 1),
                                                   ("q8_0", False, 4, 1, 70, 20), ("bf16", True, 8, 2, 66, 40),
                                                   ("q4_0", False, 2, 1, 300, 2)])
def test_many_sequences(skg, torch, fmt, bf16, hq, hk, B, draft):
    """More sequences than a wave has lanes, long ones among them that are
    split (up to 256 sequences; beyond that none is), at the seams of 64."""
    note(f"tree_attn of {B} sequences {fmt} bf16={bf16} {hq}/{hk} draft={draft}")
    rng = np.random.default_rng(B + draft)
    ctx = [int(c) for c in rng.integers(0, 12, B)]
    for b in (0, 62, 63, 64, B - 1):
        ctx[b] = int(rng.integers(500, 900))
    n = [int(t) for t in rng.integers(0, draft + 1, B)]
    n[63], n[64], n[B - 1] = draft, 1, draft
    Problem(skg, torch, fmt, ctx, n, hq, hk, 64, 16, bf16, seed=draft).check()
