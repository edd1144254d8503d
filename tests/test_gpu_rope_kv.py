"""Rotation and cache entry points against the float64 oracle (GPU).

Rotated values: within the binary32 bound of oracle.rope_tolerance.  Cache
bytes: equal, bit for bit, to the oracle's encoder on the same binary32
values; read-back values exact.
"""

import numpy as np
import pytest

import oracle
from tests._gpu import dev, host, note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def skg():
    import skinny_gemm_decode_amd as m
    return m


@pytest.fixture(scope="module")
def torch():
    import torch as t
    return t


def kinds(skg):
    return {"bf16": skg.KV_BF16, "q8_0": skg.KV_Q8_0, "q4_0": skg.KV_Q4_0}


def values(rng, shape, bf16=False):
    x = rng.standard_normal(shape).astype(np.float32)
    return oracle.formats.bf16_bits_to_f64(oracle.attention.bf16_rne(x)).astype(np.float32) if bf16 else x


def rows_on_gpu(torch, x, bf16, pad=0):
    """x [T, H, D] as a tensor whose tokens lie `pad` elements further apart than needed."""
    T, H, D = x.shape
    buf = torch.full((T, H * D + pad), float("nan"), device="cuda", dtype=torch.bfloat16 if bf16 else torch.float32)
    t = buf[:, :H * D].unflatten(1, (H, D))
    t.copy_(torch.from_numpy(x).cuda())
    return t


def back(t):
    return host(t.float())


def freqs(rot, base=10000.0):
    return (base ** (-np.arange(0, rot, 2) / rot)).astype(np.float32) if rot else np.zeros(0, np.float32)


# (T, hq, hk, D, rot, interleaved, norm, bf16, pad)
ROPE = [
    (1, 32, 32, 128, 128, True, False, False, 0),
    (1, 1, 0, 64, 64, False, True, False, 0),
    (8, 32, 8, 128, 128, False, True, False, 16),
    (3, 5, 1, 256, 64, False, True, True, 8),
    (7, 14, 2, 64, 32, True, True, True, 0),
    (5, 0, 3, 256, 256, False, False, False, 4),
    (2, 33, 17, 64, 16, False, False, True, 40),
    (4, 3, 3, 128, 0, False, True, False, 0),
    (4, 3, 3, 128, 0, False, False, True, 0),
    (131, 7, 7, 128, 96, True, True, False, 0),
    (129, 64, 8, 128, 128, False, True, True, 0),
]


@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm,bf16,pad", ROPE)
def test_qk_norm_rope(skg, torch, T, hq, hk, D, rot, inter, norm, bf16, pad):
    note(f"qk_norm_rope T={T} hq={hq} hk={hk} D={D} rot={rot} inter={inter} norm={norm} bf16={bf16}")
    rng = np.random.default_rng(T * 1000 + hq * 10 + D)
    pos = rng.integers(0, 2_000_000, T).astype(np.int32)
    pos[0] = 0 if T > 1 else 4095
    f = freqs(rot)
    out, args = {}, {}
    for name, H in (("q", hq), ("k", hk)):
        x = values(rng, (T, H, D), bf16)
        g = (1 + 0.2 * rng.standard_normal(D)).astype(np.float32) if norm and name == "q" else None
        args[name] = (x, g)
    q = rows_on_gpu(torch, args["q"][0], bf16, pad) if hq else None
    k = rows_on_gpu(torch, args["k"][0], bf16, pad) if hk else None
    gq = dev(args["q"][1]) if norm else None
    kw = dict(gq=gq, eps=1e-5, norm=norm, interleaved=inter)
    posd, fd = (dev(pos), dev(f)) if rot else (None, None)
    out = skg.qk_norm_rope(q, k, posd, fd, **kw)
    for name, y, t in (("q", out[0], q), ("k", out[1], k)):
        x, g = args[name]
        if t is None:
            assert y is None
            continue
        ref = oracle.rope_ref(x, pos, f, inter, norm, g, 1e-5)
        tol = oracle.rope_tolerance(x, ref, inter, rot // 2, norm, g, 1e-5, bf16)
        err = np.abs(back(y) - ref)
        assert np.all(err <= tol), (name, float(np.max(err / tol)))
        assert np.array_equal(back(t), x), "the input changed"
    # in place, the same bits; the gaps between tokens keep theirs
    skg.qk_norm_rope(q, k, posd, fd, qo=q, ko=k, **kw)
    for y, t in ((out[0], q), (out[1], k)):
        if t is not None:
            assert torch.equal(y, t)
            if pad and T > 1:
                whole = torch.as_strided(t, (T, t.stride(0)), (t.stride(0), 1))
                assert bool(torch.isnan(whole[:T - 1, t.shape[1] * D:]).all())


def test_rope_on_parts_of_a_fused_buffer_in_place(skg, torch):
    T, hq, hk, D = 6, 8, 2, 128
    rng = np.random.default_rng(3)
    x = values(rng, (T, hq + 2 * hk, D))
    pos, f = np.arange(T, dtype=np.int32) + 70000, freqs(D)
    note("qk_norm_rope fused buffer")
    buf = dev(x)
    qo, ko = skg.qk_norm_rope(buf[:, :hq], buf[:, hq:hq + hk], dev(pos), dev(f), qo=buf[:, :hq], ko=buf[:, hq:hq + hk])
    y = back(buf)
    ref = oracle.rope_ref(x[:, :hq + hk], pos, f)
    assert np.all(np.abs(y[:, :hq + hk] - ref) <= oracle.rope_tolerance(x[:, :hq + hk], ref, False, D // 2))
    assert np.array_equal(y[:, hq + hk:], x[:, hq + hk:])


def test_rope_negative_and_extreme_positions(skg, torch):
    pos = np.array([-1, -2**31, 2**31 - 1, 2**24 + 1], dtype=np.int32)
    x, f = values(np.random.default_rng(5), (4, 1, 64)), freqs(64)
    note("qk_norm_rope extreme positions")
    y, _ = skg.qk_norm_rope(dev(x), None, dev(pos), dev(f))
    ref = oracle.rope_ref(x, pos, f)
    # 2^31 / (2 pi) turns: the binary64 angle keeps 2^31 * 2^-53 = 2^-22 of a radian
    assert np.all(np.abs(back(y) - ref) <= oracle.rope_tolerance(x, ref, False, 32) + 2.0**-22 * np.abs(x).max())


def test_zero_row_with_eps(skg, torch):
    note("qk_norm_rope zero row")
    y, _ = skg.qk_norm_rope(torch.zeros((2, 3, 128), device="cuda"), None, dev(np.zeros(2, np.int32)), dev(freqs(128)), norm=True)
    assert np.all(back(y) == 0)


# ---- cache ----------------------------------------------------------------------

def build_cache(skg, torch, fmt, heads, D, page, pages, fill=0xA5):
    c = skg.kv_cache(kinds(skg)[fmt], heads, D, page, pages)
    c.k.fill_(fill)
    c.v.fill_(fill)
    return c


def expect_bytes(fmt, heads, D, page, pages, slots, x, fill=0xA5):
    p = oracle.Pages(fmt, pages, heads, page, D, fill)
    for s, row in zip(slots, x):
        if 0 <= s < pages * page:
            p.put(int(s), row)
    return p


# Workgroups enough for two rows a thread: a last pass that is part empty, one
# that is all empty, and the smallest call of that kind.
MANY_ROPE = [
    # T, hq, hk, D, rot, interleaved, norm, bf16, pad
    (400, 33, 6, 256, 128, False, True, True, 0),
    (1100, 3, 1, 128, 128, True, False, False, 0),
    (1024, 2, 0, 64, 32, False, True, False, 16),
]


@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm,bf16,pad", MANY_ROPE)
def test_qk_norm_rope_of_many_rows(skg, torch, T, hq, hk, D, rot, inter, norm, bf16, pad):
    test_qk_norm_rope(skg, torch, T, hq, hk, D, rot, inter, norm, bf16, pad)


CACHE = [(fmt, T, heads, D, page, bf16, pad) for fmt in oracle.KV_FMTS for T, heads, D, page, bf16, pad in
         [(1, 1, 64, 16, False, 0), (1, 32, 128, 16, False, 0), (8, 5, 256, 32, True, 16), (133, 3, 128, 64, False, 4),
          (40, 2, 64, 1024, True, 0), (17, 7, 256, 16, False, 0)]]


@pytest.mark.parametrize("fmt,T,heads,D,page,bf16,pad", CACHE)
def test_store_and_load(skg, torch, fmt, T, heads, D, page, bf16, pad):
    note(f"kv_store {fmt} T={T} heads={heads} D={D} page={page} bf16={bf16}")
    rng = np.random.default_rng(T + heads + D)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 4:  # padding and slots outside the cache
        slots[[1, 3]] = [-1, pages * page]
    k, v = values(rng, (T, heads, D), bf16), values(rng, (T, heads, D), bf16) * 32
    v[0, 0, :32] = 0  # a block of zeros
    c = build_cache(skg, torch, fmt, heads, D, page, pages)
    skg.kv_store(c, rows_on_gpu(torch, k, bf16, pad), rows_on_gpu(torch, v, bf16, pad), dev(slots))
    for buf, x in ((c.k, k), (c.v, v)):
        assert np.array_equal(host(buf), expect_bytes(fmt, heads, D, page, pages, slots, x).raw.reshape(-1))
    # read back, in another order, some slots twice, some outside
    read = np.concatenate([slots[::-1], slots[:1], [-5, 2**40]]).astype(np.int64)
    for out_bf16 in (False, True):
        kt, vt = (rows_on_gpu(torch, np.full((len(read), heads, D), 7, np.float32), out_bf16, 2 * pad) for _ in range(2))
        skg.kv_load(c, dev(read), k=kt, v=vt)
        for t, x in ((kt, k), (vt, v)):
            p = expect_bytes(fmt, heads, D, page, pages, slots, x)
            inside = (read >= 0) & (read < pages * page)
            ref = np.zeros((len(read), heads, D))
            ref[inside] = p.get(read[inside])
            got = back(t)
            if out_bf16:
                ref = oracle.formats.bf16_bits_to_f64(oracle.attention.bf16_rne(ref.astype(np.float32)))
            assert np.array_equal(got, ref)


def test_rounding_borders(skg, torch):
    """Ties of the code rounding, ties of the largest element's sign (the first
    wins), subnormal and huge blocks: the oracle's bytes."""
    D = 64
    x = np.zeros((6, 1, D), np.float32)
    x[0, 0, :32] = (np.arange(32) - 15.5) * 127 / 127  # halves at d = ...
    x[0, 0, 0], x[0, 0, 31] = 127, -127
    x[1, 0, :4] = [3, -8, 8, -8]
    x[1, 0, 32:36] = [1, 8, -8, 0.5]
    x[2, 0, :] = np.linspace(-1e-7, 1e-7, D)
    x[3, 0, :] = np.linspace(-6e8, 3e8, D)
    x[4, 0, :] = 65504 * 127.0
    x[5, 0, :] = np.linspace(-2e-38, 2e-38, D)  # 1 / d overflows: no code is defined, but d is stored as 0
    for fmt in oracle.KV_FMTS:
        note(f"kv_store borders {fmt}")
        c = build_cache(skg, torch, fmt, 1, D, 16, 1)
        slots = np.arange(6, dtype=np.int64)
        skg.kv_store(c, dev(x), dev(-x), dev(slots))
        with np.errstate(over="ignore"):
            for buf, s in ((c.k, x), (c.v, -x)):
                want = expect_bytes(fmt, 1, D, 16, 1, slots[:5], s)
                got = oracle.Pages(fmt, 1, 1, 16, D)
                got.raw[:] = host(buf).reshape(got.raw.shape)
                assert np.array_equal(got.codes[:, :, :5], want.codes[:, :, :5]), fmt
                assert np.array_equal(got.scales[:, :, :5], want.scales[:, :, :5]), fmt
                if fmt != "bf16":
                    assert np.all(got.get([5]) == 0)


@pytest.mark.parametrize("fmt", ["q8_0", "q4_0"])
def test_non_finite_elements_are_stored_as_finite_values(skg, torch, fmt):
    x = values(np.random.default_rng(9), (3, 2, 64))
    x[0, 0, 3], x[1, 1, 40], x[2, 0, 7] = np.inf, np.nan, -np.inf
    note(f"kv_store non-finite {fmt}")
    c = build_cache(skg, torch, fmt, 2, 64, 16, 1)
    s = dev(np.arange(3, dtype=np.int64))
    skg.kv_store(c, dev(x), dev(x), s)
    k, v = skg.kv_load(c, s)
    assert np.all(np.isfinite(host(k))) and np.all(np.isfinite(host(v)))
    # blocks without such an element are as they would be
    want = oracle.kv_decode(fmt, *oracle.kv_encode(fmt, np.nan_to_num(x, nan=0, posinf=0, neginf=0)))
    assert np.array_equal(host(k)[0, 1], want[0, 1]) and np.array_equal(host(k)[0, 0, 32:], want[0, 0, 32:])


@pytest.mark.parametrize("fmt", oracle.KV_FMTS)
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm,bf16", [
    (1, 32, 32, 128, 128, True, False, False), (8, 32, 8, 128, 128, False, True, False),
    (5, 7, 1, 256, 128, False, True, True), (9, 10, 5, 64, 32, True, True, True), (3, 3, 3, 64, 0, False, False, False),
    (2, 64, 8, 128, 128, False, True, True)])
def test_fused_store_is_the_two_launches(skg, torch, fmt, T, hq, hk, D, rot, inter, norm, bf16):
    """q: the bits of qk_norm_rope; the cache: the bits of kv_store of the
    binary32 rotated k and of v."""
    note(f"qkv_rope_store {fmt} T={T} hq={hq} hk={hk} D={D} rot={rot} bf16={bf16}")
    rng = np.random.default_rng(T * 7 + hq)
    x = values(rng, (T, hq + 2 * hk, D), bf16)
    qkv = rows_on_gpu(torch, x, bf16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    pos = dev(rng.integers(0, 100000, T).astype(np.int32)) if rot else None
    f = dev(freqs(rot)) if rot else None
    gq, gk = (dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2)) if norm else (None, None)
    slots = rng.permutation(64)[:T].astype(np.int64)
    if T > 4:
        slots[2] = -1
    kw = dict(gq=gq, gk=gk, norm=norm, interleaved=inter)
    one, two = (build_cache(skg, torch, fmt, hk, D, 32, 2) for _ in range(2))
    qo = skg.qkv_rope_store(one, q, k, v, dev(slots), pos, f, **kw)
    q2, _ = skg.qk_norm_rope(q, None, pos, f, **kw)
    _, k2 = skg.qk_norm_rope(None, k.float().contiguous(), pos, f, **kw)
    skg.kv_store(two, k2, v.float().contiguous(), dev(slots))
    assert torch.equal(qo, q2) and torch.equal(one.k, two.k) and torch.equal(one.v, two.v)


def test_far_slots_of_a_large_cache(skg, torch):
    """Offsets past 32 bits: the last page of a buffer of over 4 GiB."""
    heads, D, page = 8, 128, 1 << 14
    pages = (1 << 32) // (heads * page * 2 * D) + 2
    note("kv_store past 4 GiB")
    c = skg.kv_cache(skg.KV_BF16, heads, D, page, pages)
    assert c.k.numel() > 1 << 32
    x = values(np.random.default_rng(1), (3, heads, D), True)
    slots = np.array([pages * page - 1, 0, (pages - 1) * page + 5], dtype=np.int64)
    skg.kv_store(c, dev(x), dev(-x), dev(slots))
    k, v = skg.kv_load(c, dev(slots))
    assert np.array_equal(host(k), x) and np.array_equal(host(v), -x)
    at = ((pages - 1) * heads + heads - 1) * page * 2 * D + (page - 1) * 2 * D
    assert np.array_equal(host(c.k[at:at + 2 * D].view(torch.bfloat16).float()), x[0, heads - 1])


def test_on_another_stream(skg, torch):
    """Outputs allocated by the call belong to the stream that it names."""
    s = torch.cuda.Stream()
    x, f = values(np.random.default_rng(2), (64, 8, 128)), freqs(128)
    xd, pos, fd = dev(x), dev(np.arange(64, dtype=np.int32)), dev(f)
    note("qk_norm_rope on another stream")
    want, _ = skg.qk_norm_rope(xd, None, pos, fd)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        y, _ = skg.qk_norm_rope(xd, None, pos, fd, stream=stream)
        s.synchronize()
        assert torch.equal(y, want)


def test_largest_token_count(skg, torch):
    """2^24 tokens, one more than the workgroups of a launch: rotation, store
    and load of one head of 64, compared at the seam and at both ends."""
    T = 1 << 24
    note("rope, store and load of 2^24 tokens")
    x = torch.randn((T, 1, 64), device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(3))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    f = freqs(64)
    at = np.array([0, 1, 77777, T - 3, T - 2, T - 1])
    rows = host(x[at].float())
    o, _ = skg.qk_norm_rope(x, None, pos, dev(f))
    ref = oracle.rope_ref(rows, at, f, False)
    assert np.all(np.abs(host(o[at].float()) - ref) <= 2.0**-8 * np.abs(ref) + 2.0**-20)
    del o
    page = 1 << 12
    c = skg.kv_cache(skg.KV_Q8_0, 1, 64, page, T // page)
    slots = torch.arange(T, device="cuda").flip(0)
    skg.kv_store(c, x, x, slots)
    k, v = skg.kv_load(c, slots, dtype=torch.bfloat16)
    want = oracle.kv_decode("q8_0", *oracle.kv_encode("q8_0", rows))
    for t in (k, v):
        assert np.all(np.abs(host(t[at].float()) - want) <= 2.0**-8 * np.abs(want))
    assert bool((k == v).all())
