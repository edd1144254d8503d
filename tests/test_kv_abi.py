"""Refusals of the rotation, cache and attention entry points (CPU): every
invalid argument is rejected on the host, before any HIP call."""

import ctypes

import pytest
import torch

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="fake-pointer validation runs only without a GPU")

BASE = 1 << 40
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def skg():
    import skinny_gemm_decode_amd as m
    return m


def ptr(mb, off=0):
    """A fake device address, megabytes apart; never dereferenced."""
    return ctypes.c_void_p(BASE + (mb << 20) + off)


def cache(skg, fmt=1, heads=4, D=128, page=16, pages=8, k=800, v=900, koff=0):
    from skinny_gemm_decode_amd.kv import _Cache
    return ctypes.byref(_Cache(fmt, heads, D, page, pages, ptr(k, koff) if k else None, ptr(v) if v else None))


def rope(skg, rot=128, inter=0, norm=0, eps=1e-6, pos=700, inv=701, gq=None, gk=None):
    from skinny_gemm_decode_amd.kv import _Rope
    return ctypes.byref(_Rope(rot, inter, norm, eps, ptr(pos) if pos else None, ptr(inv) if inv else None, gq, gk))


def test_kv_bytes(skg):
    assert skg.kv_bytes(skg.KV_Q8_0, 32, 128, 16, 10) == 10 * 32 * 16 * (128 + 8)
    assert skg.kv_bytes(skg.KV_Q4_0, 8, 64, 64, 3) == 3 * 8 * 64 * (32 + 4)
    assert skg.kv_bytes(skg.KV_BF16, 1, 256, 1 << 20, 2) == 2 * (1 << 20) * 512
    for bad in ((3, 1, 64, 16, 1), (-1, 1, 64, 16, 1), (1, 0, 64, 16, 1), (1, 65536, 64, 16, 1), (1, 1, 96, 16, 1),
                (1, 1, 64, 8, 1), (1, 1, 64, 48, 1), (1, 1, 64, 1 << 21, 1), (1, 1, 64, 16, 0), (1, 1, 64, 16, 1 << 31),
                (0, 65535, 256, 1 << 20, (1 << 31) - 1)):
        assert skg.kv_bytes(*bad) == 0, bad


@no_gpu
def test_qk_norm_rope_refusals(skg):
    f = skg.lib.skg_qk_norm_rope

    def call(dt=F32, T=4, hq=8, hk=2, D=128, q=ptr(0), ldq=1024, k=ptr(10), ldk=256, r=None, qo=ptr(20), ldqo=1024,
             ko=ptr(30), ldko=256):
        return f(dt, T, hq, hk, D, q, ldq, k, ldk, rope(skg) if r is None else r, qo, ldqo, ko, ldko, None)

    assert call() == skg.E_DEVICE  # valid: only the device is missing
    assert call(q=ptr(0), qo=ptr(0), k=ptr(10), ko=ptr(10)) == skg.E_DEVICE  # in place
    assert call(hq=0, q=None, qo=None) == skg.E_DEVICE and call(hk=0, k=None, ko=None) == skg.E_DEVICE
    assert call(dt=2) == skg.E_INVALID_ARG
    for kw in (dict(T=0), dict(T=(1 << 24) + 1), dict(D=96), dict(hq=-1), dict(hq=0, hk=0), dict(hq=65535),
               dict(ldq=1020), dict(ldq=1026), dict(ldko=128), dict(ldqo=-1024), dict(ldk=(1 << 33))):
        assert call(**kw) == skg.E_SHAPE, kw
    for rot in (-16, 8, 144, 136):
        assert call(r=rope(skg, rot=rot)) == skg.E_SHAPE
    assert call(r=rope(skg, pos=None)) == skg.E_INVALID_ARG and call(r=rope(skg, inv=None)) == skg.E_INVALID_ARG
    assert call(r=rope(skg, rot=0, pos=None, inv=None)) == skg.E_DEVICE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(r=rope(skg, norm=1, eps=eps)) == skg.E_INVALID_ARG
        assert call(r=rope(skg, norm=0, eps=eps)) == skg.E_DEVICE
    assert call(r=rope(skg, norm=1, gq=ptr(1, 4))) == skg.E_ALIGN
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None)):
        assert call(**kw) == skg.E_INVALID_ARG, kw
    for kw in (dict(q=ptr(0, 4)), dict(ko=ptr(30, 8))):
        assert call(**kw) == skg.E_ALIGN, kw
    # overlaps: shifted by a row, outputs on each other, an output on the other input
    for kw in (dict(qo=ptr(0, 4096)), dict(qo=ptr(0, 16)), dict(qo=ptr(30)), dict(ko=ptr(0)), dict(qo=ptr(10)),
               dict(qo=ptr(0), ldqo=2048)):
        assert call(**kw) == skg.E_INVALID_ARG, kw
        assert "overlap" in skg.last_error()
    # parts of one fused buffer interleave without overlapping, and may be turned in place
    fused = dict(ldq=1536, ldk=1536, ldqo=1536, ldko=1536, q=ptr(0), k=ptr(0, 4096))
    assert call(qo=ptr(0), ko=ptr(0, 4096), **fused) == skg.E_DEVICE
    assert call(qo=ptr(0), ko=ptr(0, 4096 - 512), **fused) == skg.E_INVALID_ARG


@no_gpu
def test_store_and_load_refusals(skg):
    for name in ("skg_kv_store", "skg_kv_load"):
        f = getattr(skg.lib, name)

        def call(c=None, dt=F32, T=4, k=ptr(0), ldk=512, v=ptr(10), ldv=512, slots=ptr(20)):
            c = cache(skg) if c is None else c
            if name == "skg_kv_store":
                return f(c, dt, T, k, ldk, v, ldv, slots, None)
            return f(c, dt, T, slots, k, ldk, v, ldv, None)

        assert call() == skg.E_DEVICE
        assert call(c=ctypes.c_void_p(None)) == skg.E_INVALID_ARG
        assert call(dt=-1) == skg.E_INVALID_ARG and call(c=cache(skg, fmt=3)) == skg.E_INVALID_ARG
        assert call(c=cache(skg, k=None)) == skg.E_INVALID_ARG and call(c=cache(skg, v=None)) == skg.E_INVALID_ARG
        assert call(c=cache(skg, koff=8)) == skg.E_ALIGN
        for c in (cache(skg, heads=0), cache(skg, D=32), cache(skg, page=24), cache(skg, pages=0)):
            assert call(c=c) == skg.E_SHAPE
        for kw in (dict(T=0), dict(ldk=510), dict(ldv=256)):
            assert call(**kw) == skg.E_SHAPE, kw
        for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(k=ptr(800)), dict(v=ptr(900, 1024))):
            assert call(**kw) == skg.E_INVALID_ARG, kw
        for kw in (dict(k=ptr(0, 8)), dict(slots=ptr(20, 4))):
            assert call(**kw) == skg.E_ALIGN, kw
    assert skg.lib.skg_kv_load(cache(skg), F32, 4, ptr(20), ptr(0), 512, ptr(0), 512, None) == skg.E_INVALID_ARG


@no_gpu
def test_qkv_rope_store_refusals(skg):
    f = skg.lib.skg_qkv_rope_store

    def call(c=None, dt=F32, T=4, hq=8, q=ptr(0), ldq=1024, k=ptr(10), ldk=512, v=ptr(20), ldv=512, r=None,
             slots=ptr(30), qo=ptr(40), ldqo=1024):
        return f(cache(skg) if c is None else c, dt, T, hq, q, ldq, k, ldk, v, ldv, rope(skg) if r is None else r,
                 slots, qo, ldqo, None)

    assert call() == skg.E_DEVICE and call(qo=ptr(0)) == skg.E_DEVICE
    assert call(c=cache(skg, D=64)) == skg.E_SHAPE  # rot exceeds the head
    for kw in (dict(hq=0), dict(hq=65535), dict(T=0), dict(ldq=1000), dict(ldv=256)):
        assert call(**kw) == skg.E_SHAPE, kw
    for kw in (dict(q=None), dict(v=None), dict(slots=None), dict(qo=None), dict(qo=ptr(10)), dict(qo=ptr(20, 512)),
               dict(q=ptr(800)), dict(qo=ptr(900)), dict(dt=5)):
        assert call(**kw) == skg.E_INVALID_ARG, kw


@no_gpu
def test_tree_attn_refusals(skg):
    f = skg.lib.skg_tree_attn

    def call(c=None, dt=F32, T=4, n=2, hq=8, md=2, q=ptr(0), ldq=1024, cu=ptr(50), ctx=ptr(51), table=ptr(52), width=4,
             max_kv=0, mask=ptr(53), scale=0.1, o=ptr(10), ldo=1024, oq=None, ws=ptr(60), wsb=1 << 20):
        return f(cache(skg) if c is None else c, dt, T, n, hq, md, q, ldq, cu, ctx, table, width, max_kv, mask, scale,
                 o, ldo, oq, ws, wsb, None)

    assert call() == skg.E_DEVICE and call(cu=None, mask=None) == skg.E_DEVICE and call(oq=ptr(20)) == skg.E_DEVICE
    assert call(o=None, oq=ptr(20)) == skg.E_DEVICE
    for kw in (dict(T=0), dict(n=0), dict(n=65536), dict(hq=6), dict(hq=0), dict(hq=4 * 257), dict(md=0), dict(md=65),
               dict(width=0), dict(width=(1 << 26) + 1), dict(max_kv=-1), dict(max_kv=1 << 31), dict(ldq=1000),
               dict(ldo=512), dict(cu=None, T=5)):
        assert call(**kw) == skg.E_SHAPE, kw
    for kw in (dict(dt=2), dict(q=None), dict(ctx=None), dict(table=None), dict(o=None), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(o=ptr(0)), dict(o=ptr(0, 4096)), dict(o=ptr(800)), dict(oq=ptr(0)),
               dict(oq=ptr(10, 64))):
        assert call(**kw) == skg.E_INVALID_ARG, kw
    for kw in (dict(q=ptr(0, 8)), dict(o=ptr(10, 4)), dict(oq=ptr(20, 2)), dict(cu=ptr(50, 2)), dict(mask=ptr(53, 4))):
        assert call(**kw) == skg.E_ALIGN, kw
    assert call(dt=BF16, oq=ptr(20)) == skg.E_UNSUPPORTED
    # a long cache needs a workspace: absent, short, misaligned
    size = skg.lib.skg_tree_attn_workspace(cache(skg, pages=1000), F32, 4, 2, 8, 2, 500, 0)
    assert size > 0
    long = dict(c=cache(skg, pages=1000, v=2000), width=500)
    assert call(ws=ptr(60), wsb=size, **long) == skg.E_DEVICE
    assert call(ws=ptr(60), wsb=size - 1, **long) == skg.E_INVALID_ARG
    assert call(ws=None, wsb=size, **long) == skg.E_INVALID_ARG
    assert call(ws=ptr(60, 128), wsb=size, **long) == skg.E_ALIGN
    # workspace or Q8_1 blocks over another argument
    for kw in (dict(ws=ptr(0)), dict(ws=ptr(10)), dict(ws=ptr(800)), dict(ws=ptr(2000)), dict(ws=ptr(20), oq=ptr(20, 64))):
        assert call(wsb=size, **{**long, **kw}) == skg.E_INVALID_ARG, kw
    assert call(o=None, oq=ptr(800)) == skg.E_INVALID_ARG
    # the same cache with a small bound on its keys needs none
    assert skg.lib.skg_tree_attn_workspace(cache(skg, pages=1000), F32, 4, 2, 8, 2, 500, 200) == 0


def test_binding_refuses_host_tensors(skg):
    x, i = torch.zeros(2, 4, 128), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="on the GPU"):
        skg.qk_norm_rope(x, x, i, torch.zeros(64))
    with pytest.raises(ValueError, match="required"):
        skg.qk_norm_rope(None, None, i, torch.zeros(64))
    with pytest.raises(ValueError, match="on the GPU"):
        skg.KvCache(skg.KV_Q8_0, 4, 128, 16, torch.zeros(1), torch.zeros(1))
    with pytest.raises(skg.SkgError):
        skg.KvCache(skg.KV_Q8_0, 4, 100, 16, torch.zeros(1), torch.zeros(1))
    with pytest.raises(skg.SkgError):
        skg.kv_cache(skg.KV_Q8_0, 4, 128, 17, 4)
