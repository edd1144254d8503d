"""The operators between the QKV and the output projection of a decode layer:
their cases, inputs, plain forms and the framework's calls.

* ``rope``: per-head RMSNorm of queries and keys with the position rotation.
* ``cache``: keys and values quantised into a paged cache, and read back.
* ``attn``: attention of drafted tokens (a tree, or one token) over that cache.

``own`` chooses between the plain form (elementary torch operations in 32
bits, 64 where an angle or a rounding border needs them) and the framework's
entry points.

A cache buffer is [pages][heads][chunk] bytes; a chunk holds the codes of the
page's tokens ([page][row bytes]) and then, for q8_0 and q4_0, their fp16
scales ([page][D / 32]).  Within a row of NB = D / 32 blocks, q8_0 byte
2 NB c + 2 b + e is code + 128 of element 32 b + 2 c + e, q4_0 byte NB c + b
holds element 32 b + 2 c in its low and 32 b + 2 c + 1 in its high nibble
(code + 8), and bf16 rows are in order.
"""

import math
import random

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases ------------------------------------------------------------------

def _rope(name, T, hq, hk, d, rot, style, norm, dtype, fused, far):
    return dict(name=name, op="rope", T=T, hq=hq, hk=hk, d=d, rot=rot, style=style, norm=norm, dtype=dtype,
                fused=fused, far=far)


def _cache(name, fmt, T, R, heads, d, page, dtype):
    return dict(name=name, op="cache", fmt=fmt, T=T, R=R, heads=heads, d=d, page=page, dtype=dtype)


def _attn(name, fmt, B, draft, ctx, hq, hk, d, page, dtype):
    return dict(name=name, op="attn", fmt=fmt, B=B, draft=draft, ctx=ctx, hq=hq, hk=hk, d=d, page=page, dtype=dtype)


def listed():
    return [
        # one token of a Llama-2-7B-shaped layer (32 heads of 128), rotated in pairs
        _rope("rope 1 token", 1, 32, 32, 128, 128, "pairs", False, "f32", False, 4096),
        # eight drafted tokens of a model with grouped queries and normalised heads, in the fused QKV buffer
        _rope("rope 8 drafted, normed", 8, 32, 8, 128, 128, "halves", True, "f32", True, 32768),
        # the 512-token prompt of the framework's prefill product
        _rope("rope prompt 512", 512, 32, 32, 128, 128, "pairs", False, "f32", False, 4096),
        # a long prompt of odd length at far positions, bf16, half of each head rotated
        _rope("rope prompt 8191 bf16", 8191, 32, 8, 128, 64, "halves", True, "bf16", True, 1000000),
        # eight drafted tokens written and read back: latency
        _cache("cache 8 drafted q8_0", "q8_0", 8, 8, 32, 128, 16, "f32"),
        # a 512-token prompt written and read back whole
        _cache("cache prompt 512 q4_0", "q4_0", 512, 512, 32, 128, 64, "f32"),
        # a prompt's next piece written, its whole prefix read back
        _cache("cache prefix 16383 q8_0", "q8_0", 1000, 16383, 4, 256, 32, "bf16"),
        # the first tokens of an answer: latency
        _attn("attn 1 token, 37 keys q8_0", "q8_0", 1, 1, 37, 32, 32, 128, 16, "f32"),
        # a tree of eight at the full context of a Llama-2-7B-shaped layer
        _attn("attn tree 8, 4088 keys q8_0", "q8_0", 1, 8, 4088, 32, 32, 128, 32, "f32"),
        # a batch of answers of very different lengths, grouped queries, 4-bit cache
        _attn("attn batch 16 ragged q4_0", "q4_0", 16, 1, 8000, 32, 8, 128, 64, "f32"),
        # large trees over an unquantised cache
        _attn("attn trees of 61 bf16", "bf16", 4, 61, 6001, 32, 8, 128, 16, "bf16"),
        # one token over a very long document
        _attn("attn 1 token, 131071 keys q8_0", "q8_0", 1, 1, 131071, 64, 8, 128, 128, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = rng.choice([(32, 32), (32, 8), (64, 8), (40, 8), (28, 4), (16, 16), (8, 1), (14, 2), (5, 5)])
    d = rng.choice([64, 128, 128, 128, 256])
    op = rng.choice(["rope", "cache", "attn", "attn"])
    fmt = rng.choice(["q8_0", "q4_0", "bf16"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["f32", "bf16"])
    T = _log_int(rng, 1, 8191)
    if op == "rope":
        style, norm, fused = rng.choice(["pairs", "halves"]), rng.random() < 0.5, rng.random() < 0.5
        rot = rng.choice([d, d, d // 2])
        T = max(1, min(T, (8191 * 40 * 128 * 2) // ((heads[0] + heads[1]) * d * (4 if dtype == "f32" else 2))))
        c = _rope("", T, heads[0], heads[1], d, rot, style, norm, dtype, fused, rng.choice([4096, 32768, 1000000]))
    elif op == "cache":
        R = _log_int(rng, 1, 16383)
        rows = (17000 * 4 * 256) // (2 * heads[1] * d)
        c = _cache("", fmt, max(1, min(T, rows)), max(1, min(R, rows)), heads[1], d, page, dtype)
    else:
        B, draft, ctx = _log_int(rng, 1, 48), _log_int(rng, 1, 64), _log_int(rng, 1, 131071)
        most = 131072 * 8 * 128
        while B * (ctx + draft) * heads[1] * d > most or B * draft * (ctx + draft) * heads[0] * d > 61 * 24000 * 32 * 128:
            if ctx > 1:
                ctx = max(1, ctx * 2 // 3)
            else:
                B = max(1, B * 2 // 3)
        c = _attn("", fmt, B, draft, ctx, heads[0], heads[1], d, page, dtype)
    del c["name"]
    return c


def _lens(case):
    """Context lengths and drafted tokens of the sequences: the first has the
    most of both, the others anything down to an eighth of the context."""
    r = random.Random("%d %d %d" % (case["B"], case["ctx"], case["draft"]))
    ctx = [case["ctx"]] + [_log_int(r, max(1, case["ctx"] // 8), case["ctx"]) for _ in range(case["B"] - 1)]
    n = [case["draft"]] + [r.randint(1, case["draft"]) for _ in range(case["B"] - 1)]
    return ctx, n


def _row_bytes(fmt, d):
    """Bytes of one token's row of one head: codes, scales."""
    return {"bf16": (2 * d, 0), "q8_0": (d, d // 16), "q4_0": (d // 2, d // 16)}[fmt]


def work(case):
    es = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "rope":
        n = case["T"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 2 * n * es + 4 * case["T"] + 2 * case["rot"], "flops": n * (6 if case["norm"] else 3)}
    row = sum(_row_bytes(case["fmt"], case["d"]))
    if case["op"] == "cache":
        n = (case["T"] + case["R"]) * case["heads"] * 2
        return {"bytes": n * (case["d"] * es + row) + 8 * (case["T"] + case["R"]), "flops": n * case["d"] * 3}
    ctx, n = _lens(case)
    keys = sum(c + t for c, t in zip(ctx, n))
    pairs = sum(t * (c + t) for c, t in zip(ctx, n))
    return {"bytes": keys * case["hk"] * 2 * row + 2 * sum(n) * case["hq"] * case["d"] * es,
            "flops": 4 * pairs * case["hq"] * case["d"]}


# ---- the cache's encoding in elementary operations --------------------------

def _half_away(p):
    p = p.double()
    return torch.sign(p) * torch.floor(p.abs() + 0.5)


def _encode(fmt, x):
    """float32 [..., D] -> (code bytes [..., row], scale bytes [..., 2 D / 32] or None)."""
    lead, D = x.shape[:-1], x.shape[-1]
    if fmt == "bf16":
        return x.to(torch.bfloat16).contiguous().view(torch.uint8), None
    b = x.reshape(*lead, D // 32, 32)
    if fmt == "q8_0":
        d = b.abs().amax(-1, keepdim=True) / 127
    else:
        at = b.abs().argmax(-1, keepdim=True)
        d = b.gather(-1, at) / -8
    inv = torch.where(d != 0, 1 / d, torch.zeros_like(d))
    q = _half_away(b * inv)
    q = q.clamp(-127, 127) + 128 if fmt == "q8_0" else (q + 8).clamp(0, 15)
    q = q.to(torch.uint8).reshape(*lead, D // 32, 16, 2).transpose(-3, -2)  # [16][NB][2]
    q = q.reshape(*lead, D) if fmt == "q8_0" else (q[..., 0] | (q[..., 1] << 4)).reshape(*lead, D // 2)
    s = d[..., 0].clamp(-65504, 65504).to(torch.float16).contiguous().view(torch.uint8)
    return q.contiguous(), s


def _decode(fmt, codes, scales):
    """The inverse of _encode, as float32 [..., D]."""
    if fmt == "bf16":
        return codes.contiguous().view(torch.bfloat16).float()
    lead, nb = codes.shape[:-1], scales.shape[-1] // 2
    if fmt == "q8_0":
        q = codes.reshape(*lead, 16, nb, 2).float() - 128
    else:
        c = codes.reshape(*lead, 16, nb)
        q = torch.stack((c & 15, c >> 4), -1).float() - 8
    s = scales.contiguous().view(torch.float16).float()
    return (q.transpose(-3, -2) * s[..., None, None]).reshape(*lead, nb * 32)


def _planes(case, buf):
    """Views of a cache buffer: codes [pages, heads, page, row], scales [pages, heads, page, 2 NB]."""
    row, sc = _row_bytes(case["fmt"], case["d"])
    page, split = case["page"], case["page"] * row
    return (buf[:, :, :split].unflatten(-1, (page, row)), buf[:, :, split:].unflatten(-1, (page, sc)) if sc else None)


def _filled(case, pages, heads, gen):
    """A cache buffer that holds rows of normally distributed values."""
    page, d = case["page"], case["d"]
    x = torch.randn((pages, heads, page, d), device="cuda", generator=gen)
    codes, scales = _encode(case["fmt"], x)
    parts = [codes.reshape(pages, heads, -1)] + ([] if scales is None else [scales.reshape(pages, heads, -1)])
    return torch.cat(parts, -1).contiguous()


# ---- inputs -------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, gen)
    if case["op"] == "cache":
        return _prepare_cache(case, gen)
    return _prepare_attn(case, gen, rng)


def _prepare_rope(case, gen):
    T, hq, hk, d, dt = case["T"], case["hq"], case["hk"], case["d"], _DT[case["dtype"]]
    if case["fused"]:  # q, k and v of a token side by side, as one projection writes them
        qkv = torch.randn((T, hq + 2 * hk, d), device="cuda", generator=gen).to(dt)
        q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    else:
        q = torch.randn((T, hq, d), device="cuda", generator=gen).to(dt)
        k = torch.randn((T, hk, d), device="cuda", generator=gen).to(dt)
    start = torch.randint(0, case["far"] - T + 1 if case["far"] > T else 1, (1,), device="cuda", generator=gen)
    pos = (start + torch.arange(T, device="cuda")).to(torch.int32)
    inv_freq = (10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])).float()
    gains = (1 + 0.1 * torch.randn((2, d), device="cuda", generator=gen)) if case["norm"] else (None, None)
    return dict(case=case, q=q, k=k, pos=pos, inv_freq=inv_freq, gq=gains[0], gk=gains[1])


def _prepare_cache(case, gen):
    T, R, heads, d, page = case["T"], case["R"], case["heads"], case["d"], case["page"]
    pages = -(-max(T, R) // page) + 3
    order = torch.randperm(pages, device="cuda", generator=gen)

    def slots(n, first):
        at = first + torch.arange(n, device="cuda")
        return order[at // page] * page + at % page

    k = torch.randn((T, heads, d), device="cuda", generator=gen).to(_DT[case["dtype"]])
    v = torch.randn((T, heads, d), device="cuda", generator=gen).to(_DT[case["dtype"]])
    return dict(case=case, kc=_filled(case, pages, heads, gen), vc=_filled(case, pages, heads, gen), k=k, v=v,
                write=slots(T, max(T, R) - T + 5), read=slots(R, max(T, R) - R + 5))


def _prepare_attn(case, gen, rng):
    B, hq, hk, d, page = case["B"], case["hq"], case["hk"], case["d"], case["page"]
    ctx, n = _lens(case)
    width = max(-(-(c + t) // page) for c, t in zip(ctx, n))
    used = [-(-(c + t) // page) for c, t in zip(ctx, n)]
    pages = sum(used) + 1
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).cpu()
    table, at = torch.zeros((B, width), dtype=torch.int32), 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    mask, cu = [], [0]
    for t in n:  # a random tree: every node sees its ancestors and itself
        tree = []
        for i in range(t):
            parent = rng.randint(max(-1, i - 8), i - 1)
            tree.append((1 << i) | (tree[parent] if parent >= 0 else 0))
        mask += tree
        cu.append(cu[-1] + t)
    mask = torch.tensor([m - (1 << 64) if m >> 63 else m for m in mask], dtype=torch.int64)
    q = (2 * torch.randn((cu[-1], hq, d), device="cuda", generator=gen)).to(_DT[case["dtype"]])
    return dict(case=case, kc=_filled(case, pages, hk, gen), vc=_filled(case, pages, hk, gen), q=q,
                table=table.cuda(), ctx=torch.tensor(ctx, dtype=torch.int32).cuda(),
                cu=torch.tensor(cu, dtype=torch.int32).cuda(), mask=mask.cuda(), scale=1 / math.sqrt(d))


# ---- one pass -----------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rope": _plain_rope, "cache": _plain_cache, "attn": _plain_attn}[op](state)


def _own(state, op):
    import skinny_gemm_decode_amd as skg

    case = state["case"]
    if op == "rope":
        return skg.qk_norm_rope(state["q"], state["k"], state["pos"], state["inv_freq"], gq=state["gq"],
                                gk=state["gk"], eps=1e-6, norm=case["norm"], interleaved=case["style"] == "pairs")
    if "cache" not in state:  # the handle, which a program makes once for its buffers
        fmt = {"bf16": skg.KV_BF16, "q8_0": skg.KV_Q8_0, "q4_0": skg.KV_Q4_0}[case["fmt"]]
        state["cache"] = skg.KvCache(fmt, case["heads" if op == "cache" else "hk"], case["d"], case["page"],
                                     state["kc"], state["vc"])
    if op == "cache":
        skg.kv_store(state["cache"], state["k"], state["v"], state["write"])
        return skg.kv_load(state["cache"], state["read"], dtype=_DT[case["dtype"]])
    return skg.tree_attn(state["cache"], state["q"], state["table"], state["ctx"], cu=state["cu"],
                         mask=state["mask"], max_draft=case["draft"], scale=state["scale"])


def _plain_rope(state):
    case = state["case"]
    half, rot = case["rot"] // 2, case["rot"]
    angle = state["pos"].double()[:, None] * state["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, g):
        y = x.float()
        if case["norm"]:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * g
        t = y[..., :rot]
        if case["style"] == "pairs":
            a, b = t[..., 0::2], t[..., 1::2]
            t = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = t[..., :half], t[..., half:]
            t = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((t, y[..., rot:]), -1).to(x.dtype)

    return turned(state["q"], state["gq"]), turned(state["k"], state["gk"])


def _plain_cache(state):
    case = state["case"]
    fmt, page, dt = case["fmt"], case["page"], _DT[case["dtype"]]

    def through(buf, x):
        codes, scales = _planes(case, buf)
        c, s = _encode(fmt, x.float())
        w, r = state["write"], state["read"]
        codes[w // page, :, w % page] = c
        if s is not None:
            scales[w // page, :, w % page] = s
        return _decode(fmt, codes[r // page, :, r % page], None if s is None else scales[r // page, :, r % page]).to(dt)

    return through(state["kc"], state["k"]), through(state["vc"], state["v"])


def _plain_attn(state):
    case, q, ctx, cu = state["case"], state["q"], state["ctx"].long(), state["cu"].long()
    hq, hk, d = case["hq"], case["hk"], case["d"]
    B, n = case["B"], case["draft"]
    pages = state["table"].long()

    def keys(buf):  # [B, heads, keys, d]
        codes, scales = _planes(case, buf)
        x = _decode(case["fmt"], codes[pages], None if scales is None else scales[pages])
        return x.permute(0, 2, 1, 3, 4).reshape(B, hk, -1, d)

    k, v = keys(state["kc"]), keys(state["vc"])
    tok = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[seq]
    qp = q.new_zeros((B, n, hq, d), dtype=torch.float32)
    qp[seq, i] = q.float()
    mp = state["mask"].new_zeros((B, n))
    mp[seq, i] = state["mask"]
    qp = qp.reshape(B, n, hk, hq // hk, d).transpose(1, 2).reshape(B, hk, -1, d)
    s = qp @ k.transpose(-1, -2) * state["scale"]
    at = torch.arange(k.shape[2], device=q.device) - ctx[:, None]  # place among the drafted
    sees = (at < 0)[:, None] | ((at >= 0) & (at < 64))[:, None] & ((mp[..., None] >> at.clamp(0, 63)[:, None]) & 1).bool()
    sees = sees[:, None, :, None].expand(B, hk, n, hq // hk, -1).reshape(s.shape)
    s = s.masked_fill(~sees, -math.inf)
    e = torch.where(sees, torch.exp(s - s.amax(-1, keepdim=True)), torch.zeros_like(s))
    o = e @ v / e.sum(-1, keepdim=True)
    o = o.reshape(B, hk, n, hq // hk, d).transpose(1, 2).reshape(B, n, hq, d)
    return o[seq, i].to(q.dtype)


# ---- the definitions in 64 bits, written apart from the forms above -----------

def exact(case, seed):
    state = prepare(case, seed)
    return {"rope": _exact_rope, "cache": _exact_cache, "attn": _exact_attn}[case["op"]](case, state)


def _exact_rope(case, state):
    rot = case["rot"]
    phase = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                        torch.outer(state["pos"].double(), state["inv_freq"].double()))

    def one(x, g):
        y = x.double()
        if case["norm"]:
            y = y * torch.rsqrt(y.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6) * g.double()
        pairs = y[..., :rot].unflatten(-1, (rot // 2, 2) if case["style"] == "pairs" else (2, rot // 2))
        if case["style"] != "pairs":
            pairs = pairs.transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase[:, None])
        if case["style"] != "pairs":
            z = z.transpose(-1, -2)
        y[..., :rot] = z.reshape(*y.shape[:-1], rot)
        return y

    return one(state["q"], state["gq"]), one(state["k"], state["gk"])


def _element_places(d):
    """Place in a row's order of (c, b, e) of each element 32 b + 2 c + e."""
    nb = d // 32
    at = np.empty(d, dtype=np.int64)
    for c in range(16):
        for b in range(nb):
            for e in (0, 1):
                at[32 * b + 2 * c + e] = 2 * nb * c + 2 * b + e
    return at


def _exact_rows(case, chunks):
    """Values of the rows in chunks [n, heads, chunk bytes] as float64 [n, heads, page, d]."""
    fmt, d, page = case["fmt"], case["d"], case["page"]
    n, heads, _ = chunks.shape
    if fmt == "bf16":
        return chunks.contiguous().view(torch.bfloat16).reshape(n, heads, page, d).double()
    at = torch.from_numpy(_element_places(d)).to(chunks.device)
    size = d if fmt == "q8_0" else d // 2
    codes = chunks[..., :page * size].reshape(n, heads, page, size)
    scale = chunks[..., page * size:].contiguous().view(torch.float16).reshape(n, heads, page, d // 32).double()
    if fmt == "q8_0":
        q = codes[..., at].double() - 128.0
    else:
        q = torch.bitwise_right_shift(codes[..., at // 2], (4 * (at % 2)).to(torch.uint8)).bitwise_and(15).double() - 8.0
    return q * scale.repeat_interleave(32, -1)


def _exact_cache(case, state):
    """The stored values by the quantiser's definition, whose steps are single
    binary32 operations; rows that no write touched are the cache's own."""
    fmt, page = case["fmt"], case["page"]
    f32 = np.float32

    def quantised(x):
        if fmt == "bf16":
            return x.to(torch.bfloat16).double().cpu().numpy()
        b = x.float().cpu().numpy().reshape(*x.shape[:-1], -1, 32)
        if fmt == "q8_0":
            d = np.abs(b).max(-1, keepdims=True) / f32(127)
        else:
            d = np.take_along_axis(b, np.abs(b).argmax(-1)[..., None], -1) / f32(-8)
        with np.errstate(divide="ignore"):
            inv = np.where(d == 0, f32(0), f32(1) / d)
        p = (b * inv).astype(np.float64)
        q = np.trunc(p + np.copysign(0.5, p))
        q = np.clip(q, -127, 127) if fmt == "q8_0" else np.clip(q, -8, 7)
        return (q * np.clip(d, -65504, 65504).astype(np.float16).astype(np.float64)).reshape(x.shape)

    def one(buf, x):
        r, w = state["read"].cpu().numpy(), state["write"].cpu().numpy()
        whole = _exact_rows(case, buf)[torch.from_numpy(r // page).cuda(), :, torch.from_numpy(r % page).cuda()].cpu().numpy()
        new, place = quantised(x), {int(s): j for j, s in enumerate(w)}
        for j, s in enumerate(r):
            if int(s) in place:
                whole[j] = new[place[int(s)]]
        return torch.from_numpy(whole)

    return one(state["kc"], state["k"]), one(state["vc"], state["v"])


def _exact_attn(case, state):
    hq, hk, d = case["hq"], case["hk"], case["d"]
    ctx, n = _lens(case)
    out, first = [], 0
    for b in range(case["B"]):
        total = ctx[b] + n[b]
        pages = state["table"][b, :-(-total // case["page"])].long()
        k, v = (_exact_rows(case, buf[pages]).permute(1, 0, 2, 3).reshape(hk, -1, d)[:, :total] for buf in (state["kc"], state["vc"]))
        bits = [int(m) for m in state["mask"][first:first + n[b]]]
        sees = torch.ones((n[b], total), dtype=torch.bool)
        for i, m in enumerate(bits):
            for j in range(n[b]):
                sees[i, ctx[b] + j] = bool((m >> j) & 1)
        sees = sees.cuda()
        for i in range(n[b]):
            q = state["q"][first + i].double().reshape(hk, hq // hk, d)
            s = torch.matmul(q, k.transpose(1, 2)) * state["scale"]
            p = torch.softmax(torch.where(sees[i], s, torch.full_like(s, -math.inf)), -1)
            out.append(torch.matmul(p, v).reshape(hq, d))
        first += n[b]
    return torch.stack(out)
