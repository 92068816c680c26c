"""What is measured of the operators around a decoder layer's products: keys and
values appended to the 4-bit cache with norms and rotation on the way, attention
over that cache with a sliding window and visible first tokens, the residual's
addition with a norm to 8 bits, and the gated activation to 8 bits.

`own` False computes each operator from elementary torch operations in 32 bits
(64 where a sum decides a border between two codes); `own` True makes the
library's calls.  Definitions:
  append   v = x / sqrt(mean(x^2) + eps) w, rotation of its first `rot` values;
           q rounded once, k and v stored per 64 values as
             z = f16(min), s = f16((max - min) / 15), c = clip(rint((x - z) / s), 0, 15)
  window   token at position p sees j <= p with j < sinks or j > p - window
  norm     h = x + r, y = (h f32(1 / sqrt(mean(h^2) + eps))) w
  gated    y = act(gate) up
  8 bits   s = max|y| / 127 (1 for a row of zeros), c = clip(rint(y / s), -127, 127)
"""
import math
import random

import torch

own = False
DEV = "cuda:0"
GROUP = 64
EPS = 1e-6
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # a decode step's new token of one chat, 1B heads, as slices of the fused q|k|v product
        dict(name="append_1tok", kind="append", dtype="f16", out="f16", tokens=1, hq=32, hkv=8, d=64, rot=64,
             pairs="half", norm=False, page=64, run=1),
        # the new tokens of a serving batch, 3B heads with norms
        dict(name="append_batch", kind="append", dtype="bf16", out="bf16", tokens=48, hq=24, hkv=8, d=128, rot=128,
             pairs="half", norm=True, page=64, run=1),
        # an odd chunk, partial rotation of neighbouring pairs, fp32 products, in runs that begin inside pages
        dict(name="append_odd_partial", kind="append", dtype="f32", out="f16", tokens=777, hq=20, hkv=5, d=64, rot=32,
             pairs="neighbour", norm=True, page=32, run=100),
        # a prompt chunk, 3B heads with norms
        dict(name="append_chunk", kind="append", dtype="bf16", out="bf16", tokens=8192, hq=24, hkv=8, d=128, rot=128,
             pairs="half", norm=True, page=64, run=8192),
        # one token of a long chat that keeps 4096 tokens and the first four, 1B heads
        dict(name="window_1tok", kind="window", dtype="f16", hq=32, hkv=8, d=64, page=64, seqs=1, q=1, ctx=32768,
             window=4096, sinks=4, mix=0),
        # a serving batch of uneven lengths with an idle place, 3B heads
        dict(name="window_batch_ragged", kind="window", dtype="bf16", hq=24, hkv=8, d=128, page=64, seqs=48, q=1,
             ctx=12000, window=2048, sinks=4, mix=1),
        # a chunk of a long prompt, 1B heads, a window and a few sinks that both end inside a block
        dict(name="window_chunk_1b", kind="window", dtype="f16", hq=32, hkv=8, d=64, page=128, seqs=1, q=2048, ctx=8192,
             window=1000, sinks=20, mix=0),
        # several prompts of uneven lengths from their first token, 3B heads, no sinks
        dict(name="window_prompts_ragged", kind="window", dtype="bf16", hq=24, hkv=8, d=128, page=64, seqs=5, q=1777,
             ctx=1777, window=512, sinks=0, mix=3),
        # one token between two products, 1B width
        dict(name="norm_1tok", kind="norm", dtype="f16", res="f32", tokens=1, k=2048, pad=0),
        # a prompt chunk, 16-bit residual
        dict(name="norm_chunk", kind="norm", dtype="f16", res="bf16", tokens=8192, k=4096, pad=0),
        # one token's gate|up product, 1B width
        dict(name="gated_1tok", kind="gated", dtype="f16", act="silu", tokens=1, k=8192, fused=True),
        # a prompt chunk's gate|up product, 1B width
        dict(name="gated_chunk", kind="gated", dtype="f16", act="silu", tokens=8192, k=8192, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "window", "window", "norm", "gated"])
    d, hkv = rng.choice([64, 128]), rng.choice([1, 2, 5, 8, 16])
    if kind == "append":
        hq = hkv * rng.choice([1, 2, 3, 4])
        dt = rng.choice(["f16", "bf16", "f32"])
        tokens = min(_log(rng, 1, 8192), 8192 * 40 * 128 * 2 // ((hq + 2 * hkv) * d * SIZE[dt]))
        return dict(kind=kind, dtype=dt, out=rng.choice(["f16", "bf16"]), tokens=tokens, hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, 16, 48]), pairs=rng.choice(["half", "neighbour"]),
                    norm=rng.choice([True, False]), page=rng.choice([32, 64, 128, 256]),
                    run=rng.choice([1, 3, 100, tokens]))
    if kind == "window":
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        hq = hkv * group if hkv * group <= 48 else hkv
        mode = rng.choice(["one", "one", "few", "chunk"])
        window, sinks = _log(rng, 1, 8192), rng.choice([0, 1, 4, 33, 200])
        if mode == "chunk":
            seqs, q = rng.choice([1, 1, 2, 3]), _log(rng, 17, 2048)
            ctx = min(q + _log(rng, 1, 8192), 8192)
            while seqs * q * min(ctx, window + sinks) * hq * d > 2048 * 1020 * 32 * 64:
                q, seqs = max(1, q // 2), max(1, seqs - 1)
        else:
            q = 1 if mode == "one" else rng.randint(2, 9)
            seqs = _log(rng, 1, 64)
            budget = 48 * 2052 * 8 * 128 // (hkv * d)  # visible tokens of the largest listed batch
            window = max(1, min(window, budget // seqs - 200))
            ctx = max(q, _log(rng, 1, 32768 if seqs == 1 else 12000))
        return dict(kind=kind, dtype=rng.choice(["f16", "bf16"]), hq=hq, hkv=hkv, d=d, page=rng.choice([32, 64, 128]),
                    seqs=seqs, q=q, ctx=ctx, window=window, sinks=sinks, mix=0 if seqs == 1 else rng.randint(1, 10 ** 6))
    dt = rng.choice(["f16", "bf16", "f32"])
    if kind == "norm":
        k = _log(rng, 64, 16384)
        k -= k % rng.choice([1, 1, 8, 64])
        return dict(kind=kind, dtype=dt, res=rng.choice(["", "f32", "f16", "bf16"]), k=k,
                    tokens=max(1, min(_log(rng, 1, 8192), 8192 * 2048 // k)), pad=rng.choice([0, 0, 8, 5]))
    k = _log(rng, 64, 28672)
    k -= k % rng.choice([1, 1, 8, 64])
    return dict(kind=kind, dtype=dt, act=rng.choice(["silu", "gelu_tanh"]), k=k,
                tokens=max(1, min(_log(rng, 1, 8192), 8192 * 4096 // k)), fused=rng.choice([True, False]))


# ---------------------------------------------------------------- inputs ----

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _lens(case):
    """New and cached tokens (new ones included) of each sequence; fixed by the
    case, so that its work is too."""
    n, q, ctx = case["seqs"], case["q"], case["ctx"]
    if case["mix"] == 0 or n == 1:
        return [q] * n, [ctx] * n
    rng = random.Random(case["mix"])
    qs, ls = [], []
    for i in range(n):
        qi = q if q < 10 else rng.randint(max(1, q // 4), q)
        li = qi if q == ctx else max(qi, int(ctx * rng.uniform(0.1, 1.0)))
        qs.append(qi)
        ls.append(li)
    qs[0], ls[0] = q, ctx
    if n >= 4 and q < 10:
        ls[-1] = 0  # an idle place of the batch: its rows see nothing
    return qs, ls


def _append_inputs(case, seed):
    g = _generator(seed)
    t, hq, hkv, d, rot, page = (case[x] for x in ("tokens", "hq", "hkv", "d", "rot", "page"))
    qkv = _randn(g, t, hq + 2 * hkv, d)
    # keys come with channels that have a mean of their own
    sign = 2.0 * torch.randint(0, 2, (hkv, d), generator=g, device=DEV) - 1.0
    mean = sign * (0.8 + 0.4 * torch.rand(hkv, d, generator=g, device=DEV))
    qkv[:, hq:hq + hkv] = 2.0 * (mean + 0.25 * qkv[:, hq:hq + hkv])
    qkv = qkv.to(DT[case["dtype"]])
    maxpos = 32768
    start = torch.randint(0, maxpos, (2,), generator=g, device=DEV)  # two sequences at places of their own
    i = torch.arange(t, device=DEV)
    pos = (i + torch.where(i < (t + 1) // 2, start[0], start[1])) % maxpos
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    ang = torch.arange(maxpos, dtype=torch.float64, device=DEV).unsqueeze(1) * inv
    # runs of consecutive tokens, each from a place of its own inside its first page
    run = min(case["run"], t)
    runs = (t + run - 1) // run
    per = (run + page - 1) // page + 1
    perm = torch.randperm(runs * per, generator=g, device=DEV)
    at = torch.randint(0, page, (runs,), generator=g, device=DEV) if run < t else torch.zeros(runs, dtype=torch.long, device=DEV)
    where = at[i // run] + i % run
    slots = perm[(i // run) * per + where // page] * page + where % page
    wq = wk = None
    if case["norm"]:
        wq, wk = 1.0 + 0.2 * _randn(g, d), 1.0 + 0.1 * _randn(g, d)
    return dict(case=case, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cos=ang.cos().float(),
                sin=ang.sin().float(), pos=pos, slots=slots, pages=runs * per, wq=wq, wk=wk)


def _window_inputs(case, seed):
    g = _generator(seed)
    qs, ls = _lens(case)
    hkv, d, dtype, page = case["hkv"], case["d"], DT[case["dtype"]], case["page"]
    need = [(length + page - 1) // page for length in ls]
    total = sum(need) + 1
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(ls), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = perm[at:at + c]
        at += c
    q = (_randn(g, sum(qs), case["hq"], d) * 1.2).to(dtype)
    chan = torch.rand(3, hkv, d, generator=g, device=DEV)
    k = (_randn(g, total * page, hkv, d) * (0.3 + chan[0]) + 2.0 * (chan[1] - 0.5)).to(dtype)
    v = (_randn(g, total * page, hkv, d) * (0.2 + chan[2])).to(dtype)
    return qs, ls, table, total, q, k, v


def _row_inputs(case, seed):
    g = _generator(seed)
    t, k, dt = case["tokens"], case["k"], DT[case["dtype"]]
    if case["kind"] == "gated":
        gu = _randn(g, t, 2 * k).to(dt)
        gate, up = gu[:, :k], gu[:, k:]
        return (gate, up) if case["fused"] else (gate.contiguous(), up.contiguous())
    # hidden states with a few channels far larger than the rest
    big = torch.where(torch.rand(k, generator=g, device=DEV) < 0.005, 20.0, 1.0)
    x = (_randn(g, t, k + case["pad"])).to(dt)[:, :k]
    r = (_randn(g, t, k) * big).to(DT[case["res"]]) if case["res"] else None
    return x, r, 1.0 + 0.2 * _randn(g, k)


def _plain_cache(slots, hkv, d):
    e = dict(dtype=torch.uint8, device=DEV)
    f = dict(dtype=torch.float16, device=DEV)
    return {w + p: (torch.zeros(slots, hkv, d // 2, **e) if p == "c" else torch.zeros(slots, hkv, d // GROUP, **f))
            for w in "kv" for p in "csz"}


def _quantise(x):
    """x [n, heads, d] -> codes uint8 [n, heads, d], s and z f16 [n, heads, d / 64]"""
    n, h, d = x.shape
    y = x.float().reshape(n, h, d // GROUP, GROUP)
    lo, hi = y.amin(-1), y.amax(-1)
    z = lo.clamp(-65504.0, 65504.0).to(torch.float16)
    fifteen = torch.full_like(lo, 15.0)  # a tensor: the quotient is one IEEE division
    s = ((hi - lo) / fifteen).clamp(max=65504.0).to(torch.float16)
    sf, zf = s.float().unsqueeze(-1), z.float().unsqueeze(-1)
    c = torch.where(sf > 0, torch.round((y - zf) / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(y))
    return c.clamp(0, 15).to(torch.uint8).view(n, h, d), s, z


def _plain_write(cache, k, v, slots):
    for w, x in (("k", k), ("v", v)):
        c, s, z = _quantise(x)
        cache[w + "c"][slots] = c[..., 0::2] | (c[..., 1::2] << 4)  # two codes to a byte
        cache[w + "s"][slots] = s
        cache[w + "z"][slots] = z


def _plain_read(cache, slots):
    res = []
    for w in "kv":
        b, s, z = cache[w + "c"][slots], cache[w + "s"][slots], cache[w + "z"][slots]
        y = torch.stack((b & 15, b >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
        res.append((z.float().unsqueeze(-1) + s.float().unsqueeze(-1) * y).flatten(-2))
    return res


def _new_cache(pages, page, hkv, d):
    if own:
        from ultra_bit_weight_amd import sherry

        return sherry.Kv4Cache(pages, page, hkv, d, device=DEV)
    return _plain_cache(pages * page, hkv, d)


def _fill(cache, k, v):
    slots = torch.arange(k.shape[0], device=DEV)
    if own:
        from ultra_bit_weight_amd import sherry

        sherry.kv4_write(cache, k, v, slots)
    else:
        _plain_write(cache, k, v, slots)


def _prepare_window(case, seed):
    qs, ls, table, total, q, k, v = _window_inputs(case, seed)
    page, sinks, window = case["page"], case["sinks"], case["window"]
    cache = _new_cache(total, page, case["hkv"], case["d"])
    _fill(cache, k, v)
    st = dict(case=case, cache=cache, q=q, table=table, scale=case["d"] ** -0.5, qs=qs, ls=ls,
              lens=torch.tensor(ls, dtype=torch.int32, device=DEV),
              cu=torch.tensor([sum(qs[:i]) for i in range(len(qs) + 1)], dtype=torch.int32, device=DEV))
    if own:
        from ultra_bit_weight_amd import sherry

        st["out"] = torch.empty_like(q)
        st["lse"] = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=DEV)
        st["ws"] = sherry.kv4_attn_workspace(cache, q.shape[0], q.shape[1], len(ls), max(qs), max(ls), window=window,
                                             sinks=sinks)
        return st
    # the plain form's plan: each sequence's visible tokens and rows, padded to the batch
    js = []
    for n, length in zip(qs, ls):
        first = max(0, length - n - window + 1)
        js.append(list(range(min(sinks, first, length))) + list(range(min(first, length), length)))
    wide, most = max(1, max(len(j) for j in js)), max(qs)
    tok = torch.tensor([j + [1 << 30] * (wide - len(j)) for j in js], device=DEV)
    seq = torch.arange(len(ls), device=DEV).unsqueeze(1)
    there = tok < (1 << 30)
    safe = torch.where(there, tok, 0)
    st["slots"] = torch.where(there, table[seq, safe // page].long() * page + safe % page, 0)
    i = torch.arange(most, device=DEV).unsqueeze(0)
    n, length = torch.tensor(qs, device=DEV).unsqueeze(1), torch.tensor(ls, device=DEV).unsqueeze(1)
    st["tok"] = tok
    st["pos"] = torch.where(i < n, length - n + i, -1)
    st["row"] = torch.where(i < n, st["cu"][:-1].long().unsqueeze(1) + i, 0)
    st["live"] = i < n
    return st


def prepare(case, seed):
    if case["kind"] == "window":
        return _prepare_window(case, seed)
    if case["kind"] == "append":
        st = _append_inputs(case, seed)
        st["cache"] = _new_cache(st["pages"], case["page"], case["hkv"], case["d"])
        st["q_out"] = torch.empty(st["q"].shape, dtype=DT[case["out"]], device=DEV)
        st["k_out"], st["v_out"] = (torch.empty(st["k"].shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        return st
    t, k = case["tokens"], case["k"]
    ins = _row_inputs(case, seed)
    st = dict(case=case, ins=ins, codes=torch.empty(t, k, dtype=torch.int8, device=DEV),
              scale=torch.empty(t, dtype=torch.float32, device=DEV),
              values=torch.empty(t, k, dtype=torch.bfloat16, device=DEV))
    if case["kind"] == "norm" and ins[1] is not None:
        st["sum"] = torch.empty_like(ins[1])
    return st


# ------------------------------------------------------------------ runs ----

def _run_window(st):
    q, case = st["q"], st["case"]
    if own:
        from ultra_bit_weight_amd import sherry

        sherry.kv4_attn(st["cache"], q, st["table"], st["lens"], cu_q=st["cu"], max_q=max(st["qs"]), max_kv=max(st["ls"]),
                        scale=st["scale"], out=st["out"], lse=st["lse"], workspace=st["ws"], window=case["window"],
                        sinks=case["sinks"])
        return {"out": st["out"], "lse": st["lse"]}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    grp = hq // hkv
    seqs, wide = st["slots"].shape
    most = st["row"].shape[1]
    k, v = (x.view(seqs, wide, hkv, d) for x in _plain_read(st["cache"], st["slots"].flatten()))
    x = q[st["row"]].float().view(seqs, most, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, grp * most, d)
    s = torch.matmul(x, k.permute(0, 2, 3, 1).contiguous()) * st["scale"]
    tok, pos = st["tok"].unsqueeze(1), st["pos"].unsqueeze(2)
    seen = (tok <= pos) & ((tok < case["sinks"]) | (tok > pos - case["window"]))  # [seqs, most, wide]
    s.view(seqs, hkv, grp, most, wide).masked_fill_(~seen[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3).contiguous()) / torch.where(total > 0, total, 1.0)
    o = o.view(seqs, hkv, grp, most, d).permute(0, 3, 1, 2, 4).reshape(seqs, most, hq, d)
    lse = (m + torch.log(total)).view(seqs, hkv, grp, most).permute(0, 3, 1, 2).reshape(seqs, most, hq)
    return {"out": o[st["live"]].to(q.dtype), "lse": lse[st["live"]]}


def _run_append(st):
    case, cache = st["case"], st["cache"]
    if own:
        from ultra_bit_weight_amd import sherry

        sherry.kv4_append(cache, st["q"], st["k"], st["v"], st["cos"], st["sin"], st["pos"], st["slots"],
                          q_weight=st["wq"], k_weight=st["wk"], eps=EPS, interleaved=case["pairs"] == "neighbour",
                          q_out=st["q_out"])
        sherry.kv4_read(cache, st["slots"], k_out=st["k_out"], v_out=st["v_out"])
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    rot = case["rot"]
    cos, sin = st["cos"][st["pos"]].unsqueeze(1), st["sin"][st["pos"]].unsqueeze(1)

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        y = x[..., :rot]
        if case["pairs"] == "neighbour":
            a, b = y[..., 0::2], y[..., 1::2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((y, x[..., rot:]), -1)

    _plain_write(cache, turned(st["k"], st["wk"]), st["v"], st["slots"])
    k, v = _plain_read(cache, st["slots"])
    return {"q": turned(st["q"], st["wq"]).to(DT[case["out"]]), "k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _to_8_bits(y):
    top = y.abs().amax(-1, keepdim=True)
    s = torch.where(top == 0, 1.0, top / torch.full_like(top, 127.0))
    return torch.round(y / s).clamp(-127, 127), s.squeeze(-1)


def _values(st):  # what the 8-bit codes stand for
    return torch.mul(st["codes"], st["scale"].unsqueeze(1), out=st["values"])


def _run_norm(st):
    x, r, w = st["ins"]
    if own:
        from ultra_bit_weight_amd import sherry

        sherry.rms_norm_quant(x, w, residual=r, eps=EPS, residual_out=st.get("sum"), q_out=st["codes"],
                              scale_out=st["scale"])
        return {"values": _values(st), "scale": st["scale"], "residual": st.get("sum")}
    h = x.float() if r is None else x.float() + r.float()
    inv = torch.rsqrt(h.double().square().mean(-1, keepdim=True) + EPS).float()
    c, s = _to_8_bits(h * inv * w)
    return {"values": (c * s.unsqueeze(1)).to(torch.bfloat16), "scale": s,
            "residual": None if r is None else h.to(r.dtype)}


def _run_gated(st):
    gate, up = st["ins"]
    if own:
        from ultra_bit_weight_amd import sherry

        sherry.gated_quant(gate, up, activation=st["case"]["act"], q_out=st["codes"], scale_out=st["scale"])
        return {"values": _values(st), "scale": st["scale"]}
    g = gate.float()
    if st["case"]["act"] == "silu":
        a = g / (1.0 + torch.exp(-g))
    else:
        a = 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))
    c, s = _to_8_bits(a * up.float())
    return {"values": (c * s.unsqueeze(1)).to(torch.bfloat16), "scale": s}


def run(state):
    return {"window": _run_window, "append": _run_append, "norm": _run_norm,
            "gated": _run_gated}[state["case"]["kind"]](state)


# ------------------------------------------------------------------ work ----

def _row_bytes(hkv, d):  # a cached token: 4-bit K and V, and f16 scale and zero point per 64 values
    return hkv * (d + 8 * (d // GROUP))


def work(case):
    if case["kind"] in ("norm", "gated"):
        t, k = case["tokens"], case["k"]
        if case["kind"] == "gated":
            return {"bytes": t * k * (2 * SIZE[case["dtype"]] + 1) + 4 * t, "flops": 8 * t * k}
        res = 2 * SIZE[case["res"]] if case["res"] else 0
        return {"bytes": t * k * (SIZE[case["dtype"]] + res + 1) + 4 * t + 4 * k, "flops": 7 * t * k}
    hkv, hq, d = case["hkv"], case["hq"], case["d"]
    if case["kind"] == "append":
        t, size = case["tokens"], SIZE[case["dtype"]]
        packed = t * _row_bytes(hkv, d)
        byts = t * hq * d * (size + SIZE[case["out"]]) + 2 * t * hkv * d * size + packed
        byts += packed + 2 * t * hkv * d * 2  # read back
        return {"bytes": byts + t * (4 * case["rot"] + 24) + (8 * d if case["norm"] else 0),
                "flops": t * ((hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0)) + 16 * hkv * d)}
    qs, ls = _lens(case)
    window, sinks = case["window"], case["sinks"]
    pairs = cached = 0
    for n, length in zip(qs, ls):
        for p in range(length - n, length):
            if p >= 0:
                lo = max(0, p - window + 1)
                pairs += p + 1 - lo + min(sinks, lo)
        first = max(0, length - n - window + 1)
        cached += max(0, length - first) + min(sinks, first, length)
    t = sum(qs)
    byts = cached * _row_bytes(hkv, d) + 2 * t * hq * d * SIZE[case["dtype"]] + 4 * t * hq
    return {"bytes": byts + 4 * (cached // case["page"] + 2 * len(ls) + 1), "flops": 4 * d * hq * pairs}


# ----------------------------------------------------------- the 64-bit definition

def _exact_stored(x):
    """The values that the cache stands for: z and s in f16 as the format has
    them, the code from its 64-bit quotient."""
    n, h, d = x.shape
    y = x.double().reshape(n, h, -1, GROUP)
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    z = lo.clamp(-65504, 65504).half().double()
    s = ((hi - lo) / 15).clamp(max=65504).half().double()
    c = torch.where(s > 0, ((y - z) / s).round().clamp(0, 15), torch.zeros_like(y))
    return (z + s * c).reshape(n, h, d)


def _exact_window(case, seed):
    qs, ls, table, _, q, k, v = _window_inputs(case, seed)
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    # the quantiser's steps are 32-bit ones: its input is, too
    kk, vv = _exact_stored32(k), _exact_stored32(v)
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for i, (n, length) in enumerate(zip(qs, ls)):
        if length:
            j = torch.arange(length, device=DEV)
            p = torch.arange(length - n, length, device=DEV)[:, None]
            allowed = (j[None, :] <= p) & ((j[None, :] < case["sinks"]) | (j[None, :] + case["window"] > p))
            use = allowed.any(0)
            rows = (table[i].long()[j // page] * page + j % page)[use]
            allowed = allowed[:, use]
            for h in range(hkv):
                kh, vh = kk[rows, h].double(), vv[rows, h].double()
                for x in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                    s = (q[at:at + n, x].double() @ kh.t()) * case["d"] ** -0.5
                    s = torch.where(allowed, s, torch.full_like(s, -math.inf))
                    part = torch.logsumexp(s, -1)
                    lse[at:at + n, x] = part
                    w = torch.where(allowed.any(-1, keepdim=True), torch.exp(s - part[:, None]), torch.zeros_like(s))
                    out[at:at + n, x] = w @ vh
        at += n
    return {"out": out, "lse": lse}


def _exact_stored32(x):
    """_exact_stored with the code decided by its 32-bit quotient."""
    n, h, d = x.shape
    y = x.float().reshape(n, h, -1, GROUP)
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    z = lo.clamp(-65504, 65504).half().float()
    s = ((hi - lo).double() / 15).float().clamp(max=65504).half().float()
    t = ((y - z).double() / s.double()).float()
    c = torch.where(s > 0, t.round().clamp(0, 15), torch.zeros_like(t))
    return (z + s * c).reshape(n, h, d)  # s c has 15 bits: its sum with z is off by one 32-bit rounding


def _exact_append(case, seed):
    st = _append_inputs(case, seed)
    rot, res = case["rot"], {}
    i = torch.arange(rot // 2, device=DEV)
    a, b = (2 * i, 2 * i + 1) if case["pairs"] == "neighbour" else (i, i + rot // 2)
    c, s = (st[n].double()[st["pos"]][:, None, :] for n in ("cos", "sin"))
    for name, w in (("q", st["wq"]), ("k", st["wk"])):
        x = st[name].double()
        if w is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["d"] + EPS) * w.double()
        y = x.clone()
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        res[name] = y
    return {"q": res["q"], "k": _exact_stored(res["k"]), "v": _exact_stored(st["v"])}


def _exact_rows(case, seed):
    ins = _row_inputs(case, seed)
    res = None
    if case["kind"] == "norm":
        x, r, w = ins
        y = x.double() if r is None else x.double() + r.double()
        res = None if r is None else y
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / case["k"] + EPS) * w.double()
    else:
        g = ins[0].double()
        if case["act"] == "silu":
            y = g * torch.sigmoid(g) * ins[1].double()
        else:
            y = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)) * ins[1].double()
    s = y.abs().max(-1, keepdim=True).values / 127
    s = torch.where(s == 0, torch.ones_like(s), s)
    out = {"values": (y / s).round() * s, "scale": s[:, 0]}
    return {**out, "residual": res} if case["kind"] == "norm" else out


def exact(case, seed):
    if case["kind"] == "window":
        return _exact_window(case, seed)
    return _exact_append(case, seed) if case["kind"] == "append" else _exact_rows(case, seed)
