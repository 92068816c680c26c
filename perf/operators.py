"""What is measured of the attention operators: rotation and norms of queries
and keys, the 4-bit key/value cache (written and read back), and attention over
that cache.

`own` False computes each operator from elementary torch operations in 32 bits;
`own` True makes the library's calls.  Quantisation rule of the cache, for 64
consecutive values x of one token and head:
    z = f16(min x), s = f16((max x - min x) / 15), both clamped to +-65504
    c = clip(rint((x - z) / s), 0, 15), 0 where s == 0   (fp32 steps)
    value = z + s c
"""
import random

import torch

own = False
DEV = "cuda:0"
GROUP = 64
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # one token of a chat just begun, 1B heads
        dict(name="attn_1tok_short", kind="attn", dtype="f16", hq=32, hkv=8, d=64, page=32, seqs=1, q=1, ctx=200, mix=0),
        # one reader of a very long document, 1B heads: few rows, a long axis
        dict(name="attn_1tok_long", kind="attn", dtype="f16", hq=32, hkv=8, d=64, page=64, seqs=1, q=1, ctx=131072,
             mix=0),
        # a serving batch of uneven lengths with an idle place, 3B heads
        dict(name="attn_batch_ragged", kind="attn", dtype="bf16", hq=24, hkv=8, d=128, page=64, seqs=48, q=1, ctx=12000,
             mix=1),
        # checking a few drafted tokens per sequence (one key head per query head)
        dict(name="attn_draft_5tok", kind="attn", dtype="bf16", hq=16, hkv=16, d=128, page=32, seqs=9, q=5, ctx=4099,
             mix=2),
        # a chunk of a long prompt, 1B heads
        dict(name="attn_chunk_1b", kind="attn", dtype="f16", hq=32, hkv=8, d=64, page=128, seqs=1, q=2048, ctx=8192,
             mix=0),
        # several prompts of uneven lengths from their first token, 3B heads
        dict(name="attn_prompts_ragged", kind="attn", dtype="bf16", hq=24, hkv=8, d=128, page=64, seqs=5, q=1777,
             ctx=1777, mix=3),
        # rotation alone of one token's q and k, 1B heads, as slices of the fused q|k|v product
        dict(name="rope_1tok", kind="rope", dtype="f16", out="f16", tokens=1, hq=32, hkv=8, d=64, rot=64, pairs="half",
             norm=False, maxpos=131072),
        # norms and rotation of a long prompt chunk, 3B heads
        dict(name="rope_chunk", kind="rope", dtype="bf16", out="bf16", tokens=8192, hq=24, hkv=8, d=128, rot=128,
             pairs="half", norm=True, maxpos=32768),
        # an odd token count, partial rotation of neighbouring pairs, fp32 products to fp16
        dict(name="rope_odd_partial", kind="rope", dtype="f32", out="f16", tokens=777, hq=20, hkv=5, d=96, rot=32,
             pairs="neighbour", norm=True, maxpos=4096),
        # one decode step's new tokens of a batch into the cache, and back
        dict(name="kv_append_batch", kind="kv", mode="append", dtype="f16", hkv=8, d=64, page=64, tokens=48, run=1),
        # a prompt chunk into the cache, and back
        dict(name="kv_append_chunk", kind="kv", mode="append", dtype="bf16", hkv=8, d=128, page=64, tokens=8192,
             run=8192),
        # a stored prefix read back in 16 bits
        dict(name="kv_gather_prefix", kind="kv", mode="gather", dtype="f16", hkv=8, d=64, page=32, tokens=20011,
             run=20011),
    ]


def _log(rng, lo, hi):
    import math

    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "rope", "kv"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 5, 8, 16])
    if kind == "attn":
        group = rng.choice([1, 2, 3, 4, 7, 8, 16])
        hq = hkv * group
        if hq > 48:
            hq = hkv
        mode = rng.choice(["one", "one", "few", "chunk"])
        budget = 48 * 12000 * 8 * 128 // (hkv * d)  # cached tokens of the largest listed case
        if mode == "chunk":
            q = _log(rng, 17, 2048)
            seqs = rng.choice([1, 1, 2, 3])
            ctx = min(q + _log(rng, 1, 8192), 8192)
            q = min(q, ctx)
            while seqs * q * ctx * hq * d > 2048 * 8192 * 32 * 64:
                q, seqs = max(1, q // 2), max(1, seqs - 1)
        else:
            q = 1 if mode == "one" else rng.randint(2, 9)
            seqs = _log(rng, 1, 64)
            ctx = max(q, min(_log(rng, 1, 131072), budget // seqs, 40000 if seqs > 1 else 131072))
        return dict(kind="attn", dtype=rng.choice(["f16", "bf16"]), hq=hq, hkv=hkv, d=d, page=rng.choice([32, 64, 128]),
                    seqs=seqs, q=q, ctx=ctx, mix=0 if seqs == 1 else rng.randint(0, 10 ** 6))
    if kind == "rope":
        d = rng.choice([32, 64, 80, 96, 128, 256])
        rot = rng.choice([d, d, 32, 16])
        dt = rng.choice(["f16", "bf16", "f32"])
        hq = hkv * rng.choice([1, 2, 3, 4])
        tokens = min(_log(rng, 1, 8192), 8192 * 32 * 128 // ((hq + hkv) * d))
        return dict(kind="rope", dtype=dt, out=rng.choice([dt, "f16", "bf16"]), tokens=tokens, hq=hq, hkv=hkv, d=d,
                    rot=rot, pairs=rng.choice(["half", "neighbour"]), norm=rng.choice([True, False]),
                    maxpos=rng.choice([4096, 32768, 131072]))
    tokens = min(_log(rng, 1, 20000), 8192 * 8 * 128 // (hkv * d))
    return dict(kind="kv", mode=rng.choice(["append", "append", "gather"]), dtype=rng.choice(["f16", "bf16", "f32"]),
                hkv=hkv, d=d, page=rng.choice([32, 64, 128]), tokens=tokens,
                run=rng.choice([1, 3, 100, tokens]))


# ---------------------------------------------------------------- inputs ----

def _lens(case):
    """Lengths of the sequences: new tokens and cached tokens (new ones
    included) of each; fixed by the case, so that its work is too."""
    n, q, ctx = case["seqs"], case["q"], case["ctx"]
    if case["mix"] == 0 or n == 1:
        return [q] * n, [ctx] * n
    rng = random.Random(case["mix"])
    qs, ls = [], []
    for i in range(n):
        qi = q if q < 10 else rng.randint(max(1, q // 4), q)
        li = max(qi, int(ctx * rng.uniform(0.1, 1.0)))
        if case["q"] == case["ctx"]:  # prompts from their first token
            li = qi
        qs.append(qi)
        ls.append(li)
    qs[0], ls[0] = q, ctx
    if n >= 4 and q < 10:
        ls[-1] = 0  # an idle place of the batch: its rows see nothing
    return qs, ls


def _pages(case, lens, g):
    page = case["page"]
    need = [(length + page - 1) // page for length in lens]
    width = max(1, max(need))
    total = sum(need) + 1
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(need):
        table[i, :c] = perm[at:at + c]
        at += c
    return table, total


def _kv_values(n, hkv, d, dtype, g, g_chan):
    """Keys with channels of their own scale and offset, as rotated keys have; values plain."""
    k = torch.randn(n, hkv, d, generator=g, device=DEV)
    k = k * (0.3 + g_chan[0]) + 2.0 * (g_chan[1] - 0.5)
    v = torch.randn(n, hkv, d, generator=g, device=DEV) * (0.2 + g_chan[2])
    return k.to(dtype), v.to(dtype)


def _quantise(x):
    """x [n, heads, d] -> codes uint8 [n, heads, d], s and z f16 [n, heads, d / 64]"""
    n, h, d = x.shape
    y = x.float().view(n, h, d // GROUP, GROUP)
    lo, hi = y.amin(-1), y.amax(-1)
    z = lo.clamp(-65504.0, 65504.0).to(torch.float16)
    fifteen = torch.full_like(lo, 15.0)  # a tensor: the quotient is one IEEE division
    s = ((hi - lo) / fifteen).clamp(max=65504.0).to(torch.float16)
    sf, zf = s.float().unsqueeze(-1), z.float().unsqueeze(-1)
    c = torch.where(sf > 0, torch.round((y - zf) / torch.where(sf > 0, sf, torch.ones_like(sf))), torch.zeros_like(y))
    return c.clamp(0, 15).to(torch.uint8).view(n, h, d), s, z


def _dequantise(c, s, z):
    n, h, d = c.shape
    y = c.float().view(n, h, d // GROUP, GROUP)
    return (z.float().unsqueeze(-1) + s.float().unsqueeze(-1) * y).view(n, h, d)


def _nibbles(c):  # two codes to a byte
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _codes(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _plain_cache(slots, hkv, d):
    e = dict(dtype=torch.uint8, device=DEV)
    f = dict(dtype=torch.float16, device=DEV)
    return {w + p: (torch.zeros(slots, hkv, d // 2, **e) if p == "c" else torch.zeros(slots, hkv, d // GROUP, **f))
            for w in "kv" for p in "csz"}


def _plain_write(cache, k, v, slots):
    for w, x in (("k", k), ("v", v)):
        c, s, z = _quantise(x)
        cache[w + "c"][slots] = _nibbles(c)
        cache[w + "s"][slots] = s
        cache[w + "z"][slots] = z


def _plain_read(cache, slots):
    return [_dequantise(_codes(cache[w + "c"][slots]), cache[w + "s"][slots], cache[w + "z"][slots]) for w in "kv"]


def _new_cache(pages, page, hkv, d):
    if own:
        from ultra_bit_weight_amd import sherry

        return sherry.Kv4Cache(pages, page, hkv, d, device=DEV)
    return _plain_cache(pages * page, hkv, d)


def _fill(cache, k, v, slots):
    if own:
        from ultra_bit_weight_amd import sherry

        sherry.kv4_write(cache, k, v, slots)
    else:
        _plain_write(cache, k, v, slots)


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _attn_inputs(case, seed):
    g = _generator(seed)
    qs, ls = _lens(case)
    hkv, d, dtype = case["hkv"], case["d"], DT[case["dtype"]]
    chan = torch.rand(3, hkv, d, generator=g, device=DEV)
    table, total = _pages(case, ls, g)
    q = (torch.randn(sum(qs), case["hq"], d, generator=g, device=DEV) * 1.2).to(dtype)
    n = total * case["page"]
    step = max(1, (1 << 26) // (hkv * d))

    def chunks():
        for a in range(0, n, step):
            b = min(n, a + step)
            k, v = _kv_values(b - a, hkv, d, dtype, g, chan)
            yield a, b, k, v
    return qs, ls, table, total, q, chunks


def _prepare_attn(case, seed):
    qs, ls, table, total, q, chunks = _attn_inputs(case, seed)
    cache = _new_cache(total, case["page"], case["hkv"], case["d"])
    for a, b, k, v in chunks():
        _fill(cache, k, v, torch.arange(a, b, device=DEV))
    st = dict(case=case, cache=cache, q=q, table=table, scale=case["d"] ** -0.5, qs=qs, ls=ls,
              lens=torch.tensor(ls, dtype=torch.int32, device=DEV),
              cu=torch.tensor([sum(qs[:i]) for i in range(len(qs) + 1)], dtype=torch.int32, device=DEV))
    if own:
        from ultra_bit_weight_amd import sherry

        st["out"] = torch.empty_like(q)
        st["lse"] = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=DEV)
        st["ws"] = sherry.kv4_attn_workspace(cache, q.shape[0], q.shape[1], len(ls), max(qs), max(ls))
    else:
        page = case["page"]
        st["slots"] = [(table[i, :(n + page - 1) // page].long().unsqueeze(1) * page
                        + torch.arange(page, device=DEV)).flatten()[:n] for i, n in enumerate(ls)]
    return st


def _rope_inputs(case, seed):
    g = _generator(seed)
    t, hq, hkv, d, rot = (case[x] for x in ("tokens", "hq", "hkv", "d", "rot"))
    qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=g, device=DEV).to(DT[case["dtype"]])
    if t == 1:
        pos = torch.randint(0, case["maxpos"], (1,), generator=g, device=DEV)
    else:  # a chunk at some offset, and a second sequence behind it
        a = torch.randint(0, case["maxpos"], (2,), generator=g, device=DEV)
        pos = (torch.arange(t, device=DEV) + torch.where(torch.arange(t, device=DEV) < t // 2, a[0], a[1])) % case["maxpos"]
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    ang = torch.arange(case["maxpos"], dtype=torch.float64, device=DEV).unsqueeze(1) * inv
    wq = wk = None
    if case["norm"]:
        wq = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        wk = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
    return dict(case=case, q=qkv[:, :hq * d].view(t, hq, d), k=qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
                cos=ang.cos().float(), sin=ang.sin().float(), pos=pos, wq=wq, wk=wk)


def _kv_inputs(case, seed):
    g = _generator(seed)
    t, hkv, d, page = (case[x] for x in ("tokens", "hkv", "d", "page"))
    chan = torch.rand(3, hkv, d, generator=g, device=DEV)
    k, v = _kv_values(t, hkv, d, DT[case["dtype"]], g, chan)
    # runs of consecutive tokens, each from a place of its own inside its first page
    run = min(case["run"], t)
    runs = (t + run - 1) // run
    per = (run + page - 1) // page + 1
    pages = runs * per
    perm = torch.randperm(pages, generator=g, device=DEV)
    at = torch.randint(0, page, (runs,), generator=g, device=DEV) if case["mode"] == "append" and run < t else \
        torch.zeros(runs, dtype=torch.long, device=DEV)
    i = torch.arange(t, device=DEV)
    where = at[i // run] + i % run
    slots = perm[(i // run) * per + where // page] * page + where % page
    return k, v, slots, pages


def prepare(case, seed):
    if case["kind"] == "attn":
        return _prepare_attn(case, seed)
    if case["kind"] == "rope":
        st = _rope_inputs(case, seed)
        if own:
            out = DT[case["out"]]
            st["q_out"] = torch.empty(st["q"].shape, dtype=out, device=DEV)
            st["k_out"] = torch.empty(st["k"].shape, dtype=out, device=DEV)
        return st
    k, v, slots, pages = _kv_inputs(case, seed)
    cache = _new_cache(pages, case["page"], case["hkv"], case["d"])
    if case["mode"] == "gather":
        _fill(cache, k, v, slots)
    st = dict(case=case, cache=cache, k=k, v=v, slots=slots)
    if own:
        out = torch.float16 if case["mode"] == "gather" else k.dtype
        st["k_out"], st["v_out"] = (torch.empty(k.shape, dtype=out, device=DEV) for _ in range(2))
    return st


# ------------------------------------------------------------------ runs ----

def _run_attn(st):
    q, case = st["q"], st["case"]
    if own:
        from ultra_bit_weight_amd import sherry

        sherry.kv4_attn(st["cache"], q, st["table"], st["lens"], cu_q=st["cu"], max_q=max(st["qs"]), max_kv=max(st["ls"]),
                        scale=st["scale"], out=st["out"], lse=st["lse"], workspace=st["ws"])
        return {"out": st["out"], "lse": st["lse"]}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    grp = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float32, device=DEV)
    lse = torch.full(q.shape[:2], float("-inf"), device=DEV)
    at = 0
    for n, length, slots in zip(st["qs"], st["ls"], st["slots"]):
        if length:
            k, v = _plain_read(st["cache"], slots)  # [length, hkv, d]
            x = q[at:at + n].float().view(n, hkv, grp, d).permute(1, 2, 0, 3).reshape(hkv, grp * n, d)
            s = torch.matmul(x, k.permute(1, 2, 0).contiguous()) * st["scale"]
            if n > 1:
                late = torch.arange(length, device=DEV) > (torch.arange(n, device=DEV) + length - n).unsqueeze(1)
                s.view(hkv, grp, n, length).masked_fill_(late, float("-inf"))
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
            p = torch.exp(s - m)
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p, v.permute(1, 0, 2).contiguous()) / torch.where(total > 0, total, torch.ones_like(total))
            out[at:at + n] = o.view(hkv, grp, n, d).permute(2, 0, 1, 3).reshape(n, hq, d)
            lse[at:at + n] = (m + torch.log(total)).view(hkv, grp, n).permute(2, 0, 1).reshape(n, hq)
        at += n
    return {"out": out.to(q.dtype), "lse": lse}


def _rotate(x, cos, sin, rot, neighbour):
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if neighbour else (y[..., :rot // 2], y[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((a, b), -1).flatten(-2) if neighbour else torch.cat((a, b), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _run_rope(st):
    case = st["case"]
    if own:
        from ultra_bit_weight_amd import sherry

        sherry.qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], st["pos"], q_weight=st["wq"], k_weight=st["wk"],
                            eps=1e-6, interleaved=case["pairs"] == "neighbour", q_out=st["q_out"], k_out=st["k_out"])
        return [st["q_out"], st["k_out"]]
    cos, sin = st["cos"][st["pos"]].unsqueeze(1), st["sin"][st["pos"]].unsqueeze(1)
    res = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        res.append(_rotate(x, cos, sin, case["rot"], case["pairs"] == "neighbour").to(DT[case["out"]]))
    return res


def _run_kv(st):
    case, cache = st["case"], st["cache"]
    out = torch.float16 if case["mode"] == "gather" else st["k"].dtype
    if own:
        from ultra_bit_weight_amd import sherry

        if case["mode"] == "append":
            sherry.kv4_write(cache, st["k"], st["v"], st["slots"])
        sherry.kv4_read(cache, st["slots"], k_out=st["k_out"], v_out=st["v_out"])
        return [st["k_out"], st["v_out"]]
    if case["mode"] == "append":
        _plain_write(cache, st["k"], st["v"], st["slots"])
    return [x.to(out) for x in _plain_read(cache, st["slots"])]


def run(state):
    return {"attn": _run_attn, "rope": _run_rope, "kv": _run_kv}[state["case"]["kind"]](state)


# ------------------------------------------------------------------ work ----

def _row_bytes(hkv, d):  # a cached token: 4-bit K and V, and f16 scale and zero point per 64 values
    return hkv * (d + 8 * (d // GROUP))


def work(case):
    hkv, d = case["hkv"], case["d"]
    if case["kind"] == "attn":
        qs, ls = _lens(case)
        hq, t = case["hq"], sum(qs)
        pairs = sum(max(0, sum(max(0, length - n + i + 1) for i in range(n))) for n, length in zip(qs, ls))
        table = sum((length + case["page"] - 1) // case["page"] for length in ls)
        byts = sum(ls) * _row_bytes(hkv, d) + 2 * t * hq * d * SIZE[case["dtype"]] + 4 * t * hq + 4 * (table + 2 * len(ls) + 1)
        return {"bytes": byts, "flops": 4 * d * hq * pairs}
    if case["kind"] == "rope":
        t, h = case["tokens"], case["hq"] + hkv
        w = 8 * d if case["norm"] else 0
        return {"bytes": t * h * d * (SIZE[case["dtype"]] + SIZE[case["out"]]) + t * (4 * case["rot"] + 8) + w,
                "flops": t * h * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    t = case["tokens"]
    packed = t * _row_bytes(hkv, d)
    if case["mode"] == "gather":
        return {"bytes": packed + 2 * t * hkv * d * 2 + 8 * t, "flops": 2 * 2 * t * hkv * d}
    return {"bytes": 2 * packed + 4 * t * hkv * d * SIZE[case["dtype"]] + 16 * t, "flops": 8 * 2 * t * hkv * d}


# ----------------------------------------------------------- the 64-bit definition

def _exact_stored(x):
    """The values that the cache stands for, in 64 bits: z and s rounded to
    f16 as the format has them, the code decided by its fp32 quotient (64-bit
    quotients of 32-bit numbers, rounded to 32)."""
    n, h, d = x.shape
    y = x.double().reshape(n, h, -1, GROUP)
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    z = lo.clamp(-65504, 65504).half().double()
    s = ((hi - lo).float().double() / 15).float().clamp(max=65504).half().double()
    t = ((y - z).float().double() / s).float().double()
    c = torch.where(s > 0, t.round().clamp(0, 15), torch.zeros_like(t))
    return (z + s * c).reshape(n, h, d)


def _exact_attn(case, seed):
    qs, ls, table, total, q, chunks = _attn_inputs(case, seed)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    if total * page * hkv * d > 3 * 2 ** 29:
        return None
    ks, vs = [], []
    for _, _, k, v in chunks():
        ks.append(_exact_stored(k).float() if total * page * hkv * d > 2 ** 29 else _exact_stored(k))
        vs.append(_exact_stored(v).float() if total * page * hkv * d > 2 ** 29 else _exact_stored(v))
    kk, vv = torch.cat(ks), torch.cat(vs)
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -float("inf"), dtype=torch.float64, device=DEV)
    at = 0
    for i, (n, length) in enumerate(zip(qs, ls)):
        if length:
            j = torch.arange(length, device=DEV)
            rows = table[i].long()[j // page] * page + j % page
            allowed = j[None, :] <= torch.arange(n, device=DEV)[:, None] + (length - n)
            for h in range(hq):
                kh, vh = kk[rows, h // (hq // hkv)].double(), vv[rows, h // (hq // hkv)].double()
                s = (q[at:at + n, h].double() @ kh.t()) * case["d"] ** -0.5
                s = torch.where(allowed, s, torch.full_like(s, -float("inf")))
                part = torch.logsumexp(s, -1)
                lse[at:at + n, h] = part
                seen = allowed.any(-1)
                out[at:at + n, h] = torch.where(seen[:, None], torch.exp(s - part[:, None]) @ vh,
                                                torch.zeros(n, d, dtype=torch.float64, device=DEV))
        at += n
    return {"out": out, "lse": lse}


def _exact_rope(case, seed):
    st = _rope_inputs(case, seed)
    rot, res = case["rot"], []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["d"] + 1e-6) * w.double()
        i = torch.arange(rot // 2, device=DEV)
        a, b = (2 * i, 2 * i + 1) if case["pairs"] == "neighbour" else (i, i + rot // 2)
        c, s = (st[n].double()[st["pos"]][:, None, :] for n in ("cos", "sin"))
        y = x.clone()
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        res.append(y)
    return res


def exact(case, seed):
    if case["kind"] == "attn":
        return _exact_attn(case, seed)
    if case["kind"] == "rope":
        return _exact_rope(case, seed)
    k, v, _, _ = _kv_inputs(case, seed)
    return [_exact_stored(k), _exact_stored(v)]
