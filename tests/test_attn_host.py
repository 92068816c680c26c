"""Refusals of the attention entry points on the host: the C ABI before any HIP
call, the binding from tensor metadata (no GPU needed)."""
import ctypes

import pytest
import torch

from tests.test_abi_host import A, BF16, EALIGN, EDEVICE, EDTYPE, EINVAL, ESHAPE, F16, F32, I8, LIB, OK, lib  # noqa: F401
from ultra_bit_weight_amd import sherry


def cache(data=A, n_pages=10, page_size=64, heads=8, d=64):
    return sherry.Kv4CacheDesc(data, n_pages, page_size, heads, d)


def heads(x=A, y=A + 0x1000, w=None, xt=512, xh=64, yt=512, yh=64, n=8):
    return sherry.Heads(x, y, w, xt, xh, yt, yh, n)


def rope(lib, q=None, k=0, x_dt=F16, y_dt=F16, n=4, d=64, rot=64, inter=0, cos=A, sin=A, max_pos=100, pos=A, eps=1e-6):
    return lib.sherry_qk_norm_rope(q if q is not None else heads(), heads() if k == 0 else k, x_dt, y_dt, n, d, rot,
                                   inter, cos, sin, max_pos, pos, eps, None)


def test_rope_refusals(lib):  # noqa: F811
    assert rope(lib) == EDEVICE  # valid: the first HIP call finds no gfx950 here
    assert rope(lib, k=None) == EDEVICE
    assert rope(lib, n=0, pos=None) == OK
    assert rope(lib, n=-1) == EINVAL
    for bad in (dict(cos=None), dict(sin=None), dict(pos=None), dict(max_pos=0), dict(d=0), dict(rot=0),
                dict(q=heads(x=None)), dict(q=heads(y=None)), dict(k=heads(n=0))):
        assert rope(lib, **bad) == EINVAL, bad
    assert lib.sherry_qk_norm_rope(None, None, F16, F16, 4, 64, 64, 0, A, A, 10, A, 1e-6, None) == EINVAL
    for bad in (dict(x_dt=I8), dict(y_dt=I8), dict(x_dt=99)):
        assert rope(lib, **bad) == EDTYPE, bad
    for bad in (dict(d=72, rot=16), dict(d=272, rot=16), dict(rot=24), dict(rot=80), dict(q=heads(xt=-8)),
                dict(q=heads(yh=32)), dict(q=heads(yt=56)), dict(q=heads(n=70000)), dict(n=2 ** 31),
                dict(q=heads(xt=2 ** 41)), dict(n=2 ** 30)):
        assert rope(lib, **bad) == ESHAPE, bad
    for bad in (dict(q=heads(x=A + 2)), dict(k=heads(y=A + 8)), dict(q=heads(xt=516)), dict(q=heads(w=A + 4)),
                dict(cos=A + 4), dict(sin=A + 8), dict(pos=A + 4)):
        assert rope(lib, **bad) == EALIGN, bad


def test_kv4_bytes(lib):  # noqa: F811
    assert lib.sherry_kv4_bytes(10, 64, 8, 64) == 10 * 8 * 2 * (32 * 64 + 256)
    assert lib.sherry_kv4_bytes(3, 256, 5, 128) == 3 * 5 * 8 * (32 * 128 + 512)
    for bad in ((0, 64, 8, 64), (10, 16, 8, 64), (10, 48, 8, 64), (10, 512, 8, 64), (10, 64, 0, 64), (10, 64, 8, 96),
                (10, 64, 8, 0), (2 ** 60, 64, 8, 64), (10, 64, 70000, 64), (-1, 64, 8, 64)):
        assert lib.sherry_kv4_bytes(*bad) == 0, bad


@pytest.mark.parametrize("fn", ["sherry_kv4_write", "sherry_kv4_read"])
def test_kv4_rows_refusals(lib, fn):  # noqa: F811
    def f(c=0, k=A, v=A, dt=F16, n=4, kt=512, kh=64, vt=512, vh=64, slots=A):
        return getattr(lib, fn)(cache() if c == 0 else c, k, v, dt, n, kt, kh, vt, vh, slots, None)
    assert f() == EDEVICE
    assert f(n=0, k=None, v=None, slots=None) == OK
    for bad in (dict(n=-1), dict(c=None), dict(k=None), dict(v=None), dict(slots=None), dict(c=cache(data=None)),
                dict(c=cache(n_pages=0)), dict(c=cache(heads=-2))):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(dt=I8), dict(dt=-1)):
        assert f(**bad) == EDTYPE, bad
    for bad in (dict(c=cache(page_size=48)), dict(c=cache(d=96)), dict(kt=-8), dict(vh=-64), dict(n=2 ** 31),
                dict(n=2 ** 30), dict(kt=2 ** 42)):
        assert f(**bad) == ESHAPE, bad
    for bad in (dict(k=A + 2), dict(v=A + 8), dict(kt=516), dict(vh=68), dict(slots=A + 4), dict(c=cache(data=A + 8))):
        assert f(**bad) == EALIGN, bad
    # overlapping tokens or heads are fine to read from, not to write to
    expect = EDEVICE if fn == "sherry_kv4_write" else ESHAPE
    assert f(kt=0) == expect and f(vh=0) == expect


def attn(lib, c=0, q=A, dt=F16, n=4, hq=32, qt=2048, qh=64, cu=A, seqs=4, max_q=1, max_kv=100000, table=A, width=16,
         stride=16, lens=A, scale=0.125, out=A, ot=2048, oh=64, lse=A, ws=A, ws_bytes=2 ** 30):
    return lib.sherry_kv4_attn(cache() if c == 0 else c, q, dt, n, hq, qt, qh, cu, seqs, max_q, max_kv, table, width,
                               stride, lens, scale, out, ot, oh, lse, ws, ws_bytes, None)


def test_attn_refusals(lib):  # noqa: F811
    assert attn(lib) == EDEVICE
    assert attn(lib, lse=None, cu=None) == EDEVICE
    assert attn(lib, n=0, q=None, out=None) == OK
    assert attn(lib, seqs=0, q=None, out=None) == OK
    for bad in (dict(c=None), dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(width=0),
                dict(n=-1), dict(seqs=-1), dict(max_q=0), dict(max_kv=-1), dict(hq=0), dict(ws=None)):
        assert attn(lib, **bad) == EINVAL, bad
    for bad in (dict(dt=F32), dict(dt=I8), dict(dt=17)):
        assert attn(lib, **bad) == EDTYPE, bad
    for bad in (dict(hq=30), dict(c=cache(d=80)), dict(cu=None, n=5), dict(qt=-8), dict(ot=32), dict(oh=32),
                dict(stride=-1), dict(width=2 ** 25), dict(ws_bytes=64), dict(n=2 ** 31), dict(hq=2 ** 20),
                dict(max_q=2 ** 30), dict(seqs=2 ** 30, max_q=64)):
        assert attn(lib, **bad) == ESHAPE, bad
    for bad in (dict(q=A + 2), dict(out=A + 8), dict(qt=2052), dict(oh=68), dict(table=A + 2), dict(lens=A + 1),
                dict(cu=A + 2), dict(lse=A + 2), dict(ws=A + 8), dict(c=cache(data=A + 4))):
        assert attn(lib, **bad) == EALIGN, bad


def test_attn_workspace(lib):  # noqa: F811
    """Long single sequences are split (a workspace), full batches are not;
    what it says is what the call takes."""
    c = cache()
    one = lib.sherry_kv4_attn_workspace(c, 1, 32, 1, 1, 100000)
    assert one > 0 and one % 4 == 0
    assert lib.sherry_kv4_attn_workspace(c, 1, 32, 1, 1, 100) == 0
    assert lib.sherry_kv4_attn_workspace(c, 4096, 32, 4096, 1, 100000) == 0
    assert attn(lib, n=1, seqs=1, max_kv=100000, ws_bytes=one) == EDEVICE
    assert attn(lib, n=1, seqs=1, max_kv=100000, ws_bytes=one - 1) == ESHAPE
    assert attn(lib, n=1, seqs=1, max_kv=100, ws=None, ws_bytes=0) == EDEVICE
    for bad in ((None, 1, 32, 1, 1, 1000), (c, 0, 32, 1, 1, 1000), (c, 1, 30, 1, 1, 1000), (c, 1, 32, 0, 1, 1000),
                (c, 1, 32, 1, 0, 1000), (c, 1, 32, 1, 1, -1), (cache(d=32), 1, 32, 1, 1, 1000)):
        assert lib.sherry_kv4_attn_workspace(*bad) == 0, bad


# ------------------------------------------------------------ the binding ---

def T(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_rope(lib):  # noqa: F811
    q, k, cs, pos = T(4, 8, 64), T(4, 2, 64), T(10, 32, dtype=torch.float32), T(4, dtype=torch.int64)

    def f(q=q, k=k, cos=cs, sin=cs, pos=pos, **kw):
        return sherry.qk_norm_rope(q, k, cos, sin, pos, **kw)
    with pytest.raises(ValueError, match="on the GPU"):
        f()
    for bad in (dict(q=T(4, 512)), dict(k=T(5, 2, 64)), dict(k=T(4, 2, 32)), dict(k=T(4, 2, 64, dtype=torch.float32)),
                dict(q=T(4, 64, 8).transpose(1, 2)), dict(cos=T(10, 32)), dict(sin=T(9, 32, dtype=torch.float32)),
                dict(cos=T(32, 10, dtype=torch.float32).t(), sin=T(32, 10, dtype=torch.float32).t()),
                dict(pos=T(3, dtype=torch.int64)), dict(pos=T(4, dtype=torch.int32)),
                dict(pos=T(8, dtype=torch.int64)[::2]), dict(q_weight=T(64)), dict(q_weight=T(32, dtype=torch.float32)),
                dict(k=None, k_weight=T(64, dtype=torch.float32)), dict(q_out=T(4, 8, 32)),
                dict(k_out=T(4, 8, 64)), dict(q_out=T(4, 8, 64), k_out=T(4, 2, 64, dtype=torch.float32)),
                dict(q=T(4, 8, 64, dtype=torch.float64)), dict(out_dtype=torch.float64)):
        with pytest.raises(ValueError):
            f(**bad)


def test_binding_refuses_cache(lib):  # noqa: F811
    with pytest.raises(ValueError, match="no cache"):
        sherry.Kv4Cache(4, 48, 8, 64, device="cpu")
    with pytest.raises(ValueError):
        sherry.Kv4Cache(4, 64, 8, 64, data=T(100, dtype=torch.uint8))
    with pytest.raises(ValueError):
        sherry.Kv4Cache(4, 64, 8, 64, data=T(2 ** 20))
    c = sherry.Kv4Cache(4, 64, 8, 64, device="cpu")
    k, slots = T(3, 8, 64), T(3, dtype=torch.int64)
    for f in (lambda: sherry.kv4_write(c, k, k, slots), lambda: sherry.kv4_read(c, slots)):
        with pytest.raises(ValueError, match="on the GPU"):
            f()
    for bad in ((k[:2], k, slots), (k, T(3, 8, 128), slots), (k, k, slots.int()), (k, k.float(), slots),
                (k.double(), k.double(), slots), (k, k, T(6, dtype=torch.int64)[::2]), (k, k, slots[None]),
                (T(3, 64, 8).transpose(1, 2), k, slots)):
        with pytest.raises(ValueError):
            sherry.kv4_write(c, *bad)
    with pytest.raises(ValueError):
        sherry.kv4_read(c, slots, k_out=T(3, 8, 32))
    with pytest.raises(ValueError):
        sherry.kv4_read(c, slots, k_out=T(3, 8, 64), v_out=T(3, 8, 64, dtype=torch.float32))


def test_binding_refuses_attn(lib):  # noqa: F811
    c = sherry.Kv4Cache(4, 64, 2, 64, device="cpu")
    i32 = torch.int32
    base = dict(q=T(3, 8, 64), page_table=T(3, 5, dtype=i32), kv_lens=T(3, dtype=i32))
    with pytest.raises(ValueError, match="on the GPU"):
        sherry.kv4_attn(c, **base)
    for bad in (dict(q=T(3, 8, 128)), dict(q=T(3, 8, 64, dtype=torch.float32)), dict(page_table=T(3, 5, dtype=torch.int64)),
                dict(page_table=T(5, 3, dtype=i32).t()), dict(kv_lens=T(4, dtype=i32)), dict(kv_lens=T(6, dtype=i32)[::2]),
                dict(cu_q=T(3, dtype=i32)), dict(cu_q=T(4, dtype=torch.int64)), dict(out=T(3, 8, 32)),
                dict(out=T(3, 8, 64, dtype=torch.bfloat16)), dict(lse=T(8, 3, dtype=torch.float32)),
                dict(lse=T(3, 8)), dict(workspace=T(100)[::2])):
        with pytest.raises(ValueError):
            sherry.kv4_attn(c, **{**base, **bad})


def test_binding_refuses_other_types(lib):  # noqa: F811
    """Things that are not tensors or numbers, and another count of axes."""
    c = sherry.Kv4Cache(4, 64, 2, 64, device="cpu")
    k, slots = T(3, 2, 64), T(3, dtype=torch.int64)
    for bad in (([1.0], k, slots), (k, None, slots), (k, k, [0, 1, 2])):
        with pytest.raises(TypeError, match="must be a torch.Tensor"):
            sherry.kv4_write(c, *bad)
    q, cs, pos = T(3, 4, 64), T(10, 32, dtype=torch.float32), T(3, dtype=torch.int64)
    with pytest.raises(TypeError, match="cos must be"):
        sherry.qk_norm_rope(q, None, None, cs, pos)
    with pytest.raises(TypeError):
        sherry.qk_norm_rope(q, None, cs, cs, pos, eps="small")
    base = dict(q=q, page_table=T(3, 5, dtype=torch.int32), kv_lens=T(3, dtype=torch.int32), workspace=T(0))
    for bad in (dict(kv_lens=[1, 2, 3]), dict(max_q=1.5), dict(scale="1"), dict(cu_q=(0, 1, 2, 3)), dict(lse=7)):
        with pytest.raises(TypeError):
            sherry.kv4_attn(c, **{**base, **bad})
    for bad in (dict(q=T(3, 256)), dict(page_table=T(15, dtype=torch.int32))):
        with pytest.raises(ValueError, match="must be"):
            sherry.kv4_attn(c, **{**base, **bad})
        with pytest.raises(ValueError, match="must be"):
            sherry.kv4_attn(c, **{**base, **bad, "workspace": None})


@pytest.mark.parametrize("hkv,group,d", [(8, 4, 64), (1, 16, 128), (8, 3, 128), (40, 1, 64), (2, 7, 128)])
def test_default_workspace_serves_default_calls(lib, hkv, group, d):  # noqa: F811
    """kv4_attn_workspace without max_q and max_kv holds what kv4_attn without
    them asks for: one token a sequence without cu_q, all tokens with it, and a
    max_kv of whatever the table holds."""
    c = sherry.Kv4Cache(4, 64, hkv, d, device="cpu")
    hq = hkv * group
    lengths = sorted({*range(1, 40), *(int(1.17 ** i) for i in range(1, 140))})
    for seqs in (1, 2, 3, 7, 16, 48, 191, 300):
        for n in {seqs, seqs + 1, 3 * seqs, 40 * seqs}:
            ws = sherry.kv4_attn_workspace(c, n, hq, seqs).numel()
            for max_q in {1, n} if n == seqs else {n}:
                known = sherry.kv4_attn_workspace(c, n, hq, seqs, max_q).numel()
                needs = [lib.sherry_kv4_attn_workspace(c.desc, n, hq, seqs, max_q, length) for length in lengths]
                assert max(needs) <= known <= ws, (seqs, n, max_q)


def test_workspace_bound(lib):  # noqa: F811
    """The need is not monotone in the batch (fewer sequences can need more), and
    SHERRY_KV4_ATTN_WORKSPACE_MAX is above every call's."""
    import re

    from tests.test_abi_host import HEADER

    most = eval(re.search(r"SHERRY_KV4_ATTN_WORKSPACE_MAX \(\(size_t\)(.*)\)", open(HEADER).read()).group(1))
    assert most == sherry.KV4_ATTN_WORKSPACE_MAX
    c = cache()
    one = [lib.sherry_kv4_attn_workspace(c, n, 32, n, 1, 131072) for n in (48, 191, 192)]
    assert one[2] == 0 < one[0] < one[1]
    top = 0
    for hkv in (1, 2, 5, 8, 16, 63, 128, 511, 513):
        for group in (1, 3, 4, 8, 16, 33):
            for d in (64, 128):
                c = cache(heads=hkv, d=d)
                for seqs in (1, 2, 5, 8, 31, 63, 65, 191, 511):
                    for max_q in (1, 2, 5, 16, 17, 33, 65, 100, 128, 129, 256, 257, 512, 513, 1024, 2047, 2048, 2049, 20000):
                        need = lib.sherry_kv4_attn_workspace(c, seqs * max_q, hkv * group, seqs, max_q, 1 << 30)
                        top = max(top, need)
    assert most // 2 < top <= most


@pytest.mark.parametrize("device", [0, 1, "cuda:0", torch.device("cuda", 0), "cpu", None])
def test_cache_goes_to_the_device_asked_for(lib, device, monkeypatch):  # noqa: F811
    """Device 0 by its index is device 0, not the current one."""
    asked, zeros = [], torch.zeros

    def on_host(*a, **kw):
        asked.append(kw.pop("device"))
        return zeros(*a, **kw)
    monkeypatch.setattr(sherry.torch, "zeros", on_host)
    sherry.Kv4Cache(4, 64, 2, 64, device=device)
    assert asked == ["cuda" if device is None else device]
