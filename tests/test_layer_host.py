"""Refusals of the operators around a layer's products on the host: the C ABI
before any HIP call, the binding from tensor metadata (no GPU needed)."""
import pytest
import torch

from tests.test_abi_host import A, EALIGN, EDEVICE, EDTYPE, EINVAL, ESHAPE, F16, F32, I8, LIB, OK, lib  # noqa: F401
from tests.test_attn_host import T, cache, heads
from ultra_bit_weight_amd import sherry


def norm(lib, x=A, dt=F16, m=4, k=2048, ldx=2048, r=A, ldr=2048, ro=A, ldro=2048, rdt=F32, w=A, eps=1e-6, q=A, ldq=2048,
         s=A):
    return lib.sherry_rms_norm_quant(x, dt, m, k, ldx, r, ldr, ro, ldro, rdt, w, eps, q, ldq, s, None)


def test_norm_refusals(lib):  # noqa: F811
    assert norm(lib) == EDEVICE  # valid: the first HIP call finds no gfx950 here
    assert norm(lib, r=None, ro=None, rdt=99, ldr=0, ldro=0) == EDEVICE
    assert norm(lib, m=0, x=None, w=None, q=None, s=None) == OK
    for bad in (dict(m=-1), dict(k=0), dict(k=-5), dict(x=None), dict(w=None), dict(q=None), dict(s=None), dict(r=None),
                dict(ro=None), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm(lib, **bad) == EINVAL, bad
    for bad in (dict(dt=I8), dict(dt=99), dict(rdt=I8), dict(rdt=-3)):
        assert norm(lib, **bad) == EDTYPE, bad
    for bad in (dict(ldx=2047), dict(ldr=2047), dict(ldro=0), dict(ldq=-1), dict(ldx=2 ** 41), dict(m=2 ** 21),
                dict(k=2 ** 31, ldx=2 ** 31, ldr=2 ** 31, ldro=2 ** 31, ldq=2 ** 31)):
        assert norm(lib, **bad) == ESHAPE, bad
    for bad in (dict(x=A + 1), dict(r=A + 2), dict(ro=A + 1), dict(w=A + 2), dict(s=A + 2)):
        assert norm(lib, **bad) == EALIGN, bad
    # any element alignment, any row stride, any k
    assert norm(lib, x=A + 2, r=A + 4, q=A + 1, w=A + 4, k=1, ldx=1, ldr=3, ldro=5, ldq=7) == EDEVICE


def gated(lib, g=A, ldg=16384, u=A, ldu=16384, dt=F16, m=4, k=8192, act=0, q=A, ldq=8192, s=A):
    return lib.sherry_gated_quant(g, ldg, u, ldu, dt, m, k, act, q, ldq, s, None)


def test_gated_refusals(lib):  # noqa: F811
    assert gated(lib) == EDEVICE and gated(lib, act=1) == EDEVICE
    assert gated(lib, m=0, g=None, u=None, q=None, s=None) == OK
    for bad in (dict(m=-1), dict(k=0), dict(g=None), dict(u=None), dict(q=None), dict(s=None), dict(act=2), dict(act=-1),
                dict(act=2, m=0)):
        assert gated(lib, **bad) == EINVAL, bad
    assert gated(lib, dt=I8) == EDTYPE and gated(lib, dt=77) == EDTYPE
    for bad in (dict(ldg=8191), dict(ldu=0), dict(ldq=8191), dict(ldq=-8192), dict(m=2 ** 21), dict(ldu=2 ** 41)):
        assert gated(lib, **bad) == ESHAPE, bad
    for bad in (dict(g=A + 1), dict(u=A + 3), dict(s=A + 1)):
        assert gated(lib, **bad) == EALIGN, bad
    assert gated(lib, g=A + 2, q=A + 3, k=5, ldg=5, ldu=6, ldq=5) == EDEVICE


def append(lib, c=0, q=0, k=0, v=A, vt=512, vh=64, x_dt=F16, y_dt=F16, n=4, rot=64, inter=0, cos=A, sin=A, max_pos=100,
           pos=A, eps=1e-6, slots=A):
    k = heads(y=None, yt=0, yh=0) if k == 0 else k
    return lib.sherry_kv4_append(cache() if c == 0 else c, heads(n=32, xt=2048, yt=2048) if q == 0 else q, k, v, vt, vh,
                                 x_dt, y_dt, n, rot, inter, cos, sin, max_pos, pos, eps, slots, None)


def test_append_refusals(lib):  # noqa: F811
    def keys(**kw):
        return heads(**{**dict(y=None, yt=0, yh=0), **kw})
    assert append(lib) == EDEVICE
    assert append(lib, q=None, y_dt=99) == EDEVICE
    assert append(lib, n=0, q=None, k=None, v=None, c=None) == OK
    for bad in (dict(n=-1), dict(c=None), dict(k=None), dict(k=heads()), dict(k=keys(x=None)), dict(v=None), dict(cos=None),
                dict(sin=None), dict(pos=None), dict(slots=None), dict(max_pos=0), dict(rot=0), dict(q=heads(x=None)),
                dict(q=heads(y=None)), dict(q=heads(n=0)), dict(c=cache(data=None)), dict(c=cache(n_pages=0))):
        assert append(lib, **bad) == EINVAL, bad
    for bad in (dict(x_dt=I8), dict(y_dt=I8), dict(x_dt=-1)):
        assert append(lib, **bad) == EDTYPE, bad
    for bad in (dict(rot=24), dict(rot=80), dict(k=keys(n=4)), dict(k=keys(xt=-8)), dict(vt=-8), dict(vh=2 ** 41),
                dict(q=heads(yh=32)), dict(q=heads(yt=56)), dict(n=2 ** 31), dict(n=2 ** 25), dict(c=cache(d=96)),
                dict(c=cache(page_size=16)), dict(max_pos=2 ** 41), dict(q=heads(n=70000))):
        assert append(lib, **bad) == ESHAPE, bad
    for bad in (dict(v=A + 2), dict(vt=516), dict(k=keys(x=A + 8)), dict(k=keys(w=A + 4)), dict(q=heads(x=A + 2)),
                dict(cos=A + 4), dict(sin=A + 8), dict(pos=A + 4), dict(slots=A + 4), dict(c=cache(data=A + 8))):
        assert append(lib, **bad) == EALIGN, bad


def window(lib, c=0, q=A, dt=F16, n=4, hq=32, seqs=4, max_q=1, max_kv=100000, width=1600, window=100, sinks=4, out=A, ws=A,
           ws_bytes=2 ** 30, lens=A):
    return lib.sherry_kv4_attn_window(cache() if c == 0 else c, q, dt, n, hq, 2048, 64, A, seqs, max_q, max_kv, A, width,
                                      width, lens, 0.125, window, sinks, out, 2048, 64, A, ws, ws_bytes, None)


def test_window_refusals(lib):  # noqa: F811
    assert window(lib) == EDEVICE
    for fine in (dict(sinks=0), dict(window=1), dict(window=2 ** 62, sinks=2 ** 62), dict(sinks=2 ** 40)):
        assert window(lib, **fine) == EDEVICE, fine
    assert window(lib, n=0, q=None) == OK
    for bad in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(q=None), dict(out=None), dict(c=None),
                dict(lens=None), dict(max_q=0)):
        assert window(lib, **bad) == EINVAL, bad
    assert window(lib, dt=F32) == EDTYPE
    for bad in (dict(hq=30), dict(width=2 ** 25), dict(n=1, seqs=1, window=50000, ws_bytes=64)):
        assert window(lib, **bad) == ESHAPE, bad


def test_window_workspace(lib):  # noqa: F811
    """Sized by what a window leaves, at most by what the call without one needs
    where rows see less; the call takes what it says."""
    f = lib.sherry_kv4_attn_window_workspace
    c = cache()
    assert f(c, 1, 32, 1, 1, 100000, 100, 4) == 0
    long = f(c, 1, 32, 1, 1, 100000, 50000, 4)
    assert long > 0 and window(lib, n=1, seqs=1, window=50000, ws_bytes=long) == EDEVICE
    assert window(lib, n=1, seqs=1, window=50000, ws_bytes=long - 1) == ESHAPE
    assert window(lib, n=1, seqs=1, window=100, ws=None, ws_bytes=0) == EDEVICE
    for big in (100000, 2 ** 30, 2 ** 62):
        assert f(c, 1, 32, 1, 1, 100000, big, 0) == lib.sherry_kv4_attn_workspace(c, 1, 32, 1, 1, 100000)
    for bad in ((None, 1, 32, 1, 1, 1000, 10, 0), (c, 0, 32, 1, 1, 1000, 10, 0), (c, 1, 32, 1, 1, 1000, 0, 0),
                (c, 1, 32, 1, 1, 1000, 10, -1), (c, 1, 30, 1, 1, 1000, 10, 0)):
        assert f(*bad) == 0, bad


@pytest.mark.parametrize("hkv,group,d", [(8, 4, 64), (1, 16, 128), (40, 1, 64), (2, 7, 128)])
def test_window_workspace_bounds(lib, hkv, group, d):  # noqa: F811
    """The default workspace of the binding serves default calls with any cached
    length, and KV4_ATTN_WORKSPACE_MAX every one of at most n_seqs max_q tokens."""
    c = sherry.Kv4Cache(4, 64, hkv, d, device="cpu")
    hq = hkv * group
    lengths = sorted({*range(1, 40), *(int(1.3 ** i) for i in range(1, 76))})
    for seqs in (1, 3, 16, 191):
        for n in {seqs, 3 * seqs, 40 * seqs}:
            for w, sinks in ((1, 0), (100, 4), (1000, 20), (5000, 0), (2 ** 40, 2 ** 40)):
                ws = sherry.kv4_attn_workspace(c, n, hq, seqs, window=w, sinks=sinks).numel()
                for max_q in {1, n} if n == seqs else {n}:
                    needs = [lib.sherry_kv4_attn_window_workspace(c.desc, n, hq, seqs, max_q, length, w, sinks)
                             for length in lengths]
                    assert max(needs) <= min(ws, sherry.KV4_ATTN_WORKSPACE_MAX), (seqs, n, max_q, w)


# ------------------------------------------------------------ the binding ---

def test_binding_refuses_norm(lib):  # noqa: F811
    x, w, r = T(4, 64), T(64, dtype=torch.float32), T(4, 64, dtype=torch.float32)
    for fine in (dict(), dict(residual=r), dict(x=T(4, 100)[:, :64]), dict(residual=T(4, 64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="on the GPU"):
            sherry.rms_norm_quant(**{**dict(x=x, weight=w), **fine})
    for bad in (dict(x=T(64)), dict(x=T(2, 4, 64)), dict(x=T(64, 4).t()), dict(x=T(4, 64, dtype=torch.float64)),
                dict(weight=T(64)), dict(weight=T(63, dtype=torch.float32)), dict(weight=T(128, dtype=torch.float32)[::2]),
                dict(residual=T(4, 63)), dict(residual=T(64, 4).t()), dict(residual=T(4, 64, dtype=torch.int32)),
                dict(residual=r, residual_out=T(4, 64)), dict(residual=r, residual_out=T(3, 64, dtype=torch.float32)),
                dict(residual_out=r), dict(q_out=T(4, 64)), dict(q_out=T(4, 65, dtype=torch.int8)),
                dict(scale_out=T(4)), dict(scale_out=T(8, dtype=torch.float32)[::2])):
        with pytest.raises(ValueError):
            sherry.rms_norm_quant(**{**dict(x=x, weight=w), **bad})
    wide = T(4 * 64 + 64, dtype=torch.float32)  # the same memory with two row strides
    with pytest.raises(ValueError, match="another row stride"):
        sherry.rms_norm_quant(x, w, residual=wide[:256].view(4, 64), residual_out=wide.view(4, 80)[:, :64])
    for bad in (dict(weight=None), dict(weight=[1.0] * 64), dict(residual=5), dict(eps="0")):
        with pytest.raises(TypeError):
            sherry.rms_norm_quant(**{**dict(x=x, weight=w), **bad})


def test_binding_refuses_gated(lib):  # noqa: F811
    gu = T(4, 128)
    for fine in ((gu[:, :64], gu[:, 64:]), (T(4, 64), T(4, 64))):
        with pytest.raises(ValueError, match="on the GPU"):
            sherry.gated_quant(*fine)
    g = T(4, 64)
    for bad in (dict(gate=T(64)), dict(up=T(4, 63)), dict(up=T(4, 64, dtype=torch.float32)), dict(up=T(64, 4).t()),
                dict(gate=g.double(), up=g.double()), dict(activation="relu"), dict(activation=0), dict(q_out=T(4, 64)),
                dict(scale_out=T(3, dtype=torch.float32))):
        with pytest.raises(ValueError):
            sherry.gated_quant(**{**dict(gate=g, up=g), **bad})
    with pytest.raises(TypeError):
        sherry.gated_quant(g, None)


def test_binding_refuses_append(lib):  # noqa: F811
    c = sherry.Kv4Cache(4, 64, 2, 64, device="cpu")
    q, k, cs, pos = T(3, 8, 64), T(3, 2, 64), T(10, 32, dtype=torch.float32), T(3, dtype=torch.int64)
    base = dict(q=q, k=k, v=k, cos=cs, sin=cs, positions=pos, slots=pos)
    for fine in (dict(), dict(q=None), dict(out_dtype=torch.float32), dict(q_out=T(3, 8, 64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="on the GPU"):
            sherry.kv4_append(c, **{**base, **fine})
    for bad in (dict(q=T(3, 512)), dict(q=T(2, 8, 64)), dict(q=T(3, 8, 64, dtype=torch.float32)), dict(k=T(3, 4, 64)),
                dict(k=T(3, 2, 128)), dict(v=T(3, 2, 64, dtype=torch.float32)), dict(v=T(4, 2, 64)),
                dict(v=T(3, 64, 2).transpose(1, 2)), dict(cos=T(10, 32)), dict(sin=T(9, 32, dtype=torch.float32)),
                dict(positions=T(4, dtype=torch.int64)), dict(positions=pos.int()), dict(slots=T(2, dtype=torch.int64)),
                dict(slots=T(6, dtype=torch.int64)[::2]), dict(q_weight=T(64)), dict(k_weight=T(32, dtype=torch.float32)),
                dict(q=None, q_weight=T(64, dtype=torch.float32)), dict(q=None, q_out=T(3, 8, 64)),
                dict(q_out=T(3, 8, 32)), dict(q_out=T(3, 8, 64), out_dtype=torch.float32), dict(out_dtype=torch.int8),
                dict(k=k.double(), v=k.double(), q=q.double())):
        with pytest.raises(ValueError):
            sherry.kv4_append(c, **{**base, **bad})
    for bad in (dict(v=None), dict(slots=[0, 1, 2]), dict(cos=None), dict(eps="x")):
        with pytest.raises(TypeError):
            sherry.kv4_append(c, **{**base, **bad})


def test_binding_refuses_window(lib):  # noqa: F811
    c = sherry.Kv4Cache(4, 64, 2, 64, device="cpu")
    base = dict(q=T(3, 8, 64), page_table=T(3, 5, dtype=torch.int32), kv_lens=T(3, dtype=torch.int32), workspace=T(0))
    with pytest.raises(ValueError, match="on the GPU"):
        sherry.kv4_attn(c, **base, window=10, sinks=2)
    with pytest.raises(ValueError, match="sinks need a window"):
        sherry.kv4_attn(c, **base, sinks=2)
    for bad in (dict(window=1.5), dict(window="4"), dict(window=4, sinks=None), dict(window=4, sinks=0.5)):
        with pytest.raises(TypeError):
            sherry.kv4_attn(c, **base, **bad)


@pytest.mark.parametrize("hkv,group,d,seqs,q", [(8, 8, 64, 6, 13), (2, 8, 128, 8, 53), (1, 4, 64, 22, 25), (2, 2, 128, 49, 25),
                                                (16, 2, 128, 2, 29), (3, 1, 64, 2, 705), (2, 3, 64, 2, 221), (1, 16, 64, 15, 62),
                                                (1, 1, 128, 3, 725), (8, 4, 64, 1, 512), (8, 3, 128, 1, 512), (1, 1, 64, 1, 33)])
def test_window_workspace_grows_with_max_kv(lib, hkv, group, d, seqs, q):  # noqa: F811
    """What is asked for at one max_kv serves every smaller one, also where that takes
    other tiles; the default serves all."""
    c = sherry.Kv4Cache(4, 64, hkv, d, device="cpu")
    f = lib.sherry_kv4_attn_window_workspace
    for w, sinks in ((7, 3000), (83, 3000), (201, 3000), (518, 100), (757, 4), (2256, 0), (4074, 4), (9000, 50)):
        needs = [f(c.desc, seqs * q, hkv * group, seqs, q, kv, w, sinks)
                 for kv in [*range(1, 2199, 13), 2199, 2200, 2201, *range(2500, 9200, 97), 1 << 20, 1 << 30]]
        for kv, a, b in zip(range(len(needs)), needs, needs[1:]):
            assert a <= b, (w, sinks, kv, a, b)
        assert needs[-1] <= min(sherry.kv4_attn_workspace(c, seqs * q, hkv * group, seqs, q, window=w, sinks=sinks).numel(),
                                sherry.KV4_ATTN_WORKSPACE_MAX)
