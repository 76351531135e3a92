"""Argument checks of the operators around the chunked scan, in the binding and
behind the C ABI, on the CPU: nothing here launches a kernel."""
import ctypes

import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from ssd_chunked_scan_chunk_amd import _lib

Bz, L, C, W = 2, 10, 24, 4
BF, F32 = torch.bfloat16, torch.float32


def conv_args(**kw):
    d = dict(x=torch.zeros(Bz, L, C, dtype=BF), weight=torch.zeros(C, W), bias=torch.zeros(C),
             initial_window=torch.zeros(Bz, W - 1, C, dtype=BF), seqlens=torch.zeros(Bz, dtype=torch.int32))
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,match", [
    (dict(x=torch.zeros(L, C, dtype=BF)), "3-D"),
    (dict(x=torch.zeros(Bz, C, L, dtype=BF).transpose(1, 2)), "rows of x"),
    (dict(weight=torch.zeros(C)), "2-D"),
    (dict(weight=torch.zeros(C - 1, W)), "weight has shape"),
    (dict(weight=torch.zeros(C, W, dtype=BF)), "weight has dtype"),
    (dict(bias=torch.zeros(C + 1)), "bias has shape"),
    (dict(initial_window=torch.zeros(Bz, W, C, dtype=BF)), "initial_window has shape"),
    (dict(initial_window=torch.zeros(Bz, W - 1, C)), "initial_window has dtype"),
    (dict(seqlens=torch.zeros(Bz, dtype=torch.int64)), "seqlens has dtype"),
    (dict(seqlens=torch.zeros(Bz + 1, dtype=torch.int32)), "seqlens has shape"),
    (dict(pieces=(20, 3)), "pieces must be"),
    (dict(pieces=(6, 6, 6, 6)), "pieces must be"),
    (dict(pieces=(24, 0)), "pieces must be"),
    (dict(y=torch.zeros(Bz, L, C)), "y has dtype"),
    (dict(pieces=(20, 4), y=(torch.zeros(Bz, L, 20, dtype=BF),)), "y has 1 pieces"),
    (dict(), "on the GPU"),
])
def test_conv_fwd(kw, match):
    with pytest.raises(ValueError, match=match):
        ssd.short_conv_fwd(**conv_args(**kw))


@pytest.mark.parametrize("kw,match", [
    (dict(dy=None), "dy is required"),
    (dict(dy=torch.zeros(Bz, L, C)), "dy has dtype"),
    (dict(dy=torch.zeros(Bz, L, C - 1, dtype=BF)), "dy has shape"),
    (dict(dy=(torch.zeros(Bz, L, C - 1, dtype=BF), torch.zeros(Bz, L, 2, dtype=BF))), "pieces must be"),
    (dict(dfinal_window=torch.zeros(Bz, W - 1, C)), "dfinal_window has dtype"),
    (dict(workspace=torch.zeros(8, dtype=torch.uint8)), "workspace holds"),
])
def test_conv_bwd(kw, match):
    d = conv_args()
    d.setdefault("dy", torch.zeros(Bz, L, C, dtype=BF))
    d.update(kw)
    with pytest.raises(ValueError, match=match):
        ssd.short_conv_bwd(**d)


@pytest.mark.parametrize("kw,match", [
    (dict(window=None), "window is required"),
    (dict(window=torch.zeros(Bz, W, C, dtype=BF)), "window has shape"),
    (dict(x=torch.zeros(Bz, 1, C, dtype=BF)), "2-D"),
])
def test_conv_step(kw, match):
    d = dict(window=torch.zeros(Bz, W - 1, C, dtype=BF), x=torch.zeros(Bz, C, dtype=BF), weight=torch.zeros(C, W))
    d.update(kw)
    with pytest.raises(ValueError, match=match):
        ssd.short_conv_step(**d)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def conv_desc(**kw):
    d = dict(batch=2, seqlen=100, channels=64, width=4, x_bstride=6400, x_rstride=64, piece=(64, 0, 0), npieces=1,
             dtype=_lib.SSD_BF16, silu=1, reserved=0)
    d.update(kw)
    return _lib.ConvDesc(*[d[k] for k in ("batch", "seqlen", "channels", "width", "x_bstride", "x_rstride", "piece",
                                          "npieces", "dtype", "silu", "reserved")])


P = [ctypes.c_void_p(1 << k) for k in range(20, 44)]   # aligned, far apart, never dereferenced


def pieces(*p):
    return (ctypes.c_void_p * 3)(*p)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), _lib.SSD_ERR_SHAPE), (dict(channels=0), _lib.SSD_ERR_SHAPE),
    (dict(width=1), _lib.SSD_ERR_UNSUPPORTED), (dict(width=5), _lib.SSD_ERR_UNSUPPORTED),
    (dict(dtype=3), _lib.SSD_ERR_DTYPE), (dict(silu=2), _lib.SSD_ERR_SHAPE), (dict(reserved=1), _lib.SSD_ERR_SHAPE),
    (dict(npieces=0), _lib.SSD_ERR_SHAPE), (dict(npieces=4), _lib.SSD_ERR_SHAPE),
    (dict(piece=(60, 0, 0)), _lib.SSD_ERR_SHAPE), (dict(piece=(60, 4, 0)), _lib.SSD_ERR_SHAPE),
    (dict(piece=(65, -1, 0), npieces=2), _lib.SSD_ERR_SHAPE),
    (dict(x_rstride=-64), _lib.SSD_ERR_SHAPE), (dict(x_rstride=1 << 62), _lib.SSD_ERR_UNSUPPORTED),
    (dict(x_bstride=1 << 62), _lib.SSD_ERR_UNSUPPORTED), (dict(batch=1 << 40), _lib.SSD_ERR_UNSUPPORTED),
    (dict(seqlen=1 << 50), _lib.SSD_ERR_UNSUPPORTED),
    (dict(seqlen=1 << 31, channels=1 << 24, piece=(1 << 24, 0, 0)), _lib.SSD_ERR_UNSUPPORTED),
    (dict(batch=65535, seqlen=1, channels=65537, piece=(65535, 2, 0), npieces=2), _lib.SSD_ERR_UNSUPPORTED),
])
def test_conv_abi_shapes(lib, kw, code):
    d, n = conv_desc(**kw), ctypes.c_size_t()
    assert lib.ssd_short_conv_fwd(d, P[0], P[1], None, None, None, pieces(P[2]), None, None) == code
    assert lib.ssd_last_error() != b""
    assert lib.ssd_short_conv_bwd_workspace_bytes(d, n) == code


def test_conv_abi_pointers(lib):
    d, n = conv_desc(), ctypes.c_size_t()
    fwd = lambda x=P[0], w=P[1], b=None, w0=None, ls=None, y=pieces(P[2]), w1=None, d=d: \
        lib.ssd_short_conv_fwd(d, x, w, b, w0, ls, y, w1, None)
    assert fwd(x=None) == fwd(w=None) == fwd(y=pieces()) == _lib.SSD_ERR_NULL
    assert lib.ssd_short_conv_fwd(None, P[0], P[1], None, None, None, pieces(P[2]), None, None) == _lib.SSD_ERR_NULL
    odd = ctypes.c_void_p((1 << 20) + 1)
    assert fwd(x=odd) == fwd(w=odd) == fwd(y=pieces(odd)) == fwd(w0=odd) == fwd(ls=odd) == _lib.SSD_ERR_ALIGN
    assert fwd(y=pieces(P[0])) == fwd(w1=P[2]) == fwd(w0=P[3], w1=P[3]) == _lib.SSD_ERR_ALIAS
    two = conv_desc(piece=(32, 32, 0), npieces=2)
    assert fwd(y=pieces(P[2]), d=two) == _lib.SSD_ERR_NULL
    assert fwd(y=pieces(P[2], P[2]), d=two) == _lib.SSD_ERR_ALIAS
    # nothing to do: no launch
    assert fwd(d=conv_desc(batch=0), x=None) == fwd(d=conv_desc(seqlen=0), x=None) == _lib.SSD_OK

    assert lib.ssd_short_conv_bwd_workspace_bytes(d, n) == 0 and n.value >= 2 * 5 * 64 * 4
    bwd = lambda dy=pieces(P[2]), b=None, dx=P[3], dw=P[4], db=None, ws=P[5], wsz=n.value, d=d: \
        lib.ssd_short_conv_bwd(d, P[0], P[1], b, None, None, dy, None, dx, dw, db, None, ws, wsz, None)
    assert bwd(dy=pieces()) == bwd(dx=None) == bwd(dw=None) == bwd(b=P[6]) == bwd(db=P[6]) == _lib.SSD_ERR_NULL
    assert bwd(ws=None) == bwd(wsz=n.value - 1) == _lib.SSD_ERR_WORKSPACE
    assert bwd(ws=ctypes.c_void_p((1 << 25) + 4)) == _lib.SSD_ERR_ALIGN
    assert bwd(dx=P[0]) == bwd(dw=P[3]) == bwd(ws=P[3]) == _lib.SSD_ERR_ALIAS

    one = conv_desc(seqlen=1)
    step = lambda w=P[3], y=pieces(P[2]), d=one: lib.ssd_short_conv_step(d, w, P[0], P[1], None, y, None)
    assert step(d=d) == _lib.SSD_ERR_SHAPE
    assert step(w=None) == _lib.SSD_ERR_NULL
    assert step(w=P[0]) == step(y=pieces(P[0])) == _lib.SSD_ERR_ALIAS
    assert step(d=conv_desc(batch=0, seqlen=1)) == _lib.SSD_OK


# ---- per-channel scan ---------------------------------------------------------------
D, N, G = 24, 16, 2


def scan_args(lead=(Bz, L), **kw):
    d = dict(u=torch.zeros(*lead, D, dtype=BF), delta=torch.zeros(*lead, D, dtype=BF), A=torch.zeros(D, N),
             B=torch.zeros(*lead, G, N, dtype=BF), C=torch.zeros(*lead, G, N, dtype=BF))
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,match", [
    (dict(u=torch.zeros(L, D, dtype=BF)), "u must be"),
    (dict(u=torch.zeros(Bz, D, L, dtype=BF).transpose(1, 2)), "rows of u"),
    (dict(delta=None), "delta is required"),
    (dict(delta=torch.zeros(Bz, L, D)), "delta has dtype"),
    (dict(A=torch.zeros(D)), "A must be"),
    (dict(A=torch.zeros(D + 1, N)), "A has shape"),
    (dict(A=torch.zeros(D, N, dtype=BF)), "A has dtype"),
    (dict(B=torch.zeros(Bz, L, N, dtype=BF)), "B must be"),
    (dict(B=torch.zeros(Bz, L, G, N + 1, dtype=BF)), "B has shape"),
    (dict(C=torch.zeros(Bz, L, 1, N, dtype=BF)), "C has shape"),
    (dict(C=torch.zeros(Bz, L, N, G, dtype=BF).transpose(2, 3)), "rows of C"),
    (dict(gate=torch.zeros(Bz, L, D + 1, dtype=BF)), "gate has shape"),
    (dict(skip=torch.zeros(D, dtype=BF)), "skip has dtype"),
    (dict(delta_bias=torch.zeros(D, 1)), "delta_bias has shape"),
    (dict(initial_state=torch.zeros(Bz, D, N, dtype=BF)), "initial_state has dtype"),
    (dict(final_state=torch.zeros(Bz, N, D)), "final_state has shape"),
    (dict(y=torch.zeros(Bz, L, D)), "y has dtype"),
    (dict(seqlens=torch.zeros(Bz)), "seqlens has dtype"),
    (dict(), "on the GPU"),
])
def test_scan_fwd(kw, match):
    with pytest.raises(ValueError, match=match):
        ssd.channel_scan_fwd(**scan_args(**kw))


@pytest.mark.parametrize("kw,match", [
    (dict(state=None), "state is required"),
    (dict(state=torch.zeros(Bz, D, N, dtype=BF)), "state has dtype"),
    (dict(u=torch.zeros(Bz, 1, D, dtype=BF)), "u must be"),
    (dict(y=torch.zeros(Bz, D)), "y has dtype"),
])
def test_channel_step(kw, match):
    d = scan_args((Bz,), state=torch.zeros(Bz, D, N))
    d.update(kw)
    with pytest.raises(ValueError, match=match):
        ssd.channel_step(**d)


def chan_desc(**kw):
    d = dict(batch=2, seqlen=100, channels=64, dstate=16, ngroups=2, u_bstride=6400, u_rstride=64, delta_bstride=6400,
             delta_rstride=64, gate_bstride=6400, gate_rstride=64, B_bstride=3200, B_rstride=32, C_bstride=3200,
             C_rstride=32, dtype=_lib.SSD_BF16, softplus=1)
    d.update(kw)
    return _lib.ChannelDesc(*d.values())


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), _lib.SSD_ERR_SHAPE), (dict(seqlen=-1), _lib.SSD_ERR_SHAPE), (dict(channels=0), _lib.SSD_ERR_SHAPE),
    (dict(dstate=0), _lib.SSD_ERR_SHAPE), (dict(dstate=65), _lib.SSD_ERR_UNSUPPORTED),
    (dict(ngroups=3), _lib.SSD_ERR_SHAPE), (dict(dtype=2), _lib.SSD_ERR_DTYPE), (dict(softplus=2), _lib.SSD_ERR_SHAPE),
    (dict(B_rstride=-1), _lib.SSD_ERR_SHAPE), (dict(C_bstride=1 << 60), _lib.SSD_ERR_UNSUPPORTED),
    (dict(batch=1 << 20), _lib.SSD_ERR_UNSUPPORTED), (dict(channels=1 << 30), _lib.SSD_ERR_UNSUPPORTED),
    (dict(seqlen=1 << 40), _lib.SSD_ERR_UNSUPPORTED), (dict(seqlen=(1 << 30) + 1), _lib.SSD_ERR_UNSUPPORTED),
    (dict(channels=1 << 17, ngroups=1 << 17), _lib.SSD_ERR_UNSUPPORTED),
    (dict(u_rstride=(1 << 24) + 1), _lib.SSD_ERR_UNSUPPORTED),
    (dict(batch=1 << 15, channels=1 << 12), _lib.SSD_ERR_UNSUPPORTED),
])
def test_scan_abi_shapes(lib, kw, code):
    d, n = chan_desc(**kw), ctypes.c_size_t()
    none = [None] * 5
    assert lib.ssd_channel_scan_fwd(d, *P[:5], *none, P[6], None, None, 0, None) == code
    assert lib.ssd_last_error() != b""
    assert lib.ssd_channel_scan_fwd_workspace_bytes(d, n) == code


def test_scan_abi_pointers(lib):
    n, odd = ctypes.c_size_t(), ctypes.c_void_p((1 << 20) + 1)
    d = chan_desc()
    assert lib.ssd_channel_scan_fwd_workspace_bytes(d, n) == 0
    ws = ctypes.c_void_p(1 << 45)

    def fwd(d=d, wsz=n.value, ws=ws, **kw):
        a = dict(zip(("u", "delta", "A", "B", "C"), P), skip=None, gate=None, bias=None, h0=None, lens=None, y=P[6],
                 fin=None)
        a.update(kw)
        return lib.ssd_channel_scan_fwd(d, *a.values(), ws, wsz, None)

    for k in ("u", "delta", "A", "B", "C", "y"):
        assert fwd(**{k: None}) == _lib.SSD_ERR_NULL
        assert fwd(**{k: odd}) == _lib.SSD_ERR_ALIGN
    for k in ("skip", "gate", "bias", "h0", "lens", "fin"):
        assert fwd(**{k: odd}) == _lib.SSD_ERR_ALIGN
    assert fwd(y=P[0]) == fwd(fin=P[2]) == fwd(h0=P[7], fin=P[7]) == fwd(fin=P[6]) == _lib.SSD_ERR_ALIAS
    assert fwd(d=chan_desc(batch=0), u=None, y=None) == fwd(d=chan_desc(seqlen=0), y=None) == _lib.SSD_OK
    # a single step has no stride between steps
    assert fwd(d=chan_desc(seqlen=1, u_rstride=1 << 39), u=None) == _lib.SSD_ERR_NULL
    # a long sequence of few channels is cut into segments, which need a workspace
    long = chan_desc(batch=1, seqlen=1 << 16, u_bstride=0)
    assert lib.ssd_channel_scan_fwd_workspace_bytes(long, n) == 0
    assert n.value > 0
    assert fwd(d=long, ws=None) == fwd(d=long, wsz=n.value - 1) == _lib.SSD_ERR_WORKSPACE
    assert fwd(d=long, wsz=n.value, ws=ctypes.c_void_p((1 << 45) + 4)) == _lib.SSD_ERR_ALIGN
    assert fwd(d=long, wsz=n.value, ws=P[6]) == _lib.SSD_ERR_ALIAS

    one = chan_desc(seqlen=1)
    step = lambda st=P[8], y=P[6], d=one: lib.ssd_channel_step(d, st, *P[:5], None, None, None, y, None)
    assert step(d=d) == _lib.SSD_ERR_SHAPE
    assert step(st=None) == step(y=None) == _lib.SSD_ERR_NULL
    assert step(st=P[0]) == step(y=P[8]) == _lib.SSD_ERR_ALIAS
    assert step(d=chan_desc(batch=0, seqlen=1)) == _lib.SSD_OK


@pytest.mark.parametrize("kw,match", [
    (dict(dy=None), "dy is required"),
    (dict(dy=torch.zeros(Bz, L, D)), "dy has dtype"),
    (dict(dy=torch.zeros(Bz, D, L, dtype=BF).transpose(1, 2)), "dy must be contiguous"),
    (dict(dfinal_state=torch.zeros(Bz, D, N, dtype=BF)), "dfinal_state has dtype"),
    (dict(initial_state=torch.zeros(Bz, D + 1, N)), "initial_state has shape"),
    (dict(workspace=torch.zeros(16, dtype=torch.uint8)), "workspace holds"),
    (dict(seqlens=torch.zeros(Bz, dtype=torch.int64)), "seqlens has dtype"),
    (dict(), "on the GPU"),
])
def test_scan_bwd(kw, match):
    d = scan_args(dy=torch.zeros(Bz, L, D, dtype=BF))
    d.update(kw)
    with pytest.raises(ValueError, match=match):
        ssd.channel_scan_bwd(**d)


def test_scan_bwd_abi(lib):
    n, odd = ctypes.c_size_t(), ctypes.c_void_p((1 << 20) + 1)
    names = ("du", "ddelta", "dgate", "dB", "dC", "dA", "dskip", "ddelta_bias", "dinitial_state")
    ws = ctypes.c_void_p(1 << 46)

    def bwd(d=chan_desc(), wsz=None, ws=ws, dy=P[5], skip=None, gate=None, bias=None, dh=None, u=P[0], **kw):
        assert lib.ssd_channel_scan_bwd_workspace_bytes(d, n) == 0
        g = dict(zip(names, (P[6], P[7], None, P[8], P[9], P[10], None, None, None)))
        g.update(kw)
        grads = _lib.ChannelGrads(*[v.value if v is not None else None for v in g.values()])
        return lib.ssd_channel_scan_bwd(d, u, *P[1:5], skip, gate, bias, None, None, dy, dh, grads, ws,
                                        n.value if wsz is None else wsz, None)

    for k in ("du", "ddelta", "dB", "dC", "dA"):
        assert bwd(**{k: None}) == _lib.SSD_ERR_NULL
        assert bwd(**{k: odd}) == _lib.SSD_ERR_ALIGN
        assert bwd(**{k: P[0]}) == _lib.SSD_ERR_ALIAS
    assert bwd(dy=None) == _lib.SSD_ERR_NULL
    # gradients of optional inputs: given exactly with them
    for k, i in (("dgate", "gate"), ("dskip", "skip"), ("ddelta_bias", "bias")):
        assert bwd(**{k: P[12]}) == bwd(**{i: P[12]}) == _lib.SSD_ERR_NULL
    assert bwd(dy=odd) == bwd(dh=odd) == bwd(dinitial_state=odd) == _lib.SSD_ERR_ALIGN
    assert bwd(du=P[5]) == bwd(du=P[7]) == bwd(ws=P[6]) == bwd(dinitial_state=P[10]) == _lib.SSD_ERR_ALIAS
    assert bwd(wsz=8) == bwd(ws=None) == _lib.SSD_ERR_WORKSPACE
    assert bwd(ws=ctypes.c_void_p((1 << 46) + 8)) == _lib.SSD_ERR_ALIGN
    assert lib.ssd_channel_scan_bwd(chan_desc(), *P[:5], None, None, None, None, None, P[5], None, None, ws, 1 << 40,
                                    None) == _lib.SSD_ERR_NULL
    # more rows than a launch of the sums of dB and dC reaches
    big = chan_desc(batch=1, seqlen=1 << 30, u_bstride=0)
    assert lib.ssd_channel_scan_bwd_workspace_bytes(big, n) == _lib.SSD_ERR_UNSUPPORTED
