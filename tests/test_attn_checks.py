"""Argument checks of linear attention and the group norm, in the binding and
behind the C ABI, on the CPU: nothing here launches a kernel."""
import ctypes

import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from ssd_chunked_scan_chunk_amd import _lib

Bz, L, H, K, Dk, Dv, C = 2, 10, 4, 2, 24, 16, 24
BF, F32 = torch.bfloat16, torch.float32


def attn_args(**kw):
    d = dict(q=torch.zeros(Bz, L, H, Dk, dtype=BF), k=torch.zeros(Bz, L, K, Dk, dtype=BF),
             v=torch.zeros(Bz, L, K, Dv, dtype=BF), log_decay=torch.zeros(H))
    d.update(kw)
    return d


SHARED = [
    (dict(q=torch.zeros(L, H, Dk, dtype=BF)), "4-D"),
    (dict(q=torch.zeros(Bz, L, Dk, H, dtype=BF).transpose(2, 3)), "rows of q"),
    (dict(q=torch.zeros(Bz, L, H, 2 * Dk, dtype=BF)[..., :Dk]), "rows of q"),
    (dict(k=None), "k must be a 4-D"),
    (dict(k=torch.zeros(Bz, L, K, Dk + 1, dtype=BF)), "k has shape"),
    (dict(k=torch.zeros(Bz, L, K, Dk)), "k has dtype"),
    (dict(v=torch.zeros(Bz, L, K + 1, Dv, dtype=BF)), "v has shape"),
    (dict(v=torch.zeros(Bz, L + 1, K, Dv, dtype=BF)), "v has shape"),
    (dict(log_decay=None), "log_decay is required"),
    (dict(log_decay=torch.zeros(H + 1)), "log_decay has shape"),
    (dict(log_decay=torch.zeros(H, dtype=BF)), "log_decay has dtype"),
    (dict(log_decay=torch.zeros(2 * H)[::2]), "contiguous"),
    (dict(initial_state=torch.zeros(Bz, H, Dk, Dv)), "initial_state has shape"),
    (dict(initial_state=torch.zeros(Bz, H, Dv, Dk, dtype=BF)), "initial_state has dtype"),
    (dict(seqlens=torch.zeros(Bz, dtype=torch.int64)), "seqlens has dtype"),
    (dict(seqlens=torch.zeros(Bz + 1, dtype=torch.int32)), "seqlens has shape"),
    (dict(), "on the GPU"),
]


@pytest.mark.parametrize("kw,match", SHARED + [
    (dict(y=torch.zeros(Bz, L, H, Dv)), "y has dtype"),
    (dict(y=torch.zeros(Bz, L, H, Dk, dtype=BF)), "y has shape"),
    (dict(final_state=torch.zeros(Bz, K, Dv, Dk)), "final_state has shape"),
])
def test_attn_fwd(kw, match):
    with pytest.raises(ValueError, match=match):
        ssd.linear_attn_fwd(**attn_args(**kw))


@pytest.mark.parametrize("kw,match", SHARED + [
    (dict(dy=None), "dy is required"),
    (dict(dy=torch.zeros(Bz, L, H, Dv)), "dy has dtype"),
    (dict(dy=torch.zeros(Bz, L, K, Dv, dtype=BF)), "dy has shape"),
    (dict(dfinal_state=torch.zeros(Bz, H, Dk, Dv)), "dfinal_state has shape"),
    (dict(workspace=torch.zeros(8, dtype=torch.uint8)), "workspace holds"),
])
def test_attn_bwd(kw, match):
    with pytest.raises(ValueError, match=match):
        ssd.linear_attn_bwd(**attn_args(**dict(dict(dy=torch.zeros(Bz, L, H, Dv, dtype=BF)), **kw)))


@pytest.mark.parametrize("kw,match", [
    (dict(state=None), "state is required"),
    (dict(state=torch.zeros(Bz, H, Dk, Dv)), "state has shape"),
    (dict(q=torch.zeros(Bz, 1, H, Dk, dtype=BF)), "3-D"),
    (dict(y=torch.zeros(Bz, H, Dv)), "y has dtype"),
    (dict(), "on the GPU"),
])
def test_attn_step(kw, match):
    a = {n: t[:, 0] if n != "log_decay" else t for n, t in attn_args().items()}
    with pytest.raises(ValueError, match=match):
        ssd.linear_attn_step(**dict(dict(a, state=torch.zeros(Bz, H, Dv, Dk)), **kw))


def test_types():
    with pytest.raises(TypeError):
        ssd.linear_attn_fwd(**attn_args(q=torch.zeros(Bz, L, H, Dk, dtype=torch.float16)))
    with pytest.raises(TypeError):
        ssd.group_norm_fwd(torch.zeros(2, C, dtype=torch.float16), 2)
    with pytest.raises(TypeError):
        ssd.linear_attn_fwd(**attn_args(seqlens=[1, 2]))


NORM = [
    (dict(x=torch.zeros(C, dtype=BF)), "x must be"),
    (dict(x=torch.zeros(Bz, C, L, dtype=BF).transpose(1, 2)), "rows of x"),
    (dict(weight=torch.zeros(C - 1)), "weight has shape"),
    (dict(weight=torch.zeros(C, dtype=BF)), "weight has dtype"),
    (dict(bias=torch.zeros(C + 1)), "bias has shape"),
    (dict(gate=torch.zeros(Bz, L, C)), "gate has dtype"),
    (dict(gate=torch.zeros(Bz, L, C + 1, dtype=BF)), "gate has shape"),
    (dict(gate_first=True), "gate_first needs a gate"),
    (dict(seqlens=torch.zeros(Bz, dtype=torch.int64)), "seqlens has dtype"),
    (dict(), "on the GPU"),
]


@pytest.mark.parametrize("kw,match", NORM + [
    (dict(y=torch.zeros(Bz, L, C)), "y has dtype"),
    (dict(x=torch.zeros(Bz, C, dtype=BF), seqlens=torch.zeros(Bz, dtype=torch.int32)), "seqlens needs x"),
])
def test_norm_fwd(kw, match):
    with pytest.raises(ValueError, match=match):
        ssd.group_norm_fwd(**dict(dict(x=torch.zeros(Bz, L, C, dtype=BF), groups=3), **kw))


@pytest.mark.parametrize("kw,match", NORM[1:] + [
    (dict(dy=None), "dy is required"),
    (dict(dy=torch.zeros(Bz, L, C)), "dy has dtype"),
    (dict(dy=torch.zeros(Bz, L, 2 * C, dtype=BF)[..., :C]), "contiguous"),
    (dict(workspace=torch.zeros(8, dtype=torch.uint8)), "workspace holds"),
])
def test_norm_bwd(kw, match):
    base = dict(x=torch.zeros(Bz, L, C, dtype=BF), groups=3, dy=torch.zeros(Bz, L, C, dtype=BF))
    with pytest.raises(ValueError, match=match):
        ssd.group_norm_bwd(**dict(base, **kw))


@pytest.mark.parametrize("groups", [0, -1, 5])
def test_groups(groups):
    with pytest.raises(ssd.SSDError, match="SSD_ERR_SHAPE"):
        ssd.group_norm_bwd_workspace_bytes(torch.zeros(Bz, L, C, dtype=BF), groups)


def test_workspace_queries():
    a = attn_args()
    assert ssd.linear_attn_fwd_workspace_bytes(**a) == 0
    # shared heads: the heads' dk and dv, rounded up to 256 bytes each
    up = lambda n: -(-n // 256) * 256   # noqa: E731
    assert ssd.linear_attn_bwd_workspace_bytes(**a) == up(Bz * L * H * Dk * 4) + up(Bz * L * H * Dv * 4)
    one = attn_args(q=torch.zeros(1, 4096, 1, 32, dtype=BF), k=torch.zeros(1, 4096, 1, 32, dtype=BF),
                    v=torch.zeros(1, 4096, 1, 48, dtype=BF), log_decay=torch.zeros(1))
    n = ssd.linear_attn_fwd_workspace_bytes(**one)
    assert n > 0 and n % (32 * 48 * 4) == 0
    assert ssd.linear_attn_bwd_workspace_bytes(**one) >= 2 * n
    assert ssd.group_norm_bwd_workspace_bytes(torch.zeros(Bz, L, C), 3) % (2 * C * 4) == 0
    assert ssd.group_norm_bwd_workspace_bytes(torch.zeros(0, L, C), 3) == 0


# ---- behind the C ABI ------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    return _lib.load()


F = [ctypes.c_void_p(1 << k) for k in range(30, 46)]     # aligned, far apart, never dereferenced


def attn_desc(**kw):
    d = dict(batch=2, seqlen=100, nheads=8, kv_heads=4, key_dim=64, value_dim=32, q_bstride=51200, q_rstride=512,
             k_bstride=25600, k_rstride=256, v_bstride=12800, v_rstride=128, scale=1.0, dtype=_lib.SSD_BF16)
    d.update(kw)
    return _lib.LinearAttnDesc(*(d[n] for n, _ in _lib.LinearAttnDesc._fields_))


def attn_fwd(lib, d, q=F[0], k=F[1], v=F[2], ld=F[3], first=None, lens=None, y=F[4], last=None, ws=None, wsz=0):
    return lib.ssd_linear_attn_fwd(d, q, k, v, ld, first, lens, y, last, ws, wsz, None)


def attn_bwd(lib, d, q=F[0], k=F[1], v=F[2], ld=F[3], first=None, lens=None, dy=F[4], dlast=None, dq=F[5], dk=F[6],
             dv=F[7], dfirst=None, ws=F[8], wsz=1 << 40):
    return lib.ssd_linear_attn_bwd(d, q, k, v, ld, first, lens, dy, dlast, dq, dk, dv, dfirst, ws, wsz, None)


def attn_step(lib, d, state=F[5], q=F[0], k=F[1], v=F[2], ld=F[3], y=F[4]):
    return lib.ssd_linear_attn_step(d, state, q, k, v, ld, y, None)


ATTN_BAD = [
    (dict(batch=-1), _lib.SSD_ERR_SHAPE), (dict(seqlen=-1), _lib.SSD_ERR_SHAPE), (dict(nheads=0), _lib.SSD_ERR_SHAPE),
    (dict(kv_heads=0), _lib.SSD_ERR_SHAPE), (dict(kv_heads=3), _lib.SSD_ERR_SHAPE), (dict(key_dim=0), _lib.SSD_ERR_SHAPE),
    (dict(value_dim=0), _lib.SSD_ERR_SHAPE), (dict(dtype=7), _lib.SSD_ERR_DTYPE),
    (dict(key_dim=257), _lib.SSD_ERR_UNSUPPORTED), (dict(value_dim=257), _lib.SSD_ERR_UNSUPPORTED),
    (dict(batch=65536), _lib.SSD_ERR_UNSUPPORTED), (dict(seqlen=(1 << 30) + 1), _lib.SSD_ERR_UNSUPPORTED),
    (dict(nheads=65536, kv_heads=65536), _lib.SSD_ERR_UNSUPPORTED),
    (dict(q_rstride=-1), _lib.SSD_ERR_SHAPE), (dict(v_bstride=-1), _lib.SSD_ERR_SHAPE),
    (dict(k_rstride=(1 << 24) + 1), _lib.SSD_ERR_UNSUPPORTED), (dict(k_bstride=1 << 62), _lib.SSD_ERR_UNSUPPORTED),
    (dict(batch=65535, nheads=128, kv_heads=128), _lib.SSD_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", ATTN_BAD)
def test_attn_descriptors(lib, kw, code):
    d, n = attn_desc(**kw), ctypes.c_size_t(5)
    assert lib.ssd_linear_attn_fwd_workspace_bytes(d, n) == code and lib.ssd_last_error()
    assert lib.ssd_linear_attn_bwd_workspace_bytes(d, n) == code and n.value == 5
    assert attn_fwd(lib, d) == code and attn_bwd(lib, d) == code
    if not {"seqlen", "k_rstride"} & set(kw):   # of one row: the same refusal
        assert attn_step(lib, attn_desc(**dict(dict(seqlen=1), **kw))) == code


def test_attn_pointers(lib):
    d, odd = attn_desc(), ctypes.c_void_p((1 << 33) + 1)
    N, A, W, X = _lib.SSD_ERR_NULL, _lib.SSD_ERR_ALIGN, _lib.SSD_ERR_WORKSPACE, _lib.SSD_ERR_ALIAS
    for name in ("q", "k", "v", "ld", "y"):
        assert attn_fwd(lib, d, **{name: None}) == N and attn_fwd(lib, d, **{name: odd}) == A
    for name in ("first", "last", "lens"):
        assert attn_fwd(lib, d, **{name: odd}) == A
    for name in ("q", "k", "v", "ld", "dy", "dq", "dk", "dv"):
        assert attn_bwd(lib, d, **{name: None}) == N and attn_bwd(lib, d, **{name: odd}) == A
    for name in ("first", "dlast", "dfirst", "lens"):
        assert attn_bwd(lib, d, **{name: odd}) == A
    assert attn_bwd(lib, d, ws=None) == W and attn_bwd(lib, d, wsz=16) == W
    assert attn_bwd(lib, d, ws=ctypes.c_void_p((1 << 38) + 8)) == A
    # outputs over inputs, over each other, over the workspace
    assert attn_fwd(lib, d, y=F[2]) == X and attn_fwd(lib, d, last=F[4]) == X
    assert attn_fwd(lib, d, first=F[6], last=F[6]) == X
    for name in ("dq", "dk", "dv", "dfirst"):
        assert attn_bwd(lib, d, **{name: F[0]}) == X and attn_bwd(lib, d, **{name: F[8]}) == X
    assert attn_bwd(lib, d, dk=F[5]) == X and attn_bwd(lib, d, ws=F[4]) == X
    long = attn_desc(seqlen=1 << 16, batch=1)
    assert attn_fwd(lib, long) == W                       # segments need a workspace
    assert attn_step(lib, d) == _lib.SSD_ERR_SHAPE        # a step is one row
    one = attn_desc(seqlen=1)
    for name in ("state", "q", "k", "v", "ld", "y"):
        assert attn_step(lib, one, **{name: None}) == N and attn_step(lib, one, **{name: odd}) == A
    assert attn_step(lib, one, y=F[5]) == X and attn_step(lib, one, state=F[0]) == X
    assert attn_fwd(lib, None) == N and lib.ssd_linear_attn_fwd_workspace_bytes(d, None) == N
    # nothing to do needs nothing
    assert attn_fwd(lib, attn_desc(batch=0), q=None, k=None, v=None, y=None) == _lib.SSD_OK
    assert attn_fwd(lib, attn_desc(seqlen=0), q=None, k=None, v=None, y=None) == _lib.SSD_OK
    assert attn_bwd(lib, attn_desc(batch=0), q=None, k=None, v=None, dy=None, dq=None, dk=None, dv=None) == _lib.SSD_OK


def norm_desc(**kw):
    d = dict(batch=2, seqlen=100, channels=96, groups=3, x_bstride=9600, x_rstride=96, gate_bstride=9600, gate_rstride=96,
             eps=1e-5, dtype=_lib.SSD_BF16, center=1, silu=1, gate_first=0, reserved=0)
    d.update(kw)
    return _lib.GroupNormDesc(*(d[n] for n, _ in _lib.GroupNormDesc._fields_))


def norm_fwd(lib, d, x=F[0], w=F[1], b=F[2], gate=F[3], lens=None, y=F[4]):
    return lib.ssd_group_norm_fwd(d, x, w, b, gate, lens, y, None)


def norm_bwd(lib, d, x=F[0], w=F[1], b=F[2], gate=F[3], lens=None, dy=F[4], dx=F[5], dgate=F[6], dw=F[7], db=F[8],
             ws=F[9], wsz=1 << 40):
    return lib.ssd_group_norm_bwd(d, x, w, b, gate, lens, dy, dx, dgate, dw, db, ws, wsz, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), _lib.SSD_ERR_SHAPE), (dict(channels=0), _lib.SSD_ERR_SHAPE), (dict(groups=0), _lib.SSD_ERR_SHAPE),
    (dict(groups=5), _lib.SSD_ERR_SHAPE), (dict(dtype=9), _lib.SSD_ERR_DTYPE), (dict(center=2), _lib.SSD_ERR_SHAPE),
    (dict(silu=-1), _lib.SSD_ERR_SHAPE), (dict(gate_first=2), _lib.SSD_ERR_SHAPE), (dict(reserved=1), _lib.SSD_ERR_SHAPE),
    (dict(eps=-1e-5), _lib.SSD_ERR_SHAPE), (dict(eps=float("nan")), _lib.SSD_ERR_SHAPE),
    (dict(eps=float("inf")), _lib.SSD_ERR_SHAPE),
    (dict(channels=16385, groups=1), _lib.SSD_ERR_UNSUPPORTED), (dict(batch=65536), _lib.SSD_ERR_UNSUPPORTED),
    (dict(batch=4, seqlen=1 << 30), _lib.SSD_ERR_UNSUPPORTED),
    (dict(x_rstride=-1), _lib.SSD_ERR_SHAPE), (dict(gate_bstride=1 << 60), _lib.SSD_ERR_UNSUPPORTED),
])
def test_norm_descriptors(lib, kw, code):
    d, n = norm_desc(**kw), ctypes.c_size_t(5)
    assert lib.ssd_group_norm_bwd_workspace_bytes(d, n) == code and n.value == 5 and lib.ssd_last_error()
    assert norm_fwd(lib, d) == code and norm_bwd(lib, d) == code


def test_norm_pointers(lib):
    d, odd = norm_desc(), ctypes.c_void_p((1 << 33) + 1)
    N, A, W, X = _lib.SSD_ERR_NULL, _lib.SSD_ERR_ALIGN, _lib.SSD_ERR_WORKSPACE, _lib.SSD_ERR_ALIAS
    assert norm_fwd(lib, d, x=None) == N and norm_fwd(lib, d, y=None) == N
    for name in ("x", "w", "b", "gate", "lens", "y"):
        assert norm_fwd(lib, d, **{name: odd}) == A
    for name in ("x", "dy", "dx", "dgate", "dw", "db", "gate", "w", "b"):    # a gradient exactly for what is given
        assert norm_bwd(lib, d, **{name: None}) == N
    for name in ("x", "w", "b", "gate", "lens", "dy", "dx", "dgate", "dw", "db"):
        assert norm_bwd(lib, d, **{name: odd}) == A
    assert norm_fwd(lib, norm_desc(gate_first=1), gate=None) == N
    assert norm_bwd(lib, d, ws=None) == W and norm_bwd(lib, d, wsz=64) == W
    assert norm_fwd(lib, d, y=F[0]) == X and norm_fwd(lib, d, y=F[3]) == X
    for name in ("dx", "dgate", "dw", "db", "ws"):
        assert norm_bwd(lib, d, **{name: F[4]}) == X
    assert norm_bwd(lib, d, dgate=F[5]) == X and norm_bwd(lib, d, dw=F[9]) == X
    assert norm_fwd(lib, None) == N and lib.ssd_group_norm_bwd_workspace_bytes(d, None) == N
    assert norm_fwd(lib, norm_desc(batch=0), x=None, gate=None, y=None) == _lib.SSD_OK


@pytest.mark.parametrize("batch,nheads,fits", [(1, 1000, True), (65535, 21, True), (65535, 22, False), (22, 65535, False)])
def test_attn_launch_size(lib, batch, nheads, fits):
    # 512 threads for each of two slices and three walks of a pair: at most 2^32 items of a launch
    d, size = attn_desc(batch=batch, seqlen=1, nheads=nheads, kv_heads=1, key_dim=1, value_dim=1), ctypes.c_size_t()
    for name in ("fwd", "bwd"):
        code = getattr(lib, "ssd_linear_attn_%s_workspace_bytes" % name)(ctypes.byref(d), ctypes.byref(size))
        assert code == (0 if fits else _lib.SSD_ERR_UNSUPPORTED)
