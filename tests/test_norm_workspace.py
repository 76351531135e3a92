"""The group norm's backward holds parts of dweight and dbias in its workspace: without either it needs none."""
import ctypes

import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from ssd_chunked_scan_chunk_amd import _lib
from test_attn_checks import F, norm_bwd, norm_desc

NONE = dict(w=None, b=None, dw=None, db=None)


def test_without_parameters_none_is_asked_for():
    # dx over dy is refused after the workspace has been looked at: nothing is launched
    lib, d = _lib.load(), norm_desc()
    X, W = _lib.SSD_ERR_ALIAS, _lib.SSD_ERR_WORKSPACE
    assert norm_bwd(lib, d, dx=F[4], ws=None, wsz=0, **NONE) == X
    assert norm_bwd(lib, d, dx=F[4], ws=None, wsz=0, **dict(NONE, w=F[1], dw=F[7])) == W
    assert norm_bwd(lib, d, dx=F[4], ws=None, wsz=0, **dict(NONE, b=F[2], db=F[8])) == W
    n = ctypes.c_size_t()
    assert lib.ssd_group_norm_bwd_workspace_bytes(d, n) == _lib.SSD_OK and n.value > 0   # what the parameters need


def test_without_parameters_none_is_allocated(monkeypatch):
    def empty(*a, **kw):
        raise AssertionError("a workspace was allocated")

    x = torch.zeros(2, 10, 24)
    monkeypatch.setattr(torch, "empty", empty)
    with pytest.raises(ValueError, match="on the GPU"):
        ssd.group_norm_bwd(x, 3, x)
    with pytest.raises(AssertionError, match="allocated"):
        ssd.group_norm_bwd(x, 3, x, weight=torch.ones(24))


@pytest.mark.gpu
@pytest.mark.parametrize("C,groups", [(96, 3), (1200, 1), (6, 3)])
def test_gradients_without_parameters(C, groups):
    g = torch.Generator().manual_seed(C)
    x, z, dy = (torch.randn(2, 30, C, generator=g).cuda() for _ in range(3))
    ws = torch.empty(ssd.group_norm_bwd_workspace_bytes(x, groups), dtype=torch.uint8, device="cuda")
    a, b = ssd.group_norm_bwd(x, groups, dy, gate=z), ssd.group_norm_bwd(x, groups, dy, gate=z, workspace=ws)
    c = ssd.group_norm_bwd(x, groups, dy, gate=z, weight=torch.ones(C, device="cuda"))
    torch.cuda.synchronize()
    assert a["dweight"] is None and a["dbias"] is None
    for n in ("dx", "dgate"):
        assert torch.equal(a[n], b[n]) and torch.equal(a[n], c[n])
