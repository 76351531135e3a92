"""GPU parity of the operators around the chunked scan in the instances that large
shapes get (layer_cases.py), against the plain 64-bit forms.  Only some sequences
are compared; of the backward only those have an upstream gradient, so that sums
over the batch are theirs alone."""
import numpy as np
import pytest
import torch

import layer_cases as cases
import layer_ref as ref
import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log
from test_gpu_channel_scan import DT, inputs, lens_of, n64, want_of

pytestmark = pytest.mark.gpu

KINDS = [("bf16", False), ("bf16", True), ("f32", True)]
SHARED = ("A", "skip", "delta_bias")   # not of a sequence


def some(Bz, L):
    """The first sequences (empty, whole, one step, one short of whole: layer_cases.lengths),
    two from the middle and the last two; fewer of long ones."""
    return sorted({b for b in ((1, 3, Bz // 2, Bz - 1) if L > 100 else
                               (0, 1, 2, 3, Bz // 3, Bz // 2, Bz - 2, Bz - 1)) if 0 <= b < Bz})


def of(d, pick):
    return {k: v if v is None or k in SHARED else v[pick] for k, v in d.items()}


@pytest.mark.parametrize("dtype,ragged", KINDS)
@pytest.mark.parametrize("Bz,L,D,N,G,plan", cases.SCAN_FWD)
def test_scan_forward(dtype, ragged, Bz, L, D, N, G, plan):
    log("channel scan fwd plan %s" % ((dtype, ragged, Bz, L, D, N, G, plan),))
    d = inputs(Bz, L, D, N, G, dtype, L + N, wide=2)
    lens = (cases.lengths(Bz, L) if Bz > 1 else [L - 3]) if ragged else None
    y, h = ssd.channel_scan_fwd(**d, softplus=True, seqlens=lens_of(lens), return_final_state=True)
    torch.cuda.synchronize()
    pick = some(Bz, L)
    # sums of dt: a thread its share of a segment's steps, then the threads' shares
    want = want_of(of(d, pick), True, [lens[b] for b in pick] if lens else None, adds=plan[1] if plan[2] > 1 else 0)
    ref.check("y", y[pick], want, dtype)
    ref.check("final_state", h[pick], want, "f32")


@pytest.mark.parametrize("dtype,ragged", KINDS)
@pytest.mark.parametrize("Bz,L,D,N,G,plan", cases.SCAN_BWD)
def test_scan_backward(dtype, ragged, Bz, L, D, N, G, plan):
    log("channel scan bwd plan %s" % ((dtype, ragged, Bz, L, D, N, G, plan),))
    d = inputs(Bz, L, D, N, G, dtype, L + N, wide=2)
    lens = ([L - 5, L] if Bz == 2 else cases.lengths(Bz, L)) if ragged else None
    pick = some(Bz, L)
    gen = torch.Generator().manual_seed(L)
    dy, dh = torch.zeros(Bz, L, D), torch.zeros(Bz, D, N)
    dy[pick] = torch.randn(len(pick), L, D, generator=gen)
    dh[pick] = torch.randn(len(pick), D, N, generator=gen)
    dy, dh = dy.to(DT[dtype]).cuda(), dh.cuda()
    g = ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=True, seqlens=lens_of(lens),
                             return_dinitial_state=True)
    torch.cuda.synchronize()
    want = want_of(of(d, pick), True, [lens[b] for b in pick] if lens else None, adds=L, dy=n64(dy[pick]),
                   dh=n64(dh[pick]))
    for k in ("du", "ddelta", "dgate", "dB", "dC"):
        ref.check(k, g[k][pick], want, dtype)
    ref.check("dinitial_state", g["dinitial_state"][pick], want, "f32")
    for k in ("dA", "dskip", "ddelta_bias"):
        ref.check(k, g[k], want, "f32")


@pytest.mark.parametrize("dtype,ragged", KINDS)
@pytest.mark.parametrize("Bz,L,pieces,W,silu,plan", cases.CONV)
def test_convolution(dtype, ragged, Bz, L, pieces, W, silu, plan):
    log("short conv plan %s" % ((dtype, ragged, Bz, L, pieces, W, silu, plan),))
    C = sum(pieces)
    gen = torch.Generator().manual_seed(L + C)
    r = lambda *s, dt=DT[dtype]: torch.randn(s, generator=gen).to(dt).cuda()
    x, weight, bias = r(Bz, L, 3 + C)[:, :, 3:], r(C, W, dt=torch.float32), r(C, dt=torch.float32)
    win, dwin, dy = r(Bz, W - 1, C), r(Bz, W - 1, C), [r(Bz, L, w) for w in pieces]
    lens = cases.lengths(Bz, L) if ragged else None
    y, end = ssd.short_conv_fwd(x, weight, bias, initial_window=win, seqlens=lens_of(lens), silu=silu, pieces=pieces,
                                return_final_window=True)
    g = ssd.short_conv_bwd(x, weight, tuple(dy), bias, initial_window=win, dfinal_window=dwin, seqlens=lens_of(lens),
                           silu=silu, return_dinitial_window=True)
    torch.cuda.synchronize()
    want = ref.conv(n64(x), n64(weight), n64(bias), n64(win), lens, silu, np.concatenate([n64(t) for t in dy], 2),
                    n64(dwin), walk=plan[2])
    ref.check("y", torch.cat(y, 2), want, dtype)
    assert np.array_equal(n64(end), want["window"])
    for k in ("dx", "dinitial_window"):
        ref.check(k, g[k], want, dtype)
    for k in ("dweight", "dbias"):
        ref.check(k, g[k], want, "f32")
