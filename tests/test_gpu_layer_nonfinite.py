"""Infinities, NaN and the type's lowest values in the operators around the chunked
scan: where the definition gives a finite result, so do the kernels, whatever the
batch is padded with.  Each call is held to one whose inputs are finite and whose
results are, by the definition, the same: the bits have to be."""
import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log
from test_gpu_channel_scan import DT, inputs, lens_of, upstream

pytestmark = pytest.mark.gpu

INF, NAN, LOWEST = float("inf"), float("nan"), torch.finfo(torch.float32).min


# ---- convolution ------------------------------------------------------------------------

def conv_inputs(Bz, L, C, W, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=DT[dtype]: torch.randn(s, generator=gen).to(dt).cuda()
    return r(Bz, L, C), r(C, W, dt=torch.float32), r(C, dt=torch.float32), r(Bz, W - 1, C), r(Bz, L, C)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("L,W", [(9, 4), (1, 2), (0, 3), (200, 4)])
def test_window_of_an_empty_sequence(dtype, silu, L, W):
    # a slot of the batch without a sequence adds nothing to dweight, whatever its window holds
    log("short conv window of an empty sequence %s" % ((dtype, silu, L, W),))
    x, weight, bias, win, dy = conv_inputs(3, L, 20, W, dtype, L)
    lens = lens_of([L, 0, L])
    run = lambda: ssd.short_conv_bwd(x, weight, dy, bias, initial_window=win, seqlens=lens, silu=silu,
                                     return_dinitial_window=True)
    g0 = run()
    win[1, :, 3], win[1, 0, 7], win[1, :, 11] = NAN, INF, -INF
    if L == 0:
        win[0, 0, 5] = INF
    g1 = run()
    torch.cuda.synchronize()
    for k in g0:
        assert bool(g1[k].isfinite().all()) and torch.equal(g0[k], g1[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("n", [1, 3, 4, 6, 40])
def test_infinity_among_the_last_inputs(dtype, W, n):
    # without the nonlinearity tap k sums dy[t] x[t - (W-1) + k], t < n: an infinite x in
    # the last step is in the last tap's sum alone, however long the batch
    log("short conv infinity among the last inputs %s" % ((dtype, W, n),))
    x, weight, bias, win, dy = conv_inputs(2, 41, 20, W, dtype, n)
    dy = dy.abs() + 0.5
    lens = lens_of([41, n])
    run = lambda: ssd.short_conv_bwd(x, weight, dy, bias, initial_window=win, seqlens=lens, silu=False)
    g0 = run()
    x[1, n - 1, 3], x[1, n - 1, 8] = INF, NAN
    g1 = run()
    torch.cuda.synchronize()
    assert torch.equal(g0["dweight"][:, :W - 1], g1["dweight"][:, :W - 1])
    assert g1["dweight"][3, W - 1] == INF and bool(g1["dweight"][8, W - 1].isnan())
    others = [c for c in range(20) if c not in (3, 8)]
    assert torch.equal(g0["dweight"][others], g1["dweight"][others])
    assert torch.equal(g0["dx"], g1["dx"]) and torch.equal(g0["dbias"], g1["dbias"])   # neither depends on x


# ---- scan -------------------------------------------------------------------------------

# in one segment and in several, sequences that end inside a batch of eight steps at every
# place, at its end, and one segment early
LENGTHS = [(n, n) for n in range(8, 17)] + [(40, n) for n in (1, 8, 13, 24, 31)] + [(300, 300), (300, 283), (300, 299)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [5, 16, 24, 40])
@pytest.mark.parametrize("L,n", LENGTHS)
def test_infinite_last_input_and_dA(dtype, N, L, n):
    # dA sums e g[t] h[t-1] dt: the state after the last step is not in it
    log("channel scan infinite last input %s" % ((dtype, N, L, n),))
    d = inputs(2, L, 40, N, 1, dtype, n, carry=False)
    dy, dh = upstream(d, dtype, 5)
    run = lambda: ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=True, seqlens=lens_of([n, L]),
                                       return_dinitial_state=True)
    g0 = run()
    d["u"][0, n - 1, 3] = INF
    g1 = run()
    torch.cuda.synchronize()
    assert bool(g0["dA"].isfinite().all()) and torch.equal(g0["dA"], g1["dA"])
    for k in ("ddelta", "dgate"):
        assert torch.equal(g0[k][:, :n - 1], g1[k][:, :n - 1]), k
    assert torch.equal(g0["du"], g1["du"]) and torch.equal(g0["dinitial_state"], g1["dinitial_state"])


MASKS = [("bf16", -INF), ("bf16", torch.finfo(torch.bfloat16).min), ("f32", -INF), ("f32", LOWEST), ("f32", -2.5e38)]


@pytest.mark.parametrize("dtype,value", MASKS)
@pytest.mark.parametrize("L,N", [(13, 16), (77, 40), (300, 5)])
def test_masked_steps(dtype, value, L, N):
    # softplus of -infinity is 0, as it is of -150 in 32 bits: such a step leaves the
    # state as it was
    log("channel scan masked steps %s" % ((dtype, value, L, N),))
    d = inputs(2, L, 40, N, 1, dtype, 3)
    dy, dh = upstream(d, dtype, 5)

    def run(v, bias):
        d["delta"][0, 4, 3] = d["delta"][1, L - 1] = d["delta"][0, 7:9, 20:] = v
        d["delta_bias"][17] = bias
        y, h = ssd.channel_scan_fwd(**d, softplus=True, return_final_state=True)
        g = ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=True, return_dinitial_state=True)
        return dict(g, y=y, h=h)

    want, got = run(-150.0, -150.0), run(value, -INF)
    torch.cuda.synchronize()
    assert torch.equal(want["h"][:, 17], d["initial_state"][:, 17])   # a channel that takes no step
    for k in want:
        assert bool(got[k].isfinite().all()) and torch.equal(want[k], got[k]), k


@pytest.mark.parametrize("dtype,value", MASKS)
def test_masked_token(dtype, value):
    log("channel step masked %s" % ((dtype, value),))
    d = inputs(3, 1, 40, 16, 1, dtype, 4)
    one = {k: v if v is None or k in ("A", "skip", "delta_bias") else v[:, 0] for k, v in d.items()
           if k != "initial_state"}
    out = []
    for v in (-150.0, value):
        one["delta"][1] = one["delta"][2, 5] = v
        state = d["initial_state"].clone()
        out.append((ssd.channel_step(state, **one, softplus=True), state))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and bool(b.isfinite().all()) for a, b in zip(*out))
    assert torch.equal(out[1][1][1], d["initial_state"][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [INF, NAN])
def test_unbounded_steps_stay_in_their_channel(dtype, value):
    # softplus of infinity is infinity, of NaN is NaN: everything of that channel from
    # there on, nothing of the others
    log("channel scan unbounded steps %s" % ((dtype, value),))
    d = inputs(2, 29, 40, 16, 1, dtype, 6)
    run = lambda: ssd.channel_scan_fwd(**d, softplus=True, return_final_state=True)
    y0, h0 = run()
    d["delta"][0, 9, 3] = value
    y1, h1 = run()
    torch.cuda.synchronize()
    assert not h1[0, 3].isfinite().any() and not y1[0, 9:, 3].isfinite().any()
    keep = torch.ones_like(y0, dtype=torch.bool)
    keep[0, 9:, 3] = False
    assert torch.equal(y0[keep], y1[keep])
    others = [c for c in range(40) if c != 3]
    assert torch.equal(h0[0, others], h1[0, others]) and torch.equal(h0[1], h1[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [-INF, LOWEST, -2.4e38])
@pytest.mark.parametrize("L,n", [(13, 13), (16, 16), (40, 21), (300, 300), (300, 150), (1000, 999)])
def test_states_that_forget_at_once(dtype, value, L, n):
    # e^{dt A} is 0 for A = -infinity and the lowest values as for -1e30, with every dt
    # here; steps past the end have dt = 0 and leave the state as it is
    log("channel scan forgetting states %s" % ((dtype, value, L, n),))
    d = inputs(2, L, 40, 16, 1, dtype, 7)
    dy, dh = upstream(d, dtype, 5)
    lens = lens_of([n, L])

    def run(v):
        d["A"][3, 5] = d["A"][11] = v
        y, h = ssd.channel_scan_fwd(**d, softplus=True, seqlens=lens, return_final_state=True)
        g = ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=True, seqlens=lens, return_dinitial_state=True)
        return dict(g, y=y, h=h)

    want, got = run(-1e30), run(value)
    torch.cuda.synchronize()
    for k in want:
        assert bool(got[k].isfinite().all()) and torch.equal(want[k], got[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_token_of_states_that_forget_at_once(dtype):
    # ... and with dt = 0 (delta of -150) such a state stays
    log("channel step forgetting states %s" % dtype)
    d = inputs(2, 1, 40, 16, 1, dtype, 8)
    one = {k: v if v is None or k in ("A", "skip", "delta_bias") else v[:, 0] for k, v in d.items()
           if k != "initial_state"}
    one["delta"][1] = -150.0
    out = []
    for v in (-1e30, LOWEST, -INF):
        one["A"][3, 5] = one["A"][11] = v
        state = d["initial_state"].clone()
        out.append((ssd.channel_step(state, **one, softplus=True), state))
    torch.cuda.synchronize()
    for y, state in out[1:]:
        assert torch.equal(y, out[0][0]) and torch.equal(state, out[0][1])
    assert torch.equal(out[0][1][1], d["initial_state"][1])
