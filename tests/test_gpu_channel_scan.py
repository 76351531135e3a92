"""GPU parity of the per-channel scan (forward, backward, single-token step)
against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
n64 = lambda t: None if t is None else t.detach().double().cpu().numpy()


def inputs(Bz, L, D, N, G, dtype, seed=0, wide=0, gate=True, skip=True, bias=True, carry=True, A=None):
    """wide: elements ahead of u and gate in the rows they are cut from."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=DT[dtype]: torch.randn(s, generator=gen).to(dt).cuda()
    f = torch.float32
    both, low = r(Bz, L, wide + 2 * D), r(Bz, L, wide + 2 * G * N)
    d = dict(u=both[..., wide:wide + D], delta=r(Bz, L, D),
             A=-(torch.arange(1, N + 1).float() * torch.exp(0.3 * torch.randn(D, N, generator=gen))).cuda()
             if A is None else A,
             B=low[..., wide:wide + G * N].unflatten(-1, (G, N)), C=low[..., wide + G * N:].unflatten(-1, (G, N)),
             skip=r(D, dt=f) if skip else None, gate=both[..., wide + D:] if gate else None,
             delta_bias=r(D, dt=f) - 3 if bias else None)
    d["initial_state"] = r(Bz, D, N, dt=f) if carry else None
    return d


def want_of(d, softplus, seqlens, adds=0, **kw):
    a = {k: n64(v) for k, v in d.items()}
    return ref.scan(a["u"], a["delta"], a["A"], a["B"], a["C"], a["skip"], a["gate"], a["delta_bias"], softplus,
                    a["initial_state"], seqlens, adds, **kw)


def lens_of(seqlens):
    return None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device="cuda")


SHAPES = [
    # Bz, L, D, N, G, wide, seqlens, softplus, gate, skip, bias, carry
    (1, 1, 16, 16, 1, 0, None, True, True, True, True, True),
    (2, 5, 64, 16, 1, 0, None, True, True, True, True, False),
    (2, 17, 70, 16, 2, 0, None, False, False, False, False, True),      # 35 channels a group
    (3, 40, 96, 12, 3, 8, [40, 0, 23], True, True, True, True, True),
    (2, 33, 20, 4, 1, 0, [33, 32], True, True, False, True, True),
    (1, 50, 33, 1, 1, 3, None, True, False, True, False, True),         # one state, odd rows
    (1, 21, 130, 7, 2, 0, None, True, True, True, True, False),
    (2, 19, 24, 32, 1, 0, [19, 1], True, True, True, True, True),
    (1, 18, 40, 64, 2, 4, None, True, True, True, True, True),
    (1, 9, 5, 33, 5, 1, None, True, True, True, True, True),            # a channel a group
    (3, 0, 16, 16, 1, 0, None, True, True, True, True, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,L,D,N,G,wide,seqlens,softplus,gate,skip,bias,carry", SHAPES)
def test_forward(dtype, Bz, L, D, N, G, wide, seqlens, softplus, gate, skip, bias, carry):
    log("channel scan fwd %s" % ((dtype, Bz, L, D, N, G, wide, seqlens, softplus, gate, skip, bias, carry),))
    d = inputs(Bz, L, D, N, G, dtype, L + D, wide, gate, skip, bias, carry)
    if not softplus:   # step sizes have to be positive for the recurrence to decay
        d["delta"] = d["delta"].abs() * 0.1
    y, h = ssd.channel_scan_fwd(**d, softplus=softplus, seqlens=lens_of(seqlens), return_final_state=True)
    torch.cuda.synchronize()
    want = want_of(d, softplus, seqlens)
    ref.check("y", y, want, dtype)
    ref.check("final_state", h, want, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,L,D,N,G,seqlens", [
    (1, 1000, 40, 16, 1, None),               # few channels: cut into segments
    (3, 900, 24, 5, 3, [900, 0, 411]),        # sequences that end inside, before and at a segment's end
    (2, 512, 64, 40, 1, [256, 512]),
])
def test_segments(dtype, Bz, L, D, N, G, seqlens):
    log("channel scan segments %s" % ((dtype, Bz, L, D, N, G, seqlens),))
    d = inputs(Bz, L, D, N, G, dtype, L, wide=2)
    assert ssd.channel_scan_fwd_workspace_bytes(d["u"], d["delta"], d["A"], d["B"], d["C"]) > 0
    y, h = ssd.channel_scan_fwd(**d, softplus=True, seqlens=lens_of(seqlens), return_final_state=True)
    torch.cuda.synchronize()
    want = want_of(d, True, seqlens, adds=L / 16)   # segments have at least 16 steps, and a sum of dt no more than L / 2
    ref.check("y", y, want, dtype)
    ref.check("final_state", h, want, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,N", [(96, 2, 16), (64, 1, 16), (16, 1, 5)])
def test_many_sequences(dtype, D, G, N):
    # two workgroups of channels for every CU and a few more, which are halved; groups
    # of 48 channels leave half a half empty
    log("channel scan many sequences %s %d %d" % (dtype, D, N))
    Bz = 520 // (2 if D == 96 else 1)
    d = inputs(Bz, 9, D, N, G, dtype, D, wide=2)
    seqlens = [(7 * b) % 10 for b in range(Bz)]
    y, h = ssd.channel_scan_fwd(**d, softplus=True, seqlens=lens_of(seqlens), return_final_state=True)
    torch.cuda.synchronize()
    pick = list(range(0, Bz, 13)) + list(range(Bz - 9, Bz))   # the last are the halved ones
    d = {k: v[pick] if k not in ("A", "skip", "delta_bias") else v for k, v in d.items()}
    want = want_of(d, True, [seqlens[b] for b in pick])
    ref.check("y", y[pick], want, dtype)
    ref.check("final_state", h[pick], want, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_step_sizes(dtype):
    # softplus over its whole range: steps that vanish, and steps so long that
    # nothing of the state is left
    log("channel scan extremes %s" % dtype)
    d = inputs(1, 24, 32, 16, 1, dtype, 3, bias=False)
    d["delta"] = torch.linspace(-100, 100, 24 * 32).view(1, 24, 32).to(DT[dtype]).cuda()
    y, h = ssd.channel_scan_fwd(**d, softplus=True, return_final_state=True)
    torch.cuda.synchronize()
    want = want_of(d, True, None)
    ref.check("y", y, want, dtype)
    ref.check("final_state", h, want, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_end_are_not_read(dtype):
    log("channel scan NaN behind the end %s" % dtype)
    d = inputs(3, 40, 48, 16, 2, dtype, 4)
    seqlens = [0, 40, 22]
    run = lambda lens: ssd.channel_scan_fwd(**d, softplus=True, seqlens=lens_of(lens), return_final_state=True)
    y0, h0 = run(seqlens)
    for k in ("u", "delta", "gate", "B", "C"):
        for b, n in enumerate(seqlens):
            d[k][b, n:] = float("nan")
    y1, h1 = run(seqlens)
    y2, _ = run([-5, 1000, 22])
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(h0, h1) and torch.equal(y0, y2)
    assert torch.equal(h0[0], d["initial_state"][0])
    assert not y0[0].any() and not y0[2, 22:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nans_stay_where_they_are(dtype):
    # an infinite input in the last step of a partial batch and a NaN in another
    # channel: the state is infinite (not NaN: the steps the kernel repeats past the end
    # add nothing), the other channels and sequences are untouched
    log("channel scan infinities %s" % dtype)
    d = inputs(2, 13, 40, 16, 1, dtype, 14, carry=False)
    run = lambda: ssd.channel_scan_fwd(**d, softplus=True, seqlens=lens_of([13, 11]), return_final_state=True)
    y0, h0 = run()
    d["u"][0, 12, 3] = float("inf")
    d["u"][1, 10, 5] = float("inf")
    d["u"][1, 4, 7] = float("nan")
    y1, h1 = run()
    torch.cuda.synchronize()
    assert bool(h1[0, 3].isinf().all()) and bool(h1[1, 5].isinf().all()) and bool(h1[1, 7].isnan().all())
    assert bool(y1[1, 4:11, 7].isnan().all()) and not y1[1, 11:].any()
    ok = torch.ones_like(y0, dtype=torch.bool)
    ok[0, 12, 3] = ok[1, 10, 5] = False
    ok[1, 4:, 7] = False
    assert torch.equal(y0[ok], y1[ok])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,D,N,G,wide,gate,skip,bias,softplus", [
    (1, 1, 1, 1, 0, False, False, False, False), (3, 64, 16, 1, 0, True, True, True, True),
    (2, 35, 12, 5, 3, True, True, True, True), (5, 20, 64, 2, 0, True, False, True, True),
    (2, 33, 7, 1, 1, True, True, True, True), (4, 96, 32, 3, 0, False, True, True, True),
    (2, 40, 8, 1, 4, True, True, True, True), (3, 21, 2, 3, 0, True, True, False, True),
])
def test_steps(dtype, Bz, D, N, G, wide, gate, skip, bias, softplus):
    # a few tokens, each checked from the state the one before left
    log("channel step %s" % ((dtype, Bz, D, N, G, wide, gate, skip, bias, softplus),))
    d = inputs(Bz, 4, D, N, G, dtype, D + N, wide, gate, skip, bias, True)
    if not softplus:
        d["delta"] = d["delta"].abs() * 0.1
    state = d.pop("initial_state").clone()
    for t in range(4):
        one = {k: v if v is None or k in ("A", "skip", "delta_bias") else v[:, t] for k, v in d.items()}
        before = state.clone()
        y = ssd.channel_step(state, **one, softplus=softplus)
        torch.cuda.synchronize()
        whole = {k: v if v is None or k in ("A", "skip", "delta_bias") else v[:, None] for k, v in one.items()}
        want = want_of(dict(whole, initial_state=before), softplus, None)
        ref.check("y", y[:, None], want, dtype)
        ref.check("final_state", state, want, "f32")


def test_prompt_then_steps():
    # the convolution and the scan together, a prompt of unequal lengths and then
    # tokens, against one pass over the whole sequences
    log("channel prompt then steps")
    Bz, L, D, N, W, more = 2, 30, 48, 16, 4, 3
    d = inputs(Bz, L + more, D, N, 1, "f32", 11, carry=False)
    x = d["u"].contiguous()
    gen = torch.Generator().manual_seed(5)
    weight, cb = torch.randn(D, W, generator=gen).cuda(), torch.randn(D, generator=gen).cuda()
    layer = {k: d[k] for k in ("A", "skip", "delta_bias")}
    seqlens = [30, 14]
    lens = lens_of(seqlens)
    xc, win = ssd.short_conv_fwd(x[:, :L], weight, cb, seqlens=lens, return_final_window=True)
    rows = {k: d[k][:, :L] for k in ("delta", "B", "C", "gate")}
    y, state = ssd.channel_scan_fwd(xc, **rows, **layer, softplus=True, seqlens=lens, return_final_state=True)
    ys = []
    for t in range(more):
        xt = ssd.short_conv_step(win, x[:, L + t], weight, cb)
        ys.append(ssd.channel_step(state, xt, **{k: d[k][:, L + t] for k in rows}, **layer, softplus=True))
    torch.cuda.synchronize()
    for b, n in enumerate(seqlens):
        at = list(range(n)) + list(range(L, L + more))
        c = ref.conv(n64(x[b:b + 1, at]), n64(weight), n64(cb), None, None, True)
        a = {k: n64(d[k][b:b + 1, at]) for k in rows}
        want = ref.scan(c["y"], a["delta"], n64(d["A"]), a["B"], a["C"], n64(d["skip"]), a["gate"],
                        n64(d["delta_bias"]))
        got = torch.cat([y[b, :n], torch.stack([v[b] for v in ys])])
        # the convolution's own error enters through u: at most 40 roundings of
        # values up to max|u|, against sums of them
        scale = np.abs(want["y"]).max()
        assert np.abs(n64(got) - want["y"][0]).max() <= 2e-5 * scale
        assert np.abs(n64(state[b]) - want["final_state"][0]).max() <= 2e-5 * np.abs(want["final_state"]).max()


def test_repeats_streams_and_graphs():
    log("channel scan streams and graphs")
    d = inputs(2, 70, 80, 16, 1, "bf16", 6, wide=16)
    one = {k: v if v is None or k in ("A", "skip", "delta_bias") else v[:, 3] for k, v in d.items()
           if k != "initial_state"}
    state = d["initial_state"].clone()

    def run():
        y, h = ssd.channel_scan_fwd(**d, softplus=True, return_final_state=True)
        s = state.clone()
        return y, h, ssd.channel_step(s, **one, softplus=True), s

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(3):
        for t in held:
            t.fill_(7)
        graph.replay()
        again = run()
        torch.cuda.synchronize()
        for got in (other, held, again):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- backward -----------------------------------------------------------------------

def upstream(d, dtype, seed, carry=True):
    gen = torch.Generator().manual_seed(seed)
    Bz, L, D = d["u"].shape
    dy = torch.randn(Bz, L, D, generator=gen).to(DT[dtype]).cuda()
    return dy, torch.randn(Bz, D, d["A"].shape[1], generator=gen).cuda() if carry else None


def check_backward(d, dtype, softplus, seqlens, dy, dh, adds=0):
    g = ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=softplus, seqlens=lens_of(seqlens),
                             return_dinitial_state=True)
    torch.cuda.synchronize()
    want = want_of(d, softplus, seqlens, adds=adds, dy=n64(dy), dh=n64(dh))
    for k in ("du", "ddelta", "dgate", "dB", "dC"):
        if k != "dgate" or d["gate"] is not None:
            ref.check(k, g[k], want, dtype)
    for k, given in (("dA", True), ("dskip", d["skip"] is not None), ("ddelta_bias", d["delta_bias"] is not None),
                     ("dinitial_state", True)):
        if given:
            ref.check(k, g[k], want, "f32")
        else:
            assert g[k] is None
    assert d["gate"] is not None or g["dgate"] is None
    return g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,L,D,N,G,wide,seqlens,softplus,gate,skip,bias,carry", SHAPES)
def test_backward(dtype, Bz, L, D, N, G, wide, seqlens, softplus, gate, skip, bias, carry):
    log("channel scan bwd %s" % ((dtype, Bz, L, D, N, G, wide, seqlens, softplus, gate, skip, bias, carry),))
    d = inputs(Bz, L, D, N, G, dtype, L + D, wide, gate, skip, bias, carry)
    if not softplus:
        d["delta"] = d["delta"].abs() * 0.1
    dy, dh = upstream(d, dtype, L, carry)
    check_backward(d, dtype, softplus, seqlens, dy, dh)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,L,D,N,G,seqlens", [(1, 1000, 40, 16, 1, None), (3, 600, 24, 5, 3, [600, 0, 411]),
                                                (2, 320, 64, 40, 1, [160, 320])])
def test_backward_long(dtype, Bz, L, D, N, G, seqlens):
    # few channels and many steps: segments that sequences end inside, before and at the end of
    log("channel scan bwd long %s" % ((dtype, Bz, L, D, N, G, seqlens),))
    d = inputs(Bz, L, D, N, G, dtype, L, wide=2)
    dy, dh = upstream(d, dtype, L)
    check_backward(d, dtype, True, seqlens, dy, dh, adds=L)


def test_backward_against_differences():
    # fp32 gradients against central differences of the 64-bit forward along
    # random directions
    log("channel scan bwd differences")
    d = inputs(2, 21, 10, 5, 2, "f32", 8)
    seqlens = [21, 13]
    dy, dh = upstream(d, "f32", 9)
    g = check_backward(d, "f32", True, seqlens, dy, dh)
    names = {"u": "du", "delta": "ddelta", "A": "dA", "B": "dB", "C": "dC", "skip": "dskip", "gate": "dgate",
             "delta_bias": "ddelta_bias", "initial_state": "dinitial_state"}
    base = {k: n64(d[k]) for k in names}

    def loss(v):
        o = ref.scan(v["u"], v["delta"], v["A"], v["B"], v["C"], v["skip"], v["gate"], v["delta_bias"], True,
                     v["initial_state"], seqlens)
        return (o["y"] * n64(dy)).sum() + (o["final_state"] * n64(dh)).sum()

    rng = np.random.default_rng(1)
    for k, gk in names.items():
        r = rng.standard_normal(base[k].shape)
        step = 1e-5
        num = (loss({**base, k: base[k] + step * r}) - loss({**base, k: base[k] - step * r})) / (2 * step)
        ours = n64(g[gk])
        # truncation ~ step^2, cancellation ~ 1e-16 |loss| / step, the gradient's own fp32 error
        assert abs(num - (ours * r).sum()) <= 1e-5 * (np.abs(ours * r).sum() + 1), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_rows_behind_the_end(dtype):
    log("channel scan bwd NaN behind the end %s" % dtype)
    d = inputs(3, 40, 48, 16, 2, dtype, 4)
    seqlens = [0, 40, 22]
    dy, dh = upstream(d, dtype, 5)
    run = lambda: ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=True, seqlens=lens_of(seqlens),
                                       return_dinitial_state=True)
    g0 = run()
    for t in (d["u"], d["delta"], d["gate"], d["B"], d["C"], dy):
        for b, n in enumerate(seqlens):
            t[b, n:] = float("nan")
    g1 = run()
    torch.cuda.synchronize()
    for k in g0:
        assert torch.equal(g0[k], g1[k]), k
    for k in ("du", "ddelta", "dgate", "dB", "dC"):
        assert not g0[k][0].any() and not g0[k][2, 22:].any(), k
    assert torch.equal(g0["dinitial_state"][0], dh[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,N", [(13, 16), (77, 40)])   # in one segment and in several
def test_backward_infinities_stay_where_they_are(dtype, L, N):
    # an infinite u in the last step of a partial batch touches its channel, and of the
    # sums over channels its own step (dB and, through the state, dC)
    log("channel scan bwd infinities %s %d %d" % (dtype, L, N))
    d = inputs(2, L, 40, N, 1, dtype, 14, carry=False)
    dy, dh = upstream(d, dtype, 5)
    run = lambda: ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=True, return_dinitial_state=True)
    g0 = run()
    d["u"][0, L - 1, 3] = float("inf")
    g1 = run()
    torch.cuda.synchronize()
    others = [c for c in range(40) if c != 3]
    for k in ("du", "ddelta", "dgate"):
        assert torch.equal(g0[k][..., others], g1[k][..., others]) and torch.equal(g0[k][1], g1[k][1]), k
    for k in ("dA", "dskip", "ddelta_bias"):
        assert torch.equal(g0[k][others], g1[k][others]), k
    for k in ("dB", "dC"):
        assert torch.equal(g0[k][0, :L - 1], g1[k][0, :L - 1]) and torch.equal(g0[k][1], g1[k][1]), k
        assert not g1[k][0, L - 1].isfinite().any(), k
    assert torch.equal(g0["du"][0, :, 3], g1["du"][0, :, 3])   # no gradient of u depends on u
    assert torch.equal(g0["dinitial_state"], g1["dinitial_state"])


def test_backward_repeats_streams_and_graphs():
    log("channel scan bwd streams and graphs")
    for L in (70, 900):
        d = inputs(2, L, 80, 16, 1, "bf16", 6, wide=16)
        dy, dh = upstream(d, "bf16", 7)
        run = lambda: ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=True, return_dinitial_state=True)
        want = run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = run()
        for _ in range(3):
            for t in held.values():
                t.fill_(7)
            graph.replay()
            again = run()
            torch.cuda.synchronize()
            for got in (other, held, again):
                for k in want:
                    assert torch.equal(got[k], want[k]), (L, k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_sequences(dtype):
    # an empty batch: nothing but the parameters' gradients, which are zero
    log("channel scan empty batch %s" % dtype)
    d = inputs(0, 9, 24, 16, 1, dtype)
    y, h = ssd.channel_scan_fwd(**d, softplus=True, return_final_state=True)
    g = ssd.channel_scan_bwd(**d, dy=torch.zeros_like(d["u"]), softplus=True, return_dinitial_state=True)
    torch.cuda.synchronize()
    assert y.shape == (0, 9, 24) and h.shape == (0, 24, 16)
    for k in ("dA", "dskip", "ddelta_bias"):
        assert g[k].shape[0] == 24 and not g[k].any(), k


def test_convolution_into_the_chunked_scan():
    # the convolution's pieces are the chunked scan's X, B and C, forward and
    # backward, a prompt and then tokens
    log("short conv into the chunked scan")
    Bz, L, H, P, N, G, W = 2, 150, 4, 64, 64, 1, 4
    gen = torch.Generator().manual_seed(3)
    r = lambda *s, dt=torch.bfloat16: torch.randn(s, generator=gen).to(dt).cuda()
    pieces = (H * P, G * N, G * N)
    rows = r(Bz, L + 1, 32 + sum(pieces))
    x, weight, bias = rows[:, :, 32:], r(sum(pieces), W, dt=torch.float32) * 0.5, r(sum(pieces), dt=torch.float32) * 0.1
    a = -torch.rand(Bz, L + 1, H, generator=gen).cuda() * 0.2
    split = lambda ys, *lead: (ys[0].view(*lead, H, P), ys[1].view(*lead, G, N), ys[2].view(*lead, G, N))
    ys, win = ssd.short_conv_fwd(x[:, :L], weight, bias, pieces=pieces, return_final_window=True)
    X, B, C = split(ys, Bz, L)
    a0 = a[:, :L].contiguous()
    Y, S = ssd.chunk_scan_fwd(X, a0, B, C, 64, return_final_state=True)
    dY = r(Bz, L, H, P)
    g = ssd.chunk_scan_bwd(X, a0, B, C, dY, 64)
    gc = ssd.short_conv_bwd(x[:, :L], weight, tuple(g[k].view(Bz, L, -1) for k in ("dX", "dB", "dC")), bias)
    xt, Bt, Ct = split(ssd.short_conv_step(win, x[:, L], weight, bias, pieces=pieces), Bz)
    y1 = ssd.step(S, xt, a[:, L].contiguous(), Bt, Ct)
    torch.cuda.synchronize()
    # the convolution itself is exact to its tolerance ...
    w = ref.conv(n64(x), n64(weight), n64(bias), None, None, True)
    ref.check("y", torch.cat([torch.cat(ys, 2), torch.cat([t.reshape(Bz, 1, -1) for t in (xt, Bt, Ct)], 2)], 1), w,
              "bf16")
    # ... and the scan sees exactly its output: one oracle run over prompt and token
    import oracle
    X64, B64, C64 = (np.concatenate([n64(p), n64(q)[:, None]], 1) for p, q in ((X, xt), (B, Bt), (C, Ct)))
    Yr, Sr = oracle.fwd(X64, n64(a), B64, C64)
    got = np.concatenate([n64(Y), n64(y1)[:, None]], 1)
    assert np.abs(got - Yr).max() <= 2e-2 * np.abs(Yr).max()     # the chunked scan's own tolerance
    assert np.abs(n64(S) - Sr).max() <= 2e-2 * np.abs(Sr).max()
    dyc = np.concatenate([n64(g[k]).reshape(Bz, L, -1) for k in ("dX", "dB", "dC")], 2)
    wb = ref.conv(n64(x[:, :L]), n64(weight), n64(bias), None, None, True, dyc)
    ref.check("dx", gc["dx"], wb, "bf16")
    ref.check("dweight", gc["dweight"], wb, "f32")
    ref.check("dbias", gc["dbias"], wb, "f32")


def test_large_strides_and_many_steps():
    # batches far apart in memory (offsets past 2^31 elements), a sequence of 9000
    # steps, the last batch alone live
    log("channel scan far batches")
    if torch.cuda.get_device_properties(0).total_memory < (48 << 30):
        pytest.skip("needs 24 GiB of device memory")
    far = (1 << 31) + 64                       # elements between batches of u
    L, D = 9000, 32
    d = inputs(2, L, D, 4, 1, "bf16", 12, gate=True)
    buf = torch.empty(far + L * D, dtype=torch.bfloat16, device="cuda")
    u = torch.as_strided(buf, (2, L, D), (far, D, 1))
    u.copy_(d["u"])
    want = ssd.channel_scan_fwd(**d, softplus=True)[0]
    got = ssd.channel_scan_fwd(**dict(d, u=u), softplus=True)[0]
    x, _ = ssd.short_conv_fwd(u, d["A"], d["skip"])
    x0, _ = ssd.short_conv_fwd(d["u"].contiguous(), d["A"], d["skip"])
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(x, x0)
