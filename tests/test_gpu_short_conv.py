"""GPU parity of the short causal convolution (forward, backward, single-token
step) against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inputs(Bz, L, C, W, dtype, seed=0, wide=0, bias=True, window=True, pieces=None):
    """wide: elements ahead of x in the rows it is cut from."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=DT[dtype]: torch.randn(s, generator=g).to(dt).cuda()
    rows = r(Bz, L, wide + C)
    return dict(x=rows[:, :, wide:], weight=r(C, W, dt=torch.float32), bias=r(C, dt=torch.float32) if bias else None,
                win=r(Bz, W - 1, C) if window else None, dwin=r(Bz, W - 1, C) if window else None,
                dy=[r(Bz, L, w) for w in (pieces or (C,))])


def both(d, seqlens, silu, pieces, dtype):
    lens = None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    y, win = ssd.short_conv_fwd(d["x"], d["weight"], d["bias"], initial_window=d["win"], seqlens=lens, silu=silu,
                                pieces=pieces, return_final_window=True)
    g = ssd.short_conv_bwd(d["x"], d["weight"], tuple(d["dy"]) if pieces else d["dy"][0], d["bias"],
                           initial_window=d["win"], dfinal_window=d["dwin"], seqlens=lens, silu=silu,
                           return_dinitial_window=True)
    torch.cuda.synchronize()
    want = ref.conv(n64(d["x"]), n64(d["weight"]), n64(d["bias"]), n64(d["win"]), seqlens, silu,
                    np.concatenate([n64(t) for t in d["dy"]], 2), n64(d["dwin"]))
    ref.check("y", torch.cat(y, 2) if pieces else y, want, dtype)
    assert np.array_equal(n64(win), want["window"])
    for k in ("dx", "dinitial_window"):
        ref.check(k, g[k], want, dtype)
    ref.check("dweight", g["dweight"], want, "f32")
    if d["bias"] is None:
        assert g["dbias"] is None
    else:
        ref.check("dbias", g["dbias"], want, "f32")
    return y, win, g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,L,C,W,wide,pieces,seqlens,silu,bias,window", [
    (1, 1, 8, 4, 0, None, None, True, True, True),          # one step: less than the window
    (2, 2, 16, 4, 0, None, None, True, False, False),
    (1, 33, 8, 2, 8, None, None, False, True, True),        # one step past a wavefront's walk
    (2, 129, 520, 4, 0, (512, 8), None, True, True, True),  # one past a workgroup's, two pieces
    (3, 300, 96, 3, 32, (64, 16, 16), [300, 0, 170], True, True, True),
    (4, 40, 24, 4, 0, None, [1, 2, 3, 40], True, True, True),   # sequences shorter than the window
    (4, 40, 24, 4, 0, None, [1, 2, 0, 32], False, False, False),
    (2, 65, 7, 4, 0, None, [65, 64], True, True, True),     # odd: one channel at a time
    (2, 70, 136, 4, 5, (131, 5), None, True, True, True),   # pieces and rows at odd places
    (1, 5, 1, 3, 0, None, None, True, True, False),
    (3, 40, 24, 4, 1, (17, 3, 4), [40, 0, 9], True, True, True),    # a piece narrower than a thread's channels
    (2, 400, 1031, 4, 3, (1021, 5, 5), None, True, True, True),     # ends of pieces inside a thread's channels
    (1, 2100, 64, 4, 0, None, None, True, True, True),
    (3, 0, 16, 4, 0, None, None, True, True, True),         # no steps at all: the windows go through
])
def test_against_definition(dtype, Bz, L, C, W, wide, pieces, seqlens, silu, bias, window):
    log("short conv %s" % ((dtype, Bz, L, C, W, wide, pieces, seqlens, silu, bias, window),))
    d = inputs(Bz, L, C, W, dtype, seed=L + C, wide=wide, bias=bias, window=window, pieces=pieces)
    both(d, seqlens, silu, pieces, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_end_are_not_read(dtype):
    log("short conv NaN behind the end %s" % dtype)
    d = inputs(3, 50, 40, 4, dtype, seed=3)
    seqlens = [50, 0, 17]
    clean = both(d, seqlens, True, None, dtype)
    for b, n in enumerate(seqlens):
        d["x"][b, n:] = float("nan")
        d["dy"][0][b, n:] = float("inf")
    lens = torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    y, win = ssd.short_conv_fwd(d["x"], d["weight"], d["bias"], initial_window=d["win"], seqlens=lens,
                                return_final_window=True)
    g = ssd.short_conv_bwd(d["x"], d["weight"], d["dy"][0], d["bias"], initial_window=d["win"],
                           dfinal_window=d["dwin"], seqlens=lens, return_dinitial_window=True)
    torch.cuda.synchronize()
    assert torch.equal(y, clean[0]) and torch.equal(win, clean[1])
    for k, v in g.items():
        assert torch.equal(v, clean[2][k]), k
    # lengths outside 0 .. seqlen count as the nearest
    lens = torch.tensor([99, -3, 17], dtype=torch.int32, device="cuda")
    y2, _ = ssd.short_conv_fwd(d["x"], d["weight"], d["bias"], initial_window=d["win"], seqlens=lens)
    assert torch.equal(y2, clean[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,W,wide,pieces", [(64, 4, 16, (32, 16, 16)), (24, 3, 0, None), (13, 2, 3, (10, 3)),
                                             (2048, 4, 0, None), (27, 4, 1, (9, 7, 11)), (5, 4, 0, None)])
def test_steps_continue_a_prompt(dtype, C, W, wide, pieces):
    # a prompt, then single tokens from its final window: the bits of one longer prompt
    log("short conv steps %s" % ((dtype, C, W, wide, pieces),))
    d = inputs(3, 12, C, W, dtype, seed=C, wide=wide)
    cat = lambda y: torch.cat(y, -1) if pieces else y
    whole, wend = ssd.short_conv_fwd(d["x"], d["weight"], d["bias"], initial_window=d["win"], pieces=pieces,
                                     return_final_window=True)
    first, win = ssd.short_conv_fwd(d["x"][:, :7], d["weight"], d["bias"], initial_window=d["win"], pieces=pieces,
                                    return_final_window=True)
    ys = [cat(ssd.short_conv_step(win, d["x"][:, t], d["weight"], d["bias"], pieces=pieces)) for t in range(7, 12)]
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([cat(first), torch.stack(ys, 1)], 1), cat(whole))
    assert torch.equal(win, wend)


def test_gradients_against_differences():
    # fp32, central differences of the forward in 64 bits along random directions
    log("short conv differences")
    d = inputs(2, 37, 12, 4, "f32", seed=5)
    seqlens = [37, 20]
    _, _, g = both(d, seqlens, True, None, "f32")
    rng = np.random.default_rng(0)
    names = {"x": "dx", "weight": "dweight", "bias": "dbias", "win": "dinitial_window"}
    base = {k: n64(d[k]) for k in names}

    def loss(v):
        o = ref.conv(v["x"], v["weight"], v["bias"], v["win"], seqlens, True)
        return (o["y"] * n64(d["dy"][0])).sum() + (o["window"] * n64(d["dwin"])).sum()

    for k, gk in names.items():
        u = rng.standard_normal(base[k].shape)
        h = 1e-5
        num = (loss({**base, k: base[k] + h * u}) - loss({**base, k: base[k] - h * u})) / (2 * h)
        ours = n64(g[gk])
        # truncation ~ h^2, cancellation ~ 1e-16 |loss| / h, and the gradient's own fp32 error
        assert abs(num - (ours * u).sum()) <= 1e-6 * (np.abs(ours * u).sum() + 1), k


def test_repeats_streams_and_graphs():
    # the same bits from repeated calls, from another stream, and from a captured
    # graph replayed between eager calls
    log("short conv streams and graphs")
    d = inputs(2, 200, 72, 4, "bf16", seed=9, wide=8)
    run = lambda: (ssd.short_conv_fwd(d["x"], d["weight"], d["bias"], initial_window=d["win"])[0],
                   ssd.short_conv_bwd(d["x"], d["weight"], d["dy"][0], d["bias"], initial_window=d["win"],
                                      return_dinitial_window=True))
    y0, g0 = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, g1 = run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, g2 = run()
    for _ in range(3):
        for t in (y2, *g2.values()):
            t.fill_(7)
        graph.replay()
        y3, g3 = run()
        torch.cuda.synchronize()
        for y, g in ((y1, g1), (y2, g2), (y3, g3)):
            assert torch.equal(y, y0)
            for k in g0:
                assert torch.equal(g[k], g0[k]), k


def test_given_outputs_and_their_surroundings():
    # outputs inside larger buffers: nothing outside them is written
    log("short conv given outputs")
    Bz, L, C, W = 2, 37, 24, 4
    for dtype in ("bf16", "f32"):
        d = inputs(Bz, L, C, W, dtype, seed=1)
        buf = torch.full((Bz * L * C + 64,), 5.0, dtype=DT[dtype], device="cuda")
        y = buf[32:32 + Bz * L * C].view(Bz, L, C)
        got, _ = ssd.short_conv_fwd(d["x"], d["weight"], d["bias"], y=y)
        want, _ = ssd.short_conv_fwd(d["x"], d["weight"], d["bias"])
        torch.cuda.synchronize()
        assert got is y and torch.equal(y, want)
        assert bool((buf[:32] == 5).all()) and bool((buf[32 + Bz * L * C:] == 5).all())
        with pytest.raises(ssd.SSDError, match="SSD_ERR_ALIAS"):
            ssd.short_conv_fwd(y, d["weight"], y=y)


def test_no_sequences():
    log("short conv empty batch")
    d = inputs(0, 9, 24, 4, "bf16")
    y, win = ssd.short_conv_fwd(d["x"], d["weight"], d["bias"], return_final_window=True)
    g = ssd.short_conv_bwd(d["x"], d["weight"], d["dy"][0], d["bias"])
    torch.cuda.synchronize()
    assert y.shape == (0, 9, 24) and win.shape == (0, 3, 24)
    assert not g["dweight"].any() and not g["dbias"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 3, 4])
def test_any_alignment(dtype, shift):
    # every tensor `shift` elements into its buffer: the same values
    log("short conv alignment %s %d" % (dtype, shift))
    d = inputs(2, 21, 16, 4, dtype, seed=shift)
    move = lambda t: torch.cat([t.new_zeros(shift), t.flatten()])[shift:].view(t.shape)
    run = lambda d, y: (ssd.short_conv_fwd(d["x"], d["weight"], d["bias"], initial_window=d["win"], y=y,
                                           return_final_window=True),
                        ssd.short_conv_bwd(d["x"], d["weight"], d["dy"][0], d["bias"], initial_window=d["win"],
                                           dfinal_window=d["dwin"], return_dinitial_window=True))
    (y, win), g = run(d, None)
    m = {k: move(v) if k != "dy" else [move(v[0])] for k, v in d.items()}
    (ym, winm), gm = run(m, move(torch.zeros_like(y)))
    torch.cuda.synchronize()
    assert torch.equal(y, ym) and torch.equal(win, winm)
    for k in g:
        # dweight and dbias: a walk covers the same steps either way
        assert torch.equal(g[k], gm[k]), k
