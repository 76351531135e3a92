"""GPU parity of linear attention with a decay per head (forward, backward,
single-token step) against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GRADS = ("dq", "dk", "dv", "dinitial_state")


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inputs(Bz, L, H, K, Dk, Dv, dtype, seed=0, wide=0, carry=True, lo=0.3, hi=200.0):
    """wide: elements ahead of q in the rows that q, k and v are cut from.  Decays of lo to hi steps."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=DT[dtype]: torch.randn(s, generator=g).to(dt).cuda()   # noqa: E731
    rows = r(Bz, L, wide + H * Dk + K * (Dk + Dv))
    q, k, v = rows[..., wide:].split([H * Dk, K * Dk, K * Dv], 2)
    spans = lo * (hi / lo) ** (torch.arange(H) / max(H - 1, 1))
    state = lambda: r(Bz, H, Dv, Dk, dt=torch.float32) if carry else None    # noqa: E731
    return dict(q=q.unflatten(2, (H, Dk)), k=k.unflatten(2, (K, Dk)), v=v.unflatten(2, (K, Dv)),
                decay=(-1 / spans).cuda(), first=state(), dlast=state(), dy=r(Bz, L, H, Dv))


def calls(d, seqlens=None, scale=None, carry=True):
    lens = None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    args = [d[n] for n in ("q", "k", "v", "decay")]
    y, state = ssd.linear_attn_fwd(*args, scale=scale, initial_state=d["first"], seqlens=lens, return_final_state=True)
    g = ssd.linear_attn_bwd(*args, d["dy"], scale=scale, initial_state=d["first"], dfinal_state=d["dlast"],
                            seqlens=lens, return_dinitial_state=True)
    return dict(y=y, final_state=state, **g)


def both(d, dtype, seqlens=None, scale=None):
    got = calls(d, seqlens, scale)
    torch.cuda.synchronize()
    want = ref.attention(*(n64(d[n]) for n in ("q", "k", "v", "decay")), scale=scale, first=n64(d["first"]),
                         seqlens=seqlens, dy=n64(d["dy"]), dlast=n64(d["dlast"]), dtype=dtype)
    for name, t in got.items():
        assert t.is_contiguous()
        ref.check(name, t, want, "f32" if "state" in name else dtype)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,L,H,K,Dk,Dv,wide,seqlens,carry", [
    (1, 1, 1, 1, 1, 1, 0, None, True),                   # the smallest of everything
    (1, 1, 2, 2, 128, 128, 0, None, False),
    (1, 64, 1, 1, 64, 64, 0, None, True),                # a whole chunk (two in fp32), one step less, one more
    (1, 63, 1, 1, 64, 64, 0, None, True),
    (2, 65, 2, 2, 128, 128, 0, None, True),
    (1, 31, 1, 1, 128, 64, 0, None, True),               # keys wider than values, and values than keys
    (1, 33, 1, 1, 64, 128, 0, None, False),
    (1, 130, 1, 1, 256, 256, 0, None, True),             # the widest
    (2, 70, 2, 1, 40, 75, 3, None, True),                # odd sizes at odd places, a shared key and value head
    (1, 70, 1, 1, 7, 3, 1, None, True),                  # rows shorter than 16 bytes
    (1, 40, 1, 1, 129, 65, 1, None, True),               # one past an instance's width
    (1, 40, 2, 2, 130, 200, 5, None, True),
    (2, 100, 6, 2, 64, 64, 0, [100, 37], True),
    (4, 80, 3, 1, 33, 64, 0, [80, 0, 1, 64], True),      # nothing, one step, a whole chunk
    (4, 80, 3, 3, 64, 33, 0, [80, 0, 1, 65], False),
    (3, 0, 2, 2, 16, 24, 0, None, True),                 # no steps: the states go through
    (1, 700, 1, 1, 32, 48, 0, None, True),               # segments
    (2, 600, 2, 1, 24, 16, 0, [600, 530], True),         # segments that end early, and in the last
    (3, 520, 1, 1, 16, 16, 0, [100, 257, 512], True),
])
def test_against_definition(dtype, Bz, L, H, K, Dk, Dv, wide, seqlens, carry):
    log("linear attention %s" % ((dtype, Bz, L, H, K, Dk, Dv, wide, seqlens, carry),))
    both(inputs(Bz, L, H, K, Dk, Dv, dtype, seed=L + Dk, wide=wide, carry=carry), dtype, seqlens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_and_scales(dtype):
    # no memory, none but a trace, no decay, growth; a scale of either sign and zero
    log("linear attention decays %s" % dtype)
    d = inputs(1, 150, 6, 6, 16, 24, dtype, seed=4)
    d["decay"] = torch.tensor([-float("inf"), -3e38, -87.0, -1e-9, 0.0, 0.004], device="cuda")
    for scale in (None, 0.0, -2.5):
        got = both(d, dtype, scale=scale)
        assert all(bool(t.isfinite().all()) for t in got.values())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_end_are_not_read(dtype):
    log("linear attention NaN behind the end %s" % dtype)
    d = inputs(3, 150, 2, 1, 24, 40, dtype, seed=3)
    seqlens = [150, 0, 70]
    clean = both(d, dtype, seqlens)
    for b, n in enumerate(seqlens):
        for name in ("q", "k", "v", "dy"):
            d[name][b, n:] = float("nan") if name != "v" else float("inf")
    got = calls(d, seqlens)
    # lengths outside 0 .. seqlen count as the nearest
    lens = torch.tensor([999, -3, 70], dtype=torch.int32, device="cuda")
    y, _ = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["decay"], initial_state=d["first"], seqlens=lens)
    torch.cuda.synchronize()
    for name, t in got.items():
        assert torch.equal(t, clean[name]), name
    assert torch.equal(y, clean["y"])
    for b, n in enumerate(seqlens):
        assert not got["y"][b, n:].any() and not got["dq"][b, n:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_is_not_finite_stays_in_its_head_and_later_chunks(dtype):
    log("linear attention NaN in one head %s" % dtype)
    d = inputs(2, 200, 3, 3, 32, 32, dtype, seed=8)
    clean = calls(d)
    d["v"][1, 130, 2, 5] = float("nan")
    got = calls(d)
    torch.cuda.synchronize()
    assert bool(got["y"][1, 130:, 2, 5].isnan().all())
    # the chunks before it, the other heads and batches: the same bits
    assert torch.equal(got["y"][:, :128], clean["y"][:, :128])
    assert torch.equal(got["y"][:, :, :2], clean["y"][:, :, :2]) and torch.equal(got["y"][0], clean["y"][0])
    for name in ("dq", "dk", "dv"):
        assert torch.equal(got[name][:, :, :2], clean[name][:, :, :2]), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,H,K,Dk,Dv,wide", [(1, 1, 1, 1, 1, 0), (3, 4, 2, 128, 128, 0), (2, 3, 1, 40, 75, 5),
                                               (2, 2, 2, 256, 256, 0), (5, 2, 2, 64, 7, 1), (1, 2, 2, 3, 256, 0)])
def test_steps_continue_a_prompt(dtype, Bz, H, K, Dk, Dv, wide):
    # a prompt, then single tokens from its state: the definition of one longer prompt
    log("linear attention steps %s" % ((dtype, Bz, H, K, Dk, Dv, wide),))
    d = inputs(Bz, 40, H, K, Dk, Dv, dtype, seed=Dk + Dv, wide=wide)
    cut = lambda t, a, b: t[:, a:b]   # noqa: E731
    y, state = ssd.linear_attn_fwd(*(cut(d[n], 0, 33) for n in "qkv"), d["decay"], initial_state=d["first"],
                                   return_final_state=True)
    ys = [ssd.linear_attn_step(state, d["q"][:, t], d["k"][:, t], d["v"][:, t], d["decay"]) for t in range(33, 40)]
    torch.cuda.synchronize()
    want = ref.attention(*(n64(d[n]) for n in ("q", "k", "v", "decay")), first=n64(d["first"]), dtype=dtype)
    ref.check("y", torch.cat([y, torch.stack(ys, 1)], 1), want, dtype)
    ref.check("final_state", state, want, "f32")


def test_the_chunked_scan_of_equal_decays():
    # beside the framework's own scan: one head to a group, the same decay in every step
    log("linear attention against the chunked scan")
    d = inputs(2, 128, 4, 4, 64, 32, "f32", seed=6)
    a = d["decay"].expand(2, 128, 4).contiguous()
    v, k, q = (d[n].contiguous() for n in "vkq")
    Y, S = ssd.chunk_scan_fwd(v, a, k, q, 64, initial_state=d["first"], return_final_state=True)
    y, s = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["decay"], scale=1.0, initial_state=d["first"],
                               return_final_state=True)
    torch.cuda.synchronize()
    want = ref.attention(*(n64(d[n]) for n in ("q", "k", "v", "decay")), scale=1.0, first=n64(d["first"]))
    ref.check("y", y, want, "f32")
    # two fp32 forms of the same sums: each within the bound of the definition
    lim = 2 * 2.0 ** -24 * 1.01 * want["~y"] + 2.0 ** -24 * np.abs(want["y"])
    assert (np.abs(n64(Y) - n64(y)) <= 4 * lim).all()
    assert (np.abs(n64(S) - n64(s)) <= 8 * 2.0 ** -24 * want["~final_state"]).all()


def test_gradients_against_differences():
    # fp32 kernels, central differences of the 64-bit forward along random directions
    log("linear attention differences")
    d = inputs(2, 40, 4, 2, 12, 20, "f32", seed=5)
    seqlens = [40, 23]
    got = both(d, "f32", seqlens)
    rng = np.random.default_rng(0)
    names = {"q": "dq", "k": "dk", "v": "dv", "first": "dinitial_state"}
    base = {n: n64(d[n]) for n in names}

    def loss(t):
        o = ref.attention(t["q"], t["k"], t["v"], n64(d["decay"]), first=t["first"], seqlens=seqlens)
        return (o["y"] * n64(d["dy"])).sum() + (o["final_state"] * n64(d["dlast"])).sum()

    for n, g in names.items():
        u = rng.standard_normal(base[n].shape)
        h = 1e-4   # the loss is linear in each: only cancellation, ~1e-16 |loss| / h, and the gradient's own error
        num = (loss({**base, n: base[n] + h * u}) - loss({**base, n: base[n] - h * u})) / (2 * h)
        ours = n64(got[g]) * u
        assert abs(num - ours.sum()) <= 1e-5 * (np.abs(ours).sum() + 1), n


@pytest.mark.parametrize("Bz,L,H,K", [(2, 200, 4, 4), (1, 700, 2, 1)])
def test_repeats_streams_and_graphs(Bz, L, H, K):
    # the same bits from repeated calls, from another stream, and from a captured
    # graph replayed between eager calls
    log("linear attention streams and graphs")
    d = inputs(Bz, L, H, K, 64, 64, "bf16", seed=9, wide=8)
    state0 = d["first"].clone()

    def run():
        state = state0.clone()
        y = ssd.linear_attn_step(state, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["decay"])
        return dict(calls(d), step=y, state=state)

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
            for n in want:
                assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_any_alignment(dtype, shift):
    # every tensor `shift` elements into its buffer: the same values
    log("linear attention alignment %s %d" % (dtype, shift))
    d = inputs(2, 70, 2, 2, 24, 40, dtype, seed=shift)
    move = lambda t: torch.cat([t.new_zeros(shift), t.flatten()])[shift:].view(t.shape)   # noqa: E731
    want = calls(d)
    m = {n: move(t) for n, t in d.items()}
    got = calls(m)
    y = move(torch.zeros_like(want["y"]))
    ssd.linear_attn_fwd(m["q"], m["k"], m["v"], m["decay"], initial_state=m["first"], y=y)
    s1, s2 = d["first"].clone(), move(d["first"])
    one = lambda s, t: ssd.linear_attn_step(s, t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], t["decay"])   # noqa: E731
    y1, y2 = one(s1, d), one(s2, m)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
    assert torch.equal(y, want["y"]) and torch.equal(y1, y2) and torch.equal(s1, s2)


def test_given_outputs_and_their_surroundings():
    log("linear attention given outputs")
    for dtype in ("bf16", "f32"):
        d = inputs(2, 70, 2, 2, 24, 41, dtype, seed=1)
        want, _ = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["decay"])
        n = want.numel()
        buf = torch.full((n + 64,), 5.0, dtype=DT[dtype], device="cuda")
        y = buf[32:32 + n].view(want.shape)
        state = torch.full_like(d["first"], 3.0)
        ws = torch.empty(max(1, ssd.linear_attn_fwd_workspace_bytes(d["q"], d["k"], d["v"], d["decay"])),
                         dtype=torch.uint8, device="cuda")
        got, fin = ssd.linear_attn_fwd(d["q"], d["k"], d["v"], d["decay"], y=y, final_state=state, workspace=ws)
        torch.cuda.synchronize()
        assert got is y and fin is state and torch.equal(y, want)
        assert bool((buf[:32] == 5).all()) and bool((buf[32 + n:] == 5).all())
        with pytest.raises(ssd.SSDError, match="SSD_ERR_ALIAS"):
            v = buf[:2 * 70 * 2 * 41].view(2, 70, 2, 41)
            ssd.linear_attn_fwd(d["q"], d["k"], v, d["decay"], y=v)


def test_no_sequences():
    log("linear attention empty batch")
    d = inputs(0, 9, 2, 1, 24, 16, "bf16")
    got = calls(d)
    state = torch.empty(0, 2, 16, 24, device="cuda")
    y = ssd.linear_attn_step(state, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["decay"])
    torch.cuda.synchronize()
    assert got["y"].shape == (0, 9, 2, 16) and got["dk"].shape == (0, 9, 1, 24) and y.shape == (0, 2, 16)
