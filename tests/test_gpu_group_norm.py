"""GPU parity of the group norm with its activation or gate (forward and
backward) against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import attn_ref as ref
import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FORMS = {"plain": dict(gate=False), "gate": dict(gate=True), "gate_first": dict(gate=True, gate_first=True),
         "rms": dict(gate=True, gate_first=True, center=False), "linear": dict(gate=False, silu=False),
         "linear gate": dict(gate=True, silu=False, center=False), "linear gate_first": dict(gate=True, silu=False,
                                                                                          gate_first=True)}


def n64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inputs(Bz, L, C, dtype, seed=0, wide=0, gate=True, affine=True, offset=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=DT[dtype]: torch.randn(s, generator=g).to(dt).cuda()   # noqa: E731
    x, z = (r(Bz, L, wide + C)[:, :, wide:] for _ in range(2))
    x += offset
    return dict(x=x, gate=z if gate else None, weight=r(C, dt=torch.float32) if affine else None,
                bias=r(C, dt=torch.float32) if affine else None, dy=r(Bz, L, C))


def calls(d, groups, seqlens=None, **form):
    lens = None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device="cuda")
    kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"], seqlens=lens, **form)
    return dict(y=ssd.group_norm_fwd(d["x"], groups, **kw), **ssd.group_norm_bwd(d["x"], groups, d["dy"], **kw))


def both(d, groups, dtype, seqlens=None, **form):
    got = calls(d, groups, seqlens, **form)
    torch.cuda.synchronize()
    want = ref.norm(n64(d["x"]), groups, n64(d["weight"]), n64(d["bias"]), n64(d["gate"]), seqlens=seqlens,
                    dy=n64(d["dy"]), **form)
    for name, t in got.items():
        if t is None:
            assert {"dgate": d["gate"], "dweight": d["weight"], "dbias": d["bias"]}[name] is None
            continue
        ref.check(name, t, want, "f32" if name in ("dweight", "dbias") else dtype)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("Bz,L,C,groups,wide,seqlens,affine", [
    (1, 1, 1, 1, 0, None, True),                     # one channel: n is 0, or a sign
    (2, 5, 12, 4, 1, None, True),                    # groups shorter than 16 bytes
    (2, 9, 64, 1, 0, None, True),                    # several rows in a wavefront
    (3, 7, 771, 3, 5, [7, 0, 3], True),              # odd sizes at odd places, unequal lengths
    (1, 3, 5120, 40, 0, None, True),                 # a head of 128 to a group
    (2, 2, 5120, 1, 0, None, False),                 # the row as one group: a workgroup
    (1, 3, 513, 1, 3, None, True),                   # one piece more than a wavefront holds (two in fp32)
    (2, 70, 72, 9, 0, [70, 33], True),
])
def test_against_definition(dtype, form, Bz, L, C, groups, wide, seqlens, affine):
    log("group norm %s" % ((dtype, form, Bz, L, C, groups, wide, seqlens, affine),))
    f = dict(FORMS[form])
    d = inputs(Bz, L, C, dtype, seed=C + L, wide=wide, gate=f.pop("gate"), affine=affine)
    both(d, groups, dtype, seqlens, **f)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,groups", [(16384, 1), (9001, 1), (4100, 1), (2 * 8200, 2)])
def test_long_groups(dtype, C, groups):
    log("group norm long %s %d %d" % (dtype, C, groups))
    both(inputs(1, 3, C, dtype, seed=C), groups, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(dtype):
    # more rows than workgroups down them: every one walks several
    log("group norm rows %s" % dtype)
    both(inputs(2, 1500, 96, dtype, seed=2), 3, dtype)
    both(inputs(1, 2100, 1032, dtype, seed=2), 1, dtype, gate_first=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_constant_rows_and_large_values(dtype):
    # no variance: n is 0 where the mean is exact, eps alone divides; values far from 0
    log("group norm constants %s" % dtype)
    d = inputs(1, 4, 128, dtype, seed=7)
    d["x"][0, 0] = 0.0
    d["x"][0, 1] = 1.0
    d["x"][0, 2] = 3.0e4
    got = both(d, 2, dtype)
    assert all(bool(t.isfinite().all()) for t in got.values())
    d["x"][0, 3] *= 1e15
    both(d, 2, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_gates(dtype):
    # gates beyond the exponential's range: silu is 0 or the gate itself
    log("group norm gates %s" % dtype)
    d = inputs(1, 3, 64, dtype, seed=7)
    d["gate"][0, 0] = 200.0
    d["gate"][0, 1] = -200.0
    for first in (False, True):
        got = both(d, 2, dtype, gate_first=first)
        assert all(bool(t.isfinite().all()) for t in got.values())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_end_are_not_read(dtype):
    log("group norm NaN behind the end %s" % dtype)
    for C, groups in ((96, 3), (1200, 1), (6, 3)):
        d = inputs(3, 30, C, dtype, seed=3)
        seqlens = [30, 0, 17]
        clean = both(d, groups, dtype, seqlens)
        for b, n in enumerate(seqlens):
            for name in ("x", "gate", "dy"):
                d[name][b, n:] = float("nan")
        got = calls(d, groups, seqlens)
        torch.cuda.synchronize()
        for name, t in got.items():
            assert torch.equal(t, clean[name]), name
        assert not got["y"][1].any() and not got["dgate"][2, 17:].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_token_is_a_row(dtype):
    log("group norm token %s" % dtype)
    d = inputs(5, 4, 384, dtype, seed=1, wide=8)
    kw = dict(weight=d["weight"], bias=d["bias"], gate=d["gate"])
    y = ssd.group_norm_fwd(d["x"], 3, **kw)
    ys = [ssd.group_norm_fwd(d["x"][:, t], 3, **dict(kw, gate=d["gate"][:, t])) for t in range(4)]
    g = ssd.group_norm_bwd(d["x"][:, 0], 3, d["dy"][:, 0].contiguous(), **dict(kw, gate=d["gate"][:, 0]))
    whole = ssd.group_norm_bwd(d["x"], 3, d["dy"], **kw)
    torch.cuda.synchronize()
    assert torch.equal(torch.stack(ys, 1), y)
    assert torch.equal(g["dx"], whole["dx"][:, 0]) and torch.equal(g["dgate"], whole["dgate"][:, 0])


def test_gradients_against_differences():
    log("group norm differences")
    for form, f in FORMS.items():
        f = dict(f)
        d = inputs(2, 6, 24, "f32", seed=5, gate=f.pop("gate"))
        got = both(d, 2, "f32", [6, 4], **f)
        rng = np.random.default_rng(0)
        names = {n: g for n, g in (("x", "dx"), ("gate", "dgate"), ("weight", "dweight"), ("bias", "dbias"))
                 if d[n] is not None}
        base = {n: n64(d[n]) for n in ("x", "gate", "weight", "bias")}

        def loss(t):
            o = ref.norm(t["x"], 2, t["weight"], t["bias"], t["gate"], seqlens=[6, 4], **f)
            return (o["y"] * n64(d["dy"])).sum()

        for n, g in names.items():
            u = rng.standard_normal(base[n].shape)
            h = 1e-5
            num = (loss({**base, n: base[n] + h * u}) - loss({**base, n: base[n] - h * u})) / (2 * h)
            ours = n64(got[g]) * u
            assert abs(num - ours.sum()) <= 1e-5 * (np.abs(ours).sum() + 1), (form, n)


def test_repeats_streams_and_graphs():
    log("group norm streams and graphs")
    for C, groups in ((384, 3), (2048, 1)):
        d = inputs(2, 200, C, "bf16", seed=9, wide=8)
        want = calls(d, groups)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = calls(d, groups)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = calls(d, groups)
        for _ in range(3):
            for t in held.values():
                t.fill_(7)
            graph.replay()
            again = calls(d, groups)
            torch.cuda.synchronize()
            for got in (other, held, again):
                for n in want:
                    assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_any_alignment(dtype, shift):
    log("group norm alignment %s %d" % (dtype, shift))
    for C, groups in ((96, 2), (1000, 1)):
        d = inputs(2, 21, C, dtype, seed=shift)
        move = lambda t: torch.cat([t.new_zeros(shift), t.flatten()])[shift:].view(t.shape)   # noqa: E731
        want = calls(d, groups)
        m = {n: move(t) for n, t in d.items()}
        got = calls(m, groups)
        n = want["y"].numel()
        buf = torch.full((n + 64 + shift,), 5.0, dtype=DT[dtype], device="cuda")
        y = buf[32 + shift:32 + shift + n].view(want["y"].shape)
        ssd.group_norm_fwd(m["x"], groups, weight=m["weight"], bias=m["bias"], gate=m["gate"], y=y)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), k
        assert torch.equal(y, want["y"])
        assert bool((buf[:32 + shift] == 5).all()) and bool((buf[32 + shift + n:] == 5).all())


def test_no_rows():
    log("group norm empty")
    for Bz, L in ((0, 9), (3, 0)):
        d = inputs(Bz, L, 24, "bf16")
        got = calls(d, 2)
        torch.cuda.synchronize()
        assert got["y"].shape == (Bz, L, 24) and not got["dweight"].any() and not got["dbias"].any()


# ---- as a layer uses them: convolution, attention, norm, prompt and tokens -----------------

def test_a_layer_of_them():
    log("convolution, linear attention and norm together")
    Bz, L, H, D = 2, 90, 4, 32
    C = H * D
    g = torch.Generator().manual_seed(0)
    r = lambda *s, dt=torch.float32: torch.randn(s, generator=g).to(dt).cuda()   # noqa: E731
    rows = r(Bz, L, 4 * C)
    filt, fbias, w, b = r(3 * C, 4), r(3 * C), r(C), r(C)
    decay = -1 / torch.tensor([4.0, 16.0, 64.0, 256.0], device="cuda")
    lens = torch.tensor([90, 41], dtype=torch.int32, device="cuda")
    heads = lambda t: t.unflatten(-1, (H, D))     # noqa: E731

    def prompt(rows, lens, window=None, state=None):
        (q, k, v), window = ssd.short_conv_fwd(rows[..., C:], filt, fbias, initial_window=window, seqlens=lens,
                                               pieces=(C, C, C), return_final_window=True)
        y, state = ssd.linear_attn_fwd(heads(q), heads(k), heads(v), decay, initial_state=state, seqlens=lens,
                                       return_final_state=True)
        out = ssd.group_norm_fwd(y.flatten(2), H, weight=w, bias=b, gate=rows[..., :C], seqlens=lens)
        return out, window, state, (q, k, v, y)

    out, window, state, (q, k, v, y) = prompt(rows, lens)
    want = ref.norm(n64(y).reshape(Bz, L, C), H, n64(w), n64(b), n64(rows[..., :C]), seqlens=[90, 41])
    ref.check("y", out, want, "f32")
    att = ref.attention(n64(heads(q)), n64(heads(k)), n64(heads(v)), n64(decay), seqlens=[90, 41])
    ref.check("y", y, att, "f32")
    ref.check("final_state", state, att, "f32")
    # the first sequence as a prompt of 80 and ten tokens
    half, win, st, _ = prompt(rows[:1, :80], None)
    tail = []
    for t in range(80, 90):
        q1, k1, v1 = ssd.short_conv_step(win, rows[:1, t, C:], filt, fbias, pieces=(C, C, C))
        y1 = ssd.linear_attn_step(st, heads(q1), heads(k1), heads(v1), decay)
        tail.append(ssd.group_norm_fwd(y1.flatten(1), H, weight=w, bias=b, gate=rows[:1, t, :C]))
    torch.cuda.synchronize()
    assert torch.equal(win, window[:1])
    # two fp32 orders of the same sums
    both_ = torch.cat([half, torch.stack(tail, 1)], 1)
    assert float((both_ - out[:1]).norm() / out[:1].norm()) < 1e-5
    assert float((st - state[:1]).norm() / state[:1].norm()) < 1e-5
    # and the gradients back to the projection's rows, against differences of the 64-bit forms
    dout = r(Bz, L, C)
    gn = ssd.group_norm_bwd(y.flatten(2), H, dout, weight=w, bias=b, gate=rows[..., :C], seqlens=lens)
    ga = ssd.linear_attn_bwd(heads(q), heads(k), heads(v), decay, heads(gn["dx"]), seqlens=lens)
    gc = ssd.short_conv_bwd(rows[..., C:], filt, tuple(ga[n].flatten(2) for n in ("dq", "dk", "dv")), fbias, seqlens=lens)
    torch.cuda.synchronize()
    import layer_ref

    def loss(rows64):
        c = layer_ref.conv(rows64[..., C:], n64(filt), n64(fbias), None, [90, 41], True)["y"]
        q, k, v = (c[..., i * C:(i + 1) * C].reshape(Bz, L, H, D) for i in range(3))
        a = ref.attention(q, k, v, n64(decay), seqlens=[90, 41])["y"]
        o = ref.norm(a.reshape(Bz, L, C), H, n64(w), n64(b), rows64[..., :C], seqlens=[90, 41])["y"]
        return (o * n64(dout)).sum()

    base = n64(rows)
    ours = np.concatenate([n64(gn["dgate"]), n64(gc["dx"])], -1)
    u = np.random.default_rng(1).standard_normal(base.shape)
    h = 1e-6
    num = (loss(base + h * u) - loss(base - h * u)) / (2 * h)
    assert abs(num - (ours * u).sum()) <= 1e-4 * np.abs(ours * u).sum()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,C,groups", [(3000, 2, 2), (2500, 64, 8), (1500, 120, 1), (700, 24, 3), (257, 3, 1)])
def test_many_rows_of_few_channels(dtype, L, C, groups):
    # rows beside each other in a workgroup, whose parameters' gradients it adds up itself
    log("group norm many rows %s" % ((dtype, L, C, groups),))
    for form in ("gate", "plain"):
        d = inputs(2, L, C, dtype, seed=C, gate=form == "gate")
        both(d, groups, dtype, [L, L // 2 + 1])


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_padding_is_zero_whatever_the_parameters(gate, gate_first):
    # eps 0, and parameters that are not finite: rows behind the end are zeros all the same
    if gate_first and not gate:
        return
    log("group norm padding")
    for C, groups in ((96, 3), (1200, 1), (6, 3)):
        d = inputs(2, 9, C, "bf16", seed=1, gate=gate)
        d["weight"][:2] = float("inf")
        d["bias"][1:3] = float("nan")
        got = calls(d, groups, [9, 4], eps=0.0, gate_first=gate_first)
        torch.cuda.synchronize()
        for name in ("y", "dx") + (("dgate",) if gate else ()):
            assert not got[name][1, 4:].any(), name
