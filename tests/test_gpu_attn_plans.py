"""GPU parity of linear attention at shapes whose plans cut sequences into segments, with pairs
walked whole beside them, and far apart in memory; the plain 64-bit form runs for all
(batch, head) pairs at once, with the tolerances of attn_ref."""
import threading

import pytest
import torch

import attn_cases as cases
import ssd_chunked_scan_chunk_amd as ssd
from attn_ref import HALF, U
from gpu_util import log
from test_gpu_linear_attn import calls, inputs

pytestmark = pytest.mark.gpu


def walks(a, c, x, decay, first, lens, lead, dtype, scale_w=1.0):
    """attn_ref's walk for pairs [n, L, size] at once, in time order; steps past lens are zeros."""
    n, L = a.shape[:2]
    S = torch.zeros(n, x.shape[2], c.shape[2], dtype=torch.float64, device="cuda")
    if first is not None:
        S = first / decay[:, None, None] ** (1 - lead)
    M, chunk = S.abs(), 64 if dtype == "bf16" else 32
    cuts = 2.0 ** -26 / U if dtype == "bf16" else 0.0
    half = 2.0 ** -17 / U if dtype == "bf16" else 0.0
    y = torch.zeros(n, L, x.shape[2], dtype=torch.float64, device="cuda")
    ey = torch.zeros_like(y)
    g = decay[:, None, None]
    for t in range(L):
        on = (t < lens)[:, None, None]
        inj = scale_w * x[:, t, :, None] * c[:, t, None, :]
        S = torch.where(on, g * S + inj, S)
        M = torch.where(on, g * M + inj.abs(), M)
        steps = 2 * (t + 1) + 5 * (t // chunk + 2) + 10 + cuts
        y[:, t] = (S * a[:, t, None, :]).sum(2) * on[:, :, 0]
        ey[:, t] = (M * a[:, t, None, :].abs()).sum(2) * (steps + 2 * a.shape[2] + 2 * chunk + half) * on[:, :, 0]
    return y, ey, S, M * (2 * lens + 5 * (lens // chunk + 2) + 10 + cuts)[:, None, None]


def check(name, got, want, err, dtype):
    lim = U * err + HALF[dtype] * (want.abs() + U * err) + 1e-30
    over = ((got.double() - want).abs() / lim).max().item() if got.numel() else 0.0
    assert bool(got.isfinite().all()) and over <= 1, "%s %s: %.3g of the tolerance" % (name, dtype, over)


def expected(d, lens, dtype, bwd):
    """Pairs' y and final state, or gradients; with their errors."""
    q, k, v, dy = (d[n].double() for n in ("q", "k", "v", "dy"))
    Bz, L, H, Dk = q.shape
    K, Dv = v.shape[2:]
    scale, each = Dk ** -0.5, H // K
    pairs = lambda t: t.transpose(1, 2).flatten(0, 1)                           # noqa: E731
    q, dy, k, v = pairs(q), pairs(dy), *(pairs(t.repeat_interleave(each, 2)) for t in (k, v))
    decay = d["decay"].double().exp().repeat(Bz)
    n = torch.tensor(lens, device="cuda").repeat_interleave(H)
    first, dlast = (d[s].double().flatten(0, 1) for s in ("first", "dlast"))
    back = lambda t: t.unflatten(0, (Bz, H)).transpose(1, 2)                    # noqa: E731
    state = lambda t: t.unflatten(0, (Bz, H))                                   # noqa: E731
    if not bwd:
        y, ey, S, eS = walks(q, k, v, decay, first, n, 1, dtype)
        return {"y": (scale * back(y), scale * back(ey)), "final_state": (state(S), state(eS))}
    at = (n[:, None] - 1 - torch.arange(L, device="cuda")).clamp(min=0)         # against time, from the end
    turn = lambda t: t.gather(1, at[:, :, None].expand_as(t)) * (torch.arange(L, device="cuda") < n[:, None])[:, :, None]   # noqa: E731
    shared = lambda t: back(t).unflatten(2, (K, each)).sum(3)                   # noqa: E731
    y, ey, _, _ = walks(dy, v, k, decay, first.transpose(1, 2), n, 1, dtype)
    out = {"dq": (scale * back(y), scale * back(ey))}
    y, ey, G, eG = walks(turn(k), turn(q), turn(dy), decay, dlast, n, 0, dtype, scale)
    more = lambda t: shared(turn(t).abs()) * 2 * each                           # noqa: E731
    out["dv"] = shared(turn(y)), shared(turn(ey)) + more(y)
    g = decay[:, None, None]
    out["dinitial_state"] = state(G * g), state((eG + 4 * G.abs()) * g)
    y, ey, _, _ = walks(turn(v), turn(dy), turn(q), decay, dlast.transpose(1, 2), n, 0, dtype, scale)
    out["dk"] = shared(turn(y)), shared(turn(ey)) + more(y)
    return out


@pytest.mark.parametrize("Bz,L,H,K,Dk,Dv,dtype,bwd,plan", cases.PLANS)
@pytest.mark.parametrize("ragged", [False, True])
def test_plans(Bz, L, H, K, Dk, Dv, dtype, bwd, plan, ragged):
    log("linear attention plan %s" % ((Bz, L, H, K, Dk, Dv, dtype, bwd, plan, ragged),))
    d = inputs(Bz, L, H, K, Dk, Dv, dtype, seed=H, wide=8, lo=20.0, hi=2000.0)
    # ends inside a segment: the sequences' last and, in pairs that are cut, the second
    lens = [L - 3, plan[1] + 37][:Bz] if ragged else [L] * Bz
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda") if ragged else None
    args = [d[n] for n in ("q", "k", "v", "decay")]
    if bwd:
        got = ssd.linear_attn_bwd(*args, d["dy"], initial_state=d["first"], dfinal_state=d["dlast"], seqlens=seqlens,
                                  return_dinitial_state=True)
    else:
        y, state = ssd.linear_attn_fwd(*args, initial_state=d["first"], seqlens=seqlens, return_final_state=True)
        got = {"y": y, "final_state": state}
    torch.cuda.synchronize()
    for name, (want, err) in expected(d, lens, dtype, bwd).items():
        check(name, got[name], want, err, "f32" if "state" in name else dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bz,L,H,K,Dk,Dv", [(2, 330, 2, 1, 203, 131), (2, 330, 3, 3, 109, 99), (2, 200, 2, 2, 5, 250),
                                            (2, 330, 2, 2, 134, 64), (2, 200, 4, 2, 63, 9), (2, 330, 1, 1, 250, 222)])
def test_rows_of_any_length(dtype, Bz, L, H, K, Dk, Dv):
    # last pieces that are not whole, in both slices of columns, over many chunks
    log("linear attention rows %s" % ((dtype, Bz, L, H, K, Dk, Dv),))
    d = inputs(Bz, L, H, K, Dk, Dv, dtype, seed=Dk, wide=3, lo=20.0, hi=2000.0)
    lens = [L - 1, 97]
    got = calls(d, lens)
    torch.cuda.synchronize()
    for bwd in (False, True):
        for name, (want, err) in expected(d, lens, dtype, bwd).items():
            check(name, got[name], want, err, "f32" if "state" in name else dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_apart(dtype):
    # batches more than 2^32 bytes apart, and steps of the longest stride: offsets beyond 32 bits
    log("linear attention far apart %s" % dtype)
    d = inputs(2, 70, 2, 1, 64, 64, dtype, seed=2)
    want = calls(d)
    size = d["q"].element_size()
    buf = torch.empty((1 << 24) * 69 + 4096 + (1 << 33) // size, dtype=d["q"].dtype, device="cuda")
    far = lambda t: buf.as_strided(t.shape, ((1 << 33) // size, 1 << 24, t.shape[3], 1))   # noqa: E731
    for n in ("q", "k", "v"):
        m = dict(d, **{n: far(d[n]).copy_(d[n])})
        got = calls(m)
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), (n, name)


def test_threads_and_graphs_side_by_side():
    # two threads on streams of their own, and two captured graphs with workspaces of their own, in turn
    log("linear attention threads and graphs")
    ds = [inputs(2, 700, 3, 1, 64, 64, "bf16", seed=s, wide=8) for s in (1, 2)]
    wants = [calls(d) for d in ds]
    torch.cuda.synchronize()
    found = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got = calls(ds[i])
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(got[n], wants[i][n]) for n in got):
                    found[i] = False
                    return
        found[i] = True

    jobs = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for j in jobs:
        j.start()
    for j in jobs:
        j.join()
    assert found == [True, True]
    graphs, helds = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph, d in zip(graphs, ds):
        with torch.cuda.graph(graph):
            helds.append(calls(d))
    for order in ((0, 1), (1, 0), (0, 1)):
        for i in order:
            for t in helds[i].values():
                t.fill_(7)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in order:
            for n in wants[i]:
                assert torch.equal(helds[i][n], wants[i][n]), (i, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_a_workspace_held_before_does_not_matter(dtype):
    # of NaN: segments that end early, shared heads, sequences of nothing; the norm's parts
    log("linear attention and group norm, workspaces of NaN %s" % dtype)
    d = inputs(3, 900, 4, 2, 64, 40, dtype, seed=4, wide=8)
    args = [d[n] for n in ("q", "k", "v", "decay")]
    lens = torch.tensor([900, 0, 333], dtype=torch.int32, device="cuda")
    nans = lambda n: torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # noqa: E731
    kw = dict(initial_state=d["first"], seqlens=lens)
    fwd, bwd = ssd.linear_attn_fwd_workspace_bytes(*args), ssd.linear_attn_bwd_workspace_bytes(*args)
    assert fwd > 0 and bwd > 0
    y, s = ssd.linear_attn_fwd(*args, return_final_state=True, **kw)
    y2, s2 = ssd.linear_attn_fwd(*args, return_final_state=True, workspace=nans(fwd), **kw)
    kw.update(dfinal_state=d["dlast"], return_dinitial_state=True)
    g, g2 = ssd.linear_attn_bwd(*args, d["dy"], **kw), ssd.linear_attn_bwd(*args, d["dy"], workspace=nans(bwd), **kw)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2) and all(torch.equal(g[n], g2[n]) for n in g)
    x, w = d["dy"].flatten(2), torch.ones(160, device="cuda")
    for groups in (1, 4, 40):
        kw = dict(weight=w, bias=w, seqlens=lens)
        ws = nans(ssd.group_norm_bwd_workspace_bytes(x, groups))
        g, g2 = ssd.group_norm_bwd(x, groups, y.flatten(2), **kw), ssd.group_norm_bwd(x, groups, y.flatten(2), workspace=ws, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(g[n], g2[n]) for n in ("dx", "dweight", "dbias"))
