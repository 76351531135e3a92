"""Linear attention in float32 at the ends of the range that bf16 parts leave it: all 24 bits down to
magnitudes of 2^-110, values up to 3.38e38, and NaN, kept to their head, for what is beyond."""
import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log
from test_gpu_attn_parts import LIMIT, U, one_each, pairs_of, values
from test_gpu_linear_attn import calls, inputs

pytestmark = pytest.mark.gpu


def one_product_each(n, Dk, Dv, k_by, q_by, v_by, scale, whole=False):
    """Results of a single product each, as in test_gpu_attn_parts: their errors, y and the state."""
    g = torch.Generator().manual_seed(n)
    meets, decay = pairs_of(n, g), torch.tensor([-1 / 500.0])
    k, kv = one_each(g, n, Dk, torch.arange(n))
    q, qv = one_each(g, n, Dk, meets)
    v = values(g, n, Dv)
    if whole:                                  # powers of two
        k, q, v, kv, qv = (t.sign() for t in (k, q, v, kv, qv))
    up = lambda t, by: (t * by)[None, :, None].cuda()   # noqa: E731
    y, last = ssd.linear_attn_fwd(up(q, q_by), up(k, k_by), up(v, v_by), decay.cuda(), scale=scale, return_final_state=True)
    torch.cuda.synchronize()
    k, q, v = (k_by * kv).double(), (q_by * qv).double(), (v * v_by).double()
    back = torch.arange(n) - meets
    w = scale * torch.where(back >= 0, torch.exp(decay.double() * back.clamp(min=0)), 0) * q * k[meets]
    want = w[:, None] * v[meets]
    S = torch.exp(decay.double() * (n - 1 - torch.arange(n))) * k * v.t()
    y, last = y[0, :, 0].double().cpu(), last[0, 0, :, :n].double().cpu()
    assert not y[want == 0].any()
    on = want != 0
    return ((y - want).abs()[on] / want.abs()[on]).max().item() / U, ((last - S).abs() / S.abs()).max().item() / U


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (256, 256)])
@pytest.mark.parametrize("name", ["keys", "values", "scores"])
def test_small_magnitudes(Dk, Dv, name):
    # the last bit of the third part is 2^-23 of a value: at 2^-110 it is 2^-133, the smallest bf16
    def errors(e):
        if name == "keys":
            return one_product_each(64, Dk, Dv, 2.0 ** e, 2.0 ** -e, 1.0, 1.0)
        if name == "values":
            return one_product_each(64, Dk, Dv, 1.0, 1.0, 2.0 ** e, 2.0 ** -e)
        return one_product_each(64, Dk, Dv, 2.0 ** e, 1.0, 1.0, 2.0 ** -e)

    log("linear attention, small %s" % ((Dk, Dv, name),))
    assert max(errors(-110)) <= LIMIT
    # further down a factor is off by up to half of 2^-133, 256 halves of a step of fp32 at 2^-118;
    # on the way to y three factors may be that small: the row, the decayed row or score, the state
    assert max(errors(-118)) <= LIMIT + 3 * 256


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 128), (256, 256)])
def test_large_magnitudes(Dk, Dv):
    log("linear attention, large %s" % ((Dk, Dv),))
    largest = float(torch.tensor(3.38e38))
    assert max(one_product_each(64, Dk, Dv, 1.0, 1.0, largest, 0.5, whole=True)) <= LIMIT


@pytest.mark.parametrize("name", ["q", "k", "v", "dy", "first"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), 3.4e38])
def test_beyond_is_nan_in_its_head(name, value):
    log("linear attention, beyond the range %s" % ((name, value),))
    d = inputs(2, 100, 3, 3, 40, 24, "f32", seed=6)
    clean = calls(d)
    before = d["first"][1, 2, 5, 7].clone()
    if name == "first":
        d["first"][1, 2, 5, 7] = value
    else:
        d[name][1, 50, 2, 5] = value
    got = calls(d)
    torch.cuda.synchronize()
    hit = {"q": ("y", "dk", "dv", "dinitial_state"), "k": ("final_state", "dv", "dq"), "v": ("y", "final_state", "dk", "dq"),
           "dy": ("dq", "dk", "dv", "dinitial_state"), "first": ("y", "dq")}[name]
    if name == "first":     # a state goes on in fp32, its parts only into y: infinite, or what it decays to
        want = clean["final_state"][1, 2, 5, 7] + (value - float(before)) * torch.exp(100 * d["decay"][2])
        assert bool(torch.isclose(got["final_state"][1, 2, 5, 7], want, rtol=1e-5, atol=0))
    if value == 3.4e38:     # a state takes the decayed row, e^(-49/200) of it here: within the range
        hit = tuple(n for n in hit if "state" not in n)
    for n, t in got.items():
        head = (slice(None), 2) if "state" in n else (slice(None), slice(None), 2)
        assert n not in hit or bool(t[head][1].isnan().any()), n
        a, b = t.clone(), clean[n].clone()      # the other heads and the other batch: the same bits
        a[head][1], b[head][1] = 0, 0
        assert torch.equal(a, b), n
    # chunks of 32 steps: those before are untouched, and after in dk and dv, whose chunks count from
    # the end: step 50 of 100 is the 49th from there, in the chunk of the 32nd to the 63rd, steps 36 to 67
    if name in ("q", "k", "v"):
        assert torch.equal(got["y"][:, :32], clean["y"][:, :32])
    if name in ("q", "k", "v", "dy"):
        assert torch.equal(got["dv"][:, 68:], clean["dv"][:, 68:])
