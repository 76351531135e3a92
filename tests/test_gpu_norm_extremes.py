"""Group norm with gates of the lowest and largest finite values (a mask sets the lowest) and infinities."""
import pytest
import torch

from gpu_util import log
from test_gpu_group_norm import DT, calls, inputs

pytestmark = pytest.mark.gpu

SIZES = [(96, 3), (1200, 1), (6, 3), (771, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,groups", SIZES)
@pytest.mark.parametrize("gate_first", [False, True])
def test_masked_gates(dtype, C, groups, gate_first):
    # silu and its slope are 0 from -104 on: single channels, a whole group and a whole row at the lowest
    # value give the bits that -200 gives there
    log("group norm masked gates %s" % ((dtype, C, groups, gate_first),))
    d = inputs(3, 5, C, dtype, seed=C)
    m = C // groups
    want, got = {}, {}
    for low, out in ((-200.0, want), (torch.finfo(DT[dtype]).min, got)):
        d["gate"][0, 1, ::3] = low
        d["gate"][1, 2, :m] = low
        d["gate"][2, 4] = low
        out.update(calls(d, groups, gate_first=gate_first))
    torch.cuda.synchronize()
    for n in want:
        assert bool(got[n].isfinite().all()) and torch.equal(got[n], want[n]), n
    if not gate_first:
        assert not got["y"][2, 4].any() and not got["dgate"][2, 4].any() and not got["dx"][2, 4].any()
    else:
        assert not got["dx"][2, 4].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,groups", SIZES)
def test_largest_gates(dtype, C, groups):
    # silu is the gate itself and its slope 1: as without the activation, where nothing overflows
    log("group norm largest gates %s" % ((dtype, C, groups),))
    d = inputs(1, 3, C, dtype, seed=C)
    d["x"] *= 2.0 ** -60
    d["dy"] *= 2.0 ** -60
    d["weight"], d["bias"] = d["weight"] * 2.0 ** -60, d["bias"] * 2.0 ** -60
    d["gate"][:] = torch.finfo(DT[dtype]).max
    got, want = calls(d, groups), calls(d, groups, silu=False)
    torch.cuda.synchronize()
    for n in want:
        assert bool(got[n].isfinite().all()) and torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,groups", SIZES)
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("name", ["x", "gate", "dy"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_infinities_stay_in_their_group(dtype, C, groups, gate_first, name, value):
    log("group norm infinities %s" % ((dtype, C, groups, gate_first, name, value),))
    d = inputs(2, 5, C, dtype, seed=C)
    clean = calls(d, groups, gate_first=gate_first)
    m = C // groups
    d[name][1, 3, 1] = value                   # of the first group of one row
    got = calls(d, groups, gate_first=gate_first)
    torch.cuda.synchronize()
    for n in ("y", "dx", "dgate"):
        a, b = got[n].clone(), clean[n].clone()
        a[1, 3, :m], b[1, 3, :m] = 0, 0
        assert torch.equal(a, b), n
    for n in ("dweight", "dbias"):
        assert torch.equal(got[n][m:], clean[n][m:]), n
    if name == "dy":
        assert torch.equal(got["y"], clean["y"])
    # where the definition has no finite value, none is made up
    bad = {"x": "y", "gate": "y", "dy": "dx"}[name]
    assert not bool(got[bad][1, 3, 1].isfinite())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,groups", SIZES)
def test_squares_beyond_the_range(dtype, C, groups):
    # sums of squares that overflow leave n = 0, the row's bias; in that group alone
    log("group norm squares %s" % ((dtype, C, groups),))
    d = inputs(2, 5, C, dtype, seed=C, gate=False)
    m = C // groups
    clean = calls(d, groups, silu=False)
    d["x"][1, 3, 0] = 1e25
    got = calls(d, groups, silu=False)
    torch.cuda.synchronize()
    assert torch.equal(got["y"][1, 3, :m], d["bias"][:m].to(DT[dtype]))
    a, b = got["y"].clone(), clean["y"].clone()
    a[1, 3, :m], b[1, 3, :m] = 0, 0
    assert torch.equal(a, b) and all(bool(t.isfinite().all()) for t in got.values() if t is not None)
