"""Linear attention in float32, whose factors are multiplied as three bf16 parts each: that all
24 bits of them count, at every width, in y and in each gradient.

Where a result is a sum over many steps and elements, the bound of its sum hides what a lost
part would cost.  So here every result is a single product: the contracted rows have one element
that is not 0, each in a place of its own, and every row meets one other.

Tolerances, in halves of a step of fp32 (U, relative to the single product):
  a product of parts   13: 1 left out, as a bf16 rounding leaves at most 2^-8 of a value and the next
                       2^-17, so the three products of parts that are not formed reach 2 x 2^-25 + 2^-34;
                       6 partial products added up within an ulp each
  a power of gamma     4, a scale or a decay multiplied on 1 each
  in a chunk           score 13, its decay and scale 4 + 1 + 1, its product 13: 32
  across chunks        decayed row 4 + 1 + 1, its product 13, the powers and products of up to 3
                       chunks or segments in between 5 each, the state's product 13, its power
                       and scale 4 + 1 + 1: 53
  final_state, dinitial_state   no second product, one more power and product: below that
With two parts to a factor a product is off by up to 2^-16 + 2 x 2^-17, 512 U
(test_a_lost_part_is_seen has what these inputs make of it)."""
import numpy as np
import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log

U = 2.0 ** -24
LIMIT = 53

SIZES = [(64, 64), (128, 128), (256, 256), (64, 128), (128, 64), (256, 64), (64, 256), (99, 75)]


def values(g, *shape):
    """Of all 24 bits, between 1 and 2 in size."""
    return ((1 + torch.rand(shape, generator=g, dtype=torch.float64)) * (1 - 2 * torch.randint(0, 2, shape, generator=g))).float()


def one_each(g, n, size, at):
    """n rows with one element that is not 0, row t's at at[t]; and those elements."""
    v = values(g, n)
    rows = torch.zeros(n, size)
    rows[torch.arange(n), at] = v
    return rows, v


def pairs_of(n, g):
    """A row to meet for every row: itself, one before and one after, by turns of a permutation."""
    p = torch.randperm(n, generator=g)
    p[: n // 4] = torch.arange(n)[: n // 4][torch.randperm(n // 4, generator=g)]   # some within the first chunk
    rest = torch.tensor(sorted(set(range(n)) - set(p[: n // 4].tolist())))
    p[n // 4:] = rest[torch.randperm(len(rest), generator=g)]
    return p


def within(name, got, want):
    lim = LIMIT * U * want.abs()
    off = (got.double().cpu() - want).abs()
    assert bool((got.cpu()[want == 0] == 0).all()), name
    worst = (off[want != 0] / want.abs()[want != 0]).max().item() / U
    print("%s: %.1f U" % (name, worst), flush=True)
    assert bool((off <= lim).all()), "%s: %.1f U" % (name, worst)


@pytest.mark.gpu
@pytest.mark.parametrize("Dk,Dv", SIZES)
@pytest.mark.parametrize("span", [20.0, 500.0])
def test_every_bit_counts(Dk, Dv, span):
    log("linear attention, parts %s" % ((Dk, Dv, span),))
    n = min(Dk, Dv, 100)
    g = torch.Generator().manual_seed(Dk + Dv)
    meets = pairs_of(n, g)                    # row t of the one side meets row meets[t] of the other
    decay = torch.tensor([-1 / span])
    back = torch.arange(n) - meets            # steps between; below 0: not yet
    power = torch.where(back >= 0, torch.exp(decay.double() * back.clamp(min=0)), 0)
    scale = float(np.float32(Dk ** -0.5))
    up = lambda t: t[None, :, None].cuda()    # noqa: E731
    state = torch.zeros(1, 1, Dv, Dk).cuda()

    # queries and keys of one element each: y, dv, the states
    k, kv = one_each(g, n, Dk, torch.arange(n))
    q, qv = one_each(g, n, Dk, meets)
    v, dy = values(g, n, Dv), values(g, n, Dv)
    args = up(q), up(k), up(v), decay.cuda()
    y, last = ssd.linear_attn_fwd(*args, scale=scale, return_final_state=True)
    got = ssd.linear_attn_bwd(*args, up(dy), scale=scale, initial_state=state, return_dinitial_state=True)
    torch.cuda.synchronize()
    w = scale * power * qv.double() * kv.double()[meets]            # of row t and the one it meets
    within("y", y[0, :, 0], w[:, None] * v.double()[meets])
    dv = torch.zeros(n, Dv, dtype=torch.float64)
    dv[meets] = w[:, None] * dy.double()
    within("dv", got["dv"][0, :, 0], dv)
    S = torch.zeros(Dv, Dk, dtype=torch.float64)
    S[:, :n] = (torch.exp(decay.double() * (n - 1 - torch.arange(n))) * kv.double() * v.double().t())
    within("final_state", last[0, 0], S)
    G = torch.zeros(Dv, Dk, dtype=torch.float64)
    G[:, meets] = scale * torch.exp(decay.double() * (torch.arange(n) + 1)) * qv.double() * dy.double().t()
    within("dinitial_state", got["dinitial_state"][0, 0], G)

    # values and dy of one element each: dq and dk
    v, vv = one_each(g, n, Dv, torch.arange(n))
    dy, dv = one_each(g, n, Dv, meets)
    q, k = values(g, n, Dk), values(g, n, Dk)
    got = ssd.linear_attn_bwd(up(q), up(k), up(v), decay.cuda(), up(dy), scale=scale)
    torch.cuda.synchronize()
    w = scale * power * dv.double() * vv.double()[meets]
    within("dq", got["dq"][0, :, 0], w[:, None] * k.double()[meets])
    dk = torch.zeros(n, Dk, dtype=torch.float64)
    dk[meets] = w[:, None] * q.double()
    within("dk", got["dk"][0, :, 0], dk)


def bf16(t):
    return t.to(torch.bfloat16).float()


def product(a, b, parts):
    """a b of the largest products of ``parts`` bf16 parts of each, in 32 bits, large ones last."""
    def split(v):
        out = []
        for _ in range(parts):
            out.append(bf16(v))
            v = v - out[-1]
        return out
    a, b = split(a), split(b)
    total = torch.zeros_like(a[0] * b[0])
    for order in reversed(range(parts)):
        for i in range(order + 1):
            total = total + a[i] * b[order - i]
    return total


@pytest.mark.parametrize("Dk,Dv", SIZES)
def test_a_lost_part_is_seen(Dk, Dv):
    # the products of a chunk as above, on the CPU: with three parts within the bound, with two beyond it
    n = min(Dk, Dv, 100)
    g = torch.Generator().manual_seed(Dk + Dv)
    q, k, v = values(g, n), values(g, n), values(g, n, Dv)
    want = q.double()[:, None] * k.double()[:, None] * v.double()
    for parts, seen in ((3, False), (2, True)):
        p = product(product(q, k, parts)[:, None], v, parts)
        worst = ((p.double() - want).abs() / want.abs()).max().item() / U
        assert (worst > LIMIT) == seen, (parts, worst)
        # a score to 24 bits, and its product with two parts alone; and the other way round
        for other in (product(product(q, k, 3)[:, None], v, parts), product(product(q, k, parts)[:, None], v, 3)):
            worst = ((other.double() - want).abs() / want.abs()).max().item() / U
            assert (worst > LIMIT) == seen, (parts, worst)


def test_what_three_parts_leave_out():
    # the value whose parts shrink least: the products that are not formed are nearly a rounding, not half of one
    x = 1 + 2.0 ** -8 - 2.0 ** -17
    parts, v = [], np.float64(x)
    for _ in range(3):
        parts.append(float(bf16(torch.tensor(v, dtype=torch.float32))))
        v -= parts[-1]
    assert parts == [1.0, 2.0 ** -8, -2.0 ** -17] and v == 0
    left = sum(parts[i] * parts[j] for i in range(3) for j in range(3) if i + j > 2)
    assert 0.98 * U < abs(left) / x ** 2 <= U
