"""Rows without variance: where a group's sum is exact in fp32, its mean is, and n is 0."""
import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,groups", [(3, 4), (7, 1), (7, 5), (15, 2), (41, 3), (100, 1), (771, 3), (1001, 1), (5120, 1),
                                      (9001, 1), (16383, 1)])
def test_constant_rows_of_any_size(dtype, m, groups):
    # at most 8 bits times m below 2^14: every partial sum is exact, and so is the quotient by m
    log("group norm constant rows %s %d %d" % (dtype, m, groups))
    values = (1.0, -3.0, 1000.0, 30080.0, 0.16015625, 1.2e-3, -6.25e4)
    x = torch.tensor(values, device="cuda").to(torch.bfloat16).to(DT[dtype])[None, :, None].expand(1, -1, m * groups)
    x = x.contiguous()
    g = torch.Generator().manual_seed(m)
    bias = torch.randn(m * groups, generator=g).cuda()
    weight = torch.randn(m * groups, generator=g).cuda()
    dy = torch.ones_like(x)
    for eps in (1e-5, 1e-30):
        kw = dict(weight=weight, bias=bias, eps=eps, silu=False)
        y = ssd.group_norm_fwd(x, groups, **kw)
        got = ssd.group_norm_bwd(x, groups, dy, **kw)
        # a gradient that is constant over the group has no part besides its mean: dx is 0
        flat = ssd.group_norm_bwd(x, groups, dy, eps=eps, silu=False)
        torch.cuda.synchronize()
        assert torch.equal(y, bias.to(DT[dtype]).expand_as(y)), eps
        assert not got["dweight"].any() and not flat["dx"].any(), eps
