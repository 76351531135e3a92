"""Linear attention whose states grow, over sequences short enough that e^(seqlen log_decay) is a
float: the powers of a chunk's steps that a sequence does not have are in no result."""
import pytest
import torch

from gpu_util import log
from test_gpu_linear_attn import both, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (24, 40), (200, 256)])
@pytest.mark.parametrize("L,log_decay,seqlens", [(1, 30.0, None), (3, 6.0, None), (17, 4.0, None), (33, 2.2, None),
                                                 (40, 1.75, [40, 2]), (65, 1.2, [1, 65])])
def test_growth_over_short_sequences(dtype, Dk, Dv, L, log_decay, seqlens):
    log("linear attention growth %s" % ((dtype, Dk, Dv, L, log_decay, seqlens),))
    d = inputs(len(seqlens or [0]), L, 2, 1, Dk, Dv, dtype, seed=L + Dk)
    d["decay"] = torch.tensor([log_decay, -0.1], device="cuda")
    both(d, dtype, seqlens)
