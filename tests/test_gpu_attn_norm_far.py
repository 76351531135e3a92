"""Linear attention and group norm on rows and batches far apart in memory: the kernels that copy
whole pieces straight to LDS (steps of up to 2^22 elements, a multiple of 8 apart), those beside
them, and the norm's rows and batches more than 2^32 bytes apart."""
import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log
from test_gpu_group_norm import calls as norm_calls, inputs as norm_inputs
from test_gpu_linear_attn import calls, inputs

pytestmark = pytest.mark.gpu


def room():
    if torch.cuda.get_device_properties(0).total_memory < (64 << 30):
        pytest.skip("needs 32 GiB of device memory")


@pytest.mark.parametrize("rows", [(1 << 22) - 8, 1 << 22, (1 << 22) + 8])
@pytest.mark.parametrize("Dk,Dv", [(128, 128), (64, 64), (256, 256), (64, 128)])
def test_attention(Dk, Dv, rows):
    # aligned bf16 rows, two chunks and a part of one; q, k and v in the same far rows, batches 2^33
    # bytes apart
    log("linear attention far rows %s" % ((Dk, Dv, rows),))
    room()
    L, H, K = 150, 2, 1
    d = inputs(2, L, H, K, Dk, Dv, "bf16", seed=Dk)
    want = calls(d)
    batch = 1 << 32
    buf = torch.empty(batch + rows * (L - 1) + 2 * 256 + 256 + 256, dtype=torch.bfloat16, device="cuda")
    at = 0
    for n in ("q", "k", "v"):
        t = d[n]
        d[n] = buf.as_strided(t.shape, (batch, rows, t.shape[3], 1), at).copy_(t)
        at += t.shape[2] * t.shape[3]
    got = calls(d)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C,groups", [(96, 3), (2056, 1), (6, 3)])
@pytest.mark.parametrize("seqlens", [None, [3, 2]])
@pytest.mark.parametrize("flat", [False, True])
def test_norm(dtype, C, groups, seqlens, flat):
    # rows more than 2^32 bytes apart, the batches either as far as the rows would go on or elsewhere
    log("group norm far rows %s" % ((dtype, C, groups, seqlens, flat),))
    room()
    d = norm_inputs(2, 3, C, dtype, seed=C)
    want = norm_calls(d, groups, seqlens)
    size = d["x"].element_size()
    rows = (1 << 32) // size + 8
    batch = 3 * rows if flat else 3 * rows + 4112
    buf = torch.empty(batch + 2 * rows + 2 * C, dtype=d["x"].dtype, device="cuda")
    for n, at in (("x", 0), ("gate", C)):
        d[n] = buf.as_strided(d[n].shape, (batch, rows, 1), at).copy_(d[n])
    got = norm_calls(d, groups, seqlens)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens(dtype):
    # a token's requests more than 2^32 bytes apart
    log("tokens far apart %s" % dtype)
    room()
    d = inputs(3, 1, 4, 2, 64, 40, dtype, seed=5)
    tokens = {n: d[n][:, 0] for n in ("q", "k", "v")}
    states = d["first"].clone(), d["first"].clone()
    want = ssd.linear_attn_step(states[0], tokens["q"], tokens["k"], tokens["v"], d["decay"])
    norm = ssd.group_norm_fwd(tokens["q"].flatten(1), 4, gate=tokens["q"].flatten(1))
    batch = (1 << 32) // d["q"].element_size() + 8
    buf = torch.empty(2 * batch + 1024, dtype=d["q"].dtype, device="cuda")
    at = 0
    for n, t in tokens.items():
        tokens[n] = buf.as_strided(t.shape, (batch, t.shape[2], 1), at).copy_(t)
        at += t.shape[1] * t.shape[2]
    got = ssd.linear_attn_step(states[1], tokens["q"], tokens["k"], tokens["v"], d["decay"])
    flat = tokens["q"].as_strided((3, 256), (batch, 1))
    normed = ssd.group_norm_fwd(flat, 4, gate=flat)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(*states) and torch.equal(normed, norm)
