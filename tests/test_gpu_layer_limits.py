"""The operators around the chunked scan at the edges of what a call may be: rows and
batches as far apart as allowed, calls from two threads on streams of their own, and
two captured graphs replayed in turn."""
import threading

import pytest
import torch

import ssd_chunked_scan_chunk_amd as ssd
from gpu_util import log
from test_gpu_channel_scan import DT, inputs, upstream

pytestmark = pytest.mark.gpu


def everything(d, dy, dh, x, weight, bias, dyc):
    """Forward and backward of both operators, as one list of tensors."""
    y, h = ssd.channel_scan_fwd(**d, softplus=True, return_final_state=True)
    g = ssd.channel_scan_bwd(**d, dy=dy, dfinal_state=dh, softplus=True, return_dinitial_state=True)
    yc, win = ssd.short_conv_fwd(x, weight, bias, return_final_window=True)
    gc = ssd.short_conv_bwd(x, weight, dyc, bias, return_dinitial_window=True)
    return [y, h, yc, win, *g.values(), *gc.values()]


def call(Bz, L, D, N, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    d = inputs(Bz, L, D, N, 1, dtype, seed)
    weight, bias = torch.randn(D, 4, generator=gen).cuda(), torch.randn(D, generator=gen).cuda()
    return (d, *upstream(d, dtype, seed), d["u"].contiguous(), weight, bias,
            torch.randn(Bz, L, D, generator=gen).to(DT[dtype]).cuda())


def spread(t, rows, batches, at, buf):
    """t's values in ``buf`` from element ``at`` on, that many elements between rows and batches."""
    far = torch.as_strided(buf, t.shape, (batches, rows) + tuple(torch.empty(t.shape[2:], device="meta").stride()), at)
    far.copy_(t)
    return far


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,rows,batches", [(19, 1 << 24, 19 << 24),             # the largest step stride
                                            (70, 400, (1 << 31) + 64)])          # offsets past 2^31 elements
def test_far_rows_and_batches(dtype, L, rows, batches):
    log("layer far rows and batches %s" % ((dtype, L, rows, batches),))
    if torch.cuda.get_device_properties(0).total_memory < (64 << 30):
        pytest.skip("needs 12 GiB of device memory")
    args = call(2, L, 72, 12, dtype, 3)
    want = everything(*args)
    d = dict(args[0])
    buf = torch.empty(batches + (L - 1) * rows + 400, dtype=DT[dtype], device="cuda")
    for k, at in (("u", 0), ("delta", 72), ("gate", 144), ("B", 216), ("C", 228)):
        d[k] = spread(d[k], rows, batches, at, buf)
    x = spread(args[3], rows, batches, 241, buf)
    got = everything(d, args[1], args[2], x, *args[4:])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads():
    log("layer two threads")
    calls = [call(2, 300, 80, 16, "bf16", 1), call(3, 270, 96, 24, "f32", 2)]
    want = [everything(*a) for a in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(10):
                    got = everything(*calls[i])
                    stream.synchronize()
                    wrong.extend((i, k) for k, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
        except Exception as e:   # reported by the thread that started this one
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong[:4]


def test_two_graphs_in_turn():
    log("layer two graphs")
    calls = [call(2, 300, 80, 16, "bf16", 1), call(3, 270, 96, 24, "f32", 2)]
    want = [everything(*a) for a in calls]
    torch.cuda.synchronize()
    graphs, held = [], []
    for a in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(everything(*a))
        graphs.append(g)
    for _ in range(3):
        for t in held[0] + held[1]:
            t.fill_(7)
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        again = everything(*calls[1])
        torch.cuda.synchronize()
        for got, ref in ((held[0], want[0]), (held[1], want[1]), (again, want[1])):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
