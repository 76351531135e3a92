"""The plans of the operators around the chunked scan, on the CPU: the shapes of
layer_cases.py get the plans they are there for."""
import ctypes
import os
import shutil
import subprocess

import pytest

import layer_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ssd_chunked_scan_chunk_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "probe.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, os.path.join(ROOT, "tests", "plan_probe.cpp"),
                    os.path.join(CSRC, "shapes.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def plan(name, n, *sizes):
        out = (ctypes.c_int64 * n)()
        getattr(lib, name)(*map(ctypes.c_int64, sizes), out)
        return tuple(out)

    return plan


@pytest.mark.parametrize("Bz,L,D,N,G,want", cases.SCAN_FWD)
def test_scan_forward(probe, Bz, L, D, N, G, want):
    assert probe("probe_chan_fwd", 4, Bz, L, D, N, G) == want


@pytest.mark.parametrize("Bz,L,D,N,G,want", cases.SCAN_BWD)
def test_scan_backward(probe, Bz, L, D, N, G, want):
    assert probe("probe_chan_bwd", 3, Bz, L, D, N, G) == want


@pytest.mark.parametrize("N", range(1, 65))
def test_scan_backward_instance(probe, N):
    # the launcher takes its instance from the plan: one that exists, holds all states,
    # and writes (per batch, segment and tile, 256 threads) no more than its regions
    for Bz, L, D, G in ((1, 16, 5, 1), (2, 388, 20, 1), (3, 301, 770, 2), (770, 45, 20, 1), (4, 2048, 5120, 1)):
        cw, nr, states, ends, adjoints, sums = probe("probe_chan_bwd_regions", 6, Bz, L, D, N, G)
        assert (cw, nr) in ((64, 2), (64, 4), (32, 4), (32, 8)) and 256 // cw * nr >= N
        _, seg, nseg = probe("probe_chan_bwd", 3, Bz, L, D, N, G)
        tiles = G * -(-(D // G) // cw)
        per = Bz * nseg * tiles * 256 * nr * 4
        assert states >= per * seg // 8 and sums >= Bz * L * tiles * 2 * (256 // cw * nr) * 4
        assert ends >= (per if nseg > 1 else 0) and adjoints >= (per if nseg > 1 else 0)


@pytest.mark.parametrize("Bz,L,pieces,W,silu,want", cases.CONV)
def test_convolution(probe, Bz, L, pieces, W, silu, want):
    assert probe("probe_conv", 3, Bz, L, *(tuple(pieces) + (0, 0))[:3]) == want
