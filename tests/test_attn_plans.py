"""The plans of linear attention and the layouts of the group norm, on the CPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

import attn_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ssd_chunked_scan_chunk_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "probe.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, os.path.join(ROOT, "tests", "attn_plan_probe.cpp"),
                    os.path.join(CSRC, "shapes.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def plan(name, n, *sizes):
        out = (ctypes.c_int64 * n)()
        getattr(lib, name)(*map(ctypes.c_int64, sizes), out)
        return tuple(out)

    return plan


@pytest.mark.parametrize("Bz,L,H,K,Dk,Dv,dtype,bwd,want", cases.PLANS)
def test_attention(probe, Bz, L, H, K, Dk, Dv, dtype, bwd, want):
    assert probe("probe_attn", 4, Bz, L, H, K, Dk, Dv, dtype == "bf16", bwd)[:3] == want


@pytest.mark.parametrize("bf16", [0, 1])
@pytest.mark.parametrize("bwd", [0, 1])
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (64, 64), (64, 128), (128, 64), (128, 128), (129, 65), (256, 256)])
def test_attention_covers(probe, bf16, bwd, Dk, Dv):
    # every plan holds all steps, in segments of whole chunks, its launches and its workspace
    for Bz, L, H, K in ((0, 9, 2, 1), (1, 0, 1, 1), (1, 1, 1, 1), (1, 64, 12, 6), (2, 65, 40, 40), (8, 2048, 40, 40),
                        (1, 32768, 12, 12), (1, 1 << 20, 1, 1), (3, 1 << 30, 64, 8), (128, 4096, 64, 64),
                        (700, 3, 40, 20), (65535, 300, 20, 20)):
        whole, steps, nseg, size = probe("probe_attn", 4, Bz, L, H, K, Dk, Dv, bf16, bwd)
        pairs, case = Bz * H, (Bz, L, H, K)
        assert 0 <= whole <= pairs and nseg >= 1 and steps % 64 == 0, case
        assert steps * nseg >= L and (nseg == 1 or steps * (nseg - 1) < L), case
        assert nseg > 1 or whole == pairs, case
        slices = max(-(-d // (128 if d > 64 else 64)) for d in (Dk, Dv))
        assert (whole + (pairs - whole) * nseg) * slices * (3 if bwd else 1) * 512 < 2 ** 32, case
        assert nseg == 1 or (pairs - whole) * 256 * 256 < 2 ** 32, case
        states = (pairs - whole) * (nseg - 1) * Dk * Dv * 4 * (2 if bwd else 1)
        shared = Bz * L * H * (Dk + Dv) * 4 if bwd and K != H else 0
        assert states + shared <= size <= states + shared + 4 * 256, case


@pytest.mark.parametrize("bf16", [0, 1])
@pytest.mark.parametrize("bwd", [0, 1])
def test_norm(probe, bf16, bwd):
    full = 8 if bf16 else 4
    for m in list(range(1, 140)) + [255, 256, 257, 511, 512, 513, 2047, 2049, 4096, 5120, 8191, 8193, 16384]:
        for G in (1, 2, 3, 7, 40, 4096):
            for Bz, L in ((1, 1), (2, 3), (4, 2048), (1, 100000)):
                vec, pieces, lanes, gw, rw, threads, block, across, down, parts = \
                    probe("probe_norm", 10, Bz, L, m * G, G, bf16, bwd)
                case = (m, G, Bz, L)
                assert vec in (1, full) and vec <= m and pieces in (1, 2, 4), case
                assert threads % 64 == 0 and 64 <= threads <= 1024, case
                # a group's lanes hold it, a workgroup its groups and rows, the grid all groups
                assert (threads if block else lanes) * pieces * vec >= m, case
                assert block or (lanes <= 64 and gw * rw * lanes <= threads), case
                assert gw * across >= G > gw * (across - 1), case
                assert 1 <= down <= 32768 and (down - 1) * rw < Bz * L, case
                assert across * down * threads < 2 ** 32 and (not bwd or parts == down), case
