"""The launches of the largest calls around the product stay within a grid's limits and cover every row
(tests/sanitize/launch_checks.cpp: the library against HIP calls that launch nothing, on the CPU)."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "fp8_block_scaled_scales_amd")
CLANG = "/opt/rocm/llvm/bin/clang++"
MAX = (1 << 24) - 256

pytestmark = pytest.mark.skipif(not os.path.exists(CLANG) or not os.path.exists(os.path.join(PKG, "libdg.so")),
                                reason="needs the ROCm toolchain and the built library")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("launch") / "launch_checks")
    res = subprocess.run([CLANG, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-rdynamic",
                          os.path.join(ROOT, "tests", "sanitize", "launch_checks.cpp"), "-L" + PKG, "-l:libdg.so", "-Wl,-rpath," + PKG,
                          "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return exe


def launches(exe, *args):
    """[(workgroups, threads, first row or -1)], status; fails if a launch passes a limit."""
    res = subprocess.run([exe] + [str(a) for a in args], capture_output=True, text=True, timeout=120)
    lines = res.stdout.split("\n")
    status = int([x for x in lines if x.startswith("status")][0].split()[1])
    got = [tuple(int(v) for v in x.split()) for x in lines if x and not x.startswith("status")]
    assert res.returncode == 0, (args, got, status)
    return got, status


@pytest.mark.parametrize("cols", [16448, 65536])
@pytest.mark.parametrize("rows", [5, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, (1 << 23) + 3, MAX])
def test_norm_backward_of_long_rows(program, rows, cols):
    got, status = launches(program, "norm_bwd", rows, cols)
    assert status == 0
    if rows > 65536:  # the launches of a row per workgroup of 1024 threads, each going on where the one before ended
        by_row = [(wgs, row0) for wgs, threads, row0 in got if row0 >= 0]
        at = 0
        for wgs, row0 in by_row:
            assert row0 == at
            at += wgs
        assert at == rows


@pytest.mark.parametrize("rows,cols", [(MAX, 64), (MAX, 512), (MAX, 16384), (1 << 22, 8192), (7, MAX)])
def test_norm_backward(program, rows, cols):
    assert launches(program, "norm_bwd", rows, cols)[1] == 0


@pytest.mark.parametrize("rows,cols", [(MAX, 64), (MAX, 1024), (MAX, 4096), (1 << 22, 8192), (MAX, 16384), (MAX, 65536), (3, MAX)])
def test_norm(program, rows, cols):
    got, status = launches(program, "norm", rows, cols)
    assert status == 0 and got[0][2] == 0
    per = -(-rows // sum(g[0] for g in got))  # rows per workgroup: 1, 2 or 4
    for before, after in zip(got, got[1:]):
        assert after[2] == before[2] + before[0] * per


@pytest.mark.parametrize("rows,cols,g,block_rows", [(MAX, 4096, 64, 64), (MAX, 4096, 128, 128), (MAX, 16384, 256, 256), (MAX, 4096, 64, 1),
                                                    (MAX, 65536, 256, 1), (1, MAX, 64, 64), (5, MAX, 64, 1), (1024, 1536, 128, 128)])
def test_epilogue_backward(program, rows, cols, g, block_rows):
    assert launches(program, "epi", rows, cols, g, block_rows)[1] == 0


@pytest.mark.parametrize("M,N,K", [(MAX, 16, 128), (16, MAX, 128), (MAX, 4096, 1024), (1, 1, MAX)])
def test_residual_product(program, M, N, K):
    assert launches(program, "gemm", M, N, K)[1] == 0
