"""The launches of the calls of experts and adapters at their smallest and largest sizes stay within a grid's limits, or
the call is refused (tests/sanitize/route_launch_checks.cpp: the library against HIP calls that launch nothing)."""

import os
import subprocess

import pytest

from tests.test_launch_limits import CLANG, MAX, PKG, ROOT

pytestmark = pytest.mark.skipif(not os.path.exists(CLANG) or not os.path.exists(os.path.join(PKG, "libdg.so")),
                                reason="needs the ROCm toolchain and the built library")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("launch") / "route_launch_checks")
    res = subprocess.run([CLANG, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-rdynamic",
                          os.path.join(ROOT, "tests", "sanitize", "route_launch_checks.cpp"), "-L" + PKG, "-l:libdg.so", "-Wl,-rpath," + PKG,
                          "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return exe


def launches(exe, *args):
    """[(workgroups, threads)] and the status; fails if a launch passes a limit."""
    res = subprocess.run([exe] + [str(a) for a in args], capture_output=True, text=True, timeout=120)
    lines = res.stdout.split("\n")
    status = int([x for x in lines if x.startswith("status")][0].split()[1])
    got = [tuple(int(v) for v in x.split()) for x in lines if x and not x.startswith("status")]
    assert res.returncode == 0, (args, got, status)
    return got, status


@pytest.mark.parametrize("tokens,k,groups,align", [(1, 1, 1, 1), (4096, 1, 1024, 1), (4097, 1, 1024, 256), (MAX // 8, 8, 64, 1), (MAX, 1, 1024, 1), (1, MAX, 3, 1)])
def test_sort(program, tokens, k, groups, align):
    got, status = launches(program, "sort", tokens, k, groups, align)
    assert status == 0 and len(got) == (1 if tokens * k <= 4096 else 2) and max(g[0] for g in got) <= 256


@pytest.mark.parametrize("g", [64, 128, 256])
@pytest.mark.parametrize("tokens,k,cols,rows", [(1, 1, 256, 1), (1, 1, 1 << 23, 16), (MAX, 1, 256, MAX), (MAX // 8, 8, 7168, MAX), (MAX // 8, 8, 256, MAX),
                                                (200000, 80, 65536, MAX), (64, 1, 1 << 23, MAX), (MAX, 1, 65536, MAX), (1, 1, 256, MAX)])
def test_rows(program, tokens, k, cols, rows, g):
    for kind in (0, 1, 2):
        for block_rows in (1, g):
            got, status = launches(program, "rows", tokens, k, cols, g, block_rows, kind, rows)
            assert status == 0 or (status == -1 and not got), (status, got)
            if rows * cols <= 1 << 36:
                assert status == 0


@pytest.mark.parametrize("tokens,k,cols", [(1, 1, 8), (MAX, 1, 8), (MAX // 8, 8, 7168), (1, 8, MAX), (MAX // 8, 8, 65536)])
def test_combine_and_weights(program, tokens, k, cols):
    for kind in (0, 1, 2):
        assert launches(program, "combine", tokens, k, cols, kind)[1] == 0
        assert launches(program, "weights", tokens, k, cols, kind)[1] == 0


@pytest.mark.parametrize("rows,groups,N,K,g", [(1, 1, 1, 128, 128), (1, 1024, 1, 64, 64), (MAX, 1024, 16, 128, 128), (MAX, 1, 4096, 1024, 64), (MAX, 1024, MAX, 128, 128),
                                               (16, 1024, MAX, 256, 256), (MAX, 64, 8192, 2048, 128), (4096, 1024, 65536, 128, 128)])
def test_grouped(program, rows, groups, N, K, g):
    for layout in (0, 1):
        for sa_rows in (1, g):
            got, status = launches(program, "grouped", rows, groups, N, K, g, layout, sa_rows)
            assert (status == 0 and len(got) == 1) or (status == -1 and not got and rows * N > 1 << 36), (status, got)


@pytest.mark.parametrize("rows,groups,M,N,g", [(128, 1, 128, 128, 128), (MAX // 64 * 64, 1024, 4096, 4096, 64), (256, 1024, 65536, 65536, 256), (256, 1, 1 << 22, 256, 256),
                                               (512, 1024, 256, 256, 256), (8192, 64, 8192, 2048, 128)])
def test_wgrad(program, rows, groups, M, N, g):
    got, status = launches(program, "wgrad", rows, groups, M, N, g)
    assert (status == 0 and len(got) == 1) or (status == -1 and not got and groups * M * N > 1 << 36), (status, got)


@pytest.mark.parametrize("tokens,groups,N,K,rank", [(1, 1, 1, 8, 8), (1, 1024, 4096, 4096, 16), (MAX, 1024, 64, 64, 8), (MAX, 1, 4096, 4096, 128), (64, 128, MAX, 64, 64),
                                                    (MAX, 1024, 65536, 64, 16), (3, 1, 17, 1 << 23, 16)])
def test_lora(program, tokens, groups, N, K, rank):
    for kind in (0, 1, 2):
        got, status = launches(program, "lora", tokens, groups, N, K, rank, kind)
        assert (status == 0 and got) or (status == -1 and not got and tokens * N > 1 << 34), (status, got)
