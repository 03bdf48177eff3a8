"""bench.py's HBM traffic figures belong to the kernels that run: the hash that tags them covers every device source
that the workload's kernel is compiled from, and a change in any of them makes the figure null."""

import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "fp8_block_scaled_scales_amd", "csrc")


def closure(names):
    """The files of csrc that these include, themselves among them (the host dispatch's own headers left out)."""
    seen, todo = set(), list(names)
    while todo:
        name = todo.pop()
        if name in seen:
            continue
        seen.add(name)
        if name != "dg_host.hip":
            with open(os.path.join(CSRC, name)) as f:
                todo += re.findall(r'#include "(\w+\.h)"', f.read())
    return seen


@pytest.mark.parametrize("name", sorted(bench.TRAFFIC))
def test_hash_covers_the_kernel(name, tmp_path, monkeypatch):
    want = closure(bench.KERNEL_SOURCES[name])
    kernel = "gemm_fp8_stream" if name.startswith("decode") else "gemm_fp8_nt_big"
    assert any("__global__" in open(os.path.join(CSRC, n)).read() and kernel in open(os.path.join(CSRC, n)).read() for n in want)
    # the same hash over a copy of the tree, and another after a change in any one of the sources
    copy = tmp_path / "fp8_block_scaled_scales_amd" / "csrc"
    copy.mkdir(parents=True)
    for n in os.listdir(CSRC):
        (copy / n).write_bytes(open(os.path.join(CSRC, n), "rb").read())
    here = bench.kernel_source_hash(name)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_source_hash(name) == here
    for n in sorted(want):
        old = (copy / n).read_bytes()
        (copy / n).write_bytes(old + b"\n")
        assert bench.kernel_source_hash(name) != here, n
        (copy / n).write_bytes(old)
    assert bench.kernel_source_hash(name) == here
