"""The package without its compiled tensor binding (missing, or built for
another torch): it imports with a warning, and every call runs through the
Python checks alone, with the same refusals and the same bits."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "fp8_block_scaled_scales_amd"

PROGRAM = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import fp8_block_scaled_scales_amd as dg
assert any("_binding.so" in str(w.message) for w in seen), [str(w.message) for w in seen]
import torch
assert dg.dg_version() == 220 and dg.dg_query_tile(64, 64, 128)["bm"] > 0
x, w, s = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256), torch.zeros(1, 2)
a = torch.zeros(4, 256, dtype=torch.uint8)
for call, message in [(lambda: dg.dg_rmsnorm_quantize_fp8(x, x, w[:128]), "weight has shape"),
                      (lambda: dg.dg_rmsnorm_backward(x, x, torch.ones(5), w), "rstd has shape"),
                      (lambda: dg.dg_epilogue_backward_fp8(x, None, 2), "pre goes with"),
                      (lambda: dg.dg_gemm_fp8_residual(a, a, s, s, act=9), "act must"),
                      (lambda: dg.dg_gemm_fp8_nt(a, a, s, s), "GPU")]:
    try:
        call()
    except ValueError as e:
        assert message in str(e), e
    else:
        raise AssertionError(message)
print("imported")
"""


@pytest.mark.parametrize("binding", [None, b"", b"not a library"])
def test_import(tmp_path, binding):
    pkg = tmp_path / PKG
    pkg.mkdir()
    (pkg / "__init__.py").write_text(open(os.path.join(ROOT, PKG, "__init__.py")).read())
    os.symlink(os.path.join(ROOT, PKG, "libdg.so"), pkg / "libdg.so")
    if binding is not None:
        (pkg / "_binding.so").write_bytes(binding)
    res = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "imported" in res.stdout, res.stdout + res.stderr


@pytest.mark.gpu
def test_same_bits(monkeypatch):
    import torch

    import fp8_block_scaled_scales_amd as dg
    from tests._gpu import say
    from tests.test_gpu_layer import OUTPUTS, _buffers, _layer

    assert dg._binding.__name__.endswith("_binding")  # the compiled one
    t = _buffers(dg, 200, 512, 640, 31)
    say("a layer through the compiled binding, then without it")
    _layer(dg, t)
    torch.cuda.synchronize()
    want = {k: t[k].clone() for k in OUTPUTS}
    monkeypatch.setattr(dg, "_binding", dg._NoBinding)
    for k in OUTPUTS:
        t[k].zero_()
    _layer(dg, t)
    torch.cuda.synchronize()
    for k in OUTPUTS:
        assert torch.equal(t[k].view(torch.uint8), want[k].view(torch.uint8)), k
