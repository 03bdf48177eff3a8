"""The division of the dispatch's 16-bit values by their block's factor: for every pair of mantissas on the CPU
(tests/sanitize/quotient_checks.cpp), and every BF16 and FP16 mantissa beside every largest one on the GPU against the
quantisers, to the bit, down to factors at the ends of FP32."""

import os
import subprocess

import pytest
import torch

from tests.test_launch_limits import CLANG, ROOT

DEV = "cuda:0"


@pytest.mark.skipif(not os.path.exists(CLANG), reason="needs the ROCm toolchain")
def test_every_pair_of_mantissas(tmp_path):
    exe = str(tmp_path / "quotient_checks")
    res = subprocess.run([CLANG, "-O2", "-std=c++17", "-ffp-contract=off", os.path.join(ROOT, "tests", "sanitize", "quotient_checks.cpp"),
                          "-lm", "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and " 0 wrong" in res.stdout, res.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("xk,bits,exponents", [(torch.bfloat16, 7, (0, -1, -70, -100, -118, -126, 90, 120)), (torch.float16, 10, (0, -9, 14))])
@pytest.mark.parametrize("fmt", [0, 1])
def test_every_mantissa_on_the_gpu(xk, bits, exponents, fmt):
    import fp8_block_scaled_scales_amd as dg
    from tests._gpu import say

    n = 1 << bits
    mant = 1 + torch.arange(n, dtype=torch.float64) / n
    for e in exponents:
        say("mantissas of %s, exponent %d, format %d" % (xk, e, fmt))
        # token i: segments of g = 128 (the first 64 the largest value's, the rest smaller ones and their negatives)
        g, per = 128, 64
        segs = n // per
        x = torch.empty(n, segs, g, dtype=torch.float64)
        x[:, :, :per] = mant.reshape(1, segs, per) * 2.0 ** -1
        x[:, :, per:] = -mant.reshape(1, segs, per) * 2.0 ** -(torch.arange(per) % 12 + 1)
        x[:, :, 0] = mant[:, None]
        x = (x.reshape(n, segs * g) * 2.0 ** e).to(xk)
        assert torch.isfinite(x).all()
        x = x.to(DEV)
        for k in (1, 2):
            ids = torch.arange(n * k, dtype=torch.int32, device=DEV).reshape(n, k) % 3
            off, pos, slot = dg.dg_route_sort(ids, 3, g)
            end = int(off[-1])
            v = x[slot[:end].clamp(min=0).long() // k].float()
            v[slot[:end] < 0] = 0.0
            for br, plain in ((1, dg.dg_quantize_fp8_rows), (g, dg.dg_quantize_fp8_blocks)):
                q, s = dg.dg_route_quantize_fp8(x, pos, slot, gran=g, block_rows=br, fmt=fmt)
                wq, ws = plain(v, gran=g, fmt=fmt)
                assert torch.equal(q[:end], wq) and torch.equal(s[: ws.shape[0]], ws), (e, k, br)
