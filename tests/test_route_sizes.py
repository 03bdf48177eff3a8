"""Sizes past a C integer are refused, not cut to what is left of them in one."""

import pytest
import torch

WRAP, WRAP64 = 1 << 32, 1 << 64


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


@pytest.mark.parametrize("name,good", [
    ("dg_route_rows", (100, 2, 8, 16)), ("dg_route_sort_workspace", (5000, 2, 8)), ("dg_lora_workspace", (100, 256, 96, 16, 3)),
    ("dg_route_quantize_workspace", (100, 256, 2, 512, 128, 128))])
def test_queries(dg, name, good):
    call = getattr(dg, name)
    assert call(*good) >= 0
    for i in range(len(good)):
        for more in (WRAP, -WRAP, WRAP64, -WRAP64):
            args = list(good)
            args[i] += more
            with pytest.raises(dg.DGArgumentError, match="invalid argument"):
                call(*args)


def test_calls(dg):
    """Tensors without memory stand for those that are as long."""
    def of(*shape, dtype=torch.int32):
        return torch.empty(*shape, dtype=dtype, device="meta")

    ids = of(4, 2)
    x, y = of(1, 256, dtype=torch.bfloat16), of(64, 256, dtype=torch.bfloat16)
    k = WRAP + 2
    for fn in (lambda: dg.dg_route_sort(ids, 3, WRAP + 1), lambda: dg.dg_route_sort(ids, WRAP + 3), lambda: dg.dg_route_sort(ids, 3 - WRAP),
               lambda: dg.dg_route_sort(of(1, k), 3), lambda: dg.dg_route_quantize_fp8(x, of(1, k), of(64)), lambda: dg.dg_route_combine(y, of(1, k)),
               lambda: dg.dg_route_weight_grad(x, y, of(1, k)),
               lambda: dg.dg_lora(x, of(3, WRAP + 8, 256, dtype=x.dtype), of(3, 64, WRAP + 8, dtype=x.dtype), of(4), of(1, 1), of(1))):
        with pytest.raises(dg.DGArgumentError, match="invalid argument"):
            fn()
    for fn in (lambda: dg.dg_route_sort(ids, 3), lambda: dg.dg_route_quantize_fp8(x, of(1, 2), of(64)), lambda: dg.dg_route_combine(y, of(1, 2)),
               lambda: dg.dg_route_weight_grad(x, y, of(1, 2))):
        with pytest.raises(ValueError, match="GPU"):
            fn()
