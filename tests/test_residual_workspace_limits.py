"""dg_gemm_fp8_residual_workspace refuses the sizes that dg_gemm_fp8_residual refuses."""

import pytest

A, B, SA, SB, OUT, RES = ((i + 1) << 52 for i in range(6))  # fake device addresses, farther apart than the largest matrix


@pytest.mark.parametrize("layout", range(4))
@pytest.mark.parametrize("g", [64, 128, 256])
def test_more_tiles_than_a_grid_holds(g, layout):
    import fp8_block_scaled_scales_amd as dg

    M = N = dg.DG_MAX_DIM  # 65535^2 tiles of 256 x 256
    assert dg.lib.dg_gemm_fp8_residual(A, B, SA, SB, OUT, M, N, g, g, layout, g, 0, 0, None, 2, RES, 1, N, None, None, 0,
                                       None) == dg.DG_EINVAL
    assert dg.lib.dg_gemm_fp8_residual_workspace(M, N, g, g, layout) == dg.DG_EINVAL
    with pytest.raises(ValueError):
        dg.dg_gemm_fp8_residual_workspace(M, N, g, g, layout)
    assert dg.lib.dg_gemm_fp8_residual_workspace(M, 4096, g, g, layout) == 0
