"""dg_epilogue_backward_workspace answers for exactly the sizes that dg_epilogue_backward_fp8 takes."""

import pytest

X, PRE, Q, S, DB, WS = ((i + 1) << 52 for i in range(6))  # fake device addresses, farther apart than the largest matrix


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_scales_amd as dg

    return dg


MOST = {64: (1 << 24) - 1, 128: (1 << 22) - 1, 256: (1 << 22) - 1}  # gran x gran blocks of one call


@pytest.mark.parametrize("g", [64, 128, 256])
def test_block_limit(dg, g):
    # rows x cols of exactly the limit's number of blocks does not exist for every g: one row of blocks short of and past it
    col_blocks = 1 << 12
    most_rows = MOST[g] // col_blocks * g
    for rows, cols, fits in [(most_rows, col_blocks * g, True), (most_rows + 1, col_blocks * g, False), (most_rows - 5, col_blocks * g, True)]:
        n = dg.lib.dg_epilogue_backward_workspace(rows, cols, g, g)
        assert (n >= 0) == fits, (rows, cols, n)
        # per-row factors have no such limit
        assert dg.lib.dg_epilogue_backward_workspace(rows, cols, g, 1) >= 0
        if not fits:
            assert n == dg.DG_EINVAL
            assert dg.lib.dg_epilogue_backward_fp8(X, 1, cols, PRE, cols, 2, rows, cols, g, g, 1, None, DB, Q, S, WS, 1 << 50,
                                                   None) == dg.DG_EINVAL
            with pytest.raises(ValueError):
                dg.dg_epilogue_backward_workspace(rows, cols, g)


def test_the_largest_sizes(dg):
    assert dg.lib.dg_epilogue_backward_workspace(dg.DG_MAX_DIM, 8192, 64, 64) == dg.DG_EINVAL
    assert dg.lib.dg_epilogue_backward_workspace(dg.DG_MAX_DIM, dg.DG_MAX_DIM, 256, 256) == dg.DG_EINVAL
    assert dg.lib.dg_epilogue_backward_workspace(dg.DG_MAX_DIM, 4096, 64, 64) > 0
