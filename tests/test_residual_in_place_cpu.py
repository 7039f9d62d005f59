"""A residual in the place of the output has the output's row stride: with another one some rows would be read after
others were written over them.  Refused before any HIP call."""
import pytest

import vocabulary_cross_entropy_row_amd as lce

A, B, C, D, OUT, WS = (0x100000 * (i + 1) for i in range(6))   # never dereferenced


def linear(n, ldr, ldo):
    return lce.lib().lce_linear(A, 64, B, 64, lce.LCE_BF16, None, None, None, lce.LCE_F32, 0, OUT, ldr, n, 64, 40, OUT, ldo,
                                lce.LCE_BF16, None, 40, WS, 1 << 30, None)


def linear_blocks(n, ldr, ldo):
    return lce.lib().lce_linear_blocks(A, 64, C, 1, n, lce.LCE_E8M0, B, 64, D, 1, 1, lce.LCE_E8M0, None, lce.LCE_F32, 0, OUT, ldr,
                                       n, 64, 40, OUT, ldo, None, 40, WS, 1 << 30, None)


def linear_blocks_forward(n, ldr, ldo):
    return lce.lib().lce_linear_blocks_forward(A, 64, B, 64, None, lce.LCE_F32, OUT, ldr, n, 64, 40, OUT, ldo, None, 0, None, None, 0,
                                               None, WS, 1 << 30, None)


@pytest.mark.parametrize("call", [linear, linear_blocks, linear_blocks_forward])
@pytest.mark.parametrize("ldr,ldo", [(40, 48), (80, 40)])
def test_another_row_stride_is_refused(call, ldr, ldo):
    assert call(5, ldr, ldo) == lce.LCE_ERR_INVALID_ARG
    assert "residual in the place of out must have its row stride" in lce.lce_last_error()
