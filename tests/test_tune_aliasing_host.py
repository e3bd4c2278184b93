"""Balance gradient in place: the given gradient and the result are one matrix, not two that share their first element (rows
would be overwritten before they are read)."""
import pytest

import nvfp4_bit_block_quantize_amd as nv
from tests.test_tune_ops_host import BBWD, P, _call


@pytest.mark.parametrize("ld_in,ldd", [(64, 72), (80, 64)])
def test_in_place_with_two_leading_dimensions(ld_in, ldd):
    assert _call("nvfp4_moe_balance_backward", BBWD, dlogits_in=P, ld_in=ld_in, dlogits=P, ldd=ldd) == nv.NVFP4_ERR_SHAPE
