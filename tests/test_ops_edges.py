"""The operators' edges on the host: limits, and values that lose their meaning in 32 bits."""
import pytest

from persistent_megakernel_decode_cta_b200 import abi, build
from tests.test_ops_refusals import P, linear

UNSUPPORTED = abi.ERR["AMK_ERR_UNSUPPORTED"]
MAX_SIDE = 2**31 - 4096


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("side", [MAX_SIDE + 1, 2**31 - 32, 2**31 - 1])
@pytest.mark.parametrize("fmt", [dict(), dict(quant=1, w_scale=P), dict(quant=2, w_scale=P)])
def test_linear_refuses_sides_that_its_kernels_cannot_count(side, fmt):
    for kw in (dict(k=side, ldx=2**31), dict(n=side, ldy=2**31)):
        for m in (1, 17, 4):
            assert linear(m=m, **kw, **fmt) == UNSUPPORTED
            assert "amk_linear" in abi.lib().amk_last_error().decode()
