"""The operators' edges on the host: limits, and values that lose their meaning in 32 bits."""
import math

import pytest
import torch

import persistent_megakernel_decode_cta_b200 as amk
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


@pytest.mark.parametrize("scale", [0.0, -0.0, -1.0, 1e-50, 2.0**-150, 3.5e38, 1e39, math.inf, math.nan])
def test_a_scale_that_32_bits_do_not_hold_is_refused(scale):
    """(2^-150 and less would become 0, which stands for the default.)"""
    q = torch.zeros(1, 2, 8, dtype=torch.bfloat16)
    with pytest.raises(amk.AmkError, match="scale"):
        amk.attention(q, q, q, 0, scale=scale)


@pytest.mark.parametrize("temperature", [1e-50, 1e-7, 9.9e-7, -1.0, 1.1e6, 1e39, math.inf, math.nan])
def test_a_temperature_outside_its_range_is_refused(temperature):
    """(1e-50 would become 0, which is greedy.)"""
    t = torch.zeros(1, 4)
    with pytest.raises(amk.AmkError, match="temperature"):
        amk.verify_draft(t, torch.zeros(0, dtype=torch.int32), torch.zeros(1), temperature=temperature)


def test_values_within_their_ranges_get_to_the_next_check():
    q, t = torch.zeros(1, 2, 8, dtype=torch.bfloat16), torch.zeros(1, 4)
    for scale in (None, 1, 0.125, 2.0**-149, 2.0**128 - 2.0**104):
        with pytest.raises(amk.AmkError, match="CUDA"):
            amk.attention(q, q, q, 0, scale=scale)
    for temperature in (0, 0.0, 1e-6, 1, 1e6):
        with pytest.raises(amk.AmkError, match="CUDA"):
            amk.verify_draft(t, torch.zeros(0, dtype=torch.int32), torch.zeros(1),
                             temperature=temperature)
