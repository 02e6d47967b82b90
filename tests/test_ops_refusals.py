"""The operators' argument checks, on the host: every refused call returns its
status before any device work (the pointers are never followed), and without a
device a good call says so."""
import ctypes

import pytest

import persistent_megakernel_decode_cta_b200 as amk
from persistent_megakernel_decode_cta_b200 import abi, build

P = 1 << 20  # a pointer that only the checks look at
INVALID = abi.ERR["AMK_ERR_INVALID_ARG"]


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def linear(**kw):
    a = abi.LinearArgs(x=P, w=P, y=P, ldx=64, ldy=32, m=4, n=32, k=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return abi.lib().amk_linear(ctypes.byref(a), None)


def attention(**kw):
    a = abi.AttentionArgs(q=P, k=P, v=P, out=P, q_token_stride=128, q_head_stride=64,
                          out_token_stride=128, out_head_stride=64, k_head_stride=640,
                          k_row_stride=64, v_head_stride=640, v_row_stride=64, n_tokens=3,
                          pos=2, n_heads=2, n_kv_heads=1, head_dim=64, kv_rows=10)
    for k, v in kw.items():
        setattr(a, k, v)
    return abi.lib().amk_attention(ctypes.byref(a), None)


def verify(**kw):
    a = abi.VerifyArgs(target=P, draft=P, u=P, draft_tokens=P, tokens=P, n_accepted=P,
                       target_stride=100, draft_stride=100, n_draft=2, vocab=100,
                       temperature=1.0, workspace=P, workspace_bytes=1 << 20)
    for k, v in kw.items():
        setattr(a, k, v)
    return abi.lib().amk_verify_draft(ctypes.byref(a), None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(y=None), dict(m=-1), dict(n=0), dict(k=0), dict(quant=3),
    dict(quant=-1), dict(act=4), dict(act=-1), dict(y_type=2), dict(residual=P, ldr=31),
    dict(residual_type=5), dict(ldx=63), dict(ldy=31), dict(quant=1), dict(quant=2),
    dict(quant=2, w_scale=P, k=63, ldx=63), dict(quant=1, w_scale=P, up=P), dict(up_bias=P),
    dict(x=P + 1), dict(y=P + 1), dict(y_type=1, y=P + 2), dict(bias=P + 1),
    dict(residual=P + 2, ldr=32, residual_type=1)])
def test_linear_refuses(kw):
    assert linear(**kw) == INVALID
    assert "amk_linear" in abi.lib().amk_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(n_tokens=-1), INVALID), (dict(n_heads=0), INVALID),
    (dict(n_kv_heads=0), INVALID), (dict(n_heads=3, n_kv_heads=2), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=257), abi.ERR["AMK_ERR_UNSUPPORTED"]),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(pos=-1), abi.ERR["AMK_ERR_POS_RANGE"]), (dict(pos=8), abi.ERR["AMK_ERR_POS_RANGE"]),
    (dict(pos=2**31 - 1), abi.ERR["AMK_ERR_POS_RANGE"]),
    (dict(kv_rows=2**30 + 1), abi.ERR["AMK_ERR_UNSUPPORTED"]),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=P + 1), INVALID), (dict(out=P + 1), INVALID),
    (dict(out_head_stride=63), INVALID), (dict(out_token_stride=127), INVALID),
    (dict(out_token_stride=64, out_head_stride=191), INVALID), (dict(k_row_stride=-64), INVALID)])
def test_attention_refuses(kw, status):
    assert attention(**kw) == status
    assert "amk_attention" in abi.lib().amk_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(target=None), INVALID), (dict(u=None), INVALID), (dict(tokens=None), INVALID),
    (dict(n_accepted=None), INVALID), (dict(draft_tokens=None), INVALID),
    (dict(n_draft=-1), INVALID), (dict(n_draft=65), abi.ERR["AMK_ERR_UNSUPPORTED"]),
    (dict(vocab=0), INVALID), (dict(vocab=2**30 + 1), abi.ERR["AMK_ERR_UNSUPPORTED"]), (dict(temperature=-1.0), INVALID),
    (dict(temperature=1e-7), INVALID), (dict(temperature=float("nan")), INVALID),
    (dict(temperature=float("inf")), INVALID), (dict(target_stride=99), INVALID),
    (dict(draft_stride=99), INVALID), (dict(target=P + 2), INVALID), (dict(workspace=None), INVALID),
    (dict(workspace=P + 8), INVALID), (dict(workspace_bytes=100), INVALID)])
def test_verify_refuses(kw, status):
    assert verify(**kw) == status
    assert "amk_verify_draft" in abi.lib().amk_last_error().decode()


def test_verify_workspace_sizes():
    fn = abi.lib().amk_verify_workspace
    assert fn(-1, 10) < 0 and fn(65, 10) < 0 and fn(0, 0) < 0 and fn(0, 2**31 - 1) < 0
    assert 0 < fn(0, 1) <= fn(4, 1) <= fn(4, 128256) < 1 << 20
    assert verify(workspace_bytes=fn(2, 100) - 1) == INVALID


def test_null_arguments_and_empty_calls():
    lib = abi.lib()
    for fn in (lib.amk_linear, lib.amk_attention, lib.amk_verify_draft):
        assert fn(None, None) == INVALID
    assert linear(m=0) == abi.AMK_OK
    assert attention(n_tokens=0) == abi.AMK_OK


def test_extend_refuses():
    lib = abi.lib()
    assert lib.amk_extend(None, None, 0, 0, 0, None) == INVALID
    assert "amk_extend" in lib.amk_last_error().decode()
    assert lib.amk_ops_timeouts(None) == INVALID


def test_good_calls_without_a_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    none = abi.ERR["AMK_ERR_NO_DEVICE"]
    assert linear() == none and attention() == none and verify() == none


def test_python_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(amk.AmkError, match="not a CUDA tensor"):
        amk.linear(x, x)
    with pytest.raises(amk.AmkError, match="not a CUDA tensor"):
        amk.attention(x, x, x, 0)
    with pytest.raises(amk.AmkError, match="not a CUDA tensor"):
        amk.verify_draft(x, x, x)
