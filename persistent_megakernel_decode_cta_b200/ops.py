"""The operators of the multi-token step on torch CUDA tensors: argument checks
and marshalling for amk_linear, amk_attention and amk_verify_draft (see
include/amk.h for what they compute).

Each call enqueues on torch's current stream of the tensors' device, or on
``stream`` (a raw cudaStream_t handle), and returns at once.  Results that the
caller does not pass in are allocated by torch.  Inference only: a call that
would have to record a gradient is refused.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import AmkError, _check, abi

_I32 = 2**31 - 1
_F32_TINY, _F32_MAX = 2.0**-149, 2.0**128 - 2.0**104
_INVALID = abi.ERR["AMK_ERR_INVALID_ARG"]
_pack_linear = abi.packer(abi.LinearArgs)
_pack_attention = abi.packer(abi.AttentionArgs)
_pack_verify = abi.packer(abi.VerifyArgs)
_workspace = {}  # bytes by (drafts, vocab)
_torch = None
_lib = _raw_stream = _device = None


def _load():
    """Imports torch and loads the library, on the first call."""
    global _torch, _lib, _raw_stream, _device
    import torch
    _lib = abi.lib()
    # the current stream's handle and device without the objects around them
    # (which cost more than the launch), where this torch has them
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch


def _refuse(what: str):
    raise AmkError(_INVALID, what)


def _check_tensors(what: str, names, tensors) -> int:
    """The CUDA device that all of the tensors (or None) are on; refuses others
    and any that a gradient would have to be recorded for."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0):
            break
    else:
        if not _torch.is_grad_enabled():
            return dev
        for t in tensors:
            if t is not None and t.requires_grad:
                break
        else:
            return dev
    for name, t in zip(names, tensors):
        if t is None:
            continue
        if not t.is_cuda:
            _refuse(f"{what}: {name} is not a CUDA tensor")
        if t.get_device() != dev:
            _refuse(f"{what}: {name} is on cuda:{t.get_device()}, others on cuda:{dev}")
        if t.requires_grad:
            _refuse(f"{what}: {name} requires a gradient, which is not computed")
    _refuse(f"{what}: tensors are on no one CUDA device")


def _launch(what: str, fn, args: bytes, dev: int, stream, tensors):
    if stream is None:
        st = _raw_stream(dev)
    else:
        st = stream
        side = _torch.cuda.ExternalStream(stream, device=dev)
        for t in tensors:  # their memory is not reused before this stream is through
            if t is not None:
                t.record_stream(side)
    if dev == _device():
        rc = fn(args, st)
    else:
        with _torch.cuda.device(dev):
            rc = fn(args, st)
    if rc != abi.AMK_OK:
        _check(rc, what)


def _new(like, stream, shape, dtype):
    """A result on the device of `like`, from the pool of the stream that will
    write it."""
    if stream is None:
        return like.new_empty(shape) if like.dtype is dtype else like.new_empty(shape, dtype=dtype)
    side = _torch.cuda.ExternalStream(stream, device=like.device)
    with _torch.cuda.stream(side):
        return like.new_empty(shape, dtype=dtype)


def _rows(what: str, name: str, t, n: int):
    """(rows, row stride) of a tensor seen as [rows][n]."""
    if t.dim() == 2:
        ld, one = t.stride()
        if one == 1 or n == 1:
            rows = t.shape[0]
            if rows <= 1:
                return rows, n
            if ld < n:
                _refuse(f"{what}: the rows of {name} overlap")
            return rows, ld
    if t.is_contiguous():
        return (t.numel() // n if n else 0), n
    _refuse(f"{what}: {name} is neither contiguous nor a matrix of contiguous rows")


_LINEAR = ("x", "w", "scale", "bias", "up", "up_scale", "up_bias", "residual", "out")


def linear(x, w, *, scale=None, bias=None, act: str = "none", up=None, up_scale=None,
           up_bias=None, residual=None, out=None, out_dtype=None, stream=None):
    """``act(x @ w.T + bias)``, times ``x @ up.T + up_bias`` when ``up`` is given,
    plus ``residual`` (amk_linear).

    x: bf16 [..., k] (rows may be strided, the inputs of a row are contiguous).
    w, up: bf16 [n, k]; or int8 [n, k] with scale fp16 [n]; or packed int4,
    uint8 [n, k / 2] with scale fp16 [n, ceil(k / 128)] -- contiguous, both of
    one format.  Biases: bf16 [n].  act: "none", "silu", "gelu" or "relu".
    residual: bf16 or fp32 [..., n].  Returns bf16 or fp32 [..., n]: ``out``
    (which may be ``residual`` itself, and overlaps no input otherwise), else a
    new tensor of ``out_dtype`` (default: bf16)."""
    if _torch is None:
        _load()
    torch = _torch
    dev = _check_tensors("linear", _LINEAR, (x, w, scale, bias, up, up_scale, up_bias, residual,
                                             out))
    bf16, f32 = torch.bfloat16, torch.float32
    if x.dtype is not bf16:
        _refuse(f"linear: x is {x.dtype}, not bfloat16")
    if x.dim() < 1 or w.dim() != 2:
        _refuse("linear: x needs one dimension at least and w two")
    act_code = abi.ACT.get(act)
    if act_code is None:
        _refuse(f"linear: unknown activation {act!r}")
    xs = x.shape
    k = xs[-1]
    n = w.shape[0]
    wt = w.dtype
    if wt is bf16:
        quant, cols, sshape = 0, k, None
    elif wt is torch.int8:
        quant, cols, sshape = 1, k, (n,)
    elif wt is torch.uint8:
        if k % 2:
            _refuse("linear: int4 rows need an even number of inputs")
        quant, cols, sshape = 2, k // 2, (n, (k + 127) // 128)
    else:
        _refuse(f"linear: no weight format with {wt} elements")
    _check_weights("w", w, scale, wt, (n, cols), sshape)
    if up is not None:
        _check_weights("up", up, up_scale, wt, (n, cols), sshape)
    elif up_scale is not None or up_bias is not None:
        _refuse("linear: up_scale or up_bias without up")
    for b in (bias, up_bias):
        if b is not None and (b.dtype is not bf16 or b.shape != (n,) or not b.is_contiguous()):
            _refuse(f"linear: a bias is not contiguous bfloat16 [{n}]")
    m, ldx = _rows("linear", "x", x, k)
    shape = (m, n) if len(xs) == 2 else (*xs[:-1], n)
    if out is None:
        out = _new(x, stream, shape, out_dtype or bf16)
        ldy = n
    else:
        if out.shape != shape:
            _refuse(f"linear: out has shape {list(out.shape)}, not {list(shape)}")
        if out_dtype is not None and out.dtype is not out_dtype:
            _refuse(f"linear: out is {out.dtype}, not {out_dtype}")
        _, ldy = _rows("linear", "out", out, n)
    ot = out.dtype
    if ot is not bf16 and ot is not f32:
        _refuse(f"linear: out is {ot}, not bfloat16 or float32")
    ldr = rt = rp = 0
    if residual is not None:
        rd = residual.dtype
        if rd is not bf16 and rd is not f32:
            _refuse(f"linear: residual is {rd}, not bfloat16 or float32")
        if residual.shape != shape:
            _refuse(f"linear: residual has shape {list(residual.shape)}, not {list(shape)}")
        _, ldr = _rows("linear", "residual", residual, n)
        rt = 1 if rd is f32 else 0
        rp = residual.data_ptr()
    if m == 0:
        return out
    if m > _I32 or n > _I32 or k > _I32:
        _refuse("linear: a size above 2^31 - 1")
    args = _pack_linear(
        x.data_ptr(), w.data_ptr(), scale.data_ptr() if scale is not None else 0,
        bias.data_ptr() if bias is not None else 0, up.data_ptr() if up is not None else 0,
        up_scale.data_ptr() if up_scale is not None else 0,
        up_bias.data_ptr() if up_bias is not None else 0, rp, out.data_ptr(), ldx, ldr, ldy, m, n,
        k, quant, act_code, rt, 1 if ot is f32 else 0)
    _launch("amk_linear", _lib.amk_linear, args, dev, stream,
            (x, w, scale, bias, up, up_scale, up_bias, residual, out))
    return out


def _check_weights(name, m, s, dtype, shape, sshape):
    if m.dtype is not dtype or m.shape != shape or not m.is_contiguous():
        _refuse(f"linear: {name} is not a contiguous {dtype} {list(shape)} matrix")
    if sshape is None:
        if s is not None:
            _refuse(f"linear: bf16 {name} takes no scale")
    elif s is None or s.dtype is not _torch.float16 or s.shape != sshape or not s.is_contiguous():
        _refuse(f"linear: the scale of {name} is not contiguous float16 {list(sshape)}")


def attention(q, k, v, pos: int, *, window: int = 0, sinks: int = 0,
              scale: Optional[float] = None, out=None, stream=None):
    """Causal attention of the query tokens q (bf16 [tokens, heads, head_dim], at
    positions pos, pos + 1, ...) over the cache rows k and v (bf16 [kv_heads,
    rows, head_dim], row j = position j, as ``Decoder.kv`` returns them):
    amk_attention.  ``window`` > 0 limits a token to the last ``window`` rows
    up to its own, and to the first ``sinks`` rows.  scale: default
    1 / sqrt(head_dim).  Returns bf16 [tokens, heads, head_dim] (``out`` if
    given, which overlaps no input).  Leading dimensions may be strided; head_dim is contiguous."""
    if _torch is None:
        _load()
    if scale is None:
        scale = 0.0
    elif not _F32_TINY <= scale <= _F32_MAX:  # the call takes it in 32 bits, where 0 is the default
        _refuse("attention: scale must be positive and finite in 32 bits")
    dev = _check_tensors("attention", ("q", "k", "v", "out"), (q, k, v, out))
    bf16 = _torch.bfloat16
    if q.dtype is not bf16 or k.dtype is not bf16 or v.dtype is not bf16:
        _refuse("attention: q, k and v must be bfloat16")
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or ks != v.shape or ks[2] != qs[2]:
        _refuse("attention: q must be [tokens, heads, head_dim], k and v [kv_heads, rows, head_dim]")
    T, nh, hd = qs
    nkv, rows, _ = ks
    if out is None:
        out = _torch.empty_like(q) if stream is None else _new(q, stream, qs, bf16)
    elif out.dtype is not bf16 or out.shape != qs:
        _refuse("attention: out must be bfloat16 of q's shape")
    (qt, qh, q1), (kh, kr, k1), (vh, vr, v1), (ot, oh, o1) = (q.stride(), k.stride(), v.stride(),
                                                              out.stride())
    if hd > 1 and not q1 == k1 == v1 == o1 == 1:
        _refuse("attention: head_dim must be contiguous")
    if not 0 <= pos <= rows - T or rows > _I32:
        raise AmkError(abi.ERR["AMK_ERR_POS_RANGE"], f"attention: positions {pos} .. "
                       f"{pos + T - 1} outside the {rows} rows")
    if window < 0 or sinks < 0:
        _refuse("attention: window or sinks < 0")
    if T == 0:
        return out
    args = _pack_attention(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), qt, qh, ot, oh,
                           kh, kr, vh, vr, T, pos, nh, nkv, hd, rows,
                           # beyond any position: the same mask
                           min(window, _I32), min(sinks, _I32), scale)
    _launch("amk_attention", _lib.amk_attention, args, dev, stream, (q, k, v, out))
    return out


def verify_draft(target_logits, draft_tokens, u, *, draft_logits=None, temperature: float = 1.0,
                 tokens=None, n_accepted=None, stream=None):
    """Verifies drafted tokens against the target's distributions, from given
    random numbers, and draws the token behind the accepted ones
    (amk_verify_draft).  target_logits: fp32 [drafts + 1, vocab];
    draft_tokens: int32 [drafts]; u: fp32 [drafts + 1] in [0, 1);
    draft_logits: fp32 [drafts, vocab], or None when the draft has no
    distribution.  temperature: 0 (greedy), or 1e-6 .. 1e6.  Returns (tokens int32
    [drafts + 1], n_accepted int32 [1]) on the device (those given, which overlap
    no input, or new ones): the accepted tokens, the drawn one, then -1.  With no drafts it samples one token."""
    if _torch is None:
        _load()
    torch = _torch
    if not (temperature == 0 or 1e-6 <= temperature <= 1e6):  # less could become 0: greedy
        _refuse("verify_draft: temperature is not 0 or within [1e-6, 1e6]")
    dev = _check_tensors("verify_draft", ("target_logits", "draft_tokens", "u", "draft_logits",
                                          "tokens", "n_accepted"),
                         (target_logits, draft_tokens, u, draft_logits, tokens, n_accepted))
    f32, i32 = torch.float32, torch.int32
    ts = target_logits.shape
    if len(ts) != 2 or ts[0] < 1:
        _refuse("verify_draft: target_logits must be [drafts + 1, vocab]")
    d, vocab = ts[0] - 1, ts[1]
    if vocab > _I32 or d > _I32:
        _refuse("verify_draft: a size above 2^31 - 1")
    nbytes = _workspace.get((d, vocab))
    if nbytes is None:
        nbytes = _lib.amk_verify_workspace(d, vocab)
        if nbytes < 0:
            _check(int(nbytes), "amk_verify_workspace")
        if len(_workspace) >= 256:
            _workspace.clear()
        _workspace[d, vocab] = nbytes
    if draft_tokens.dtype is not i32 or draft_tokens.shape != (d,) or \
            not draft_tokens.is_contiguous():
        _refuse(f"verify_draft: draft_tokens is not contiguous int32 [{d}]")
    if u.dtype is not f32 or u.shape != (d + 1,) or not u.is_contiguous():
        _refuse(f"verify_draft: u is not contiguous float32 [{d + 1}]")
    tstr, one = target_logits.stride()
    if target_logits.dtype is not f32 or (one != 1 and vocab > 1):
        _refuse("verify_draft: target_logits is not float32 with contiguous rows")
    dstr = dp = 0
    if draft_logits is not None:
        if draft_logits.dtype is not f32 or draft_logits.shape != (d, vocab) or \
                (draft_logits.stride(1) != 1 and vocab > 1):
            _refuse(f"verify_draft: draft_logits is not float32 [{d}, {vocab}] with contiguous rows")
        dstr, dp = draft_logits.stride(0), draft_logits.data_ptr()
    if tokens is None:
        tokens = _new(draft_tokens, stream, (d + 1,), i32)
    elif tokens.dtype is not i32 or tokens.shape != (d + 1,) or not tokens.is_contiguous():
        _refuse(f"verify_draft: tokens is not contiguous int32 [{d + 1}]")
    if n_accepted is None:
        n_accepted = _new(draft_tokens, stream, (1,), i32)
    elif n_accepted.dtype is not i32 or n_accepted.shape != (1,):
        _refuse("verify_draft: n_accepted is not int32 [1]")
    work = _new(draft_tokens, stream, ((nbytes + 3) >> 2,), i32)
    args = _pack_verify(target_logits.data_ptr(), dp, u.data_ptr(), draft_tokens.data_ptr(),
                        tokens.data_ptr(), n_accepted.data_ptr(), tstr, dstr, d, vocab,
                        temperature, work.data_ptr(), nbytes)
    _launch("amk_verify_draft", _lib.amk_verify_draft, args, dev, stream,
            (target_logits, draft_tokens, u, draft_logits, tokens, n_accepted, work))
    return tokens, n_accepted


def ops_timeouts() -> int:
    """CTAs of the operators' kernels that gave up a wait on the current device
    since the library was loaded (amk_ops_timeouts): 0 on a sound device."""
    n = abi.c_u32(0)
    _check(abi.lib().amk_ops_timeouts(ctypes.byref(n)), "amk_ops_timeouts")
    return n.value
