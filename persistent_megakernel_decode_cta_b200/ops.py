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
from typing import Optional, Tuple

from . import AmkError, _check, abi

_I32 = 2**31 - 1
_INVALID = abi.ERR["AMK_ERR_INVALID_ARG"]
_torch = None


def _lib():
    """torch and the loaded library (both are imported on the first call)."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch, abi.lib()


def _refuse(what: str):
    raise AmkError(_INVALID, what)


def _tensors(what: str, stream, named):
    """Checks that every tensor is on one CUDA device and needs no gradient;
    returns the device index and the stream handle."""
    torch = _torch
    dev = None
    grad = torch.is_grad_enabled()
    for name, t in named:
        if t is None:
            continue
        if not t.is_cuda:
            _refuse(f"{what}: {name} is not a CUDA tensor")
        i = t.get_device()
        if dev is None:
            dev = i
        elif i != dev:
            _refuse(f"{what}: {name} is on cuda:{i}, others on cuda:{dev}")
        if grad and t.requires_grad:
            _refuse(f"{what}: {name} requires a gradient, which is not computed")
    if stream is None:
        return dev, torch.cuda.current_stream(dev).cuda_stream
    side = torch.cuda.ExternalStream(stream, device=dev)
    for _, t in named:
        if t is not None:
            t.record_stream(side)
    return dev, stream


def _call(fn, args, dev: int, stream: int, what: str):
    torch = _torch
    if dev == torch.cuda.current_device():
        rc = fn(ctypes.byref(args), stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(ctypes.byref(args), stream)
    if rc != abi.AMK_OK:
        _check(rc, what)


def _new(what, stream, shape, dtype, dev):
    """A result tensor, from the pool of the stream that will write it."""
    torch = _torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=dev)):
        return torch.empty(shape, dtype=dtype, device=f"cuda:{dev}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def linear(x, w, *, scale=None, bias=None, act: str = "none", up=None, up_scale=None,
           up_bias=None, residual=None, out=None, out_dtype=None, stream=None):
    """``act(x @ w.T + bias)``, times ``x @ up.T + up_bias`` when ``up`` is given,
    plus ``residual`` (amk_linear).

    x: bf16 [..., k] (rows may be strided, the inputs of a row are contiguous).
    w, up: bf16 [n, k]; or int8 [n, k] with scale fp16 [n]; or packed int4,
    uint8 [n, k / 2] with scale fp16 [n, ceil(k / 128)] -- contiguous, both of
    one format.  Biases: bf16 [n].  act: "none", "silu", "gelu" or "relu".
    residual: bf16 or fp32 [..., n].  Returns bf16 or fp32 [..., n]: ``out``
    (which may be ``residual``), else a new tensor of ``out_dtype`` (default:
    bf16)."""
    torch, lib = _lib()
    dev, st = _tensors("linear", stream,
                       (("x", x), ("w", w), ("scale", scale), ("bias", bias), ("up", up),
                        ("up_scale", up_scale), ("up_bias", up_bias), ("residual", residual),
                        ("out", out)))
    bf16, f32 = torch.bfloat16, torch.float32
    if x.dtype is not bf16:
        _refuse(f"linear: x is {x.dtype}, not bfloat16")
    if x.dim() < 1 or w.dim() != 2:
        _refuse("linear: x needs one dimension at least and w two")
    if act not in abi.ACT:
        _refuse(f"linear: unknown activation {act!r}")
    k = x.shape[-1]
    n = w.shape[0]
    wt = w.dtype
    if wt is bf16:
        quant, cols, sshape = abi.QUANT_BF16, k, None
    elif wt is torch.int8:
        quant, cols, sshape = abi.QUANT_W8A16, k, (n,)
    elif wt is torch.uint8:
        quant, cols, sshape = abi.QUANT_W4A16, k // 2, (n, (k + 127) // 128)
        if k % 2:
            _refuse("linear: int4 rows need an even number of inputs")
    else:
        _refuse(f"linear: no weight format with {wt} elements")
    for name, m, s in (("w", w, scale), ("up", up, up_scale)):
        if m is None:
            if s is not None:
                _refuse(f"linear: {name}_scale without {name}")
            continue
        if m.dtype is not wt or m.shape != (n, cols) or not m.is_contiguous():
            _refuse(f"linear: {name} is not a contiguous {wt} [{n}, {cols}] matrix")
        if sshape is None:
            if s is not None:
                _refuse(f"linear: bf16 {name} takes no scale")
        elif s is None or s.dtype is not torch.float16 or s.shape != sshape or \
                not s.is_contiguous():
            _refuse(f"linear: the scale of {name} is not contiguous float16 {list(sshape)}")
    if up is None and up_bias is not None:
        _refuse("linear: up_bias without up")
    for name, b in (("bias", bias), ("up_bias", up_bias)):
        if b is not None and (b.dtype is not bf16 or b.shape != (n,) or not b.is_contiguous()):
            _refuse(f"linear: {name} is not contiguous bfloat16 [{n}]")
    lead = x.shape[:-1]
    shape = (*lead, n)
    m, ldx = _rows("linear", "x", x)
    if out is None:
        out = _new("linear", stream, shape, out_dtype or bf16, dev)
    elif out_dtype is not None and out.dtype is not out_dtype:
        _refuse(f"linear: out is {out.dtype}, not {out_dtype}")
    ot = out.dtype
    if ot is not bf16 and ot is not f32:
        _refuse(f"linear: out is {ot}, not bfloat16 or float32")
    if out.shape != shape:
        _refuse(f"linear: out has shape {list(out.shape)}, not {list(shape)}")
    _, ldy = _rows("linear", "out", out)
    ldr, rt = 0, 0
    if residual is not None:
        if residual.dtype is not bf16 and residual.dtype is not f32:
            _refuse(f"linear: residual is {residual.dtype}, not bfloat16 or float32")
        if residual.shape != shape:
            _refuse(f"linear: residual has shape {list(residual.shape)}, not {list(shape)}")
        _, ldr = _rows("linear", "residual", residual)
        rt = abi.DT_F32 if residual.dtype is f32 else abi.DT_BF16
    if m == 0:
        return out
    if max(m, n, k) > _I32:
        _refuse("linear: a size above 2^31 - 1")
    a = abi.LinearArgs(x.data_ptr(), w.data_ptr(), _ptr(scale), _ptr(bias), _ptr(up),
                       _ptr(up_scale), _ptr(up_bias), _ptr(residual), out.data_ptr(), ldx, ldr,
                       ldy, m, n, k, quant, abi.ACT[act], rt,
                       abi.DT_F32 if ot is f32 else abi.DT_BF16)
    _call(lib.amk_linear, a, dev, st, "amk_linear")
    return out


def _rows(what: str, name: str, t) -> Tuple[int, int]:
    """(rows, row stride) of a tensor seen as [rows][last dimension]."""
    n = t.shape[-1]
    if t.dim() == 2 and (t.stride(1) == 1 or n == 1):
        rows, ld = t.shape[0], t.stride(0)
        if rows <= 1:
            ld = max(ld, n)
        elif ld < n:
            _refuse(f"{what}: the rows of {name} overlap")
        return rows, ld
    if t.is_contiguous():
        return (t.numel() // n if n else 0), n
    _refuse(f"{what}: {name} is neither contiguous nor a matrix of contiguous rows")


def attention(q, k, v, pos: int, *, window: int = 0, sinks: int = 0,
              scale: Optional[float] = None, out=None, stream=None):
    """Causal attention of the query tokens q (bf16 [tokens, heads, head_dim], at
    positions pos, pos + 1, ...) over the cache rows k and v (bf16 [kv_heads,
    rows, head_dim], row j = position j, as ``Decoder.kv`` returns them):
    amk_attention.  ``window`` > 0 limits a token to the last ``window`` rows
    up to its own, and to the first ``sinks`` rows.  scale: default
    1 / sqrt(head_dim).  Returns bf16 [tokens, heads, head_dim] (``out`` if
    given).  Leading dimensions may be strided; head_dim is contiguous."""
    torch, lib = _lib()
    dev, st = _tensors("attention", stream, (("q", q), ("k", k), ("v", v), ("out", out)))
    bf16 = torch.bfloat16
    if q.dtype is not bf16 or k.dtype is not bf16 or v.dtype is not bf16:
        _refuse("attention: q, k and v must be bfloat16")
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[2] != q.shape[2]:
        _refuse("attention: q must be [tokens, heads, head_dim], k and v [kv_heads, rows, head_dim]")
    T, nh, hd = q.shape
    nkv, rows, _ = k.shape
    if out is None:
        out = _new("attention", stream, (T, nh, hd), bf16, dev)
    elif out.dtype is not bf16 or out.shape != q.shape:
        _refuse("attention: out must be bfloat16 of q's shape")
    (qt, qh, q1), (kh, kr, k1), (vh, vr, v1), (ot, oh, o1) = (q.stride(), k.stride(), v.stride(),
                                                              out.stride())
    if hd > 1 and not q1 == k1 == v1 == o1 == 1:
        _refuse("attention: head_dim must be contiguous")
    if scale is not None and not 0 < scale < float("inf"):
        _refuse("attention: scale must be positive and finite")
    if not 0 <= pos <= rows - T or rows > _I32:
        raise AmkError(abi.ERR["AMK_ERR_POS_RANGE"], f"attention: positions {pos} .. "
                       f"{pos + T - 1} outside the {rows} rows")
    if window < 0 or sinks < 0:
        _refuse("attention: window or sinks < 0")
    if T == 0:
        return out
    window, sinks = min(window, _I32), min(sinks, _I32)  # beyond any position: the same mask
    a = abi.AttentionArgs(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), qt, qh, ot, oh,
                          kh, kr, vh, vr, T, pos, nh, nkv, hd, rows, window, sinks, scale or 0.0)
    _call(lib.amk_attention, a, dev, st, "amk_attention")
    return out


def verify_draft(target_logits, draft_tokens, u, *, draft_logits=None, temperature: float = 1.0,
                 tokens=None, n_accepted=None, stream=None):
    """Verifies drafted tokens against the target's distributions, from given
    random numbers, and draws the token behind the accepted ones
    (amk_verify_draft).  target_logits: fp32 [drafts + 1, vocab];
    draft_tokens: int32 [drafts]; u: fp32 [drafts + 1] in [0, 1);
    draft_logits: fp32 [drafts, vocab], or None when the draft has no
    distribution.  temperature 0 is greedy.  Returns (tokens int32
    [drafts + 1], n_accepted int32 [1]) on the device: the accepted tokens, the
    drawn one, then -1.  With no drafts it samples one token."""
    torch, lib = _lib()
    dev, st = _tensors("verify_draft", stream,
                       (("target_logits", target_logits), ("draft_tokens", draft_tokens),
                        ("u", u), ("draft_logits", draft_logits), ("tokens", tokens),
                        ("n_accepted", n_accepted)))
    if target_logits.dim() != 2 or target_logits.shape[0] < 1:
        _refuse("verify_draft: target_logits must be [drafts + 1, vocab]")
    d, vocab = target_logits.shape[0] - 1, target_logits.shape[1]
    if vocab > _I32 or d > _I32:
        _refuse("verify_draft: a size above 2^31 - 1")
    f32, i32 = torch.float32, torch.int32
    if tokens is None:
        tokens = _new("verify_draft", stream, (d + 1,), i32, dev)
    if n_accepted is None:
        n_accepted = _new("verify_draft", stream, (1,), i32, dev)
    for name, t, dtype, shape in (("draft_tokens", draft_tokens, i32, (d,)), ("u", u, f32, (d + 1,)),
                                  ("tokens", tokens, i32, (d + 1,)),
                                  ("n_accepted", n_accepted, i32, (1,))):
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            _refuse(f"verify_draft: {name} is not contiguous {dtype} {list(shape)}")
    for name, t, n in (("target_logits", target_logits, d + 1), ("draft_logits", draft_logits, d)):
        if t is not None and (t.dtype is not f32 or t.shape != (n, vocab)
                              or (vocab > 1 and t.stride(1) != 1)):
            _refuse(f"verify_draft: {name} is not float32 [{n}, {vocab}] with contiguous rows")
    nbytes = lib.amk_verify_workspace(d, vocab)
    if nbytes < 0:
        _check(int(nbytes), "amk_verify_workspace")
    ws = _new("verify_draft", stream, (nbytes,), torch.uint8, dev)
    a = abi.VerifyArgs(target_logits.data_ptr(), _ptr(draft_logits) or None, u.data_ptr(),
                       draft_tokens.data_ptr() or None, tokens.data_ptr(), n_accepted.data_ptr(),
                       target_logits.stride(0), draft_logits.stride(0) if draft_logits is not None
                       else 0, d, vocab, temperature, ws.data_ptr(), nbytes)
    _call(lib.amk_verify_draft, a, dev, st, "amk_verify_draft")
    return tokens, n_accepted
