"""Plain 64-bit forms of the multi-token step's operators for the tests, and
the error each kernel may make, derived from its arithmetic.

A bf16 result is off by half a step of the value, 2^-8 relative, an fp32 one by
2^-24; sums of n fp32 terms by at most n 2^-24 of the sum of their magnitudes
(taken twice, 2^-23: tensor cores may truncate where they align terms)."""
import math

import torch

HALF = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}


def dense(w, scale=None):
    """The 64-bit weights that codes and scales stand for."""
    if w.dtype == torch.bfloat16:
        return w.double()
    if w.dtype == torch.int8:
        return w.double() * scale.double()[:, None]
    lo, hi = (w & 15).to(torch.int64), (w >> 4).to(torch.int64)
    q = torch.stack((lo, hi), dim=2).reshape(w.shape[0], -1)
    q = torch.where(q >= 8, q - 16, q).double()
    return q * scale.double().repeat_interleave(128, 1)[:, :q.shape[1]]


def linear(x, w, scale=None, bias=None, act="none", up=None, up_scale=None, up_bias=None,
           residual=None, out_dtype=torch.bfloat16):
    """(y, tolerance) in 64 bits."""
    xd = x.double()

    def product(m, s, b):
        md = dense(m, s)
        y, mag = xd @ md.t(), xd.abs() @ md.abs().t()
        if b is not None:
            y, mag = y + b.double(), mag + b.double().abs()
        return y, (x.shape[-1] + 16) * 2.0**-23 * mag

    y, err = product(w, scale, bias)
    if act == "silu":
        y, pre = y * torch.sigmoid(y), y
    elif act == "gelu":
        y, pre = 0.5 * y * (1 + torch.erf(y / math.sqrt(2))), y
    elif act == "relu":
        y, pre = y.clamp(min=0), y
    else:
        pre = torch.zeros_like(y)
    # the activations' slopes stay below 1.13; their own fp32 evaluation is off by a few
    # units in the last place of the input, times |input| in the exponential
    err = 1.13 * err + 2.0**-21 * pre.abs() * (1 + pre.abs().clamp(max=30))
    if up is not None:
        u, uerr = product(up, up_scale, up_bias)
        err = err * (u.abs() + uerr) + y.abs() * uerr
        y = y * u
    if residual is not None:
        y = y + residual.double()
    mag = y.abs() + err
    return y, err + HALF[out_dtype] * mag + 2.0**-22 * mag


def visible(T, pos, window, sinks, device):
    i = torch.arange(pos, pos + T, device=device)[:, None]
    j = torch.arange(pos + T, device=device)[None, :]
    m = j <= i
    if window:
        m = m & ((j > i - window) | (j < sinks))
    return m


def attention(q, k, v, pos, window=0, sinks=0, scale=None):
    """(out, tolerance) in 64 bits; what a masked row holds never enters."""
    T, nh, hd = q.shape
    g = nh // k.shape[0]
    scale = scale or 1 / math.sqrt(hd)
    n = pos + T
    seen = visible(T, pos, window, sinks, q.device)
    out = torch.empty(T, nh, hd, dtype=torch.float64, device=q.device)
    tol = torch.empty_like(out)
    for h in range(nh):
        kd, vd = k[h // g, :n].double(), v[h // g, :n].double()
        qd = q[:, h].double()
        s = torch.where(seen, (qd @ kd.t()) * scale, -math.inf)
        p = torch.softmax(s, 1)
        # rows no token sees; a row that some see enters only through them
        clean = torch.where(torch.isfinite(vd), vd, 0)
        o, mag = p @ clean, p @ clean.abs()
        for j in torch.nonzero(~torch.isfinite(vd).all(1))[:, 0].tolist():
            hit = seen[:, j]
            o[hit] = o[hit] + p[hit, j, None] * torch.where(torch.isfinite(vd[j]), 0, vd[j])
        big = torch.where(seen, (qd.abs() @ torch.nan_to_num(kd).abs().t()) * scale, 0.0).amax(1)
        rel = 2 * ((hd + 8) * 2.0**-23 * big + 2.0**-20)[:, None]  # of each weight
        out[:, h], tol[:, h] = o, mag * (rel + 2.0**-8) + 2.0**-8 * o.abs() + 1e-30
    return out, tol


def verify(target, tokens, u, draft=None, temperature=1.0):
    """(tokens, n_accepted) as lists, token by token in 64 bits."""
    d, vocab = target.shape[0] - 1, target.shape[1]
    target, u = target.double().cpu(), u.double().cpu()
    tokens = tokens.cpu().tolist()
    draft = draft.double().cpu() if draft is not None else None

    def fine(row):
        return not (torch.isnan(row).any() or (row == math.inf).any() or (row == -math.inf).all())

    out = [-1] * (d + 1)
    for i in range(d + 1):
        if not fine(target[i]):
            return out, i
        if temperature == 0:
            best = int((target[i] == target[i].max()).nonzero()[0])
            if i < d and tokens[i] == best:
                out[i] = best
                continue
            out[i] = best
            return out, i
        p = torch.softmax(target[i] / temperature, 0)
        w = p
        if i < d:
            if draft is not None:
                if not fine(draft[i]):
                    return out, i
                q = torch.softmax(draft[i] / temperature, 0)
            else:
                q = torch.zeros(vocab, dtype=torch.float64)
                if 0 <= tokens[i] < vocab:
                    q[tokens[i]] = 1
            t = tokens[i]
            if 0 <= t < vocab and u[i] * q[t] < p[t]:
                out[i] = t
                continue
            w = (p - q).clamp(min=0)
            if w.sum() <= 0:
                w = p
        c = w.cumsum(0)
        hit = (c > u[d] * c[-1]).nonzero()
        out[i] = int(hit[0]) if len(hit) else int((w > 0).nonzero()[-1])
        return out, i
