"""The operators of the multi-token step, for measurement: the matrix product with its fused
epilogue (``amk.linear``), attention over the decoder's KV cache with a sliding window and sinks
(``amk.attention``) and the verification of drafted tokens (``amk.verify_draft``).

Each case is one call of one operator.  ``run`` computes it in plain torch operations, or, with
``own`` true, by the framework's entry point; ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

GROUP = 128  # inputs per int4 scale


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # one token through a 7B-shaped O-projection, added to the fp32 residual stream
        _linear("linear one token 4096", 1, 4096, 4096, "bf16", residual="f32", out="f32"),
        # five tokens (four drafts and their root) through a 1B-shaped int8 gate/up pair
        _linear("linear 5 gated int8", 5, 8192, 2048, "int8", act="silu", gated=True),
        # a short prompt through a 7B-shaped int4 down projection
        _linear("linear 77 int4 down", 77, 4096, 11008, "int4", residual="bf16"),
        # ragged prompt through a 135M-shaped FFN projection with bias
        _linear("linear 250 bias", 250, 1536, 576, "bf16", act="gelu", bias=True),
        # a long prompt through the 7B-shaped gate/up pair: the largest product of a layer
        _linear("linear 2048 gated", 2048, 11008, 4096, "bf16", act="silu", gated=True),
        # one token over a full 7B-shaped cache, no window
        _attention("attention one token", 1, 2047, 32, 32, 128),
        # five tokens over a long cache with grouped heads, all of it visible
        _attention("attention 5 long cache", 5, 32000, 32, 4, 64),
        # a ragged chunk of a prompt, 135M-shaped heads, a short window and one sink
        _attention("attention 333 window", 333, 700, 9, 3, 64, window=256, sinks=1),
        # a long prompt of the 7B shape with a window and four sinks
        _attention("attention 2048 window", 2048, 2048, 32, 32, 128, window=1024, sinks=4),
        # one token sampled from the target alone, no draft
        _verify("verify no draft", 0, 49152, 1.0, "none"),
        # four tokens drafted by a model with a distribution of its own
        _verify("verify 4 drafts", 4, 32000, 0.8, "logits"),
        # eight tokens drafted by lookup (no distribution), the largest vocabulary
        _verify("verify 8 lookup drafts", 8, 128256, 1.0, "none"),
    ]


def _linear(name, m, n, k, weights, act="none", bias=False, gated=False, residual="none",
            out="bf16"):
    c = {"op": "linear", "m": m, "n": n, "k": k, "weights": weights, "act": act, "bias": bias,
         "gated": gated, "residual": residual, "out": out}
    return dict(c, name=name) if name else c


def _attention(name, tokens, pos, heads, kv_heads, head_dim, window=0, sinks=0):
    c = {"op": "attention", "tokens": tokens, "pos": pos, "heads": heads, "kv_heads": kv_heads,
         "head_dim": head_dim, "window": window, "sinks": sinks}
    return dict(c, name=name) if name else c


def _verify(name, drafts, vocab, temperature, draft):
    c = {"op": "verify", "drafts": drafts, "vocab": vocab, "temperature": temperature,
         "draft": draft}
    return dict(c, name=name) if name else c


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "attention", "attention", "verify"])
    if op == "linear":
        weights = rng.choice(["bf16", "bf16", "int8", "int4"])
        step = {"bf16": 1, "int8": 1, "int4": 32}[weights]
        m = _log_uniform(rng, 1, 2048)
        n = _log_uniform(rng, 64, 12000)
        k = -(-_log_uniform(rng, 64, 11008) // step) * step
        # most widths of models are multiples of 64; vocabularies and cut rows are not
        if rng.random() < 0.75:
            n = -(-n // 64) * 64
        if rng.random() < 0.85:
            k = -(-k // 64) * 64
        gated = rng.random() < 0.35
        cost = 2048 * 11008 * 4096 * 2
        if m * n * k * (2 if gated else 1) > cost:
            m = max(1, cost // (n * k * (2 if gated else 1)))
        return _linear(None, m, n, k, weights,
                       act="silu" if gated else rng.choice(["none", "none", "silu", "gelu",
                                                            "relu"]),
                       bias=rng.random() < 0.3, gated=gated,
                       residual=rng.choice(["none", "f32", "bf16"]),
                       out=rng.choice(["bf16", "f32"]))
    if op == "attention":
        heads, kv_heads, head_dim = rng.choice([(32, 32, 128), (32, 4, 64), (32, 8, 64),
                                                (9, 3, 64), (32, 8, 128), (4, 2, 16)])
        tokens = rng.choice([1, 1, _log_uniform(rng, 2, 16), _log_uniform(rng, 17, 2048)])
        pos = rng.choice([0, _log_uniform(rng, 1, 4096),
                          _log_uniform(rng, 4096, 32768) if tokens <= 16 else 511])
        window = rng.choice([0, 0, _log_uniform(rng, 16, 2048)])
        sinks = rng.choice([0, 1, 4, 37]) if window else 0
        return _attention(None, tokens, pos, heads, kv_heads, head_dim, window, sinks)
    return _verify(None, rng.choice([0, 1, 2, 3, 4, 5, 6, 7, 8]), _log_uniform(rng, 256, 128256),
                   round(rng.uniform(0.5, 1.5), 2), rng.choice(["logits", "none"]))


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _weight(g, n, k, fmt):
    """N(0, 0.02) weights in the framework's formats: (codes, scales or None)."""
    w = _randn(g, n, k).mul_(0.02)
    if fmt == "bf16":
        return w.to(torch.bfloat16), None
    if fmt == "int8":
        s = (w.abs().amax(1) / 127).to(torch.float16)
        return torch.round(w / s.float()[:, None]).clamp_(-127, 127).to(torch.int8), s
    groups = -(-k // GROUP)
    w = torch.nn.functional.pad(w, (0, groups * GROUP - k)).view(n, groups, GROUP)
    s = (w.abs().amax(2) / 7).to(torch.float16)
    q = torch.round(w / s.float()[:, :, None]).clamp_(-7, 7).view(n, -1)[:, :k].to(torch.int16)
    q = q & 15
    return (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8), s


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = _randn(g, m, k).to(torch.bfloat16)  # normed activations: unit variance
        st["w"], st["scale"] = _weight(g, n, k, case["weights"])
        st["up"], st["up_scale"] = (_weight(g, n, k, case["weights"]) if case["gated"]
                                    else (None, None))
        st["bias"] = _randn(g, n).to(torch.bfloat16) if case["bias"] else None
        st["up_bias"] = (_randn(g, n).to(torch.bfloat16) if case["bias"] and case["gated"]
                         else None)
        st["residual"] = (_randn(g, m, n).to(_TYPES[case["residual"]])
                          if case["residual"] != "none" else None)
    elif case["op"] == "attention":
        t, pos, hd = case["tokens"], case["pos"], case["head_dim"]
        rows = pos + t + 64  # a cache with room for the tokens to come
        st["q"] = _randn(g, t, case["heads"], hd).to(torch.bfloat16)
        st["k"] = _randn(g, case["kv_heads"], rows, hd).to(torch.bfloat16)
        st["v"] = _randn(g, case["kv_heads"], rows, hd).to(torch.bfloat16)
    else:
        d, v = case["drafts"], case["vocab"]
        st["target"] = _randn(g, d + 1, v).mul_(2.5)
        # a draft model agrees with the target but for some noise, and draws from its own
        # distribution; tokens found by lookup agree with the target's top choices at times
        noisy = st["target"][:d] + 0.7 * _randn(g, d, v)
        st["draft"] = noisy if case["draft"] == "logits" else None
        u = torch.rand(d, v, generator=g, device="cuda").clamp_(1e-20, 1.0)
        st["tokens"] = (noisy / case["temperature"] - torch.log(-torch.log(u))
                        ).argmax(1).to(torch.int32) if d else torch.empty(
                            0, dtype=torch.int32, device="cuda")
        st["u"] = torch.rand(d + 1, generator=g, device="cuda")
    return st


# ---- one pass ----------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"linear": _plain_linear, "attention": _plain_attention,
            "verify": _plain_verify}[case["op"]](case, state)


def _run_own(case, st):
    import persistent_megakernel_decode_cta_b200 as amk
    if case["op"] == "linear":
        return amk.linear(st["x"], st["w"], scale=st["scale"], bias=st["bias"], act=case["act"],
                          up=st["up"], up_scale=st["up_scale"], up_bias=st["up_bias"],
                          residual=st["residual"], out_dtype=_TYPES[case["out"]])
    if case["op"] == "attention":
        return amk.attention(st["q"], st["k"], st["v"], case["pos"], window=case["window"],
                             sinks=case["sinks"])
    return amk.verify_draft(st["target"], st["tokens"], st["u"], draft_logits=st["draft"],
                            temperature=case["temperature"])


def _dense(w, scale, k):
    """The weights that the codes and scales stand for, in 32 bits."""
    if scale is None:
        return w.float()
    if w.dtype == torch.int8:
        return w.float() * scale.float()[:, None]
    q = torch.stack((w & 15, w >> 4), 2).view(w.shape[0], k).to(torch.int8)
    q = torch.where(q > 7, q - 16, q).float()
    return q * scale.float().repeat_interleave(GROUP, 1)[:, :k]


def _plain_linear(case, st):
    x = st["x"].float()
    y = x @ _dense(st["w"], st["scale"], case["k"]).t()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    if case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif case["act"] == "relu":
        y = torch.clamp(y, min=0)
    if case["gated"]:
        up = x @ _dense(st["up"], st["up_scale"], case["k"]).t()
        if st["up_bias"] is not None:
            up = up + st["up_bias"].float()
        y = y * up
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(_TYPES[case["out"]])


def _plain_attention(case, st):
    t, pos, heads, hd = case["tokens"], case["pos"], case["heads"], case["head_dim"]
    group = heads // case["kv_heads"]
    n = pos + t
    q = st["q"].float().transpose(0, 1)  # [heads, t, hd]
    k = st["k"][:, :n].float().repeat_interleave(group, 0)
    v = st["v"][:, :n].float().repeat_interleave(group, 0)
    s = (q @ k.transpose(1, 2)) * (1 / math.sqrt(hd))
    i = torch.arange(pos, n, device=s.device)[:, None]
    j = torch.arange(n, device=s.device)[None, :]
    seen = j <= i
    if case["window"]:
        seen = seen & ((j > i - case["window"]) | (j < case["sinks"]))
    s = torch.where(seen, s, -math.inf)
    p = torch.exp(s - s.amax(2, keepdim=True))
    o = (p @ v) / p.sum(2, keepdim=True)
    return o.transpose(0, 1).to(torch.bfloat16).contiguous()


def _softmax64(z, temperature):
    z = z.double() / temperature
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_verify(case, st):
    # 64 bits: whether a token is taken, and which one a random number falls on, are decisions
    d, v = case["drafts"], case["vocab"]
    dev = st["target"].device
    p = _softmax64(st["target"], case["temperature"])
    tok, u = st["tokens"].long(), st["u"].double()
    if d:
        if st["draft"] is not None:
            q = _softmax64(st["draft"], case["temperature"])
        else:
            q = torch.zeros(d, v, dtype=torch.float64, device=dev).scatter_(1, tok[:, None], 1.0)
        pd, qd = p[:d].gather(1, tok[:, None])[:, 0], q.gather(1, tok[:, None])[:, 0]
        n = (u[:d] * qd < pd).long().cumprod(0).sum()
        q = torch.cat((q, torch.zeros(1, v, dtype=torch.float64, device=dev)))
        row_p, row_q = p.index_select(0, n[None])[0], q.index_select(0, n[None])[0]
        r = torch.clamp(row_p - row_q, min=0)
        r = torch.where(r.sum() > 0, r, row_p)
    else:
        n = torch.zeros((), dtype=torch.long, device=dev)
        r = p[0]
    cdf = torch.cumsum(r, 0)
    nxt = (cdf <= u[d] * cdf[-1]).sum()  # the first token whose cumulative weight passes u
    i = torch.arange(d + 1, device=dev)
    drafted = torch.cat((tok, nxt[None]))
    tokens = torch.where(i < n, drafted, torch.where(i == n, nxt, -1))
    return tokens.to(torch.int32), n.to(torch.int32)[None]


# ---- the work and the definition ---------------------------------------------

def _visible(case):
    """(rows of the cache that some token sees, pairs of a token and a row that it sees)"""
    t, pos, w, s = case["tokens"], case["pos"], case["window"], case["sinks"]
    if not w:
        return pos + t, sum(pos + i + 1 for i in range(t))
    lo = max(0, pos - w + 1)
    rows = pos + t - lo + min(s, lo)
    pairs = 0
    for p in range(pos, pos + t):
        a = max(0, p - w + 1)
        pairs += p + 1 - a + min(s, a)
    return rows, pairs


def work(case):
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        mats = 2 if case["gated"] else 1
        w = {"bf16": 2 * n * k, "int8": n * k + 2 * n,
             "int4": n * k / 2 + 2 * n * -(-k // GROUP)}[case["weights"]]
        size = {"none": 0, "bf16": 2, "f32": 4}
        b = mats * w + 2 * m * k + m * n * (size[case["residual"]] + size[case["out"]])
        return {"bytes": b + (2 * n * mats if case["bias"] else 0), "flops": 2 * m * n * k * mats}
    if case["op"] == "attention":
        rows, pairs = _visible(case)
        hd = case["head_dim"]
        return {"bytes": 4 * rows * case["kv_heads"] * hd + 4 * case["tokens"] * case["heads"] * hd,
                "flops": 4 * hd * case["heads"] * pairs}
    d, v = case["drafts"], case["vocab"]
    rows = d + 1 + (d if case["draft"] == "logits" else 0)
    return {"bytes": 4 * rows * v, "flops": 4 * rows * v}


def _exact_weights(w, scale, k):
    if scale is None:
        return w.to(torch.float64)
    if w.dtype == torch.int8:
        return torch.einsum("nk,n->nk", w.to(torch.float64), scale.to(torch.float64))
    b = w.to(torch.int64)
    codes = torch.zeros(w.shape[0], k, dtype=torch.float64, device=w.device)
    codes[:, 0::2] = ((b + 8) % 16 - 8).to(torch.float64)
    codes[:, 1::2] = ((b // 16 + 8) % 16 - 8).to(torch.float64)
    at = torch.arange(k, device=w.device) // GROUP
    return codes * scale.to(torch.float64)[:, at]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        x = st["x"].to(torch.float64)
        y = torch.einsum("mk,nk->mn", x, _exact_weights(st["w"], st["scale"], case["k"]))
        y = y if st["bias"] is None else y + st["bias"].to(torch.float64)
        y = {"none": lambda z: z, "silu": lambda z: z * torch.sigmoid(z),
             "gelu": lambda z: z * torch.special.ndtr(z),
             "relu": lambda z: torch.maximum(z, torch.zeros_like(z))}[case["act"]](y)
        if case["gated"]:
            up = torch.einsum("mk,nk->mn", x, _exact_weights(st["up"], st["up_scale"], case["k"]))
            y = y * (up if st["up_bias"] is None else up + st["up_bias"].to(torch.float64))
        return y if st["residual"] is None else y + st["residual"].to(torch.float64)
    if case["op"] == "attention":
        t, pos, w = case["tokens"], case["pos"], case["window"]
        group, n = case["heads"] // case["kv_heads"], case["pos"] + case["tokens"]
        out = torch.empty(t, case["heads"], case["head_dim"], dtype=torch.float64, device="cuda")
        far = torch.arange(pos, n, device="cuda")[:, None] - torch.arange(n, device="cuda")
        hidden = far < 0
        if w:
            hidden |= (far >= w) & (torch.arange(n, device="cuda") >= case["sinks"])
        for h in range(case["heads"]):
            kk = st["k"][h // group, :n].to(torch.float64)
            s = st["q"][:, h].to(torch.float64) @ kk.t() / math.sqrt(case["head_dim"])
            a = torch.softmax(s.masked_fill(hidden, -math.inf), 1)
            out[:, h] = a @ st["v"][h // group, :n].to(torch.float64)
        return out
    return _exact_verify(case, st)


def _exact_verify(case, st):
    d, temperature = case["drafts"], case["temperature"]
    target = st["target"].cpu().numpy().astype(np.float64)
    tok, u = st["tokens"].cpu().numpy(), st["u"].cpu().numpy().astype(np.float64)

    def dist(row):
        e = np.exp((row - row.max()) / temperature)
        return e / math.fsum(e)

    out = np.full(d + 1, -1, np.int32)
    for i in range(d + 1):
        p = dist(target[i])
        weights = p
        if i < d:
            if st["draft"] is not None:
                q = dist(st["draft"][i].cpu().numpy().astype(np.float64))
            else:
                q = np.eye(1, case["vocab"], tok[i])[0]
            if u[i] * q[tok[i]] < p[tok[i]]:
                out[i] = tok[i]
                continue
            weights = np.maximum(p - q, 0)
            weights = weights if weights.sum() > 0 else p
        cdf = np.cumsum(weights)
        out[i] = np.searchsorted(cdf, u[d] * cdf[-1], side="right")
        return out, np.array([i], np.int32)
