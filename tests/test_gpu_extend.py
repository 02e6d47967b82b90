"""The multi-token step (amk_extend) and generation on the GPU, against the fp64
oracle fed the same tokens one by one.

Tolerance.  The step rounds what its matrix products take (normed residual,
rotated q, attention and SwiGLU outputs) to bf16: by at most 2^-8 of an element,
2^-8 / sqrt(3) / sqrt(7 / 3) = 1.5e-3 rms (of a binade's numbers), so each of the 2 L sublayers' outputs is off by at most 3e-3 of its own
norm (three roundings in a row, and a half for what the norms pass on), added
up like independent errors with the final norm's: 3e-3 sqrt(2 L + 1) of the
logits' norm.  A single logit's error is a sum of many independent roundings,
so nearly normal: none of the some 1e6 that are looked at here is beyond six
times the root mean square (2e-9 each).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as orc
import persistent_megakernel_decode_cta_b200 as amk
import synth_inputs as si
from tests.parity_helpers import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    pass


def tol(cfg):
    return 3e-3 * math.sqrt(2 * cfg.n_layers + 1)


def close(cfg, got, want, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    size = np.sqrt((want**2).mean())
    rms, worst = np.sqrt(((got - want)**2).mean()) / size, np.abs(got - want).max() / size
    assert rms <= tol(cfg) and worst <= 6 * tol(cfg), (
        f"{what}: error {rms:.3g} rms, {worst:.3g} at most, of the logits' root mean square; "
        f"tolerance {tol(cfg):.3g} and six times that")


def pair(cfg, seed=0):
    w = si.make_model(cfg, seed=seed, device="cuda")
    torch.cuda.synchronize()
    return amk.Decoder(cfg, w), orc.OracleModel(cfg, w), w


TINY = si.get_config("tiny")
VARIANTS = {
    "bf16": TINY, "tied": TINY.with_(tied=True), "w8a16": TINY.with_(quant="w8a16"),
    "w4a16": TINY.with_(quant="w4a16", ffn=192),
    "wide": TINY.with_(hidden=256, n_heads=8, n_kv_heads=1, head_dim=64, ffn=512),
}


@pytest.mark.parametrize("name", VARIANTS)
def test_extend_matches_the_oracle_token_by_token(name):
    cfg = VARIANTS[name]
    dec, ref, _ = pair(cfg)
    toks = si.make_prompt(cfg, 31)
    want = [ref.step(t, p)[0] for p, t in enumerate(toks)]
    # 11 tokens, one alone, a decode step between, the rest
    got = dec.extend(toks[:11], 0, n_logits=11)
    for p in range(11):
        close(cfg, got[p], want[p], f"{name} {p}")
    close(cfg, dec.extend(toks[11:12], 11)[0], want[11], f"{name} 11")
    lg = torch.empty(cfg.vocab, device="cuda")
    dec.step(toks[12], 12, logits=lg)
    close(cfg, lg, want[12], f"{name} step 12")
    got = dec.extend(toks[13:30], 13, n_logits=5)
    for i in range(5):
        close(cfg, got[i], want[25 + i], f"{name} {25 + i}")
    dec.step(toks[30], 30, logits=lg)
    close(cfg, lg, want[30], f"{name} step 30")
    dec.close()


def test_extend_over_several_chunks():
    """More tokens than run at a time, the wanted logits across the border."""
    cfg = TINY.with_(max_ctx=2100)
    dec, ref, _ = pair(cfg)
    toks = si.make_prompt(cfg, 2090)
    want = {}
    for p, t in enumerate(toks):
        r = ref.step(t, p)[0]
        if p >= 2090 - 50 or p in (1023, 1024):
            want[p] = r
    got = dec.extend(toks, 0, n_logits=50)
    for i in range(50):
        close(cfg, got[i], want[2040 + i], f"{2040 + i}")
    got = dec.extend(toks[:1025], 0, n_logits=2)
    close(cfg, got[0], want[1023], "1023")
    close(cfg, got[1], want[1024], "1024")
    dec.close()


@pytest.mark.parametrize("name,n", [("smol135", 60), ("smol135_w4", 30), ("tinyllama", 33),
                                    ("llama1b_w8", 20)])
def test_extend_full_size(name, n):
    cfg = si.get_config(name)
    dec, ref, _ = pair(cfg)
    toks = si.make_prompt(cfg, n)
    for p, t in enumerate(toks):
        r = ref.step(t, p)[0]
        if p == n - 3:
            want3 = r
    got = dec.extend(toks, 0, n_logits=3)
    close(cfg, got[0], want3, f"{name} {n - 3}")
    close(cfg, got[2], r, f"{name} {n - 1}")
    # the cache rows are the oracle's but for bf16 steps: a decode step reads them
    lg = torch.empty(cfg.vocab, device="cuda")
    dec.step(toks[0], n, logits=lg)
    close(cfg, lg, ref.step(toks[0], n)[0], f"{name} step {n}")
    dec.close()


def test_steps_after_extend_keep_their_parity():
    """The single-token path is untouched: after a reset it still matches the
    oracle to its own tolerance."""
    cfg = TINY
    dec, ref, _ = pair(cfg)
    dec.extend(si.make_prompt(cfg, 20), 0)
    dec.reset()
    lg = torch.empty(cfg.vocab, device="cuda")
    for p, t in enumerate(si.make_prompt(cfg, 8, seed=5)):
        am = dec.step(t, p, logits=lg)
        r, r_am, _ = ref.step(t, p)
        compare(cfg, lg.double().cpu().numpy(), am, r, r_am, f"pos {p}")
    dec.close()


def test_extend_refusals():
    cfg = TINY
    dec, _, _ = pair(cfg)
    lg = torch.empty((3, cfg.vocab), device="cuda")
    for toks, pos, n in (([0] * 33, 0, 1), ([0], 32, 1), ([0], -1, 1), ([cfg.vocab], 0, 1),
                         ([-1], 0, 1), ([0, 1], 0, 3), ([0, 1], 0, -1)):
        with pytest.raises(amk.AmkError):
            dec.extend(toks, pos, n_logits=n, logits=lg[:n] if n > 0 else None)
    with pytest.raises(amk.AmkError):
        dec.extend([0, 1], 0, logits=lg[:, ::2])
    assert dec.extend([], 5).shape == (0, cfg.vocab)
    dec.extend([1, 2], 0)
    with pytest.raises(amk.AmkError):  # no token was chosen
        dec.step(-1, 2)
    dec.step(3, 2)
    dec.step(-1, 3)
    side = torch.cuda.Stream()
    d2 = amk.Decoder(cfg, si.make_model(cfg, device="cuda"), stream=side.cuda_stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lg.zero_()
        with pytest.raises(amk.AmkError, match="capturing"):
            d2.extend([1], 0, logits=lg[:1])
    dec.close()
    d2.close()


def test_extend_stays_within_its_buffers():
    cfg = TINY.with_(hidden=96, ffn=200, n_heads=6, n_kv_heads=3, head_dim=16)
    w = si.make_model(cfg, device="cuda")
    dec = amk.Decoder(cfg, w, options=amk.default_options(debug_checks=1))
    for n in (1, 7, 32):
        dec.extend(si.make_prompt(cfg, n), 0, n_logits=n)
        assert dec.check_guards() == 0
    dec.close()


# ---- generation --------------------------------------------------------------------

def greedy_by_steps(dec, prompt, n):
    out, lg = [], torch.empty(dec.cfg.vocab, device="cuda")
    margins = []
    for p in range(len(prompt) + n - 1):
        t = prompt[p] if p < len(prompt) else out[-1]
        am = dec.step(t, p, logits=lg)
        if p >= len(prompt) - 1:
            top = torch.topk(lg, 2).values
            margins.append(float((top[0] - top[1]) / lg.abs().max()))
            out.append(am)
    return out, margins


@pytest.mark.parametrize("n_draft", [0, 1, 3, 8])
@pytest.mark.parametrize("same", [True, False])
def test_greedy_generation_is_the_targets_own(n_draft, same):
    cfg = TINY
    w = si.make_model(cfg, seed=0, device="cuda")
    target = amk.Decoder(cfg, w)
    draft = amk.Decoder(cfg, w if same else si.make_model(cfg, seed=1, device="cuda"))
    prompt = si.make_prompt(cfg, 6)
    want, margins = greedy_by_steps(target, prompt, 20)
    got = amk.generate(target, prompt, 20, draft=draft if n_draft else None, n_draft=n_draft,
                       temperature=0.0)
    for i, (a, b) in enumerate(zip(want, got)):
        if a != b:  # only where two logits are as near as the two paths are
            assert margins[i] <= 12 * tol(cfg), f"token {i}: {b}, not {a}"
            break
    assert len(got) == 20
    target.close()
    draft.close()


def test_sampled_generation():
    cfg = TINY
    w = si.make_model(cfg, seed=0, device="cuda")
    target = amk.Decoder(cfg, w)
    draft = amk.Decoder(cfg, si.make_model(cfg, seed=1, device="cuda"))
    prompt = si.make_prompt(cfg, 4)

    def run(seed, **kw):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return amk.generate(target, prompt, 25, temperature=0.9, generator=g, **kw)

    for kw in ({}, {"draft": draft, "n_draft": 4}):
        a, b, c = run(1, **kw), run(1, **kw), run(2, **kw)
        assert a == b and a != c and len(a) == 25
        assert all(0 <= t < cfg.vocab for t in a)
    with pytest.raises(amk.AmkError):
        amk.generate(target, prompt, 30)
    with pytest.raises(amk.AmkError):
        amk.generate(target, [], 3)
    assert amk.generate(target, prompt, 0) == []
    target.close()
    draft.close()


def test_generation_on_a_stream_of_its_own():
    cfg = TINY
    w = si.make_model(cfg, seed=0, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    target = amk.Decoder(cfg, w, stream=side.cuda_stream)
    draft = amk.Decoder(cfg, w, stream=side.cuda_stream)
    here = amk.Decoder(cfg, w)
    prompt = si.make_prompt(cfg, 5)
    want = amk.generate(here, prompt, 15, temperature=0.0)
    got = amk.generate(target, prompt, 15, draft=draft, n_draft=3, temperature=0.0)
    assert len(got) == 15 and got[0] == want[0]
    with pytest.raises(amk.AmkError):
        amk.generate(here, prompt, 3, draft=draft)
    for d in (target, draft, here):
        d.close()


# ---- sliding window ------------------------------------------------------------------

class WindowedModel:
    """The decoder in 64-bit numpy over all tokens at once, with a window and
    sinks (the oracle has none); shared by the single- and multi-token paths."""

    def __init__(self, cfg, w, window, sinks):
        self.cfg, self.window, self.sinks = cfg, window, sinks
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        self.w = {k: [f(t) for t in v] if isinstance(v, list) else f(v)
                  for k, v in w.items() if v is not None}

    def logits(self, toks):
        c, w, n = self.cfg, self.w, len(toks)

        def norm(x, g):
            return x / np.sqrt((x * x).mean(-1, keepdims=True) + c.rms_eps) * g

        half = c.head_dim // 2
        ang = np.arange(n)[:, None] * c.rope_theta ** (-np.arange(half) / half)
        cs, sn = np.cos(ang)[:, None], np.sin(ang)[:, None]

        def rope(x):
            a, b = x[..., :half], x[..., half:]
            return np.concatenate((a * cs - b * sn, b * cs + a * sn), -1)

        i, j = np.arange(n)[:, None], np.arange(n)
        seen = (j <= i) & ((j > i - self.window) | (j < self.sinks))
        bf = lambda x: torch.tensor(x).to(torch.bfloat16).double().numpy()  # noqa: E731
        x = w["embed"][toks]
        for l in range(c.n_layers):
            h = norm(x, w["attn_norm"][l])
            q = rope((h @ w["wq"][l].T).reshape(n, c.n_heads, c.head_dim))
            k = bf(rope((h @ w["wk"][l].T).reshape(n, c.n_kv_heads, c.head_dim)))
            v = bf((h @ w["wv"][l].T).reshape(n, c.n_kv_heads, c.head_dim))
            g = c.n_heads // c.n_kv_heads
            o = np.empty_like(q)
            for a in range(c.n_heads):
                s = q[:, a] @ k[:, a // g].T / math.sqrt(c.head_dim)
                s = np.where(seen, s, -np.inf)
                p = np.exp(s - s.max(1, keepdims=True))
                o[:, a] = p / p.sum(1, keepdims=True) @ v[:, a // g]
            x = x + o.reshape(n, -1) @ w["wo"][l].T
            h = norm(x, w["ffn_norm"][l])
            z = h @ w["wgate"][l].T
            x = x + (z / (1 + np.exp(-z)) * (h @ w["wup"][l].T)) @ w["wdown"][l].T
        head = w["embed"] if c.tied else w["lm_head"]
        return norm(x, w["final_norm"]) @ head.T


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (5, 3), (16, 1), (40, 4), (7, 100),
                                          (200, 2), (70, 33)])
def test_window_and_sinks(window, sinks):
    """Single- and multi-token steps of a handle with a window: against 64 bits,
    a step to the bf16 step tolerance, across several attention chunks."""
    cfg = TINY.with_(max_ctx=160)
    w = si.make_model(cfg, device="cuda")
    toks = si.make_prompt(cfg, 150)
    want = WindowedModel(cfg, w, window, sinks).logits(toks)
    lg = torch.empty(cfg.vocab, device="cuda")
    for flagged in (1, -1):
        dec = amk.Decoder(cfg, w, options=amk.default_options(
            attn_window=window, attn_sinks=sinks, flagged_waits=flagged, debug_checks=1))
        for p, t in enumerate(toks):
            dec.step(t, p, logits=lg)
            err = np.abs(lg.double().cpu().numpy() - want[p]).max() / np.abs(want[p]).max()
            assert err <= 0.5 * 1e-2, f"step {p}: {err:.3g}"
        dec.reset()
        got = dec.extend(toks[:101], 0, n_logits=101)
        for p in range(101):
            close(cfg, got[p], want[p], f"extend {p}")
        dec.step(toks[101], 101, logits=lg)
        close(cfg, lg, want[101], "step 101 behind extend")
        got = dec.extend(toks[102:], 102, n_logits=48)
        for i in range(48):
            close(cfg, got[i], want[102 + i], f"extend {102 + i}")
        assert dec.check_guards() == 0
        dec.close()


def test_window_of_the_no_allocation_step():
    cfg = TINY.with_(max_ctx=96)
    w = si.make_model(cfg, device="cuda")
    toks = si.make_prompt(cfg, 90)
    want = WindowedModel(cfg, w, 11, 2).logits(toks)
    plan = amk.Plan(cfg, torch.cuda.get_device_properties(0).multi_processor_count,
                    amk.default_options(attn_window=11, attn_sinks=2))
    ws, keep = amk.weights_struct(cfg, w)
    kv = torch.zeros((cfg.n_layers, 2, cfg.n_kv_heads, cfg.max_ctx, cfg.head_dim),
                     dtype=torch.bfloat16, device="cuda")
    lg = torch.empty(cfg.vocab, device="cuda")
    for p, t in enumerate(toks):
        amk.decode_step_noalloc(plan, ws, kv, t, p, lg, want_argmax=True)
        err = np.abs(lg.double().cpu().numpy() - want[p]).max() / np.abs(want[p]).max()
        assert err <= 0.5 * 1e-2, f"step {p}: {err:.3g}"
    plan.close()


def test_window_refusals():
    with pytest.raises(amk.AmkError):
        amk.Plan(TINY, 148, amk.default_options(attn_window=-1))
    with pytest.raises(amk.AmkError):
        amk.Plan(TINY, 148, amk.default_options(attn_window=4, attn_sinks=-1))


def test_tokens_are_read_before_the_call_returns():
    dec, _, _ = pair(TINY)
    toks = si.make_prompt(TINY, 24)
    want = dec.extend(toks, 0, n_logits=24).clone()
    pinned = torch.tensor(toks, dtype=torch.int32).pin_memory()
    got = torch.empty((24, TINY.vocab), device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)  # some 10 ms of work before it on the stream
    at = ctypes.cast(pinned.data_ptr(), ctypes.POINTER(ctypes.c_int32))
    assert amk.abi.lib().amk_extend(dec._h, at, 24, 0, 24, got.data_ptr()) == 0
    pinned.fill_(0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
