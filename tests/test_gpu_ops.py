"""The operators of the multi-token step on the GPU, against their 64-bit forms
(tests/ops_oracle.py, where the tolerances are derived)."""
import math

import pytest
import torch

import persistent_megakernel_decode_cta_b200 as amk
import synth_inputs as si
from tests import ops_oracle as oo

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    torch.backends.cuda.matmul.allow_tf32 = False


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def weights(fmt, n, k, seed):
    if fmt == "bf16":
        return randn(gen(seed), n, k, std=0.02, dtype=BF16), None
    fn = si._int8_rows if fmt == "int8" else si._int4_groups
    return fn((n, k), "cuda", seed, "w")


def close(got, want, tol, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{(err / tol)[bad].max():.3g} of the tolerance, first at "
                           f"{bad.nonzero()[0].tolist()}")


# ---- matrix product ------------------------------------------------------------

def check_linear(m, n, k, fmt, seed=0, bias=False, act="none", gated=False, residual=None,
                 out_dtype=BF16):
    g = gen(seed + 1)
    x = randn(g, m, k, dtype=BF16)
    w, s = weights(fmt, n, k, seed)
    kw = {"scale": s, "act": act}
    if bias:
        kw["bias"] = randn(g, n, dtype=BF16)
    if gated:
        kw["up"], kw["up_scale"] = weights(fmt, n, k, seed + 7)
        if bias:
            kw["up_bias"] = randn(g, n, dtype=BF16)
    if residual is not None:
        kw["residual"] = randn(g, m, n, dtype=residual)
    y = amk.linear(x, w, out_dtype=out_dtype, **kw)
    assert y.dtype == out_dtype and y.shape == (m, n)
    want, tol = oo.linear(x, w, out_dtype=out_dtype, **kw)
    close(y, want, tol, f"linear {m}x{n}x{k} {fmt}")


FORMATS = ["bf16", "int8", "int4"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 257])
def test_linear_rows(m, fmt):
    check_linear(m, 192, 256, fmt, seed=m, out_dtype=F32)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,k", [(1, 32), (3, 64), (64, 96), (127, 128), (128, 160), (129, 192),
                                 (576, 576), (500, 1536), (2048, 2048), (172, 64)])
def test_linear_sizes(n, k, fmt):
    for m in (1, 19):
        check_linear(m, n, k, fmt, seed=n + k, residual=F32, out_dtype=F32)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("k", [2, 8, 34, 172, 250, 1022])
def test_linear_unaligned_inputs(k, fmt):
    # rows that do not start at multiples of 16 bytes
    for m, n in ((1, 7), (70, 65)):
        check_linear(m, n, k, fmt, seed=k, bias=True, act="relu")


@pytest.mark.parametrize("k", [1, 3, 63, 129])
def test_linear_odd_inputs(k):
    check_linear(5, 9, k, "bf16", seed=k, out_dtype=F32)
    check_linear(5, 9, k, "int8", seed=k, out_dtype=F32)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [1, 5, 40, 130, 300])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_epilogue(m, fmt, gated):
    for act in ("none", "silu", "gelu", "relu"):
        check_linear(m, 320, 384, fmt, seed=m, bias=True, act=act, gated=gated, residual=BF16)
    check_linear(m, 320, 384, fmt, seed=m, act="silu", gated=gated, residual=F32, out_dtype=F32)


@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_large(fmt):
    check_linear(1000, 1408, 2048, fmt, act="silu", gated=True)
    check_linear(1, 4096, 11008, fmt, residual=F32, out_dtype=F32)
    check_linear(515, 2048, 8192, fmt, residual=F32, out_dtype=F32)


def test_linear_strided_rows_and_in_place_residual():
    g = gen(3)
    big = randn(g, 21, 512, dtype=BF16)
    x = big[:, 64:320]
    w, _ = weights("bf16", 96, 256, 3)
    res = randn(g, 21, 160)
    keep = res.clone()
    out = res[:, 32:128]
    want, tol = oo.linear(x, w, residual=out.clone(), out_dtype=F32)
    y = amk.linear(x, w, residual=out, out=out)
    assert y is out
    close(out, want, tol)
    assert torch.equal(res[:, :32], keep[:, :32]) and torch.equal(res[:, 128:], keep[:, 128:])
    # a base and a row stride off the 16-byte grid
    for x in (big[:, 3:259], randn(g, 21, 257, dtype=BF16)[:, :256]):
        want, tol = oo.linear(x, w)
        close(amk.linear(x, w), want, tol)


def test_linear_leading_dimensions_and_empty():
    g = gen(4)
    x = randn(g, 2, 3, 64, dtype=BF16)
    w, _ = weights("bf16", 48, 64, 4)
    y = amk.linear(x, w)
    assert y.shape == (2, 3, 48)
    want, tol = oo.linear(x.view(6, 64), w)
    close(y.view(6, 48), want, tol)
    assert amk.linear(x[:0], w).shape == (0, 3, 48)
    v = amk.linear(x[0, 0], w)
    assert v.shape == (48,) and torch.equal(v, amk.linear(x[0, :1], w)[0])


def test_linear_non_finite_inputs_stay_in_their_rows():
    g = gen(5)
    x = randn(g, 40, 256, dtype=BF16)
    w, _ = weights("bf16", 130, 256, 5)
    clean = amk.linear(x, w)
    x[7, 3] = math.inf
    x[9, 200] = math.nan
    y = amk.linear(x, w)
    rows = [i for i in range(40) if i not in (7, 9)]
    assert torch.equal(y[rows], clean[rows])
    assert not torch.isfinite(y[7].float()).any() and torch.isnan(y[9].float()).all()


@pytest.mark.parametrize("fmt,k", [("bf16", 4104), ("int8", 4112), ("int8", 5616), ("int4", 4128),
                                   ("int4", 10976)])
def test_linear_few_tokens_over_long_ragged_rows(fmt, k):
    # rows that end inside a step, behind many whole ones
    for m in (1, 5, 8, 9, 16):
        check_linear(m, 200, k, fmt, seed=m + k, gated=m % 2 == 1, out_dtype=F32)
    x = randn(gen(k), 11, k, dtype=BF16)
    w, s = weights(fmt, 200, k, k)
    clean = amk.linear(x, w, scale=s)
    x[10, k - 1] = math.nan  # the last token, whose row stands in for those behind it
    x[3, 0] = math.inf
    y = amk.linear(x, w, scale=s)
    rows = [i for i in range(11) if i not in (3, 10)]
    assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[10].float()).all()


def test_linear_repeats_bit_for_bit():
    g = gen(6)
    for m in (1, 12, 300):
        x = randn(g, m, 2048, dtype=BF16)
        for fmt in FORMATS:
            w, s = weights(fmt, 640, 2048, 6)
            a = amk.linear(x, w, scale=s, out_dtype=F32)
            for _ in range(3):
                assert torch.equal(a, amk.linear(x, w, scale=s, out_dtype=F32))


def test_linear_refuses_on_the_device():
    x = torch.zeros(2, 64, dtype=BF16, device="cuda")
    w = torch.zeros(8, 64, dtype=BF16, device="cuda")
    s = torch.ones(8, dtype=torch.float16, device="cuda")
    bad = [lambda: amk.linear(x.float(), w), lambda: amk.linear(x, w.float()),
           lambda: amk.linear(x, w[:, :63]), lambda: amk.linear(x, w, scale=s),
           lambda: amk.linear(x, w.to(torch.int8)), lambda: amk.linear(x, w, act="tanh"),
           lambda: amk.linear(x, w, up=w[:4]), lambda: amk.linear(x, w, up_bias=w[0]),
           lambda: amk.linear(x, w, bias=s), lambda: amk.linear(x, w, residual=x),
           lambda: amk.linear(x, w, out=torch.empty(2, 8, device="cuda", dtype=torch.float16)),
           lambda: amk.linear(x.t(), w), lambda: amk.linear(x, w.cpu()),
           lambda: amk.linear(x.clone().requires_grad_(), w)]
    for f in bad:
        with pytest.raises(amk.AmkError):
            f()


# ---- attention -----------------------------------------------------------------

def check_attention(T, pos, nh, nkv, hd, window=0, sinks=0, seed=0, rows=None, scale=None):
    g = gen(seed)
    rows = rows or pos + T + 5
    q = randn(g, T, nh, hd, dtype=BF16)
    k, v = randn(g, nkv, rows, hd, dtype=BF16), randn(g, nkv, rows, hd, dtype=BF16)
    # rows behind the last token are whatever the cache held
    k[:, pos + T:], v[:, pos + T:] = math.nan, math.inf
    out = amk.attention(q, k, v, pos, window=window, sinks=sinks, scale=scale)
    want, tol = oo.attention(q, k, v, pos, window, sinks, scale)
    close(out, want, tol, f"attention T {T} pos {pos} {nh}/{nkv}x{hd} w {window} s {sinks}")


HEADS = [(4, 2, 16), (9, 3, 64), (32, 4, 64), (8, 8, 128), (8, 1, 128), (6, 2, 96), (5, 5, 80),
         (4, 1, 256), (3, 1, 2), (2, 2, 7)]


@pytest.mark.parametrize("nh,nkv,hd", HEADS)
def test_attention_heads(nh, nkv, hd):
    for T, pos in ((1, 0), (1, 130), (3, 61), (40, 0), (150, 20)):
        check_attention(T, pos, nh, nkv, hd, seed=T)
        check_attention(T, pos, nh, nkv, hd, window=17, sinks=3, seed=T)


@pytest.mark.parametrize("T", [1, 2, 5, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_attention_lengths(T):
    for pos in (0, 1, 63, 64, 127, 128, 500):
        check_attention(T, pos, 6, 2, 64, seed=pos)
        check_attention(T, pos, 2, 2, 128, window=100, sinks=4, seed=pos)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 127, 128, 129, 400, 10**6])
@pytest.mark.parametrize("sinks", [0, 1, 5, 64, 130, 300])
def test_attention_masks(window, sinks):
    for T, pos in ((1, 700), (200, 300)):
        check_attention(T, pos, 4, 2, 64, window, sinks, seed=window + sinks)
    check_attention(70, 333, 2, 2, 128, window, sinks, seed=window + sinks)


@pytest.mark.parametrize("window", [500, 501, 2**30, 2**31 - 2, 2**31 - 1, 2**40])
@pytest.mark.parametrize("sinks", [0, 2**31 - 1, 2**40])
def test_attention_masks_beyond_the_last_row(window, sinks):
    for T, pos, nh, nkv, hd in ((1, 499, 4, 2, 64), (200, 300, 4, 2, 64), (200, 300, 32, 32, 64),
                                (3, 40, 2, 2, 7)):
        check_attention(T, pos, nh, nkv, hd, window, sinks, seed=sinks % 7)


@pytest.mark.parametrize("T,pos,heads,window,sinks", [
    (1, 20000, (32, 4, 64), 0, 0), (5, 32000, (32, 4, 64), 0, 0), (1, 9000, (32, 32, 128), 0, 0),
    (1, 30000, (9, 3, 64), 4096, 4), (700, 900, (8, 4, 128), 0, 0),
    (600, 3000, (9, 3, 64), 1024, 2), (2, 40000, (8, 8, 128), 20000, 64)])
def test_attention_long(T, pos, heads, window, sinks):
    check_attention(T, pos, *heads, window, sinks)


def test_attention_extreme_scores():
    """Large scores: the weights concentrate; and a scale of its own."""
    g = gen(11)
    q = randn(g, 33, 4, 64, std=30, dtype=BF16)
    k, v = randn(g, 2, 300, 64, std=30, dtype=BF16), randn(g, 2, 300, 64, dtype=BF16)
    for scale in (None, 1e-3):
        out = amk.attention(q, k, v, 200, scale=scale)
        want, tol = oo.attention(q, k, v, 200, scale=scale)
        close(out, want, tol)


@pytest.mark.parametrize("nh,nkv,hd", [(4, 2, 64), (2, 2, 128), (4, 2, 40)])
@pytest.mark.parametrize("T,pos", [(1, 90), (4, 90), (180, 90)])
def test_attention_masked_rows_hold_anything(nh, nkv, hd, T, pos):
    """NaN and infinities in rows that a token does not see do not reach it."""
    g = gen(12)
    q = randn(g, T, nh, hd, dtype=BF16)
    k, v = randn(g, nkv, 400, hd, dtype=BF16), randn(g, nkv, 400, hd, dtype=BF16)
    n = pos + T
    window, sinks = 33, 2
    k[:, n:], v[:, n:] = math.nan, math.nan
    for j in range(sinks, pos - window + 1):  # left of every window, not a sink
        k[:, j], v[:, j] = math.nan, math.inf
    out = amk.attention(q, k, v, pos, window=window, sinks=sinks)
    want, tol = oo.attention(q, k, v, pos, window, sinks)
    close(out, want, tol)
    if T > 100:  # rows that some of the tokens see poison those alone
        v[:, pos + 100] = math.nan
        k[:, pos + 20] = math.inf
        v[0, pos + 60, 1] = -math.inf
        out = amk.attention(q, k, v, pos, window=window, sinks=sinks).double()
        i = torch.arange(pos, n)
        for row in (100, 20, 60):
            p = pos + row
            hit = (i >= p) & (i < p + window)
            if row == 100:
                assert torch.isnan(out[hit]).all()
        clean = [t for t in range(T) if not any(
            pos + r <= pos + t < pos + r + window for r in (100, 20, 60))]
        kk, vv = k.clone(), v.clone()
        kk[:, pos + 20], vv[:, pos + 100], vv[0, pos + 60, 1] = 0, 0, 0
        want, tol = oo.attention(q, kk, vv, pos, window, sinks)
        close(out[clean], want[clean], tol[clean])


def test_attention_strides():
    g = gen(13)
    T, nh, nkv, hd, pos = 20, 4, 2, 64, 37
    qkv = randn(g, T, (nh + 2 * nkv) * hd, dtype=BF16)
    q = qkv[:, :nh * hd].view(T, nh, hd)
    k = randn(g, 80, nkv, 2 * hd, dtype=BF16).transpose(0, 1)[:, :, :hd]  # rows outside heads
    v = randn(g, nkv, 90, hd, dtype=BF16)[:, 4:84]
    out = torch.full((nh, T + 2, hd), 7.0, device="cuda", dtype=BF16)
    want, tol = oo.attention(q, k, v, pos, 16, 2)
    amk.attention(q, k, v, pos, window=16, sinks=2, out=out[:, :T].transpose(0, 1))
    close(out[:, :T].transpose(0, 1), want, tol)
    assert (out[:, T:] == 7).all()
    # a base off the 16-byte grid
    flat = randn(g, nkv * 80 * hd + 1, dtype=BF16)[1:].view(nkv, 80, hd)
    want, tol = oo.attention(q, flat, v, pos)
    close(amk.attention(q, flat, v, pos), want, tol)


def test_attention_refuses_on_the_device():
    q = torch.zeros(2, 4, 64, dtype=BF16, device="cuda")
    k = torch.zeros(2, 8, 64, dtype=BF16, device="cuda")
    bad = [lambda: amk.attention(q, k, k, 7), lambda: amk.attention(q, k, k, -1),
           lambda: amk.attention(q.float(), k, k, 0), lambda: amk.attention(q, k, k[:, :7], 0),
           lambda: amk.attention(q[:, :3], k, k, 0), lambda: amk.attention(q, k, k, 0, window=-1),
           lambda: amk.attention(q, k, k, 0, scale=0.0), lambda: amk.attention(q, k, k, 2**31),
           lambda: amk.attention(q, k, k.cpu(), 0),
           lambda: amk.attention(q, k, k, 0, out=q[:1]),
           lambda: amk.attention(q, k, k, 0, out=q[:1].expand(2, 4, 64))]
    for f in bad:
        with pytest.raises(amk.AmkError):
            f()
    assert amk.attention(q[:0], k, k, 8).shape == (0, 4, 64)


# ---- verification ---------------------------------------------------------------

def draft_case(d, vocab, seed, noise=0.7, std=2.5, temperature=1.0):
    g = gen(seed)
    target = randn(g, d + 1, vocab, std=std)
    draft = target[:d] + noise * randn(g, d, vocab)
    e = torch.rand(d, vocab, generator=g, device="cuda").clamp_(1e-20, 1)
    tok = (draft / max(temperature, 0.1) - (-e.log()).log()).argmax(1).int() if d else \
        torch.empty(0, dtype=torch.int32, device="cuda")
    return target, draft, tok, torch.rand(d + 1, generator=g, device="cuda")


def check_verify(target, tok, u, draft=None, temperature=1.0):
    got, n = amk.verify_draft(target, tok, u, draft_logits=draft, temperature=temperature)
    want, wn = oo.verify(target, tok, u, draft, temperature)
    assert (got.tolist(), n.tolist()) == (want, [wn])
    return wn


@pytest.mark.parametrize("vocab", [1, 2, 5, 63, 64, 257, 1000, 32000, 49152, 128256, 300001])
def test_verify_vocabularies(vocab):
    for d in (0, 1, 4, 9):
        for seed in range(3):
            target, draft, tok, u = draft_case(d, vocab, seed)
            check_verify(target, tok, u, draft)
            check_verify(target, tok, u, None, 0.8)
            check_verify(target, tok, u, draft, 0.0)


@pytest.mark.parametrize("d", [0, 1, 2, 3, 7, 8, 15, 16, 17, 40, 64])
def test_verify_counts(d):
    for seed in range(6):
        for noise in (0.05, 1.5):  # drafts that are mostly taken, and mostly not
            target, draft, tok, u = draft_case(d, 777, 100 + seed, noise=noise)
            check_verify(target, tok, u, draft)
            check_verify(target, tok, u, None)
            check_verify(target, tok, u, draft, 1.7)


def test_verify_agreement_takes_every_token():
    target, _, _, u = draft_case(6, 500, 1)
    tok = target[:6].argmax(1).int()
    assert check_verify(target, tok, u, target[:6].clone()) == 6
    assert check_verify(target, tok, u, None, 0.0) == 6


def test_verify_masked_and_tied_logits():
    inf = math.inf
    t = torch.full((3, 40), -inf, device="cuda")
    t[:, 5], t[:, 9], t[:, 30] = 1.0, 1.0, 0.0
    u = torch.tensor([0.5, 0.99, 0.3], device="cuda")
    tok = torch.tensor([9, 7], dtype=torch.int32, device="cuda")
    check_verify(t, tok, u, None)
    check_verify(t, tok, u, None, 0.0)   # ties: the lowest index
    draft = t[:2].clone()
    draft[0, 7] = 3.0                    # a token the target never takes
    check_verify(t, tok, u, draft)
    for x in (0.0, 0.25, 0.5, 0.999999, 1.0 - 2.0**-24):
        u[2] = x
        check_verify(t[:1], tok[:0], u[2:])
    # all of both distributions on one token, another one drafted: nothing is left but p
    t.fill_(-inf)
    t[:, 11] = 0.0
    check_verify(t, tok, u, t[:2].clone())
    check_verify(t, tok, u, None)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("row", [0, 2, 4])
def test_verify_rows_without_a_distribution(value, row):
    target, draft, tok, u = draft_case(4, 600, 5, noise=0.0)
    u.fill_(0.0)  # every token is accepted up to the row
    bad = target.clone()
    bad[row, 17] = value
    assert check_verify(bad, tok, u, draft) == row
    check_verify(bad, tok, u, None)
    check_verify(bad, tok, u, None, 0.0)
    bad = target.clone()
    bad[row] = -math.inf
    assert check_verify(bad, tok, u, draft) == row
    if row < 4:
        bad = draft.clone()
        bad[row, 3] = value
        assert check_verify(target, tok, u, bad) == row
    # behind the first rejection nothing matters
    bad = target.clone()
    bad[4] = math.nan
    u[0] = 0.999
    tok[0] = -1
    assert check_verify(bad, tok, u, draft) == 0


def test_verify_tokens_out_of_range_are_rejected():
    target, draft, tok, u = draft_case(3, 100, 6)
    u.fill_(0.0)
    for t in (-1, 100, 2**31 - 1, -2**31):
        tok[1] = t
        for temperature in (1.0, 0.0):
            assert check_verify(target, tok, u, draft, temperature) <= 1
            assert check_verify(target, tok, u, None, temperature) <= 1


def test_verify_strided_rows():
    target, draft, tok, u = draft_case(4, 999, 7)
    wide = torch.full((5, 2003), math.nan, device="cuda")
    wide[:, 1:1000] = target
    dwide = torch.full((4, 1001), math.nan, device="cuda")
    dwide[:, :999] = draft
    check_verify(wide[:, 1:1000], tok, u, dwide[:, :999])


def test_verify_samples_the_target_distribution():
    """Over an even grid of u the drawn tokens are the distribution itself."""
    g = gen(8)
    vocab, n = 12, 2000
    target = randn(g, 1, vocab)
    tok = torch.empty(0, dtype=torch.int32, device="cuda")
    us = (torch.arange(n, device="cuda") + 0.5) / n
    drawn = [amk.verify_draft(target, tok, us[i:i + 1])[0] for i in range(n)]
    count = torch.bincount(torch.cat(drawn).long(), minlength=vocab).double().cpu()
    p = torch.softmax(target[0].double(), 0).cpu()
    assert ((count / n - p).abs() <= 1.0 / n + 1e-7).all()  # each interval is cut at both ends


def test_verify_refuses_on_the_device():
    t = torch.zeros(3, 10, device="cuda")
    tok = torch.zeros(2, dtype=torch.int32, device="cuda")
    u = torch.zeros(3, device="cuda")
    bad = [lambda: amk.verify_draft(t.half(), tok, u), lambda: amk.verify_draft(t, tok.long(), u),
           lambda: amk.verify_draft(t, tok[:1], u), lambda: amk.verify_draft(t, tok, u[:2]),
           lambda: amk.verify_draft(t, tok, u, draft_logits=t),
           lambda: amk.verify_draft(t.t(), tok, u), lambda: amk.verify_draft(t[0], tok, u),
           lambda: amk.verify_draft(t, tok, u, temperature=-1.0),
           lambda: amk.verify_draft(t, tok, u.cpu())]
    for f in bad:
        with pytest.raises(amk.AmkError):
            f()


# ---- streams and graphs ------------------------------------------------------------

def test_operators_on_another_stream_and_in_a_graph():
    g = gen(20)
    x = randn(g, 9, 256, dtype=BF16)
    w, s = weights("int8", 128, 256, 20)
    q = randn(g, 9, 2, 64, dtype=BF16)
    kv = randn(g, 1, 64, 64, dtype=BF16)
    target, draft, tok, u = draft_case(3, 128, 20)
    y0 = amk.linear(x, w, scale=s)
    o0 = amk.attention(q, kv, kv, 40)
    t0 = amk.verify_draft(target, tok, u, draft_logits=draft)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    raw = side.cuda_stream
    y1 = amk.linear(x, w, scale=s, stream=raw)
    o1 = amk.attention(q, kv, kv, 40, stream=raw)
    t1 = amk.verify_draft(target, tok, u, draft_logits=draft, stream=raw)
    side.synchronize()
    assert torch.equal(y0, y1) and torch.equal(o0, o1)
    assert all(torch.equal(a, b) for a, b in zip(t0, t1))

    graphs = []
    for _ in range(2):  # two graphs of the same calls, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = (amk.linear(x, w, scale=s), amk.attention(q, kv, kv, 40),
                    *amk.verify_draft(target, tok, u, draft_logits=draft))
        graphs.append((graph, outs))
    for seed in (21, 22):
        x.copy_(randn(gen(seed), 9, 256, dtype=BF16))
        q.copy_(randn(gen(seed), 9, 2, 64, dtype=BF16))
        target.copy_(draft_case(3, 128, seed)[0])
        for graph, _ in graphs:
            graph.replay()
        want = (amk.linear(x, w, scale=s), amk.attention(q, kv, kv, 40),
                *amk.verify_draft(target, tok, u, draft_logits=draft))
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_operators_on_two_streams_at_once():
    """Calls that overlap on the GPU share nothing: each gives what it gives alone."""
    jobs = []
    for i in range(2):
        g = gen(30 + i)
        x = randn(g, (3, 300)[i], 1024, dtype=BF16)
        w, s = weights(("int4", "bf16")[i], 700, 1024, i)
        q = randn(g, (2, 150)[i], 8, 64, dtype=BF16)
        kv = randn(g, 2, 3000, 64, dtype=BF16)
        jobs.append((x, w, s, q, kv, draft_case(4, 5000, 40 + i)))

    def run(job, stream=None):
        x, w, s, q, kv, (target, draft, tok, u) = job
        return (amk.linear(x, w, scale=s, stream=stream),
                amk.attention(q, kv, kv, 2500, stream=stream),
                *amk.verify_draft(target, tok, u, draft_logits=draft, stream=stream))

    want = [run(j) for j in jobs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(run(jobs[i], sides[i].cuda_stream))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_views_of_one_buffer_and_a_leading_batch():
    """What a model hands over: q as a slice of a joint projection, the result
    into a slice of a wider buffer."""
    g = gen(50)
    n, nh, nkv, hd = 40, 4, 2, 64
    joint = randn(g, n, (nh + 2 * nkv) * hd, dtype=BF16)
    q = joint[:, :nh * hd].unflatten(1, (nh, hd))
    cache = randn(g, 2, nkv, 200, hd, dtype=BF16)
    wide = torch.zeros(n, 2 * nh * hd, dtype=BF16, device="cuda")
    out = wide[:, nh * hd:].unflatten(1, (nh, hd))
    want, tol = oo.attention(q, cache[0], cache[1], 100, 30, 2)
    assert amk.attention(q, cache[0], cache[1], 100, window=30, sinks=2, out=out) is out
    close(out, want, tol)
    assert (wide[:, :nh * hd] == 0).all()
    w, _ = weights("bf16", 96, nh * hd, 50)
    y = amk.linear(wide[:, nh * hd:], w, act="silu")
    want, tol = oo.linear(wide[:, nh * hd:], w, act="silu")
    close(y, want, tol)


def test_no_operator_gave_up_a_wait():
    torch.cuda.synchronize()
    assert amk.ops_timeouts() == 0
