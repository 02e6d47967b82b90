"""Generation and the multi-token step on the GPU where a caller's other work, streams or model
shapes could go wrong."""
import pytest
import torch

import persistent_megakernel_decode_cta_b200 as amk
import synth_inputs as si
from tests.test_gpu_extend import tol

pytestmark = pytest.mark.gpu

TINY = si.get_config("tiny")


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    pass


@pytest.mark.parametrize("n_draft", [0, 3])
@pytest.mark.parametrize("own", [True, False])  # a stream of the decoders' own, or the default one
def test_generation_beside_pending_work(n_draft, own):
    """Work is queued on torch's stream that still writes memory which is free again."""
    w = si.make_model(TINY, seed=0, device="cuda")
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    stream = side.cuda_stream if own else torch.cuda.default_stream().cuda_stream
    target = amk.Decoder(TINY, w, stream=stream)
    draft = amk.Decoder(TINY, w, stream=stream) if n_draft else None
    prompt = si.make_prompt(TINY, 5)

    def run(pending):
        with torch.cuda.stream(other):
            if pending:
                blocks = [torch.empty((n, TINY.vocab), device="cuda")
                          for n in (n_draft + 1, max(n_draft, 1)) for _ in range(4)]
                torch.cuda._sleep(20_000_000)  # some 10 ms
                for b in blocks:
                    b.fill_(0).select(1, 3).fill_(1e30)  # token 3 wherever it is read as logits
                del blocks, b
            return amk.generate(target, prompt, 15, draft=draft, n_draft=n_draft, temperature=0.0)

    want = run(False)
    for _ in range(3):
        assert run(True) == want
    target.close()
    if draft:
        draft.close()


def test_generation_that_fails_leaves_the_decoders_usable():
    w = si.make_model(TINY, seed=0, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    target = amk.Decoder(TINY, w, stream=side.cuda_stream)
    prompt = si.make_prompt(TINY, 5)
    want = amk.generate(target, prompt, 10, temperature=0.0)
    with pytest.raises(amk.AmkError):
        amk.generate(target, prompt, 10, temperature=-1.0)
    assert amk.generate(target, prompt, 10, temperature=0.0) == want
    target.close()


def test_extend_refuses_wide_heads_before_it_changes_anything():
    """The single-token step takes heads of 512, the attention over several tokens up to 256."""
    cfg = TINY.with_(hidden=512, n_heads=2, n_kv_heads=2, head_dim=512, max_ctx=16)
    dec = amk.Decoder(cfg, si.make_model(cfg, device="cuda"))
    dec.step(1, 0)
    before = [t.clone() for layer in range(cfg.n_layers) for t in dec.kv(layer)]
    with pytest.raises(amk.AmkError, match="UNSUPPORTED"):
        dec.extend([2, 3, 4], 0)
    torch.cuda.synchronize()
    after = [t for layer in range(cfg.n_layers) for t in dec.kv(layer)]
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    dec.step(-1, 1)  # the token that the step before chose
    dec.close()
    cfg = TINY.with_(hidden=256, n_heads=2, n_kv_heads=1, head_dim=256, max_ctx=16)
    dec = amk.Decoder(cfg, si.make_model(cfg, device="cuda"))
    assert torch.isfinite(dec.extend([2, 3, 4], 0, n_logits=3)).all()
    dec.close()


def test_two_decoders_at_once():
    """Multi-token steps, and single ones between them, of two handles that overlap on the GPU."""
    cfgs = [TINY.with_(max_ctx=600), TINY.with_(quant="w8a16", max_ctx=600)]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    decs, toks = [], []
    for cfg, side in zip(cfgs, sides):
        w = si.make_model(cfg, seed=4, device="cuda")
        torch.cuda.synchronize()
        decs.append(amk.Decoder(cfg, w, stream=side.cuda_stream))
        toks.append(si.make_prompt(cfg, 560))

    def run(i, out):
        out.append(decs[i].extend(toks[i][:500], 0, n_logits=30))
        for p in range(500, 540, 10):
            out.append(decs[i].extend(toks[i][p:p + 9], p, n_logits=9))
            lg = torch.empty(cfgs[i].vocab, device="cuda")
            decs[i].step(toks[i][p + 9], p + 9, logits=lg, want_argmax=False)
            out.append(lg)

    want = [[], []]
    for i in (0, 1):
        run(i, want[i])
        torch.cuda.synchronize()
    for _ in range(5):
        got = [[], []]
        torch.cuda.synchronize()
        for i in (0, 1):
            run(i, got[i])
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    for d in decs:
        d.close()


@pytest.mark.parametrize("n_draft", [0, 1, 3, 8])
@pytest.mark.parametrize("same", [True, False])
def test_every_greedy_token_is_the_largest_behind_its_own_prefix(n_draft, same):
    """All positions, each behind the tokens that were generated before it.  Two logits of the
    multi-token step are each off by a nearly normal error of tol() rms of the logits' own, their
    difference by sqrt(2) of that: none of the 160 that are looked at is beyond six times it."""
    w = si.make_model(TINY, seed=0, device="cuda")
    target = amk.Decoder(TINY, w)
    draft = amk.Decoder(TINY, w if same else si.make_model(TINY, seed=1, device="cuda"))
    prompt = si.make_prompt(TINY, 6)
    got = amk.generate(target, prompt, 20, draft=draft if n_draft else None, n_draft=n_draft,
                       temperature=0.0)
    target.reset()
    lg = torch.empty(TINY.vocab, device="cuda")
    for p, t in enumerate([*prompt, *got[:-1]]):
        target.step(t, p, logits=lg)
        if p >= len(prompt) - 1:
            token = got[p - len(prompt) + 1]
            behind = float(lg.max() - lg[token])
            assert behind <= 6 * 2**0.5 * tol(TINY) * float(lg.square().mean().sqrt()), (p, token)
    target.close()
    draft.close()
