"""Generation and the multi-token step on the GPU where a caller's other work, streams or model
shapes could go wrong."""
import pytest
import torch

import persistent_megakernel_decode_cta_b200 as amk
import synth_inputs as si

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
