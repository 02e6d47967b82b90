"""Token generation with a Decoder: a prompt by the multi-token step, then
sampling or speculative decoding.

Speculative decoding: a draft Decoder proposes a few tokens by single-token
steps, the target runs them (with the token before them) in one multi-token
step -- its weights are read once for all of them --, and amk_verify_draft takes
as many as leave the target's distribution what it is, plus one token of its
own.  The host reads the proposed tokens and the verdict; logits stay on the
device.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

from . import AmkError, Decoder, abi
from .ops import verify_draft

__all__ = ["generate"]


def generate(target: Decoder, prompt: Sequence[int], n_new: int, *,
             draft: Optional[Decoder] = None, n_draft: int = 4, temperature: float = 1.0,
             generator=None) -> List[int]:
    """``n_new`` tokens behind ``prompt`` (at least one token), sampled from the
    target's distribution at ``temperature`` (0: greedy).  ``draft``: a Decoder
    of the same vocabulary on the same stream that proposes ``n_draft`` tokens
    at a time; without one each token is a step of its own.  ``generator``: a
    torch CUDA generator of the random numbers.  Both decoders' caches are
    written from position 0 on."""
    import torch
    invalid = abi.ERR["AMK_ERR_INVALID_ARG"]
    seq = [int(t) for t in prompt]
    if not seq or n_new < 0 or not 0 <= n_draft <= 64:
        raise AmkError(invalid, "generate: an empty prompt, n_new < 0 or n_draft outside [0, 64]")
    decoders = [target] if draft is None else [target, draft]
    for d in decoders:
        if len(seq) + n_new > d.cfg.max_ctx + 1:  # the last new token is not run
            raise AmkError(abi.ERR["AMK_ERR_POS_RANGE"],
                           f"generate: {len(seq) + n_new} tokens, a cache of {d.cfg.max_ctx} rows")
    if draft is not None and (draft.cfg.vocab != target.cfg.vocab or
                              draft.stream != target.stream):
        raise AmkError(invalid, "generate: draft and target differ in vocabulary or stream")
    # the operators run on the decoders' stream
    stream = target.stream if target.stream != torch.cuda.current_stream().cuda_stream else None
    vocab, total = target.cfg.vocab, len(seq) + n_new
    # what the decoders write comes from their stream's pool: work that is pending
    # on torch's stream, or starts there after an error, never shares its memory
    with torch.cuda.stream(torch.cuda.ExternalStream(target.stream) if target.stream
                           else torch.cuda.default_stream()):
        logits = torch.empty((n_draft + 1, vocab), device="cuda")
        proposed = torch.empty((max(n_draft, 1), vocab), device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")

    def uniform(n):
        u = torch.rand(n, device="cuda", generator=generator)
        return u.clamp_(max=1 - 2.0**-24)  # [0, 1)

    def settle():  # torch's own writes (random numbers, tokens) before the decoders' stream
        if stream is not None:
            torch.cuda.current_stream().synchronize()

    def sample(rows, drafted, drafted_logits):
        u = uniform(len(drafted) + 1)
        settle()
        tokens, n = verify_draft(rows, drafted, u, draft_logits=drafted_logits,
                                 temperature=temperature, stream=stream)
        if stream is not None:
            torch.cuda.synchronize()
        return tokens.tolist(), int(n)

    for d in decoders:
        d.extend(seq[:-1], 0, n_logits=0)
    cached = len(seq) - 1  # tokens of seq in the target's cache; one is always left
    drafted_to = cached    # ... in the draft's
    while len(seq) < total:
        k = 0 if draft is None else min(n_draft, total - len(seq) - 1)
        if k == 0:
            target.step(seq[-1], cached, logits=logits[0], want_argmax=False)
            new, n = sample(logits[:1], none, None)
        else:
            if drafted_to < cached:
                draft.extend(seq[drafted_to:cached], drafted_to, n_logits=0)
            token, tokens = seq[-1], []
            for i in range(k):
                draft.step(token, cached + i, logits=proposed[i], want_argmax=False)
                token = sample(proposed[i:i + 1], none, None)[0][0]
                if token < 0:  # the draft has no distribution here: verify what there is
                    break
                tokens.append(token)
            k = len(tokens)
            target.extend([seq[-1], *tokens], cached, logits=logits[:k + 1])
            new, n = sample(logits[:k + 1], torch.tensor(tokens, dtype=torch.int32, device="cuda"),
                            proposed[:k])
            # the draft has run seq[-1] and its proposals but the last
            drafted_to = cached + min(n + 1, max(k, 1))
        if new[n] < 0:
            raise AmkError(invalid, "generate: the target's logits are not finite")
        seq += new[:n + 1]
        cached += n + 1
    return seq[len(prompt):]
