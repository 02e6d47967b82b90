"""generate() on decoders whose stream is not torch's current one, on the host with stand-ins for
the decoders, the verification and torch's streams: what a stream writes was allocated from its own
pool, or the pool's stream was waited for in between."""
import contextlib
import types

import pytest
import torch

from persistent_megakernel_decode_cta_b200 import speculative

CURRENT, OWN, VOCAB = 7, 5, 11


class Streams:
    """Which stream is current, and where each tensor was allocated."""

    def __init__(self, monkeypatch):
        self.now, self.settled, self.pool, self.writes = CURRENT, {}, [], []
        cuda = types.SimpleNamespace(
            current_stream=lambda *a: types.SimpleNamespace(
                cuda_stream=self.now, synchronize=lambda s=self.now: self.wait(s)),
            default_stream=lambda *a: types.SimpleNamespace(cuda_stream=0),
            ExternalStream=lambda s, **k: types.SimpleNamespace(cuda_stream=s),
            stream=self.under, synchronize=lambda *a: [self.wait(s) for s in (CURRENT, OWN)])
        monkeypatch.setattr(torch, "cuda", cuda)
        for name in ("empty", "rand", "tensor"):
            monkeypatch.setattr(torch, name, self.allocating(getattr(torch, name)))

    @contextlib.contextmanager
    def under(self, s):
        before, self.now = self.now, s.cuda_stream
        yield
        self.now = before

    def allocating(self, fn):
        def new(*args, **kw):
            kw.pop("device", None)
            kw.pop("generator", None)
            t = fn(*args, **kw)
            self.settled.setdefault(self.now, set())
            self.pool.append((t.untyped_storage().data_ptr(), t.untyped_storage().nbytes(),
                              self.now, t))
            return t
        return new

    def wait(self, stream):
        self.settled[stream] = {p for p, _, s, _ in self.pool if s == stream}

    def write(self, t, stream):
        at = t.data_ptr()
        for start, size, pool, _ in reversed(self.pool):
            if start <= at < start + max(size, 1):
                assert pool == stream or start in self.settled.get(pool, ()), \
                    f"stream {stream} writes memory of stream {pool}'s pool before waiting for it"
                self.writes.append(at)
                return
        raise AssertionError("a buffer from nowhere")


class StandIn:
    def __init__(self, streams, stream):
        self.streams, self.stream = streams, stream
        self.cfg = types.SimpleNamespace(vocab=VOCAB, max_ctx=64)

    def step(self, token, pos, logits=None, want_argmax=True):
        self.streams.write(logits, self.stream)

    def extend(self, tokens, pos, logits=None, n_logits=None):
        if logits is not None and n_logits != 0:
            self.streams.write(logits, self.stream)


@pytest.mark.parametrize("drafted", [False, True])
def test_buffers_belong_to_the_decoders_stream(monkeypatch, drafted):
    streams = Streams(monkeypatch)
    ones = torch.ones

    def verify(rows, tokens, u, **kw):
        return ones(len(tokens) + 1, dtype=torch.int32), ones(1, dtype=torch.int32) * len(tokens)

    monkeypatch.setattr(speculative, "verify_draft", verify)
    target = StandIn(streams, OWN)
    draft = StandIn(streams, OWN) if drafted else None
    assert speculative.generate(target, [1, 2, 3], 9, draft=draft, n_draft=3) == [1] * 9
    assert streams.writes
