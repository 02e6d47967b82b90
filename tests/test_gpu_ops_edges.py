"""The operators of the multi-token step on the GPU, at the edges of their variants, limits and
entry points (64-bit forms and tolerances: tests/ops_oracle.py)."""
import os
import subprocess
import sys

import pytest
import torch

import persistent_megakernel_decode_cta_b200 as amk
from tests import ops_oracle as oo
from tests.test_gpu_ops import BF16, close, gen, randn, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    torch.backends.cuda.matmul.allow_tf32 = False


# int8 weights with bf16 results and many tiles: 192 tokens to a tile, a ring of three stages
@pytest.mark.parametrize("m,n,k,gated", [(192, 18944, 1024, False), (576, 6272, 2048, False),
                                         (1000, 1408, 2048, True), (1111, 4000, 656, True)])
def test_linear_three_stage_ring(m, n, k, gated):
    x = randn(gen(m), m, k, dtype=BF16)
    w, s = weights("int8", n, k, m)
    kw = {"scale": s, "act": "silu"}
    if gated:
        kw["up"], kw["up_scale"] = weights("int8", n, k, m + 1)
    first = amk.linear(x, w, **kw)
    want, tol = oo.linear(x, w, **kw)
    close(first, want, tol, f"{m}x{n}x{k}")
    for _ in range(100):
        assert torch.equal(amk.linear(x, w, **kw), first)


def test_the_count_of_timeouts_waits_for_every_stream():
    amk.ops_timeouts()  # (a first call loads code, which may wait by itself)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # some 100 ms
        done = torch.cuda.Event()
        done.record()
    assert amk.ops_timeouts() == 0
    assert done.query()


def test_linear_as_many_rows_as_there_can_be():
    """Row indexes up to 2^31 - 2, through the kernel for any alignment (4 GB of x, and of y)."""
    m = 2**31 - 1
    x = torch.empty(m, 1, dtype=BF16, device="cuda").random_(0, 100, generator=gen(0))
    w = torch.tensor([[3.0]], dtype=BF16, device="cuda")
    y = amk.linear(x, w)
    torch.cuda.synchronize()
    step = 1 << 28
    for i in range(0, m, step):  # whole numbers up to 297: rounded once, as by torch
        assert torch.equal(y[i:i + step], (x[i:i + step].float() * 3).to(BF16))


FIRST_CALLS_CAPTURED = """
import torch
import persistent_megakernel_decode_cta_b200 as amk
from tests.test_gpu_ops import BF16, gen, randn, draft_case
x, w = randn(gen(0), 300, 256, dtype=BF16), randn(gen(1), 384, 256, std=0.1, dtype=BF16)
q, kv = randn(gen(2), 200, 32, 64, dtype=BF16), randn(gen(3), 4, 900, 64, dtype=BF16)
odd = randn(gen(4), 4, 900, 7, dtype=BF16)
target, draft, tok, u = draft_case(3, 5000, 5)
def calls():
    return [amk.linear(x, w), amk.linear(x[:3], w), amk.linear(x[:, 1:250], w[:, :249].contiguous()),
            amk.attention(q, kv, kv, 600), amk.attention(q[:2], kv, kv, 800),
            amk.attention(q[:2, :, :7], odd, odd, 800),
            *amk.verify_draft(target, tok, u, draft_logits=draft)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
assert amk.ops_timeouts() == 0
print("captured")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    """Nothing that a first call sets up (code, limits, device facts) upsets a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], cwd=root, timeout=300,
                         capture_output=True, text=True)
    assert run.returncode == 0 and "captured" in run.stdout, run.stderr[-2000:]
