"""Steps of a handle with a window, in every instance of the kernel: weight formats, lane widths,
the generic one and the one without flagged waits, against the multi-token step on the same rows
(tolerance: tests/test_gpu_extend.py), before and behind the row from which the window moves on."""
import pytest
import torch

import persistent_megakernel_decode_cta_b200 as amk
import synth_inputs as si
from tests.test_gpu_extend import close

pytestmark = pytest.mark.gpu

TINY = si.get_config("tiny").with_(max_ctx=96)
MODELS = {
    "bf16": TINY, "w8a16": TINY.with_(quant="w8a16"), "w4a16": TINY.with_(quant="w4a16", ffn=192),
    "tied int8": TINY.with_(quant="w8a16", tied=True),
    "heads of 8": TINY.with_(n_heads=4, n_kv_heads=4, head_dim=8),
    "heads of 128": TINY.with_(hidden=256, n_heads=4, n_kv_heads=2, head_dim=128, ffn=512),
    "int8 heads of 128": TINY.with_(hidden=256, n_heads=4, n_kv_heads=1, head_dim=128, ffn=512,
                                    quant="w8a16"),
    "int4 heads of 64": TINY.with_(hidden=256, n_heads=8, n_kv_heads=1, head_dim=64, ffn=512,
                                   quant="w4a16"),
}


@pytest.fixture(autouse=True)
def _cuda(cuda_ok):
    pass


@pytest.mark.parametrize("flagged", [1, -1])
@pytest.mark.parametrize("name", MODELS)
def test_windowed_steps_agree_with_extend(name, flagged):
    cfg = MODELS[name]
    w = si.make_model(cfg, seed=3, device="cuda")
    toks = si.make_prompt(cfg, 90)
    for window, sinks in ((7, 0), (20, 3), (33, 40)):
        dec = amk.Decoder(cfg, w, options=amk.default_options(
            attn_window=window, attn_sinks=sinks, flagged_waits=flagged, debug_checks=1))
        steps = torch.empty((len(toks), cfg.vocab), device="cuda")
        for p, t in enumerate(toks):
            dec.step(t, p, logits=steps[p])
        assert dec.check_guards() == 0
        dec.reset()
        got = dec.extend(toks, 0, n_logits=len(toks))
        for p in range(len(toks)):
            close(cfg, got[p], steps[p].double().cpu().numpy(), f"{name} {window} {sinks} {p}")
        dec.close()
