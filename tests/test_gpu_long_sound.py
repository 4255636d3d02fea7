"""Calls of the operators of long contexts whose results hang on an order between
warps or CTAs, and ways out of a wait.  Plain forms and tolerances are those of
the operators' own tests."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla
    from test_gpu_evict import SCALE, Weights


@pytest.mark.parametrize("heads,sq,page", [(16, 1, 64), (40, 2, 32), (128, 1, 16), (128, 3, 64), (128, 8, 256)])
def test_key_weights_of_e4m3_rows_are_those_of_the_same_rows_in_bf16(heads, sq, page):
    # The codes are expanded without rounding and the products and sums are taken
    # alike: the same bits, whichever warps of whichever CTA expanded a key.
    rng = np.random.default_rng(heads + sq)
    w = Weights([int(x) for x in rng.integers(1, 2500, 24)], heads, sq, page, True, seed=heads + sq)
    scale = SCALE * w.pages.kv_scale
    codes = w.pages.cache
    wide = torch.where(codes.view(torch.uint8) & 0x7F == 0x7F, float("nan"), codes.float()).bfloat16()
    got = {}
    for name, cache in (("bf16", wide), ("e4m3", codes)):
        for i in range(4):
            out = torch.zeros_like(w.weights)
            mla.key_weights(w.q_abs, w.q_pe, cache, w.pages.table, w.seq_lens, w.lse, out, scale=scale,
                            query_start_loc=w.qsl, decay=0.0, status=w.status)
            torch.cuda.synchronize()
            assert w.status.item() == 0
            assert torch.equal(got.setdefault("bf16", out), out), (name, i)
    w.weights = got["bf16"]
    w.old, w.decay = torch.zeros_like(w.weights), 0.0
    w.check()
