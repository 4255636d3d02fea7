"""Waits that run out in long decodes: the first cache tile never comes, with
hundreds of tiles and many units behind it, whose loads must stop where the CTA
gives up.  Each call returns promptly with the status, and the next one is right."""
import time

import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla
    from gpu_case import GpuCase, compare
    from test_gpu_shared import Case


def give_up(call, limit_ns=2_000_000):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    try:
        mla.set_decode_wait_test(True, limit_ns)
        call()
        torch.cuda.synchronize()
    finally:
        mla.set_decode_wait_test(False, 0)
    return time.perf_counter() - t0


@pytest.mark.parametrize("limit_ns", [300_000, 2_000_000])
@pytest.mark.parametrize("cache_dtype,heads,splits", [("bf16", 128, 0), ("fp8", 128, 0), ("bf16", 16, 0), ("fp8", 16, 7),
                                                      ("bf16", 128, 9)])
def test_decode(cache_dtype, heads, splits, limit_ns):
    case = synth.make_decode_case(num_heads=heads, batch=40, ctx=(500, 9000), page_size=16, cache_dtype=cache_dtype,
                                  seed=heads + splits)
    g = GpuCase(case, num_splits_max=splits)
    for _ in range(3):
        assert give_up(lambda: g.decode(splits), limit_ns) < 5.0
        assert mla.decode_status(g.workspace) & mla.DEVERR_TIMEOUT
    g.out.fill_(float("nan"))
    g.lse.fill_(float("nan"))
    g.decode(splits)
    assert mla.decode_status(g.workspace) == 0
    compare(case, g, rows=np.arange(0, case.total_q * heads, 29))


@pytest.mark.parametrize("limit_ns", [300_000, 2_000_000])
@pytest.mark.parametrize("heads,sq,fp8,splits", [(128, 1, False, 0), (16, 1, False, 0), (40, 2, False, 5), (128, 1, True, 0),
                                                 (16, 3, True, 0)])
def test_decode_shared(heads, sq, fp8, splits, limit_ns):
    rng = np.random.default_rng(heads)
    c = Case([(9000, 20), (700, 12)], [int(x) for x in rng.integers(1, 2500, 32)], heads, sq, 64, fp8, seed=heads, splits=splits)
    for _ in range(3):
        assert give_up(c.run, limit_ns) < 5.0
        assert mla.decode_status(c.workspace) & mla.DEVERR_TIMEOUT
    c.run().check()
