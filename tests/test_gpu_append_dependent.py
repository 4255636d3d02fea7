"""GPU test of the rotated append right behind kernels of the library that
write its norm weight and table (programmatic launches: it starts beside
them), which change from call to call."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla


def rnd(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("T", [1, 300])
def test_append_reads_the_norm_weight_of_the_kernel_before(T):
    g = torch.Generator(device="cuda").manual_seed(T)
    down, w = rnd(g, T, 576), rnd(g, 1, 512, 512) / 512 ** 0.5
    table = torch.randn(50, 64, generator=g, device="cuda")
    pos, slots = torch.arange(T, device="cuda") % 50, torch.arange(T, device="cuda")
    cache = torch.zeros(T, 1, 576, dtype=torch.bfloat16, device="cuda")
    weight = torch.zeros(1, 1, 512, dtype=torch.bfloat16, device="cuda")
    lat = rnd(g, 40, 512)
    got, weights = [], []
    for k in range(40):
        mla.kv_up_proj(lat[k:k + 1], w, weight)
        mla.rope_cache_write(down[:, :512], down[:, 512:], pos, table, slots, cache, norm_weight=weight.view(512))
        got.append(cache.clone())
        weights.append(weight.clone())
    torch.cuda.synchronize()
    for c, x in zip(got, weights):
        cache.zero_()
        torch.cuda.synchronize()
        mla.rope_cache_write(down[:, :512], down[:, 512:], pos, table, slots, cache, norm_weight=x.view(512).clone())
        assert torch.equal(c, cache)
    assert not torch.equal(got[0], got[1])


def test_append_reads_the_table_of_the_kernel_before():
    """A table of [positions, 64] floats as the LSE of 64 heads."""
    g = torch.Generator(device="cuda").manual_seed(9)
    T, P = 100, 30
    q, kv, pe = rnd(g, P, 64, 192), rnd(g, 200, 64, 256), rnd(g, 200, 64)
    cu_q = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    cu_kv = torch.tensor([[0, 200 - 3 * k] for k in range(40)], dtype=torch.int32, device="cuda")
    out = torch.empty(P, 64, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mla.prefill_workspace_size(1, P, 64), dtype=torch.uint8, device="cuda")
    table = torch.zeros(P, 64, device="cuda")
    down, pos, slots = rnd(g, T, 576), torch.arange(T, device="cuda") % P, torch.arange(T, device="cuda")
    cache = torch.zeros(T, 1, 576, dtype=torch.bfloat16, device="cuda")
    got, tables = [], []
    for k in range(40):
        mla.prefill(q, kv, pe, cu_q, cu_kv[k], out, ws, scale=1 / math.sqrt(192), causal=False, lse=table)
        mla.rope_cache_write(down[:, :512], down[:, 512:], pos, table, slots, cache)
        got.append(cache.clone())
        tables.append(table.clone())
    torch.cuda.synchronize()
    for c, t in zip(got, tables):
        cache.zero_()
        torch.cuda.synchronize()
        mla.rope_cache_write(down[:, :512], down[:, 512:], pos, t, slots, cache)
        assert torch.equal(c, cache)
    assert not torch.equal(got[0], got[1])
