"""GPU tests of the prompt-side operators on one token of a head-major buffer
whose heads lie far apart: the stride to a next token is never used."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla

HEADS, FAR = 128, 180000          # heads * FAR * 192 elements are beyond 2^32


def test_prefill_of_one_token_between_far_heads():
    g = torch.Generator(device="cuda").manual_seed(1)
    buf = torch.empty(HEADS, FAR, 192, dtype=torch.bfloat16, device="cuda")
    q = buf[:, 5:6].transpose(0, 1)
    q.copy_(torch.randn(1, HEADS, 192, generator=g, device="cuda"))
    keys = 700
    kv = torch.randn(keys, HEADS, 256, generator=g, device="cuda").to(torch.bfloat16)
    pe = torch.randn(keys, 64, generator=g, device="cuda").to(torch.bfloat16)
    cu_q, cu_kv = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (1, keys))
    ws = torch.empty(mla.prefill_workspace_size(1, 1, HEADS), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, 1, HEADS, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2, 1, HEADS, device="cuda")
    for i, x in enumerate((q, q.contiguous())):
        mla.prefill(x, kv, pe, cu_q, cu_kv, out[i], ws, scale=1 / math.sqrt(192), lse=lse[i])
        assert mla.prefill_status(ws) == 0
    assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1]) and out.any()


def test_append_of_one_token_between_far_heads():
    g = torch.Generator(device="cuda").manual_seed(2)
    buf = torch.empty(HEADS, FAR, 192, dtype=torch.bfloat16, device="cuda")
    q = buf[:, 7:8, 128:].transpose(0, 1)
    q.copy_(torch.randn(1, HEADS, 64, generator=g, device="cuda"))
    table = torch.randn(10, 64, generator=g, device="cuda")
    row = torch.randn(1, 576, generator=g, device="cuda").to(torch.bfloat16)
    pos, slot = torch.tensor([3], device="cuda"), torch.tensor([1], device="cuda")
    cache = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device="cuda")
    want, got = (torch.empty(1, HEADS, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    args = (row[:, :512], row[:, 512:], pos, table, slot, cache)
    mla.rope_cache_write(*args, q_pe=q.contiguous(), q_pe_out=want)
    mla.rope_cache_write(*args, q_pe=q, q_pe_out=got)
    assert torch.equal(got, want) and got.any()
    mla.rope_cache_write(*args, q_pe=q, q_pe_out=q)
    assert torch.equal(q, want)
