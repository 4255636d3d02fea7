"""GPU test of the rotated append between column ranges of the same rows.  The
same bits as between tensors of their own."""
import pytest
import torch

from test_gpu_append import Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla


@pytest.mark.parametrize("T,N", [(1, 1), (1, 16), (7, 1), (33, 20), (300, 3)])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("src,dst", [(64, 128), (128, 0), (192, 128), (8, 72)])
def test_append_rotates_queries_into_other_columns_of_their_rows(T, N, head_major, src, dst):
    c = Case(T, N, 64, False, True, seed=T + N)
    wide = torch.randn((N, T, 256) if head_major else (T, N, 256), device="cuda").to(torch.bfloat16)
    before = wide.clone()
    view = wide.transpose(0, 1) if head_major else wide
    q, q_out = view[..., src:src + 64], view[..., dst:dst + 64]
    want = torch.empty(T, N, 64, dtype=torch.bfloat16, device="cuda")
    args = (c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache)
    mla.rope_cache_write(*args, q_pe=q.clone(), q_pe_out=want, norm_weight=c.weight)
    mla.rope_cache_write(*args, q_pe=q, q_pe_out=q_out, norm_weight=c.weight)
    torch.cuda.synchronize()
    assert torch.equal(q_out, want) and not torch.equal(want, q.contiguous())
    wide[..., dst:dst + 64] = before[..., dst:dst + 64]
    assert torch.equal(wide, before)                     # no other column
