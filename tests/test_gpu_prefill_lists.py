"""GPU tests of the prefill's list of many items with cut blocks: more items
than the pairs' spans are made for, and one that would outlast all others.
Tolerances are those of the prefill's own tests."""
import pytest
import torch

from test_gpu_prefill import Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla

# 64 blocks of 16 heads are 1024 items; of 76 pairs' shares (271 to 600 units
# here) the long block has two or more, so it is cut for every head.  With more
# than 256 blocks the list is sorted by classes of length.
CUT = [([1] * 63 + [1], [1000] * 63 + [100000], 16), ([1] * 63 + [600], [1000] * 63 + [100000], 16),
       ([1] * 300 + [600], [100] * 300 + [60000], 16)]


class Poisoned(Case):
    """A case whose workspace ends where the library says it does."""
    GUARD = 1 << 16

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        n = self.ws.numel()
        self.whole = torch.full((n + self.GUARD,), 0xEE, dtype=torch.uint8, device="cuda")
        self.ws = self.whole[:n]

    def check(self, causal=True, **kw):
        super().check(causal, **kw)
        assert (self.whole[self.ws.numel():] == 0xEE).all()
        return self


@pytest.mark.parametrize("q_lens,kv_lens,heads", CUT)
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_cuts_the_long_blocks_of_a_list(q_lens, kv_lens, heads, causal):
    a = Poisoned(q_lens, kv_lens, heads, seed=41, pad_q=3, pad_kv=5).run(causal).check(causal)
    # cut items are joined in the order of their keys: the same bits every time
    out, lse = a.out.clone(), a.lse.clone()
    for _ in range(3):
        a.out.fill_(7.0)
        a.run(causal)
        torch.cuda.synchronize()
        assert torch.equal(a.out, out) and torch.equal(a.lse, lse)
    # and the same answer as without a cut
    Poisoned(q_lens, kv_lens, heads, seed=41, pad_q=3, pad_kv=5, splits=1).run(causal).check(causal)


def test_prefill_replayed_between_a_cut_and_an_uncut_list():
    q_lens, kv_lens, heads = [9] * 64, [1000] * 63 + [60000], 16
    c = Poisoned(q_lens, kv_lens, heads, seed=42).run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for lens in ([1900] * 64, [1000] * 63 + [60000], [0] * 32 + [100] * 31 + [50000], [1000] * 64, kv_lens):
        c.at_kv = [sum(lens[:i]) for i in range(65)]
        c.cu_kv.copy_(torch.tensor(c.at_kv, dtype=torch.int32))
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        g.replay()
        c.check()
