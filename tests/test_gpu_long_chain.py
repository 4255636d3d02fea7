"""Shared prefixes and eviction as a serving loop uses them: requests behind one
prefix decode a step, the weights of their own keys are accumulated, requests
over their budget are cut back to it, and the next step's rows follow the kept
ones; the whole captured and replayed."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import long_ref
    import mla_latent_kv_15_gb300 as mla

SCALE = 192 ** -0.5
HEADS, PAGE, BUDGET, SINKS, RECENT = 16, 64, 128, 2, 16


class Loop:
    """What a serving program keeps between steps."""

    def __init__(self, prefix, own, fp8, seed):
        # (pages for the rows that the steps add)
        self.pages = long_ref.Pages([prefix] + [n + 8 for n in own], PAGE, fp8, seed)
        self.B = B = len(own)
        self.prefix = prefix
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")      # noqa: E731
        self.prefix_table, self.table = self.pages.table[:1].contiguous(), self.pages.table[1:].contiguous()
        self.prefix_lens, self.prefix_requests = i32([prefix]), i32([0, B])
        self.seq = i32(own)
        self.q_abs, self.q_pe = self.pages.queries(B, HEADS)
        self.out = torch.empty(B, HEADS, 512, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty(B, HEADS, device="cuda")
        self.weights = torch.zeros(B, self.table.shape[1] * PAGE, device="cuda")
        self.keep = torch.empty(B, BUDGET, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(mla.decode_shared_workspace_size(B, 1, B, HEADS), dtype=torch.uint8, device="cuda")

    def step(self):
        p = self.pages
        mla.decode_shared(self.q_abs, self.q_pe, p.cache, self.prefix_table, self.prefix_lens, self.prefix_requests,
                          self.table, self.seq, self.out, self.ws, scale=SCALE, lse=self.lse, kv_scale=p.kv_scale)
        mla.key_weights(self.q_abs, self.q_pe, p.cache, self.table, self.seq, self.lse, self.weights, scale=SCALE,
                        kv_scale=p.kv_scale, status=self.status)
        mla.evict_select(self.weights, self.seq, self.keep, self.seq, sinks=SINKS, recent=RECENT, status=self.status)
        mla.cache_compact(p.cache, self.table, self.keep, self.seq, weights=self.weights, status=self.status)


def rows_of(loop, lengths):
    return [loop.pages.rows(1 + b, n) for b, n in enumerate(lengths)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_loop(fp8, captured):
    own = [300, 60, 129, 128, 500, 1]
    loop = Loop(777, own, fp8, 1)
    if captured:
        loop.step()                   # loads the kernels
        torch.cuda.synchronize()
        fresh = Loop(777, own, fp8, 1)
        for name in ("seq", "q_abs", "q_pe", "weights"):
            getattr(loop, name).copy_(getattr(fresh, name))
        loop.pages.cache.view(torch.uint8).copy_(fresh.pages.cache.view(torch.uint8))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loop.step()
    g = torch.Generator(device="cuda").manual_seed(7)
    lengths = list(own)
    acc = [torch.zeros(n, dtype=torch.float64, device="cuda") for n in own]
    prefix = loop.pages.rows(0)
    for step in range(4):
        before = rows_of(loop, lengths)
        q = torch.cat([loop.q_abs, loop.q_pe], dim=2).double()
        graph.replay() if captured else loop.step()
        torch.cuda.synchronize()
        assert mla.decode_status(loop.ws) == 0 and loop.status.item() == 0
        keep, got = loop.keep.cpu().numpy(), loop.seq.tolist()
        for b, n in enumerate(lengths):
            keys = torch.cat([prefix, before[b]])
            ref, lse, mag = long_ref.attention(q[b], keys, SCALE, len(keys))
            # the decode's own bars: 1e-3 on the lse, bf16 probabilities and outputs
            assert (loop.lse[b].double() - lse).abs().max() < 1e-3
            assert ((loop.out[b].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -7 * mag + 2.0 ** -8).all()
            acc[b] = acc[b] + torch.exp(SCALE * (q[b] @ before[b].t()) - lse[:, None]).sum(0)
            assert got[b] == min(n, BUDGET)
            kept = keep[b, :got[b]]
            assert (np.diff(kept) > 0).all() and (keep[b, got[b]:] == -1).all()
            if n > BUDGET:
                # what was dropped weighs no more than what stays, within the bar of the weights
                assert set(range(SINKS)) <= set(kept) and set(range(n - RECENT, n)) <= set(kept)
                middle = np.ones(n, dtype=bool)
                middle[:SINKS] = middle[n - RECENT:] = False
                stays = np.zeros(n, dtype=bool)
                stays[kept] = True
                w = acc[b].cpu().numpy()
                assert w[middle & ~stays].max() <= w[middle & stays].min() * 1.003 + 1e-9
            index = torch.as_tensor(kept.astype(np.int64), device="cuda")
            assert torch.equal(loop.pages.rows(1 + b, got[b]), before[b][index])
            acc[b] = acc[b][index]
            # each step's lse is within 1e-3
            assert ((loop.weights[b, :got[b]].double() - acc[b]).abs() <= 1.5e-3 * acc[b] + 1e-9).all()
        # the next step's rows
        lengths = [n + 1 for n in got]
        new = torch.randn(loop.B, 576, generator=g, device="cuda").bfloat16()
        slots = torch.stack([loop.pages.slots(1 + b, n)[-1] for b, n in enumerate(lengths)])
        mla.cache_write(new[:, :512].contiguous(), new[:, 512:].contiguous(), slots, loop.pages.cache, loop.pages.kv_scale)
        loop.seq.copy_(torch.tensor(lengths))
        loop.weights[torch.arange(loop.B), torch.tensor(lengths) - 1] = 0.0
        acc = [torch.cat([a, a.new_zeros(1)]) for a in acc]
