"""GPU tests of the prefill's bounded waits where nothing is wrong: a limit on
one wait does not limit the call or an item, whose lengths are the work's."""
import pytest
import torch

from test_gpu_prefill import Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla


def same_under_a_short_limit(c, limit_ns, causal):
    c.run(causal)
    torch.cuda.synchronize()
    assert mla.prefill_status(c.ws) == 0
    out, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(7.0)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    try:
        mla.set_decode_wait_test(wait_limit_ns=limit_ns)
        begin.record()
        c.run(causal)
        end.record()
        torch.cuda.synchronize()
        assert mla.prefill_status(c.ws) == 0
    finally:
        mla.set_decode_wait_test()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    return begin.elapsed_time(end) * 1e6


def test_prefill_outlasts_the_limit_of_its_waits_for_an_item():
    """Thousands of items, each far below the limit of a wait for an item (64
    times that of the others), the call above it."""
    c = Case([24576], [24576], 128, seed=61)
    took = same_under_a_short_limit(c, 150_000, True)
    assert took > 64 * 150_000, f"the call took {took / 1e6:.2f} ms: too short to tell"


def test_prefill_item_with_a_ragged_end_outlasts_the_limit_of_a_wait():
    """The last value rows of an item, which are cleared past the sequence's
    end, are awaited from the item's start."""
    c = Case([512], [60005], 8, seed=62, splits=1)
    took = same_under_a_short_limit(c, 100_000, False)
    assert took > 2 * 100_000, f"the call took {took / 1e6:.2f} ms: too short to tell"


@pytest.mark.parametrize("q_lens,kv_lens,heads", [([300], [300], 2), ([1] * 8, [3000] * 8, 16), ([1] * 40, [3000] * 40, 1),
                                                  ([600] * 3, [700] * 3, 128)])
def test_prefill_status_is_of_the_last_call(q_lens, kv_lens, heads):
    """One launch, two and three: whatever the workspace held, a clean call
    reads clean, one whose keys never arrive and one of inconsistent sums say
    so, and the next is clean again."""
    c = Case(q_lens, kv_lens, heads, seed=63)
    cu_q = c.cu_q.clone()
    for junk in (0xFF, 0x01, 0xEE):
        c.ws.fill_(junk)
        c.run()
        assert mla.prefill_status(c.ws) == 0
        try:
            mla.set_decode_wait_test(skip_first_tile=True, wait_limit_ns=2_000_000)
            c.run()
            assert mla.prefill_status(c.ws) == mla.DEVERR_TIMEOUT
        finally:
            mla.set_decode_wait_test()
        c.ws.fill_(junk)
        c.cu_q[-1] = c.q.shape[0] + 1
        c.run()
        assert mla.prefill_status(c.ws) == mla.DEVERR_BAD_QSL
        c.cu_q.copy_(cu_q)
        c.out.fill_(7.0)
        c.run().check()
