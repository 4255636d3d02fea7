"""Calls of the operators of long contexts whose results hang on an order between
warps or CTAs, and ways out of a wait.  Plain forms and tolerances are those of
the operators' own tests."""
import time

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import exact_scores
    import long_ref
    import mla_latent_kv_15_gb300 as mla
    from test_gpu_evict import SCALE, Weights, check_compact, check_select, i32, subset
    from test_gpu_shared import Case


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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths", [[3000], [900, 40], [700] * 160])        # clusters of many CTAs, of some, of one
def test_compact_wait_that_runs_out(lengths, fp8):
    rng = np.random.default_rng(len(lengths))
    keeps = [subset(rng, n, n // 2) for n in lengths]
    p = long_ref.Pages(lengths, 64, fp8, seed=91)
    keep = torch.full((len(lengths), max(len(k) for k in keeps)), -1, dtype=torch.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = torch.as_tensor(k.astype(np.int32))
    keep, lens, status = keep.cuda(), i32([len(k) for k in keeps]), i32([0])
    raw = p.cache.view(torch.uint8).view(-1, p.cache.element_size() * 576)
    before = raw.clone()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    try:
        mla.set_decode_wait_test(True, 2_000_000)
        mla.cache_compact(p.cache, p.table, keep, lens, status=status)
        torch.cuda.synchronize()
    finally:
        mla.set_decode_wait_test(False, 0)
    assert time.perf_counter() - t0 < 5.0
    assert status.item() == mla.DEVERR_TIMEOUT
    # only rows of the kept ones' places were written, and with rows of the same request
    places = torch.cat([p.slots(b, len(k)) for b, k in enumerate(keeps)])
    left = torch.ones(raw.shape[0], dtype=torch.bool, device="cuda")
    left[places] = False
    assert torch.equal(raw[left], before[left])
    for b, k in enumerate(keeps):
        at = p.slots(b, len(k))
        new = before[p.slots(b, lengths[b])[torch.as_tensor(k, device="cuda")]]
        assert ((raw[at] == new).all(1) | (raw[at] == before[at]).all(1)).all()
    check_compact(lengths, keeps, 64, fp8)           # the next call


def test_compact_takes_no_more_than_its_wait_limit_allows_for():
    # a limit far above a call's time, no row left out: nothing runs out
    try:
        mla.set_decode_wait_test(False, 50_000_000)
        check_compact([3000, 17], [np.arange(1500, 3000), np.arange(17)], 64)
    finally:
        mla.set_decode_wait_test(False, 0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bounds", [[0, 2, 50, 50], [0, 2, 50, 4], [0, -1, 2, 4], [0, 2, 1, 4], [-2147483648, 2, 2, 4],
                                    [0, 2147483647, -2147483648, 4], [0, 2, 4, 5]])
def test_key_weights_query_range_of_a_request_without_keys(bounds, fp8):
    # a request whose tokens are not within the call's counts as without query rows
    # and is reported, whether it has keys or none
    for lengths in ([300, 0, 0], [0, 300, 200], [300, 200, 0], [0, 0, 0], [300, -5, 1]):
        w = Weights([max(n, 0) for n in lengths], 16, [2, 1, 1], 64, fp8, seed=92)
        w.seq_lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        w.qsl.copy_(torch.tensor(bounds, dtype=torch.int32))
        w.run(0.5)
        torch.cuda.synchronize()
        assert w.status.item() == 8
        for b, n in enumerate(lengths):
            lo, hi = bounds[b:b + 2]
            assert torch.equal(w.weights[b, max(n, 0):], w.old[b, max(n, 0):])
            if not 0 <= lo <= hi <= 4 and n > 0:
                assert torch.equal(w.weights[b, :n], w.old[b, :n] * 0.5)
    w = Weights([300, 0, 0], 16, [2, 1, 1], 64, fp8, seed=92)
    w.run(0.5).check()                       # padded requests whose tokens are the call's


def test_key_weights_bad_query_range_of_a_late_request():
    # behind more requests than a block has threads
    w = Weights([3] * 700 + [0] * 3, 2, [1] * 702 + [2], 16, seed=93)
    w.qsl[703] = 10 ** 6
    w.run(0.0)
    torch.cuda.synchronize()
    assert w.status.item() == 8
    w.status.zero_()
    w.qsl[703] = 704
    w.run(0.0).check()


@pytest.mark.parametrize("prefix,own,heads,sq,fp8", [
    ([(300, 3), (70, 1)], [40, 1, 200, 64], 16, 1, False),
    ([(450, 2)], [100, 333], 128, 1, False),               # full rows, fewer than 512 keys
    ([(3000, 4)], [100, 7, 64, 300], 16, 1, False),        # long prefixes of 64 rows
    ([(2999, 2), (0, 1)], [100, 65, 700], 32, 1, False),
    ([(3000, 5)], [100, 7, 64, 300, 1], 128, 1, True), ([(513, 3)], [10, 700, 64], 40, 2, True),
])
def test_shared_log_sum_exp_where_scores_are_exchanged_as_they_are(prefix, own, heads, sq, fp8):
    # whole numbers, whose scores are exact in float32: codes in the exchange would
    # put rows further off (tests/test_exact_scores_cpu.py)
    c = Case(prefix, own, heads, sq, 64, fp8, seed=len(own) + heads, scale=exact_scores.SCALE)
    p = c.pages
    p.kv_scale = 1.0
    c.q_abs, c.q_pe = (exact_scores.queries(t.shape, p.g) for t in (c.q_abs, c.q_pe))
    flat = p.cache.view(-1, 576)
    for i, n in enumerate(p.lengths):
        if n:
            rows = exact_scores.keys((n, 576), p.g)
            if fp8:
                p.cache.view(torch.uint8).view(-1, 576)[p.slots(i, n)] = rows.float().to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                flat[p.slots(i, n)] = rows
    c.run().check()
    q = torch.cat([c.q_abs, c.q_pe], dim=2).double()
    for b, n in enumerate(c.own):
        g = int(np.searchsorted(c.begin, b, side="right")) - 1
        keys = torch.cat([p.rows(g), p.rows(len(prefix) + b)])
        for t in range(c.sq[b]):
            row = int(c.at[b]) + t
            s = c.scale * (q[row] @ keys[:c.prefix[g][0] + n - c.sq[b] + 1 + t].t())
            lse = torch.logsumexp(s, dim=1)
            err = (c.lse[row].double() - lse).abs()
            assert (err <= exact_scores.lse_bar(s, lse)).all(), (b, t, (err / exact_scores.lse_bar(s, lse)).max())


@pytest.mark.parametrize("decay", [0.0, 0.5])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_key_weights_of_requests_with_and_without_query_rows(page, decay):
    # None, one and several tiles of query rows a request, in either order, where
    # e4m3 codes go straight into registers: a request without rows or without keys
    # must leave the turns of those behind it as they are
    lengths, sq = [700, 0, 129, 1500, 1], [2, 0, 9, 1, 0]
    for n, t in ((lengths, sq), (lengths[::-1], sq[::-1]), ([300, 700, 0, 900, 257], [0, 9, 3, 0, 9])):
        for fp8 in (True, False):
            Weights(n, 128, t, page, fp8, seed=94).run(decay).check()


@pytest.mark.parametrize("heads,sq,fp8", [(16, 1, False), (128, 1, False), (128, 1, True), (40, 2, True)])
def test_shared_results_are_the_same_every_time(heads, sq, fp8):
    # whatever the workspace held, alone and beside another kernel
    rng = np.random.default_rng(heads)
    c = Case([(5000, 20), (700, 12)], [int(x) for x in rng.integers(1, 1500, 32)], heads, sq, 64, fp8, seed=heads + sq).run().check()
    out, lse = c.out.clone(), c.lse.clone()
    a, s = torch.randn(2048, 2048, device="cuda", dtype=torch.bfloat16), torch.cuda.Stream()
    for i in range(20):
        c.workspace.random_(0, 256) if i % 3 else c.workspace.fill_(255)
        c.out.fill_(float("nan"))
        c.lse.fill_(float("nan"))
        torch.cuda.synchronize()
        if i % 2:
            with torch.cuda.stream(s):
                a @ a
        c.run()
        torch.cuda.synchronize()
        assert mla.decode_status(c.workspace) == 0
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("width", [41000, 131072])
def test_select_in_rows_far_wider_than_the_requests(width):
    # the width decides how many CTAs a request has and where its codes are; most
    # of them then have no key, or none that competes
    g = torch.Generator(device="cuda").manual_seed(width)
    for lengths, budget, sinks, recent in (([300], 64, 4, 16), ([9000, 0, 1, 4097, 513, width], 512, 4, 64),
                                           ([700] * 90, 100, 0, 0), ([130], 129, 100, 28)):
        w = torch.full((len(lengths), width), 1e9, device="cuda")
        for b, n in enumerate(lengths):
            w[b, :n] = torch.rand(n, generator=g, device="cuda").mul(50).round()
        check_select(w, lengths, budget, sinks, recent)


@pytest.mark.parametrize("heads,fp8", [(16, False), (128, False), (16, True)])
def test_shared_with_tables_far_wider_than_the_requests(heads, fp8):
    # the width decides which kernel a call gets
    c = Case([(512, 5), (70, 3)], [10, 64, 1, 200, 333, 7, 90, 129], heads, 1, 64, fp8, seed=95)
    c.run().check()
    for name in ("prefix_table", "block_table"):
        t = getattr(c, name)
        wide = torch.full((t.shape[0], 600), -1, dtype=torch.int32, device="cuda")
        wide[:, :t.shape[1]] = t
        setattr(c, name, wide)
    c.run().check()
