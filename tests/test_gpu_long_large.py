"""The operators of long contexts where offsets pass 32 bits, where more
prefixes stand than the plan keeps places of on chip, and where calls overlap on
the GPU.  Tolerances are those of the operators' own tests."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import long_ref
    import mla_latent_kv_15_gb300 as mla
    from test_gpu_evict import SCALE, Weights, check_compact, check_select, i32, subset
    from test_gpu_shared import Case


def far_pages(lengths, page, fp8, seed):
    """Pages of a cache whose rows pass 2^32 bytes (bf16 and e4m3 alike): every
    second page of a sequence is at the cache's end."""
    p = long_ref.Pages(lengths, page, fp8, seed)
    blocks = (1 << 32) // (page * 576 * (1 if fp8 else 2)) + 200
    far = torch.zeros((blocks, page, 576), dtype=p.cache.dtype, device="cuda")
    n = p.cache.shape[0]
    assert n < 200
    moved = torch.arange(n, device="cuda")
    moved[::2] += blocks - n
    far.view(torch.uint8)[moved] = p.cache.view(torch.uint8)
    ok = p.table >= 0
    p.table[ok] = moved[p.table[ok].long()].int()
    p.cache = far
    return p


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_over_a_far_cache(fp8):
    c = Case([(700, 3), (100, 1)], [100, 64, 1, 200], 16, 1, 64, fp8, seed=21)
    c.pages = far_pages([700, 100, 100, 64, 1, 200], 64, fp8, 21)
    c.prefix_table, c.block_table = c.pages.table[:2].contiguous(), c.pages.table[2:].contiguous()
    c.run().check()


@pytest.mark.parametrize("fp8", [False, True])
def test_key_weights_over_a_far_cache_and_far_rows(fp8):
    lengths = [700, 1, 300]
    w = Weights(lengths, 16, 1, 64, fp8, seed=22)
    w.pages = far_pages(lengths, 64, fp8, 22)
    wide = torch.empty_strided((3, 705), ((1 << 30) + 3, 1), dtype=torch.float32, device="cuda")   # the last row past 2^31
    wide.copy_(w.weights[:, :1].expand(3, 705))
    w.weights = wide
    old = wide.contiguous().clone()
    w.run(0.5)
    w.old = old
    w.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_compact_over_a_far_cache_and_far_rows(fp8):
    rng = np.random.default_rng(23)
    lengths, keeps = [900, 5, 500], [subset(rng, 900, 300), np.array([0, 4]), subset(rng, 500, 499)]
    p = far_pages(lengths, 64, fp8, 23)
    want = [p.rows(b)[torch.as_tensor(k, device="cuda")] for b, k in enumerate(keeps)]
    tail = [p.rows(b)[len(k):] for b, k in enumerate(keeps)]
    keep = torch.full((3, 499), -1, dtype=torch.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = torch.as_tensor(k.astype(np.int32))
    w = torch.empty_strided((3, 900), ((1 << 30) + 3, 1), dtype=torch.float32, device="cuda")
    w.copy_(torch.rand(3, 900, device="cuda"))
    old = w.contiguous().clone()
    mla.cache_compact(p.cache, p.table, keep.cuda(), i32([len(k) for k in keeps]), weights=w)
    torch.cuda.synchronize()
    for b, k in enumerate(keeps):
        assert torch.equal(p.rows(b, len(k)), want[b])
        assert torch.equal(p.rows(b)[len(k):], tail[b])
        assert torch.equal(w[b, :len(k)], old[b, torch.as_tensor(k, device="cuda")])
        assert torch.equal(w[b, len(k):], old[b, len(k):])


def test_select_over_far_rows():
    w = torch.empty_strided((3, 5000), ((1 << 30) + 3, 1), dtype=torch.float32, device="cuda")
    w.copy_(torch.rand(3, 5000, generator=torch.Generator(device="cuda").manual_seed(24), device="cuda"))
    check_select(w, [5000, 3, 4097], 512, 4, 64)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_select_rows_at_any_word(offset):
    # rows that begin at any word of a 16-byte piece, behind words that are larger than all
    base = torch.full((4 * 1003 + 8,), 9.0, device="cuda")
    w = base[offset:offset + 4 * 1003].view(4, 1003)[:, :997]
    w.copy_(torch.rand(4, 997, generator=torch.Generator(device="cuda").manual_seed(offset), device="cuda"))
    check_select(w, [997, 996, 1, 513], 256, 0, 0)
    check_select(w, [997, 996, 1, 513], 256, 3, 7)


@pytest.mark.parametrize("heads,count", [(2, 300), (16, 700)])
def test_more_prefixes_than_the_plan_keeps(heads, count):
    # more than a block of them, some of no request, some without keys
    rng = np.random.default_rng(count)
    prefix = [(int(rng.choice([0, 1, 64, 65, 130])), int(rng.choice([0, 1, 1, 2]))) for _ in range(count)]
    B = sum(r for _, r in prefix)
    own = [int(x) for x in rng.integers(0, 70, B)]
    Case(prefix, own, heads, 1, 16, False, seed=count).run().check()
    sq = [int(x) for x in rng.integers(0, 3, B)]
    sq[0] = 1
    Case(prefix, own, heads, sq, 16, False, seed=count).run().check()


def test_a_padded_request_of_queries_that_are_not_finite():
    c = Case([(0, 4)], [100, 0, 64, 0], 16, 1, 64, seed=25)
    c.q_abs[1], c.q_pe[3] = float("nan"), float("inf")
    c.run()
    torch.cuda.synchronize()
    assert (c.out[[1, 3]] == 0).all() and (c.lse[[1, 3]] == -np.inf).all()
    w = Weights([100, 0, 64, 0], 16, 1, 64, seed=26)
    w.q_abs[1], w.q_pe[3] = float("nan"), float("inf")
    w.q[1] = w.q[3] = 0
    w.run().check()


def test_calls_at_once():
    # two of each on two streams, behind a long product that lets them pile up
    cases = [Case([(3000, 10), (100, 6)], [int(x) for x in np.random.default_rng(s).integers(1, 300, 16)], 16, 1, 64,
                  bool(s & 1), seed=s) for s in (31, 32)]
    weights = [Weights([1000, 700, 3], 32, 1, 64, bool(s & 1), seed=s) for s in (33, 34)]
    streams = [torch.cuda.Stream() for _ in cases]
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    rows = [torch.rand(2, 4000, device="cuda") for _ in cases]
    seqs = [i32([4000, 100]), i32([3999, 4000])]
    keeps = [torch.empty(2, 500, dtype=torch.int32, device="cuda") for _ in cases]
    lens = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in cases]
    caches = [long_ref.Pages([4000, 4000], 64, bool(i), seed=35 + i) for i in range(2)]
    want = [[p.rows(b) for b in range(2)] for p in caches]
    torch.cuda.synchronize()
    a @ a
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    for i, s in enumerate(streams):
        weights[i].run(0.0, stream=s)
        mla.evict_select(rows[i], seqs[i], keeps[i], lens[i], sinks=1, recent=9, stream=s)
        mla.cache_compact(caches[i].cache, caches[i].table, keeps[i], lens[i], stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()
    for w in weights:
        w.check()
    for i, p in enumerate(caches):
        host = rows[i].cpu().numpy()
        for b, n in enumerate(seqs[i].tolist()):
            index = torch.as_tensor(long_ref.select(host[b], n, 500, 1, 9), device="cuda")
            assert torch.equal(p.rows(b, len(index)), want[i][b][index])


def test_two_graphs_of_one_workspace():
    # captured calls that share a workspace, replayed in turn
    a, b = (Case([(512, 3)], [64, 100, 1], 16, 1, 64, seed=s) for s in (41, 42))
    b.workspace = a.workspace
    graphs = []
    for c in (a, b):
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for c in (a, b):
        c.out.fill_(float("nan"))
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_compact_of_one_row_many_times():
    check_compact([1000, 40], [np.full(500, 999), np.full(40, 39)], 16)
    check_compact([1000, 40], [np.full(1000, 999), np.full(40, 39)], 64, True)


@pytest.mark.parametrize("lengths,heads,sq,fp8", [
    ([700, 60, 300], 128, [20, 1, 9], False),      # more rows than lse are kept on chip, few rows, more again
    ([700, 60, 300], 128, [20, 1, 9], True),
    ([300, 129], 1024, 2, False), ([40], 1000, [33], True), ([2000, 5], 1023, 1, False),
])
def test_key_weights_of_many_rows(lengths, heads, sq, fp8):
    Weights(lengths, heads, sq, 64, fp8, seed=heads).run(0.5).check()


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_of_many_heads(fp8):
    Case([(300, 2), (65, 1)], [70, 2, 130], 1024, 1, 64, fp8, seed=51).run().check()
    Case([(300, 2), (65, 1)], [70, 30, 130], 1000, [1, 9, 2], 16, fp8, seed=52).run().check()


def test_without_the_optional_arguments():
    c = Case([(100, 2)], [20, 30], 16, 1, 64, seed=61).run().check()
    want = c.out.clone()
    c.out.fill_(float("nan"))
    c.lse.fill_(7.0)
    c.run(lse=None)
    torch.cuda.synchronize()
    assert torch.equal(c.out, want) and (c.lse == 7).all()
    w = Weights([300, 64], 16, 1, 64, seed=62)
    w.run(0.5, status=None)
    w.check()
    seq, keep, lens = i32([300, 64]), torch.empty(2, 50, dtype=torch.int32, device="cuda"), i32([0, 0])
    mla.evict_select(w.weights, seq, keep, lens)
    before = [w.pages.rows(b) for b in range(2)]
    mla.cache_compact(w.pages.cache, w.pages.table, keep, lens)
    torch.cuda.synchronize()
    for b in range(2):
        assert torch.equal(w.pages.rows(b, 50), before[b][keep[b].long()])
    assert lens.tolist() == [50, 50]


@pytest.mark.parametrize("heads,sq,own,splits", [
    (128, 1, [70, 2, 300], 1),                     # long units of full rows beside short ones, one piece each
    (40, 2, [5, 130, 64, 1], 1), (16, 1, [100] * 9, 1), (33, 2, [2, 2000], 1),
    (128, 1, [64] * 9, 0), (128, 1, [64, 3, 700], 2),
])
def test_long_units_of_many_rows(heads, sq, own, splits):
    # units on either side of the choice of how the partial scores are exchanged, in turn on one pair
    prefix = [(2300, len(own) - 1), (5000, 1)]
    Case(prefix, own, heads, sq, 64, False, seed=heads, splits=splits).run().check()
    Case(prefix, own, heads, sq, 64, True, seed=heads, splits=splits).run().check()


def test_many_long_units():
    # several a pair: 20 groups of rows behind 20000 keys, own keys of all sizes
    rng = np.random.default_rng(71)
    Case([(20000, 20), (2500, 12)], [int(x) for x in rng.integers(1, 2500, 32)], 128, 1, 64, False, seed=71).run().check()


@pytest.mark.parametrize("page", [16, 64, 256])
def test_key_weights_of_e4m3_rows_and_many_query_rows(page):
    # on either side of one tile of rows a request, with bad pages, empty and padded requests, waits that run out
    Weights([700, 0, 129, 1500, 1], 128, 3, page, True, seed=page).run(0.5).check()
    Weights([700, 0, 129, 1500, 1], 128, [2, 0, 9, 1, 0], page, True, seed=page).run(0.0, status=None)
    w = Weights([300, 200], 128, 4, page, True, seed=81)
    w.pages.table[0, 0] = 10 ** 6
    w.run()
    torch.cuda.synchronize()
    assert w.status.item() == 4 and w.weights.isfinite().all()
    w = Weights([300, 200], 128, 4, page, True, seed=82)
    try:
        mla.set_decode_wait_test(True, 2_000_000)
        w.run()
    finally:
        mla.set_decode_wait_test(False, 0)
    torch.cuda.synchronize()
    assert w.status.item() & mla.DEVERR_TIMEOUT
    w.status.zero_()
    w.run(0.0).check()


def test_key_weights_of_many_query_rows_are_the_same_every_time():
    w = Weights([3000, 2500, 900], 128, 5, 64, True, seed=83).run(0.0).check()
    want = w.weights.clone()
    for _ in range(5):
        w.run(0.0)
        torch.cuda.synchronize()
        assert torch.equal(w.weights, want)
