"""mla_key_weights, mla_evict_select and mla_cache_compact against plain forms."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import long_ref
    import mla_latent_kv_15_gb300 as mla

SCALE = 192 ** -0.5


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- key weights


class Weights:
    def __init__(self, lengths, heads, sq=1, page=64, fp8=False, seed=0, q_std=1.0, scale=SCALE, pad=5, spread=3):
        self.pages = long_ref.Pages(lengths, page, fp8, seed)
        self.lengths, self.heads, self.scale = list(lengths), heads, scale
        self.sq = [sq] * len(lengths) if isinstance(sq, int) else list(sq)
        self.at = np.concatenate([[0], np.cumsum(self.sq)])
        T = int(self.at[-1])
        self.qsl = None if sq == 1 else i32(self.at.tolist())
        self.seq_lens = i32(self.lengths)
        self.q_abs, self.q_pe = self.pages.queries(T, heads, q_std)
        self.q = torch.cat([self.q_abs, self.q_pe], dim=2).double()
        self.lse = torch.zeros(T, heads, device="cuda")
        for b, n in enumerate(self.lengths):
            keys = self.pages.rows(b)
            for t in range(self.sq[b]):
                row = int(self.at[b]) + t
                self.lse[row] = long_ref.attention(self.q[row], keys, scale, n - self.sq[b] + 1 + t)[1].float()
        wide = torch.rand(len(lengths), max(list(lengths) + [1]) + pad + spread, generator=self.pages.g, device="cuda")
        self.weights = wide[:, :wide.shape[1] - spread]      # rows further apart than they are wide
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, decay=1.0, **over):
        kw = dict(scale=self.scale, query_start_loc=self.qsl, decay=decay, kv_scale=self.pages.kv_scale, status=self.status)
        kw.update(over)
        self.old = self.weights.clone()
        self.decay = decay
        mla.key_weights(self.q_abs, self.q_pe, self.pages.cache, self.pages.table, self.seq_lens, self.lse, self.weights, **kw)
        return self

    def check(self):
        torch.cuda.synchronize()
        assert self.status.item() == 0
        for b, n in enumerate(self.lengths):
            keys = self.pages.rows(b)
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            tol = torch.zeros_like(got)
            for t in range(self.sq[b]):
                row, seen = int(self.at[b]) + t, max(0, n - self.sq[b] + 1 + t)
                s = self.scale * (self.q[row] @ keys[:seen].t())
                l = self.lse[row].double()[:, None]
                p = torch.where(l == -np.inf, 0.0, torch.exp(s - l))
                got[:seen] += p.sum(0)
                # a score: 576 products summed in float32, its product with the
                # scale and its difference to the lse rounded (2^-23 of each in
                # binary units); an exponential within 2^-21
                qk = abs(self.scale) * self.q[row].norm(dim=1, keepdim=True) * keys[:seen].norm(dim=1)
                e = 64 * 2.0 ** -24 * qk + 2.0 ** -22 * (s.abs() + torch.where(l == -np.inf, 0.0, l.abs())) + 2.0 ** -21
                tol[:seen] += (p * e).sum(0)
            old = self.decay * self.old[b, :n].double() if self.decay else torch.zeros_like(got)
            ref = old + got
            # the sum over rows in several float32 partial sums, and the last addition
            tol += (self.sq[b] * self.heads / 4 + 4) * 2.0 ** -24 * got + 2.0 ** -23 * ref
            err = (self.weights[b, :n].double() - ref).abs()
            assert (err <= tol).all(), (b, (err / tol.clamp(min=1e-30)).max(), err.max())
            assert torch.equal(self.weights[b, n:], self.old[b, n:])
        return self


WEIGHTS = [
    ([1], 16, 1, 64, False), ([777], 16, 1, 64, False), ([128, 0, 129, 127], 16, 1, 64, False),
    ([5, 300, 1000], 1, 1, 16, False), ([200, 64, 500], 40, 1, 32, False), ([500, 900], 100, 1, 128, False),
    ([1000, 3000, 17], 128, 1, 64, False), ([400, 130], 200, 1, 256, False),       # two row tiles
    ([300, 700], 128, 4, 64, False), ([50, 700, 129, 400], 40, [4, 1, 0, 3], 16, False),
    ([2, 3, 1, 600], 16, 4, 64, False),                                            # fewer keys than query tokens
    ([777], 16, 1, 64, True), ([128, 0, 129, 1500], 128, 1, 16, True), ([700, 333], 40, [3, 2], 128, True),
    ([90] * 70, 8, 1, 32, False),
]


@pytest.mark.parametrize("decay", [0.0, 0.9, 1.0])
@pytest.mark.parametrize("i", range(len(WEIGHTS)))
def test_key_weights(i, decay):
    lengths, heads, sq, page, fp8 = WEIGHTS[i]
    w = Weights(lengths, heads, sq, page, fp8, seed=i)
    if decay == 0.0:
        w.weights.fill_(float("nan"))            # not read
        w.run(decay)
        w.old = torch.where(w.old.isnan(), 0.0, w.old)
        for b, n in enumerate(lengths):
            assert w.weights[b, n:].isnan().all()
            w.weights[b, n:] = 0.0
        w.check()
    else:
        w.run(decay).check()


def test_key_weights_of_long_requests_and_more_requests_than_threads():
    Weights([40000, 3, 20000], 16, 1, 64, False, seed=1).run().check()
    Weights([int(x) for x in np.random.default_rng(2).integers(0, 60, 1200)], 2, 1, 16, False, seed=2).run().check()


def test_key_weights_sharp_and_negative_scale():
    Weights([700, 300], 16, 2, 64, False, seed=3, q_std=6.0).run(0.0).check()
    Weights([700, 300], 16, 1, 64, True, seed=4, scale=-SCALE).run().check()


def test_key_weights_add_up_to_the_rows():
    w = Weights([700, 300, 64], 32, 1, 64, False, seed=5)
    out = torch.empty(3, 32, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 32, device="cuda")
    w.pages.cache.nan_to_num_(0.0)
    ws = torch.empty(mla.decode_workspace_size(3, 3, 32), dtype=torch.uint8, device="cuda")
    mla.decode(w.q_abs, w.q_pe, w.pages.cache, w.pages.table, w.seq_lens, out, ws, scale=SCALE, lse=lse)
    w.lse = lse
    w.run(0.0)
    torch.cuda.synchronize()
    for b, n in enumerate(w.lengths):
        # the decode's lse is within 1e-3 of the exact one, its own bar
        assert abs(w.weights[b, :n].double().sum().item() - 32) < 32 * 1.1e-3


def test_key_weights_not_finite():
    # a key that is not finite: its own weight alone; a row without lse: no weight
    w = Weights([300, 200], 16, 2, 64, False, seed=6)
    w.run(0.0)
    clean = w.weights.clone()
    w.pages.cache.view(-1, 576)[w.pages.slots(0, 300)[77], 5] = float("nan")
    w.run(0.0)
    torch.cuda.synchronize()
    assert w.weights[0, 77].isnan()
    w.weights[0, 77] = clean[0, 77]
    assert torch.equal(w.weights[:, :200], clean[:, :200])
    # the last key is hidden from the first token: its NaN reaches it by the second alone
    w = Weights([300, 200], 16, 2, 64, False, seed=6)
    w.lse[1] = -np.inf
    w.run(0.0).check()
    w.pages.cache.view(-1, 576)[w.pages.slots(0, 300)[299], 5] = float("nan")
    w.q_abs[1] = 0                                # (rows that see it)
    w.run(0.0)
    torch.cuda.synchronize()
    assert w.weights[0, 299].isnan() and w.weights[0, :299].isfinite().all()


def test_key_weights_every_e4m3_code():
    # key j holds code j in one column and a code of another sign behind it; one query reads the column
    p = long_ref.Pages([256], 64, fp8=True, seed=11)
    flat = p.cache.view(torch.uint8).view(-1, 576)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    for column in (0, 65, 511, 513, 575):
        flat.zero_()
        flat[p.slots(0, 256), column] = codes
        if column + 1 < 576:
            flat[p.slots(0, 256), column + 1] = codes ^ 0x80
        q = torch.zeros(1, 1, 576, dtype=torch.bfloat16, device="cuda")
        q[0, 0, column] = 1.0
        w = torch.full((1, 256), 7.0, device="cuda")
        mla.key_weights(q[..., :512].contiguous(), q[..., 512:].contiguous(), p.cache, p.table, i32([256]),
                        torch.zeros(1, 1, device="cuda"), w, scale=1.0, decay=0.0, kv_scale=0.25)
        torch.cuda.synchronize()
        value = codes.view(torch.float8_e4m3fn).double()
        finite = value.isfinite()
        ref = torch.exp(0.25 * value)
        # one product; the exponent's rounding (2^-24 of up to 162 in binary units) and its power's 2^-21;
        # a power past float32's largest (exp 112 is 4e48) is infinite there
        over = ref > torch.finfo(torch.float32).max
        assert (w[0] == float("inf"))[finite & over].all()
        assert ((w[0].double() - ref).abs() <= (162 * 2.0 ** -23 + 2.0 ** -21) * ref + 1e-37)[finite & ~over].all()
        if column + 1 < 576:                   # NaN times zero beside it
            assert w[0][~finite].isnan().all()


def test_key_weights_device_errors():
    w = Weights([300, 200], 16, 1, 64, False, seed=7)
    w.pages.table[0, 1] = -7
    w.run()
    torch.cuda.synchronize()
    assert w.status.item() == 4 and w.weights.isfinite().all()
    w = Weights([300, 200], 16, 1, 64, False, seed=7)
    w.seq_lens[1] = 1 << 20
    w.pages.cache.nan_to_num_(0.0)
    w.run()
    torch.cuda.synchronize()
    assert w.status.item() & 2
    w = Weights([300, 200], 16, 2, 64, False, seed=7)
    w.qsl[2] = 50
    w.run(0.5)
    torch.cuda.synchronize()
    assert w.status.item() == 8
    assert torch.equal(w.weights[1, :200], w.old[1, :200] * 0.5)      # no query rows
    w = Weights([300, 200], 16, 1, 64, False, seed=7)
    w.seq_lens[0] = -3
    w.run()
    torch.cuda.synchronize()
    assert w.status.item() == 0 and torch.equal(w.weights[0], w.old[0])


def test_key_weights_wait_that_runs_out():
    for fp8 in (False, True):
        w = Weights([300, 200], 16, 1, 64, fp8, seed=8)
        try:
            mla.set_decode_wait_test(True, 2_000_000)
            w.run()
        finally:
            mla.set_decode_wait_test(False, 0)
        torch.cuda.synchronize()
        assert w.status.item() & mla.DEVERR_TIMEOUT
        w.status.zero_()
        w.run(0.0).check()


def test_key_weights_replayed_over_other_lengths():
    w = Weights([700, 300, 64], 32, 1, 64, False, seed=9).run().check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.run(0.5)
    for lengths in ([699, 1, 0], [0, 0, 0], [128, 300, 64]):
        w.lengths = w.pages.lengths = lengths
        w.seq_lens.copy_(torch.tensor(lengths))
        w.old = w.weights.clone()
        w.decay = 0.5
        g.replay()
        w.check()


@pytest.mark.parametrize("seed", range(24))
def test_key_weights_drawn(seed):
    rng = np.random.default_rng(300 + seed)
    B = int(rng.integers(1, 9))
    lengths = [int(rng.choice([0, 1, 63, 127, 128, 129, 500, 1500])) + int(rng.integers(0, 4)) for _ in range(B)]
    sq = int(rng.choice([1, 1, 2])) if rng.random() < 0.6 else [int(x) for x in rng.integers(0, 7, B)]
    if not isinstance(sq, int) and sum(sq) == 0:
        sq[0] = 1
    Weights(lengths, int(rng.choice([1, 3, 16, 17, 33, 64, 100, 128, 130])), sq, int(rng.choice([16, 32, 64, 128, 256])),
            bool(rng.random() < 0.4), seed=seed).run(float(rng.choice([0.5, 1.0]))).check()


# ------------------------------------------------------------------ selection


def run_select(weights, lengths, budget, sinks=0, recent=0, in_place=False):
    B = len(lengths)
    seq = i32(lengths)
    keep = torch.full((B, budget), -77, dtype=torch.int32, device="cuda")
    lens = seq if in_place else torch.full((B,), -77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.evict_select(weights, seq, keep, lens, sinks=sinks, recent=recent, status=status)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), lens.cpu().numpy(), status.item()


def check_select(weights, lengths, budget, sinks=0, recent=0, in_place=False):
    keep, lens, status = run_select(weights, lengths, budget, sinks, recent, in_place)
    assert status == 0
    host = weights.cpu().numpy()
    for b, n in enumerate(lengths):
        want = long_ref.select(host[b], n, budget, sinks, recent)
        assert lens[b] == min(n, budget) == len(want)
        assert np.array_equal(keep[b, :len(want)], want), b
        assert (keep[b, len(want):] == -1).all()


@pytest.mark.parametrize("lengths,budget,sinks,recent", [
    ([1], 1, 0, 0), ([5], 1, 0, 0), ([5], 1, 1, 0), ([5], 1, 0, 1), ([0, 1, 2, 3], 2, 1, 1), ([33, 32, 31], 32, 0, 0),
    ([1000, 10, 512, 513], 512, 4, 64), ([4096], 1024, 4, 64), ([20000, 8192, 1, 0, 4097], 4096, 4, 512),
    ([300], 200, 100, 100), ([70000, 3], 5000, 0, 0), ([500000], 4096, 4, 32),
    ([100] * 400, 50, 2, 3), ([3000] * 200, 100, 0, 0),
])
def test_select(lengths, budget, sinks, recent):
    g = torch.Generator(device="cuda").manual_seed(len(lengths) + budget)
    wide = torch.exp(2 * torch.randn(len(lengths), max(lengths) + 9, generator=g, device="cuda"))
    w = wide[:, :max(lengths) + 2]
    check_select(w, lengths, budget, sinks, recent)
    check_select(w, lengths, budget, sinks, recent, in_place=True)
    # ties: few values, many zeros
    w = torch.where(w < 1, 0.0, w.round().clamp(max=7))
    check_select(w, lengths, budget, sinks, recent)
    # all the same: the first ones
    check_select(torch.zeros_like(w), lengths, budget, sinks, recent)


def test_select_special_values():
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(3, 2000, generator=g, device="cuda")
    w[0, ::3] = float("inf")
    w[0, 1::7] = float("-inf")
    w[1, ::2] = float("nan")
    w[1, 1::4] = float("-inf")
    w[2] = torch.where(torch.rand(2000, generator=g, device="cuda") < 0.5, 0.0, -0.0)     # equal
    w[2, ::50] = 1e-45                                                                     # above zero
    for budget in (10, 700, 1500, 1999):
        check_select(w, [2000, 1999, 1800], budget, 2, 3)


def test_select_errors_and_rows_behind():
    w = torch.rand(2, 100, device="cuda")
    keep, lens, status = run_select(w, [200, 50], 150)
    assert status == 2 and lens.tolist() == [100, 50] and (keep[0, :100] == np.arange(100)).all()
    keep, lens, status = run_select(w, [-4, 50], 20)
    assert status == 0 and lens[0] == 0 and (keep[0] == -1).all()


@pytest.mark.parametrize("seed", range(12))
def test_select_drawn(seed):
    rng = np.random.default_rng(500 + seed)
    B = int(rng.choice([1, 2, 20, 160]))
    lengths = [int(x) for x in rng.integers(0, int(rng.choice([10, 600, 9000])), B)]
    budget = int(rng.integers(1, max(lengths) + 2))
    sinks = int(rng.integers(0, min(budget, 5) + 1))
    w = torch.rand(B, max(lengths) + 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    if seed % 2:
        w = (w * 20).round()
    check_select(w, lengths, budget, sinks, int(rng.integers(0, budget - sinks + 1)))


# ----------------------------------------------------------------- compaction


def check_compact(lengths, keeps, page, fp8=False, with_weights=True, seed=0, max_keep=None):
    p = long_ref.Pages(lengths, page, fp8, seed)
    B, most = len(lengths), max_keep or max(len(k) for k in keeps)
    keep = torch.full((B, most), -1, dtype=torch.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = torch.as_tensor(np.asarray(k, dtype=np.int32))
    width = max(lengths) + 3
    wide = torch.rand(B, width + 5, device="cuda")
    weights = wide[:, :width] if with_weights else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = p.cache.view(torch.uint8).clone() if fp8 else p.cache.view(torch.int16).clone()
    flat = want.view(-1, 576)
    wwant = wide.clone()
    for b, k in enumerate(keeps):
        slots = p.slots(b, lengths[b])
        src = torch.as_tensor(np.asarray(k, dtype=np.int64), device="cuda")
        rows = flat[slots[src]].clone()
        flat[slots[:len(k)]] = rows
        if with_weights:
            wwant[b, :len(k)] = wide[b, src].clone()
    mla.cache_compact(p.cache, p.table, keep.cuda(), i32([len(k) for k in keeps]), weights=weights, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert torch.equal(p.cache.view(want.dtype), want)
    assert torch.equal(wide, wwant)


def subset(rng, n, k):
    return np.sort(rng.choice(n, k, replace=False))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256, 1, 100])
def test_compact(page, fp8):
    rng = np.random.default_rng(page)
    lengths = [1000, 1, 64, 333, 700, 5]
    keeps = [subset(rng, 1000, 400), [0], np.arange(64), subset(rng, 333, 332), np.arange(300, 700), []]
    check_compact(lengths, keeps, page, fp8, seed=page)
    check_compact(lengths, keeps, page, fp8, with_weights=False, seed=page, max_keep=500)


@pytest.mark.parametrize("fp8", [False, True])
def test_compact_sizes(fp8):
    rng = np.random.default_rng(3)
    check_compact([8192], [subset(rng, 8192, 2048)], 64, fp8)                       # one request over several CTAs
    check_compact([20000], [subset(rng, 20000, 19000)], 64, fp8)                    # many waves
    check_compact([3000] * 90, [subset(rng, 3000, int(k)) for k in rng.integers(0, 3000, 90)], 64, fp8)
    check_compact([200] * 400, [subset(rng, 200, 100) for _ in range(400)], 16, fp8)


def test_compact_any_order_from_behind():
    # indices need not ascend: at or behind their place is enough
    rng = np.random.default_rng(4)
    n, k = 3000, 1500
    keep = np.array([int(rng.integers(i, n)) for i in range(k)])
    check_compact([n, n], [keep, np.full(k, n - 1)], 64)


def test_compact_device_errors():
    p = long_ref.Pages([300, 300], 64, seed=5)
    before = p.cache.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = i32([[0, 0, 5, 10 ** 6, -3, 7], [200, 201, 202, 203, 204, 205]])
    table = p.table.clone()
    table[1, 3] = 10 ** 6                           # the pages of 192..255
    mla.cache_compact(p.cache, table, keep, i32([6, 6]), status=status)
    torch.cuda.synchronize()
    assert status.item() == 16 | 4
    s0 = p.slots(0, 300)
    want = before.view(-1, 576).clone()
    want[s0[2]], want[s0[5]] = want[s0[5]].clone(), want[s0[7]].clone()
    assert torch.equal(p.cache.view(torch.int16), want.view(before.shape).view(torch.int16))
    status.zero_()
    mla.cache_compact(p.cache, p.table, i32([[1, 2], [0, 1]]), i32([9, -2]), status=status)
    torch.cuda.synchronize()
    assert status.item() == 2


def test_compact_and_select_captured():
    rng = np.random.default_rng(6)
    p = long_ref.Pages([900, 500], 64, seed=6)
    w = torch.rand(2, 900, device="cuda")
    seq = i32([900, 500])
    keep = torch.empty(2, 300, dtype=torch.int32, device="cuda")
    lens = torch.empty(2, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    mla.evict_select(w, seq, keep, lens, sinks=2, recent=20)          # (loads the kernels before the capture)
    mla.cache_compact(p.cache.clone(), p.table, keep, lens, weights=w.clone())
    with torch.cuda.graph(g):
        mla.evict_select(w, seq, keep, lens, sinks=2, recent=20)
        mla.cache_compact(p.cache, p.table, keep, lens, weights=w)
    for lengths in ([900, 500], [100, 301]):
        fresh = torch.randn(p.cache.shape, device="cuda").bfloat16()
        p.cache.copy_(fresh)
        w.copy_(torch.from_numpy(rng.random((2, 900), dtype=np.float32)))
        host = w.cpu().numpy()
        seq.copy_(torch.tensor(lengths))
        g.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(lengths):
            want = torch.as_tensor(long_ref.select(host[b], n, 300, 2, 20), device="cuda")
            assert torch.equal(p.cache.view(-1, 576)[p.slots(b, len(want))], fresh.view(-1, 576)[p.slots(b, n)[want]])
            assert np.array_equal(w[b, :len(want)].cpu().numpy(), host[b, want.cpu().numpy()])
