"""mla_decode_shared against a plain 64-bit form over the concatenated keys."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import long_ref
    import mla_latent_kv_15_gb300 as mla

LKV = 512
SCALE = 192 ** -0.5


class Case:
    """prefix: [(keys, requests)], own: keys of each request, sq: query tokens
    of each request (one number: all the same)."""

    def __init__(self, prefix, own, heads, sq=1, page=64, fp8=False, seed=0, std=1.0, q_std=1.0, splits=0, scale=SCALE):
        lengths = [p for p, _ in prefix] + list(own)
        self.prefix, self.own, self.heads, self.splits, self.scale = prefix, list(own), heads, splits, scale
        self.sq = [sq] * len(own) if isinstance(sq, int) else list(sq)
        assert sum(r for _, r in prefix) == len(own) == len(self.sq)
        self.pages = long_ref.Pages(lengths, page, fp8, seed, std)
        G = len(prefix)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")      # noqa: E731
        self.prefix_table, self.block_table = self.pages.table[:G].contiguous(), self.pages.table[G:].contiguous()
        self.prefix_lens, self.seq_lens = i32([p for p, _ in prefix]), i32(self.own)
        self.begin = np.concatenate([[0], np.cumsum([r for _, r in prefix])])
        self.prefix_requests = i32(self.begin.tolist())
        self.at = np.concatenate([[0], np.cumsum(self.sq)])
        self.T = int(self.at[-1])
        self.qsl = None if sq == 1 else i32(self.at.tolist())
        self.q_abs, self.q_pe = self.pages.queries(self.T, heads, q_std)
        self.out = torch.full((self.T, heads, LKV), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, heads), float("nan"), device="cuda")
        self.workspace = torch.empty(mla.decode_shared_workspace_size(len(own), G, self.T, heads, splits),
                                     dtype=torch.uint8, device="cuda")

    def run(self, **over):
        kw = dict(scale=self.scale, query_start_loc=self.qsl, lse=self.lse, num_splits=self.splits,
                  kv_scale=self.pages.kv_scale)
        kw.update(over)
        mla.decode_shared(self.q_abs, self.q_pe, self.pages.cache, self.prefix_table, self.prefix_lens,
                          self.prefix_requests, self.block_table, self.seq_lens, self.out, self.workspace, **kw)
        return self

    def check(self, status=0):
        torch.cuda.synchronize()
        assert mla.decode_status(self.workspace) == status
        G = len(self.prefix)
        q = torch.cat([self.q_abs, self.q_pe], dim=2).double()
        pre = [self.pages.rows(g) for g in range(G)]
        for b, (n, sq) in enumerate(zip(self.own, self.sq)):
            if sq == 0:
                continue
            g = int(np.searchsorted(self.begin, b, side="right")) - 1
            keys = torch.cat([pre[g], self.pages.rows(G + b)])
            P = self.prefix[g][0]
            knorm = keys.norm(dim=1).max().item() if len(keys) else 0.0
            vmax = keys[:, :LKV].abs().max().item() if len(keys) else 0.0
            for t in range(sq):
                row = int(self.at[b]) + t
                ref, lse, mag = long_ref.attention(q[row], keys, self.scale, P + max(0, n - sq + 1 + t))
                # A score: the exchanged half of it within 1.5 of 32766 steps of
                # half its range (at most |q| |k|), 576 products summed in float32
                # (2^-23 of |q| |k| each, far from reached), and the logarithm of
                # the sum within 2^-20 of it
                qk = abs(self.scale) * q[row].norm(dim=1) * knorm
                e = qk * (1.5 / 32766 + 576 * 2.0 ** -24)
                err = (self.lse[row].double() - lse).abs()
                fin = lse.isfinite()
                assert torch.equal(self.lse[row].isfinite(), fin)
                assert (self.lse[row][~fin] == -np.inf).all()
                assert (err[fin] <= (e + 2.0 ** -20 * lse.abs() + 2.0 ** -18)[fin]).all(), (b, t, err[fin].max())
                # An output: bf16 probabilities (2^-8 each), scores, the partials'
                # 16-bit codes (2^-12 of the largest of 32 values), one rounding
                tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * e[:, None] + 2.0 ** -16) * mag + 2.0 ** -11 * vmax
                bad = (self.out[row].double() - ref).abs() > tol
                assert not bad.any(), (b, t, (self.out[row].double() - ref).abs().max(), bad.sum())
        return self


SMALL = [
    # (prefixes, own, heads, sq, page, fp8, splits)
    ([(100, 1)], [1], 16, 1, 64, False, 0),                                  # one request
    ([(512, 4)], [1, 17, 64, 65], 16, 1, 64, False, 0),
    ([(1, 3)], [1, 2, 3], 1, 1, 16, False, 0),                               # one head, one prefix key
    ([(0, 3)], [5, 0, 200], 16, 1, 64, False, 0),                            # no prefix; a padded request
    ([(77, 3)], [0, 0, 9], 16, 1, 32, False, 0),                             # requests without own keys
    ([(130, 2), (0, 1), (700, 0), (65, 3)], [3, 100, 64, 1, 129, 5], 8, 1, 64, False, 0),   # a prefix of nobody
    ([(300, 5)], [10, 4, 33, 128, 64], 40, [4, 2, 0, 1, 3], 16, False, 0),   # mixed query tokens, none
    ([(1000, 6)], [40] * 6, 128, 1, 64, False, 0),
    ([(257, 3)], [70, 2, 300], 200, 2, 128, False, 0),                       # more than 128 rows a token
    ([(640, 9)], [64] * 9, 20, 1, 256, False, 0),
    ([(900, 4)], [100, 200, 1, 64], 32, 2, 64, False, 1),
    ([(900, 4)], [100, 200, 1, 64], 32, 2, 64, False, 7),                    # forced pieces: more than are merged at once
    ([(512, 4)], [1, 17, 64, 65], 16, 1, 64, True, 0),
    ([(4097, 7), (1500, 6)], [2, 777, 50, 64, 128, 4, 9, 100, 300, 2, 65, 63, 31], 40, 2, 16, True, 0),
    ([(130, 2), (0, 1), (65, 3)], [3, 100, 64, 1, 129, 5], 128, 1, 32, True, 3),
]


@pytest.mark.parametrize("i", range(len(SMALL)))
def test_shared(i):
    prefix, own, heads, sq, page, fp8, splits = SMALL[i]
    Case(prefix, own, heads, sq, page, fp8, seed=i, splits=splits).run().check()


@pytest.mark.parametrize("fp8", [False, True])
def test_sharp_scores_and_negative_scale(fp8):
    Case([(700, 3)], [100, 1, 64], 16, 1, 64, fp8, seed=3, q_std=6.0).run().check()
    Case([(700, 3)], [100, 1, 64], 16, 1, 64, fp8, seed=4, scale=-SCALE).run().check()


def test_many_requests_and_groups():
    # more groups of rows than the plan keeps in shared memory
    rng = np.random.default_rng(5)
    own = [int(x) for x in rng.integers(1, 40, 1100)]
    Case([(200, 500), (64, 600)], own, 3, 1, 16, False, seed=5).run().check()


def test_same_as_decode_over_concatenated_pages():
    # a prefix that fills its pages: the concatenated table is a plain decode
    c = Case([(256, 4)], [100, 64, 1, 200], 16, 1, 64, False, seed=6).run().check()
    table = torch.cat([c.prefix_table.expand(4, -1)[:, :4], c.block_table], dim=1).contiguous()
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    ws = torch.empty(mla.decode_workspace_size(4, 4, 16), dtype=torch.uint8, device="cuda")
    c.pages.cache.nan_to_num_(0.0)
    mla.decode(c.q_abs, c.q_pe, c.pages.cache, table, c.seq_lens + 256, out, ws, scale=SCALE, lse=lse)
    # each side within its own roundings
    assert (lse - c.lse).abs().max() < 1e-3
    assert (out.float() - c.out.float()).abs().max() < 2e-2 * c.out.float().abs().max() + 1e-2


def test_rows_outside_every_request_are_left():
    c = Case([(100, 2)], [20, 30], 16, 2, 64, seed=7)
    # query_start_loc covers tokens 0..2 only
    c.qsl = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    c.at, c.sq = np.array([0, 1, 3]), [1, 2]
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    c.run().check()
    assert (c.out[3] == 7).all() and (c.lse[3] == 7).all()


def test_device_errors():
    good = ([(300, 2), (64, 1)], [20, 30, 200])
    # a bad page reads as zeros and is reported; the others' rows are not touched
    c = Case(*good, 16, seed=8)
    c.prefix_table[0, 2] = 10 ** 6
    c.run()
    torch.cuda.synchronize()
    assert mla.decode_status(c.workspace) == 4 and c.out.isfinite().all()
    # lengths beyond their tables are cut
    for name in ("prefix_lens", "seq_lens"):
        c = Case(*good, 16, seed=8)
        getattr(c, name)[0] = 1 << 20
        c.run()
        torch.cuda.synchronize()
        assert mla.decode_status(c.workspace) & 2
    # inconsistent requests or query rows: nothing is written
    for begin in ([0, 2, 2], [1, 2, 3], [0, 3, 2], [0, -1, 3], [0, 2, 1 << 30]):
        c = Case(*good, 16, seed=8)
        c.prefix_requests.copy_(torch.tensor(begin))
        c.run()
        torch.cuda.synchronize()
        assert mla.decode_status(c.workspace) == 8 and c.out.isnan().all() and c.lse.isnan().all()
    for qsl in ([0, 1, 2, 4], [0, 2, 1, 3], [-1, 1, 2, 3]):
        c = Case(*good, 16, seed=8)
        c.qsl = torch.tensor(qsl, dtype=torch.int32, device="cuda")
        c.run()
        torch.cuda.synchronize()
        assert mla.decode_status(c.workspace) == 8 and c.out.isnan().all()
    c = Case(*good, 16, seed=8)
    c.prefix_lens[0] = -5
    c.prefix[0] = (0, 2)
    c.pages.lengths[0] = 0
    c.run().check()


def test_captured_and_replayed_over_other_lengths():
    c = Case([(512, 3), (300, 2)], [64, 100, 1, 200, 129], 32, 1, 64, seed=9).run().check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for prefix, own, begin in (((400, 77), [64, 50, 0, 130, 1], [0, 3, 5]), ((1, 0), [1, 1, 1, 1, 1], [0, 1, 5]),
                               ((512, 300), [64, 100, 1, 200, 129], [0, 5, 5])):
        c.prefix = [(p, b - a) for p, a, b in zip(prefix, begin, begin[1:])]
        c.own, c.begin = own, np.array(begin)
        c.pages.lengths = list(prefix) + own
        c.prefix_lens.copy_(torch.tensor(prefix))
        c.seq_lens.copy_(torch.tensor(own))
        c.prefix_requests.copy_(torch.tensor(begin))
        c.pages.cache.nan_to_num_(0.0)
        c.out.fill_(float("nan"))
        g.replay()
        c.check()


def test_same_bits_beside_other_work():
    c = Case([(3000, 20), (100, 12)], [int(x) for x in np.random.default_rng(1).integers(1, 300, 32)], 16, 1, 64, seed=10)
    c.run().check()
    want, lse = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    a = torch.randn(2048, 2048, device="cuda", dtype=torch.bfloat16)
    for _ in range(10):
        with torch.cuda.stream(side):
            a @ a
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and torch.equal(c.lse, lse)


def test_other_stream():
    c = Case([(512, 3)], [64, 100, 1], 16, 1, 64, seed=11)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    c.check()


@pytest.mark.parametrize("seed", range(24))
def test_drawn(seed):
    rng = np.random.default_rng(100 + seed)
    G = int(rng.choice([1, 1, 2, 3]))
    prefix = [(int(rng.choice([0, 1, 63, 64, 65, 500, 1000])) + int(rng.integers(0, 40)) * int(rng.random() < 0.5),
               int(rng.integers(0, 6))) for _ in range(G)]
    if sum(r for _, r in prefix) == 0:
        prefix[0] = (prefix[0][0], 2)
    B = sum(r for _, r in prefix)
    heads = int(rng.choice([1, 2, 5, 16, 20, 40, 64, 128]))
    sq = int(rng.choice([1, 1, 2])) if rng.random() < 0.6 else [int(x) for x in rng.integers(0, 5, B)]
    if not isinstance(sq, int) and sum(sq) == 0:
        sq[0] = 1
    own = [int(rng.choice([0, 1, 16, 63, 64, 130, 300])) + int(rng.integers(0, 5)) for _ in range(B)]
    Case(prefix, own, heads, sq, int(rng.choice([16, 32, 64, 128, 256])), bool(rng.random() < 0.4), seed=seed,
         splits=int(rng.choice([0, 0, 0, 1, 3]))).run().check()


def test_wait_that_runs_out_is_reported():
    c = Case([(512, 3)], [64, 100, 1], 16, 1, 64, seed=12)
    try:
        mla.set_decode_wait_test(True, 2_000_000)
        c.run()
    finally:
        mla.set_decode_wait_test(False, 0)
    torch.cuda.synchronize()
    assert mla.decode_status(c.workspace) & mla.DEVERR_TIMEOUT
    c.run().check()
