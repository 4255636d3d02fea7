"""GPU tests of the expanded attention against float64 on the same bf16 inputs.

Tolerance.  A score is a sum of 192 products in float32; with each addition off
by at most 2^-23 of the running magnitude it is off by at most
e = 192 * 2^-23 * scale * sum |q||k|, and sum |q||k| * scale stays below 14 for
the normal inputs drawn here (below 14 * sharp with the query scaled): e <=
3.3e-4 * sharp.  The probabilities and their sum are then off by e relative
each, the bf16 rounding of a probability by 2^-8, so that an output is off by
at most (2^-8 + 2 e + 2^-18) of the mean magnitude of the values it averages,
plus its own rounding of 2^-8; the LSE by e, and 2^-20 of its value.
"""
import math

import numpy as np
import pytest
import torch

import prompt_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla

SCALE = 1.0 / math.sqrt(192)


def starts(n):
    return [0] + list(np.cumsum(n))


class Case:
    def __init__(self, q_lens, kv_lens, heads, seed=0, sharp=1.0, pad_q=0, pad_kv=0, splits=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

        self.sharp, self.splits = sharp, splits
        self.at_q, self.at_kv = starts(q_lens), starts(kv_lens)
        T, Tk = self.at_q[-1] + pad_q, self.at_kv[-1] + pad_kv
        self.q, self.kv, self.k_pe = rnd(T, heads, 192, scale=sharp), rnd(Tk, heads, 256), rnd(Tk, 576)[:, 512:]
        self.cu_q = torch.tensor(self.at_q, dtype=torch.int32, device="cuda")
        self.cu_kv = torch.tensor(self.at_kv, dtype=torch.int32, device="cuda")
        self.out = torch.full((T, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((T, heads), 7.0, device="cuda")
        n = mla.prefill_workspace_size(len(q_lens), T, heads, splits) if T else 256
        self.ws = torch.full((n,), 0xEE, dtype=torch.uint8, device="cuda")

    def run(self, causal=True, scale=SCALE, stream=None):
        mla.prefill(self.q, self.kv, self.k_pe, self.cu_q, self.cu_kv, self.out, self.ws, scale=scale, causal=causal,
                    lse=self.lse, num_splits=self.splits, stream=stream)
        return self

    def check(self, causal=True, scale=SCALE):
        torch.cuda.synchronize()
        assert mla.prefill_status(self.ws) == 0
        n = self.at_q[-1]
        out, lse, mag = prompt_ref.prefill_torch(self.q, self.kv, self.k_pe, self.at_q, self.at_kv, scale, causal)
        got, gl = self.out[:n].double(), self.lse[:n].double()
        assert torch.isfinite(got).all()
        e = 3.3e-4 * self.sharp * scale / SCALE
        bound = 2.0 ** -8 * out[:n].abs() + (2.0 ** -8 + 2 * e + 2.0 ** -18) * mag[:n]
        excess = ((got - out[:n]).abs() - bound).max().item() if n else 0.0
        assert excess <= 0, f"output {excess:.3g} over its bound"
        empty = lse[:n] == -math.inf
        assert torch.equal(gl == -math.inf, empty) and (got[empty] == 0).all()
        err = (gl - lse[:n])[~empty].abs()
        assert (err <= e + 2.0 ** -20 * lse[:n][~empty].abs()).all(), f"LSE off by {err.max().item():.3g}"
        # rows behind the last sequence are left as they were
        assert (self.out[n:] == 7.0).all() and (self.lse[n:] == 7.0).all()
        return self


SHAPES = [
    ([1], [1], 1), ([1], [1], 16), ([1], [300], 3), ([2], [2], 1), ([37], [37], 16), ([127], [127], 2),
    ([128], [128], 3), ([129], [129], 2), ([255], [255], 1), ([256], [256], 2), ([257], [257], 2), ([1000], [1000], 2),
    ([1, 1, 1, 1], [1, 0, 129, 5000], 16), ([5, 0, 300, 1], [5, 7, 300, 0], 5), ([0, 0, 3], [0, 9, 3], 2),
    ([100], [1500], 4), ([300], [2000], 3), ([513], [700], 7), ([700], [300], 3), ([64] * 20, [64] * 20, 2),
    ([33, 65, 200, 1, 17], [400, 65, 260, 900, 17], 20), ([2], [6000], 128), ([40], [7000], 1), ([1500], [1500], 40),
]


@pytest.mark.parametrize("q_lens,kv_lens,heads", SHAPES)
@pytest.mark.parametrize("causal", [True, False])
def test_prefill(q_lens, kv_lens, heads, causal):
    Case(q_lens, kv_lens, heads, seed=sum(q_lens) + sum(kv_lens) + heads, pad_q=3, pad_kv=5).run(causal).check(causal)


@pytest.mark.parametrize("q_lens,kv_lens,heads,splits", [
    ([1], [700], 2, 3), ([300], [900], 2, 4), ([1, 40, 600], [50, 1000, 600], 3, 5), ([256], [2000], 1, 100),
    ([10, 0, 3], [0, 5, 400], 2, 2), ([700], [300], 2, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_forced_splits(q_lens, kv_lens, heads, splits, causal):
    Case(q_lens, kv_lens, heads, seed=splits, splits=splits, pad_q=1).run(causal).check(causal)


@pytest.mark.parametrize("sharp", [8.0, 40.0])
def test_prefill_sharp_scores(sharp):
    """Scores of a few sharp peaks: the running reference rises often."""
    Case([300, 70], [800, 70], 4, seed=5, sharp=sharp).run().check()


def test_prefill_rising_scores():
    """Keys sorted so that every tile raises every row's maximum by far more
    than the rescaling threshold, and the reverse."""
    for sign in (1.0, -1.0):
        c = Case([200], [1000], 2, seed=6)
        ramp = sign * torch.linspace(-30, 30, 1000, device="cuda")
        c.q[..., 128:] = 0
        c.q[..., 128] = 1.0
        c.k_pe[:, 0] = (ramp / SCALE).to(torch.bfloat16)
        c.sharp = 4.0       # sum |q||k| * scale is below 44 here
        c.run().check()


def test_prefill_many_sequences():
    g = np.random.Generator(np.random.PCG64(3))
    q = [int(x) for x in g.integers(0, 20, 700)]
    kv = [int(x) for x in g.integers(0, 40, 700)]
    Case(q, kv, 2, seed=7).run().check()


def test_prefill_large_scale_and_small_scale():
    for scale in (1e-6, 0.5):
        c = Case([150], [400], 2, seed=8)
        c.run(scale=scale).check(scale=scale)


def test_prefill_strided_layouts():
    """Head-major queries and keys, column ranges of wider rows."""
    c = Case([90, 200], [300, 200], 3, seed=9)
    want = c.run().out.clone()
    torch.cuda.synchronize()
    c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((500, 3, 320), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., 32:288] = c.kv
    c.kv = wide[..., 32:288]
    c.k_pe = c.k_pe.contiguous()
    c.out.fill_(7.0)
    c.run().check()
    assert torch.equal(c.out, want)


def test_prefill_garbage_outside_the_sequences():
    """Key rows of no sequence and of the next sequence may hold NaN, and so
    may query rows behind the last one."""
    c = Case([70, 130], [100, 333], 3, seed=10, pad_q=40, pad_kv=60)
    c.q[200:], c.kv[433:], c.k_pe[433:] = float("nan"), float("nan"), float("inf")
    c.run().check()
    # the second sequence's keys are NaN: the first is not touched by them
    c.kv[100:433] = float("nan")
    c.run()
    torch.cuda.synchronize()
    first = Case([70], [100], 3)
    first.q, first.kv, first.k_pe = c.q[:70], c.kv[:100], c.k_pe[:100]
    first.out, first.lse, first.ws = c.out[:70], c.lse[:70], c.ws
    first.check()
    assert torch.isnan(c.out[70:200]).all()


@pytest.mark.parametrize("splits", [0, 3])
def test_prefill_non_finite_keys_reach_only_the_rows_that_see_them(splits):
    """Infinities and NaN in values and keys of one sequence: a row before them
    is what it is without them, in every output."""
    c = Case([300, 20], [420, 20], 2, seed=16, splits=splits)
    clean = c.kv.clone()
    c.kv[200, 0, 130] = float("inf")          # a value: query rows 80.. of sequence 0 see key 200
    c.kv[333, 1, 255] = float("nan")          # rows 213..
    c.kv[422, 1, 140] = float("-inf")         # sequence 1, rows 2..
    c.kv[419, 0, 5] = float("nan")            # a key: row 299 alone
    c.run()
    torch.cuda.synchronize()
    bad = ~torch.isfinite(c.out)
    want = torch.zeros_like(bad)
    want[80:300, 0, 2] = True
    want[213:300, 1, 127] = True
    want[302:320, 1, 12] = True
    want[299, 0] = True
    assert torch.equal(bad, want)
    kv, c.kv = c.kv, clean
    ref, lse, mag = prompt_ref.prefill_torch(c.q, c.kv, c.k_pe, c.at_q, c.at_kv, SCALE, True)
    err = (c.out.double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 6.6e-4 + 2.0 ** -18) * mag)[~want].all()
    fine = torch.isfinite(c.lse)
    assert not fine[299, 0] and fine.sum() == fine.numel() - 1
    assert ((c.lse.double() - lse).abs() <= 3.3e-4 + 2.0 ** -20 * lse.abs())[fine].all()


@pytest.mark.parametrize("rows", [100, 200])
def test_prefill_non_finite_keys_of_short_sequences(rows):
    """The same for sequences of one query tile, whose key tiles alternate."""
    c = Case([rows], [500], 2, seed=18)
    clean = c.kv.clone()
    c.kv[470, 0, 130] = float("inf")
    c.kv[390 + 3, 1, 200] = float("nan")       # seen by every row when rows is 100
    c.run()
    torch.cuda.synchronize()
    want = torch.zeros_like(c.out, dtype=torch.bool)
    i = torch.arange(rows, device="cuda")
    want[:, 0, 2] = i >= 470 - (500 - rows)
    want[:, 1, 72] = i >= 393 - (500 - rows)
    assert torch.equal(~torch.isfinite(c.out), want) and torch.isfinite(c.lse).all()
    ref, lse, mag = prompt_ref.prefill_torch(c.q, clean, c.k_pe, c.at_q, c.at_kv, SCALE, True)
    err = (c.out.double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 6.6e-4 + 2.0 ** -18) * mag)[~want].all()


@pytest.mark.parametrize("q_lens,kv_lens,heads", [([1] * 8, [8191, 4097, 1, 777, 6000, 129, 8000, 0], 16),
                                                  ([512], [9000], 20), ([600, 1, 256, 257], [600, 9001, 3000, 2570], 8),
                                                  ([1], [20000], 1), ([3000], [3000], 9), ([256] * 9, [256] * 9, 70)])
def test_prefill_balanced_over_the_pairs(q_lens, kv_lens, heads):
    """Few items: each is cut where the pairs' spans end, in pieces of any
    number of tiles."""
    Case(q_lens, kv_lens, heads, seed=19).run(True).check(True)
    Case(q_lens, kv_lens, heads, seed=20).run(False).check(False)


def test_prefill_is_deterministic():
    c = Case([300, 1, 40], [900, 4000, 2000], 16, seed=11).run()
    torch.cuda.synchronize()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.out.fill_(0)
        c.ws.fill_(0xAB)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("q_lens,kv_lens,heads", [([1] * 8, [8191, 4097, 1, 777, 6000, 129, 8000, 0], 16),
                                                  ([100, 256, 17, 200], [3000, 700, 2000, 999], 40),
                                                  ([700, 300, 1000], [700, 900, 1000], 64)])
def test_prefill_gives_the_same_bits_every_time(q_lens, kv_lens, heads):
    """Loads, products and softmax meet in another order in every run."""
    c = Case(q_lens, kv_lens, heads, seed=17).run().check()
    out, lse = c.out.clone(), c.lse.clone()
    busy = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    for k in range(60):
        if k % 2:
            with torch.cuda.stream(side):
                busy.zero_()
        c.out.fill_(0)
        c.run()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    torch.cuda.synchronize()


def test_prefill_captured_and_replayed_over_other_lengths():
    c = Case([100, 50], [400, 50], 4, seed=12).run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    g.replay()
    c.check()
    c.at_q, c.at_kv = [0, 20, 150], [0, 330, 450]
    c.cu_q.copy_(torch.tensor(c.at_q, dtype=torch.int32))
    c.cu_kv.copy_(torch.tensor(c.at_kv, dtype=torch.int32))
    c.out.fill_(7.0)
    g.replay()
    c.check()


def test_prefill_on_two_streams_with_a_workspace_each():
    a, b = Case([400], [400], 8, seed=13), Case([1, 1], [3000, 5], 8, seed=14)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(stream=s1)
        b.run(stream=s2)
    a.check()
    b.check()


def test_prefill_inconsistent_sums_are_flagged_and_write_nothing():
    for cu_q, cu_kv, bit in (([0, 50, 40], [0, 50, 90], mla.DEVERR_BAD_QSL), ([0, 50, 101], [0, 50, 90], mla.DEVERR_BAD_QSL),
                             ([-1, 50, 90], [0, 50, 90], mla.DEVERR_BAD_QSL), ([0, 50, 90], [0, 95, 90], mla.DEVERR_BAD_SEQ_LEN),
                             ([0, 50, 90], [0, 50, 91], mla.DEVERR_BAD_SEQ_LEN)):
        c = Case([50, 50], [50, 40], 2, seed=15)
        c.cu_q.copy_(torch.tensor(cu_q, dtype=torch.int32))
        c.cu_kv.copy_(torch.tensor(cu_kv, dtype=torch.int32))
        c.run()
        torch.cuda.synchronize()
        assert mla.prefill_status(c.ws) == bit
        assert (c.out == 7.0).all() and (c.lse == 7.0).all()
    Case([50, 50], [50, 40], 2, seed=15).run().check()


@pytest.mark.parametrize("q_lens,kv_lens,heads", [([1] * 32, [16] * 32, 5), ([1] * 33, [15] * 33, 5), ([600, 0, 40], [512, 0, 0], 7),
                                                  ([3, 500, 1], [100, 412, 0], 100), ([3, 500, 1], [100, 412, 1], 100)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_around_the_sizes_without_a_plan(q_lens, kv_lens, heads, causal):
    """Up to 32 sequences over up to 512 key rows take one launch."""
    c = Case(q_lens, kv_lens, heads, seed=21, pad_q=2).run(causal).check(causal)
    c.cu_q[-1] = c.q.shape[0] + 1
    c.out.fill_(7.0)
    c.run(causal)
    torch.cuda.synchronize()
    assert mla.prefill_status(c.ws) == mla.DEVERR_BAD_QSL and (c.out == 7.0).all()


def test_prefill_without_rows_or_keys():
    Case([0, 0], [3, 4], 2).run()                       # no query row: nothing to do
    c = Case([5, 300], [0, 0], 2).run()                 # no key at all
    c.check()
    c = Case([5], [9], 2)
    mla.prefill(c.q, c.kv, c.k_pe, c.cu_q, c.cu_kv, c.out, c.ws, scale=SCALE)    # no LSE wanted
    torch.cuda.synchronize()
    assert (c.lse == 7.0).all() and not (c.out == 7.0).all()


@pytest.mark.parametrize("q_lens,kv_lens,heads", [([300], [300], 2), ([700, 1], [900, 5000], 16), ([4000], [4000], 40)])
def test_prefill_waits_are_bounded(q_lens, kv_lens, heads):
    """Keys that never arrive: the waits for them run out, the call returns and
    says so, and the next one is clean."""
    c = Case(q_lens, kv_lens, heads, seed=22)
    try:
        mla.set_decode_wait_test(skip_first_tile=True, wait_limit_ns=2_000_000)
        c.run()
        torch.cuda.synchronize()
        assert mla.prefill_status(c.ws) & mla.DEVERR_TIMEOUT
    finally:
        mla.set_decode_wait_test()
    c.run().check()


def test_prefill_mending_rows_outlasts_the_wait_limit():
    """An infinity that only the last row sees: the rows beside it are computed
    again over 16000 keys, which takes longer than the waits' limit set here;
    the time does not count as a wait that ran out."""
    heads, keys = 170, 16000
    c = Case([300], [keys], heads, seed=31, splits=1)
    clean = c.kv.clone()
    c.kv[keys - 1, :, 128] = float("inf")
    try:
        mla.set_decode_wait_test(wait_limit_ns=2_000_000)
        c.run()
        torch.cuda.synchronize()
        assert mla.prefill_status(c.ws) == 0
    finally:
        mla.set_decode_wait_test()
    assert (c.out[299, :, 0] == float("inf")).all()
    c.out[299, :, 0] = 0
    assert torch.isfinite(c.out).all()
    for h in (0, 80, 169):
        ref, lse, mag = prompt_ref.prefill_torch(c.q[:, h:h + 1], clean[:, h:h + 1], c.k_pe, c.at_q, c.at_kv, SCALE, True)
        err = (c.out[:299, h:h + 1].double() - ref[:299]).abs()
        assert (err <= 2.0 ** -8 * ref[:299].abs() + (2.0 ** -8 + 6.6e-4 + 2.0 ** -18) * mag[:299]).all()


@pytest.mark.parametrize("q_lens,kv_lens,heads", [
    ([1] * 8, [8191, 4097, 1, 777, 6000, 129, 8000, 0], 16), ([512], [9000], 20), ([600, 1, 256, 257], [600, 9001, 3000, 2570], 8),
    ([1], [70000], 1), ([1] * 31 + [300], [0] * 31 + [5000], 3), ([0, 3, 0, 700, 2], [900, 3, 5, 2900, 1], 5),
    ([5000], [5000], 7), ([16] * 32, [130, 2000] * 16, 2), ([1, 513], [1300, 1024], 37), ([2, 3], [600, 513], 150),
    ([260] * 3, [1025, 1030, 1100], 60), ([1] * 20, [1024 + 130 * i for i in range(20)], 30)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_with_and_without_a_plan(q_lens, kv_lens, heads, causal):
    """Up to 32 sequences the pairs find and cut their items by themselves; with
    more (empty ones here) a plan does.  The pieces are the same, and so are
    the results to the bit."""
    a = Case(q_lens, kv_lens, heads, seed=32).run(causal).check(causal)
    none = [0] * 33
    b = Case(q_lens + none, kv_lens + none, heads, seed=32).run(causal)
    torch.cuda.synchronize()
    assert mla.prefill_status(b.ws) == 0
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
