"""GPU tests of the prefill whose values say which key they belong to, and of
values that are not finite across the cuts.

A value row is zero but for one dim, the key's tile (or its place in the tile)
modulo 128, so an output is a sum of probabilities of a few tiles' keys, all
terms positive: a tile that is lost, repeated or taken for another one changes
it by 3 % or more (100000 keys: up to seven tiles a dim, weighted 1 to 7).

Tolerance, all relative to the output.  Probabilities are rounded to bf16
(2^-8) and so is the output (2^-8); a score is off by at most e = 3.3e-4 for
the normal inputs drawn here, in numerator and sum; float32 sums of up to
100000 positive terms, 16 to a product, are off by at most 6250 * 2^-23, with
the sum of the probabilities (814 additions in a row) below 2^-10.
"""
import math

import pytest
import torch

import prompt_ref
from test_gpu_prefill import SCALE, Case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla

REL = (1 + 2.0 ** -8) * (1 + 2.0 ** -8) * (1 + 6.6e-4 + 2.0 ** -10) - 1


def mark(c, kv_lens, dims, weights):
    """Value rows of key j of each sequence: weights(j) in dim dims(j)."""
    c.kv[..., 128:] = 0
    for k0, n in zip(c.at_kv, kv_lens):
        j = torch.arange(n, device="cuda")
        c.kv[k0 + j, :, 128 + dims(j)] = weights(j).to(torch.bfloat16)[:, None]


def check(c, causal):
    torch.cuda.synchronize()
    assert mla.prefill_status(c.ws) == 0
    want, lse, _ = prompt_ref.prefill_torch(c.q, c.kv, c.k_pe, c.at_q, c.at_kv, SCALE, causal)
    excess = (c.out.double() - want).abs() - REL * want
    assert excess.max().item() <= 0, f"output {excess.max().item():.3g} over its bound"
    seen = ~lse.isinf()
    assert ((c.lse.double() - lse).abs() <= 3.3e-4 + 2.0 ** -20 * lse.abs())[seen].all()


@pytest.mark.parametrize("q_lens,kv_lens,heads,splits", [
    ([1], [20000], 1, 0), ([1], [70000], 1, 0), ([1], [70000], 1, 7), ([40], [70000], 3, 0), ([1], [16384], 5, 1),
    ([1] * 8, [8191, 4097, 1, 777, 6000, 129, 8000, 0], 16, 0), ([512], [9000], 20, 0), ([600], [9001], 3, 4),
    ([700, 1, 300], [900, 5000, 20000], 16, 0), ([3000], [3000], 9, 0), ([1] * 63 + [600], [1000] * 63 + [100000], 16, 0),
    ([256] * 9, [256] * 9, 70, 0)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_takes_every_key_tile_once(q_lens, kv_lens, heads, splits, causal):
    c = Case(q_lens, kv_lens, heads, seed=51, splits=splits)
    mark(c, kv_lens, lambda j: j // 128 % 128, lambda j: 1.0 + j // 16384)
    check(c.run(causal), causal)


@pytest.mark.parametrize("q_lens,kv_lens,heads", [([1], [300], 2), ([37], [37], 16), ([129, 1], [1500, 1001], 3),
                                                  ([512], [513], 2), ([257], [1023], 70), ([5] * 40, [17 * i for i in range(40)], 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_takes_every_key_of_a_tile_once(q_lens, kv_lens, heads, causal):
    c = Case(q_lens, kv_lens, heads, seed=52)
    mark(c, kv_lens, lambda j: j % 128, lambda j: 1.0 + j // 128)
    check(c.run(causal), causal)


@pytest.mark.parametrize("low", [0, 1, 3])
@pytest.mark.parametrize("splits", [0, 1, 4])
def test_prefill_value_that_is_not_finite_counts_wherever_the_keys_are_cut(low, splits):
    """A quarter of the keys scores 150 below the others, so that all its
    probabilities are zeros in float32.  An infinity among their values makes
    the output not finite all the same (0 * inf), in one piece or cut."""
    keys = 4096
    c = Case([1, 2], [keys, keys], 1, seed=53, splits=splits)
    level = torch.zeros(keys, device="cuda")
    level[1024 * low:1024 * (low + 1)] = -150.0
    c.q[..., 128:] = 0
    c.q[..., 128] = 1.0
    c.k_pe[:, 0] = (level.repeat(2) / SCALE).to(torch.bfloat16)
    c.kv[1024 * low + 100, 0, 128 + 5] = float("inf")          # of the first sequence
    c.kv[1024 * low + 300, 0, 128 + 77] = float("nan")
    c.run()
    torch.cuda.synchronize()
    want = torch.zeros_like(c.out, dtype=torch.bool)
    want[0, 0, 5] = want[0, 0, 77] = True
    assert torch.equal(~torch.isfinite(c.out), want)
    assert torch.isfinite(c.lse).all()
