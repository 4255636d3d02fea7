"""The bar of tests/exact_scores.py tells the two ways of exchanging partial
scores apart: codes pass it."""
import pytest
import torch

import exact_scores


@pytest.mark.parametrize("keys", [70, 300, 3000])
def test_codes_are_further_off_than_the_bar(keys):
    g = torch.Generator().manual_seed(keys)
    q, k = exact_scores.queries((64, 576), g).double(), exact_scores.keys((keys, 576), g).double()
    s = exact_scores.SCALE * (q @ k.t())
    lse = torch.logsumexp(s, dim=1)
    bar = exact_scores.lse_bar(s, lse)
    assert bar.max() < 3e-5
    off = (exact_scores.coded_lse(q, k) - lse).abs() > bar
    assert off.double().mean() > (0.5 if keys < 3000 else 0.1)      # (of 64 rows; one is enough)


def test_scores_of_float32_are_exact():
    g = torch.Generator().manual_seed(1)
    q, k = exact_scores.queries((64, 576), g), exact_scores.keys((300, 576), g)
    assert torch.equal((q.float() @ k.float().t()).double(), q.double() @ k.double().t())
    assert torch.equal(k.float().to(torch.float8_e4m3fn).double(), k.double())
