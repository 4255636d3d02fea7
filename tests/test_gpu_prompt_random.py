"""Drawn configurations of the prompt-side operators: lengths around the tile,
block and span sizes, any head count, forced and automatic splits.  The
tolerances are those of each operator's own tests."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import test_gpu_append
    import test_gpu_kv_proj
    import test_gpu_prefill
    import mla_latent_kv_15_gb300 as mla


def near(rng, bases, spread):
    return max(0, int(rng.choice(bases)) + int(rng.integers(-spread, spread + 1)))


def prefill_case(seed):
    rng = np.random.default_rng(seed)
    batch = int(rng.integers(1, 7)) if rng.random() < 0.8 else int(rng.integers(20, 60))
    q, kv, left = [], [], 40_000_000
    heads = int(rng.choice([1, 2, 3, 5, 8, 16, 20, 40, 70]))
    for _ in range(batch):
        a = near(rng, [0, 1, 16, 64, 128, 256, 512, 600, 1024], 3 if rng.random() < 0.7 else 60)
        b = near(rng, [0, 16, 100, 128, 256, 384, 512, 1000, 2048], 3 if rng.random() < 0.7 else 60)
        b = b + a if rng.random() < 0.5 else b
        if a * b * heads > left:
            a, b = a % 17, b % 300
        left -= a * b * heads
        q.append(a)
        kv.append(b)
    splits = int(rng.choice([0, 0, 0, 1, 2, 5]))
    return q, kv, heads, splits, bool(rng.random() < 0.6), float(rng.choice([1.0, 1.0, 4.0]))


def run_prefill(seed):
    q, kv, heads, splits, causal, sharp = prefill_case(seed)
    if sum(q) == 0:
        q[0] = 5
    test_gpu_prefill.Case(q, kv, heads, seed=seed, sharp=sharp, splits=splits, pad_q=2, pad_kv=1).run(causal).check(causal)


@pytest.mark.parametrize("seed", range(40))
def test_drawn_prefill(seed):
    run_prefill(seed)


@pytest.mark.parametrize("seed", range(16))
def test_drawn_kv_up_proj(seed):
    rng = np.random.default_rng(1000 + seed)
    T = near(rng, [1, 16, 64, 128, 256, 512, 1500], 20) + 1
    N, D = int(rng.integers(1, 50)), int(rng.choice([8, 64, 72, 128, 192, 256, 256, 320]))
    lat, w = test_gpu_kv_proj.data(T, N, D, seed, bool(rng.random() < 0.5))
    kv = torch.full((T, N, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    mla.kv_up_proj(lat[:, :512], w, kv)
    torch.cuda.synchronize()
    test_gpu_kv_proj.check(kv, lat, w)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_append(seed):
    rng = np.random.default_rng(2000 + seed)
    test_gpu_append.test_append(int(rng.integers(1, 400)), int(rng.choice([0, 1, 7, 31, 32, 33, 64, 100])),
                                int(rng.choice([16, 32, 64, 128, 256])), *(bool(x) for x in rng.random(4) < 0.5))
