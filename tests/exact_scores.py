"""Inputs of whole numbers whose scores are exact in float32 however they are
summed, and how far off a row's log-sum-exp may then be where the partial scores
of two CTAs are exchanged as they are: by exponentials, sums and logarithm alone."""
import torch

SCALE = 2.0 ** -8
CODES = 32766                # steps of half the range of 32 keys' partial scores, where they are exchanged as codes


def queries(shape, g):
    return torch.randint(-64, 65, shape, generator=g, device=g.device).to(torch.bfloat16)


def keys(shape, g):
    """Exact in bf16 and in e4m3; with the queries above no partial score passes
    576 * 64 * 2 < 2^17."""
    return torch.randint(-2, 3, shape, generator=g, device=g.device).to(torch.bfloat16)


def lse_bar(scores, lse):
    """Of rows [rows, keys] of scaled scores in float64.  In binary units: scale *
    log2 e, the product with it, and the difference to the maximum are rounded
    (2^-24 of twice the largest score each); the powers of two are within 2^-22,
    their sum that of 16 pairs a tile of 64 keys, of the tiles and of their pieces
    (2^-24 for each step, twice); the logarithm within 2^-22 of 1 or of itself; the
    result is rounded twice."""
    top = scores.abs().amax(dim=1)
    steps = 2 * (16 + 2 * (scores.shape[1] / 64 + 2))
    log_sum = (lse - scores.amax(dim=1)).abs()
    return (3 * 2.0 ** -24 * 2 * top + 2.0 ** -22 + steps * 2.0 ** -24 + 2.0 ** -22 * log_sum.clamp(min=1)
            + 2 * 2.0 ** -24 * lse.abs())


def coded_lse(q, k):
    """What the log-sum-exp becomes where each CTA of a pair has half the columns
    (256 latent, 32 rope ones) and the first gets the other's partial scores as
    codes: 64-bit otherwise.  q [rows, 576], k [keys, 576]."""
    half = [list(range(256 * r, 256 * r + 256)) + list(range(512 + 32 * r, 544 + 32 * r)) for r in (0, 1)]
    mine, other = (q[:, h] @ k[:, h].t() for h in half)
    for a in range(0, k.shape[0], 32):
        part = other[:, a:a + 32]
        hi, lo = part.amax(dim=1, keepdim=True), part.amin(dim=1, keepdim=True)
        step = ((hi - lo) / 2 / CODES).clamp(min=1e-30)
        other[:, a:a + 32] = (hi + lo) / 2 + ((part - (hi + lo) / 2) / step).round() * step
    return torch.logsumexp(SCALE * (mine + other), dim=1)
