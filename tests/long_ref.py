"""Plain 64-bit forms of the operators of long contexts (shared prefixes, key
weights, eviction), and their inputs, for the tests."""
from __future__ import annotations

import numpy as np
import torch

LKV, ROPE, DQK = 512, 64, 576
SCALE = 192 ** -0.5


class Pages:
    """A paged cache whose rows behind each sequence's last key, and whose
    pages of no sequence, hold NaN."""

    def __init__(self, lengths, page, fp8=False, seed=0, std=1.0, spare=3, kv_scale=6.0 / 448.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lengths, self.page, self.fp8 = list(lengths), page, fp8
        counts = [-(-n // page) for n in lengths]
        blocks = sum(counts) + spare
        perm = torch.randperm(blocks, generator=g, device="cuda").cpu()
        self.table = torch.full((len(lengths), max(counts + [1])), -1, dtype=torch.int32)
        cache = torch.full((blocks, page, DQK), float("nan"), dtype=torch.bfloat16, device="cuda")
        at = 0
        for i, n in enumerate(lengths):
            self.table[i, :counts[i]] = perm[at:at + counts[i]].to(torch.int32)
            at += counts[i]
        self.table = self.table.cuda()
        for i, n in enumerate(lengths):
            if n:
                cache.view(-1, DQK)[self.slots(i, n)] = (torch.randn(n, DQK, generator=g, device="cuda") * std).bfloat16()
        self.kv_scale = kv_scale if fp8 else 1.0
        if fp8:
            codes = (cache.float() / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            codes.view(torch.uint8)[cache.isnan()] = 0x7F
            cache = codes
        self.cache, self.g = cache, g

    def slots(self, i, n):
        at = torch.arange(n, device="cuda")
        return self.table[i, at // self.page].long() * self.page + at % self.page

    def rows(self, i, n=None):
        """Rows of sequence i in float64."""
        n = self.lengths[i] if n is None else n
        flat = self.cache.view(torch.uint8).view(-1, DQK) if self.fp8 else self.cache.view(-1, DQK)
        rows = flat[self.slots(i, n)]
        return rows.view(torch.float8_e4m3fn).double() * self.kv_scale if self.fp8 else rows.double()

    def queries(self, tokens, heads, std=1.0):
        q = [(torch.randn(tokens, heads, d, generator=self.g, device="cuda") * std).bfloat16() for d in (LKV, ROPE)]
        return q


def attention(q, keys, scale, seen):
    """q [heads, 576], keys [n, 576] in float64: (out, lse, mean absolute
    weighted value) over the first `seen` keys."""
    seen = max(0, min(seen, keys.shape[0]))
    if seen == 0:
        z = torch.zeros(q.shape[0], LKV, dtype=torch.float64, device=q.device)
        return z, torch.full((q.shape[0],), -np.inf, dtype=torch.float64, device=q.device), z
    s = scale * (q @ keys[:seen].t())
    lse = torch.logsumexp(s, dim=1)
    p = torch.exp(s - lse[:, None])
    return p @ keys[:seen, :LKV], lse, p @ keys[:seen, :LKV].abs()


def select(weights, n, budget, sinks, recent):
    """Kept indices of one request (numpy float32 weights, n keys)."""
    if n <= budget:
        return np.arange(n)
    lo, hi = sinks, n - recent
    w = weights[lo:hi].astype(np.float64)
    w = np.where(np.isnan(w), -np.inf, w)
    below = np.isnan(weights[lo:hi])             # NaN below -inf
    order = np.lexsort((np.arange(hi - lo), -w, below))
    middle = np.sort(order[:budget - sinks - recent]) + lo
    return np.concatenate([np.arange(lo), middle, np.arange(hi, n)])
