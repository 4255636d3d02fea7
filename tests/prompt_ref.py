"""Plain 64-bit forms of the prompt-side operators (numpy), for the tests."""
from __future__ import annotations

import numpy as np

LKV, ROPE, NOPE, VDIM = 512, 64, 128, 128


def rotate(x, cos, sin, interleaved):
    """x [..., 64] with cos, sin [..., 32] broadcast against its pairs."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    out = np.empty_like(x)
    if interleaved:
        out[..., 0::2], out[..., 1::2] = ra, rb
    else:
        out[..., :32], out[..., 32:] = ra, rb
    return out


def append_rows(kv_c, k_pe, positions, table, weight, eps, interleaved):
    """[c | rot(k_pe)] rows in float64."""
    c = kv_c
    if weight is not None:
        c = kv_c / np.sqrt(np.mean(kv_c ** 2, axis=1, keepdims=True) + eps) * weight
    t = table[positions]
    return np.concatenate([c, rotate(k_pe, t[:, :32], t[:, 32:], interleaved)], axis=1)


def prefill(q, kv, k_pe, cu_q, cu_kv, scale, causal, live=None):
    """(out, lse, mean absolute weighted value) of packed sequences in float64;
    keys a row does not see contribute nothing, whatever they hold.  ``live``:
    rows of q that belong to a sequence (others are left NaN)."""
    T, N, _ = q.shape
    out = np.full((T, N, VDIM), np.nan)
    mag = np.full((T, N, VDIM), np.nan)
    lse = np.full((T, N), np.nan)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_kv[b], cu_kv[b + 1]
        sq, sk = q1 - q0, k1 - k0
        for i in range(sq):
            n = sk if not causal else min(sk, max(0, sk - sq + 1 + i))
            if n == 0:
                out[q0 + i], mag[q0 + i], lse[q0 + i] = 0.0, 0.0, -np.inf
                continue
            k, v = kv[k0:k0 + n, :, :NOPE], kv[k0:k0 + n, :, NOPE:]
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (np.einsum("nd,jnd->nj", q[q0 + i, :, :NOPE], k) + q[q0 + i, :, NOPE:] @ k_pe[k0:k0 + n].T)
                m = s.max(axis=1, keepdims=True)
                p = np.exp(s - m)
                tot = p.sum(axis=1, keepdims=True)
                out[q0 + i] = np.einsum("nj,jnd->nd", p / tot, v)
                mag[q0 + i] = np.einsum("nj,jnd->nd", p / tot, np.abs(v))
                lse[q0 + i] = (m + np.log(tot))[:, 0]
    return out, lse, mag


def prefill_torch(q, kv, k_pe, cu_q, cu_kv, scale, causal):
    """The same on the tensors' device in torch float64 (finite inputs)."""
    import torch
    T, N, _ = q.shape
    out = torch.zeros((T, N, VDIM), dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lse = torch.full((T, N), -np.inf, dtype=torch.float64, device=q.device)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_kv[b], cu_kv[b + 1]
        sq, sk = q1 - q0, k1 - k0
        if sq == 0 or sk == 0:
            continue
        for h in range(N):
            x, y = q[q0:q1, h].double(), kv[k0:k1, h].double()
            s = scale * (x[:, :NOPE] @ y[:, :NOPE].t() + x[:, NOPE:] @ k_pe[k0:k1].double().t())
            if causal:
                i = torch.arange(sq, device=q.device)[:, None] + sk - sq
                s = s.masked_fill(torch.arange(sk, device=q.device)[None] > i, -np.inf)
            l = torch.logsumexp(s, dim=1)
            p = torch.exp(s - torch.where(l.isinf(), 0.0, l)[:, None])
            out[q0:q1, h], mag[q0:q1, h], lse[q0:q1, h] = p @ y[:, NOPE:], p @ y[:, NOPE:].abs(), l
    return out, lse, mag
