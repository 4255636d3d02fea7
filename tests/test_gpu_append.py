"""GPU tests of the rotated, normalised cache append against a 64-bit form.

Tolerance: a stored value is the float32 result rounded once, so it is off by
at most 2^-8 (bf16) or 2^-4 (e4m3, plus half its subnormal step 2^-10 of the
scale) of the value; the float32 arithmetic before it adds at most 2^-21 of
the magnitudes that enter: a rotation is two products and a sum, a norm is a
512-term sum of squares (each lane adds 16 and five shuffles join them: under
24 roundings of 2^-24 in the sum, half of that after the root), a root, a
division and two products.
"""
import numpy as np
import pytest
import torch

import prompt_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla

LKV, ROPE, DQK = 512, 64, 576


def f64(t):
    return t.detach().double().cpu().numpy()


def make_table(n, seed=0):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64.0)
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)).cuda()


class Case:
    def __init__(self, T, N, page, fp8, norm, seed, wide=True):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

        self.down = rnd(T, 64 + DQK if wide else DQK)
        self.kv_c, self.k_pe = self.down[:, -DQK:-ROPE], self.down[:, -ROPE:]
        self.q = rnd(T, max(N, 1), 192)
        self.table = make_table(5000)
        self.positions = torch.randint(0, 5000, (T,), generator=g, device="cuda")
        blocks = -(-T // page) + 3
        self.cache = rnd(blocks, page, DQK)
        self.kv_scale = 1.0
        if fp8:
            self.kv_scale = 0.013
            self.cache = self.cache.to(torch.float8_e4m3fn)
        self.slots = torch.randperm(blocks * page, generator=g, device="cuda")[:T].contiguous()
        self.weight = (1 + 0.2 * torch.randn(LKV, generator=g, device="cuda")).to(torch.bfloat16) if norm else None

    def rows(self, interleaved, eps=1e-6):
        w = None if self.weight is None else f64(self.weight)
        return prompt_ref.append_rows(f64(self.kv_c), f64(self.k_pe), self.positions.cpu().numpy(), f64(self.table), w,
                                      eps, interleaved)

    def magnitude(self, rows):
        """Bound of what enters each value: a rotated value's partners."""
        m = np.abs(rows).copy()
        pe = np.abs(f64(self.k_pe))
        m[:, LKV:] = pe.max(axis=1, keepdims=True) * 2
        return m


def near(got, ref, mag, half_step, floor=0.0):
    err = np.abs(got - ref)
    bound = half_step * np.abs(ref) + floor + 2.0 ** -21 * mag * (1 + half_step)
    assert np.all(err <= bound), f"worst excess {np.max(err - bound):.3g}"


@pytest.mark.parametrize("T,N,page,fp8,norm,interleaved,latent", [
    (1, 16, 64, False, True, True, False), (1, 1, 16, True, True, False, True), (7, 3, 16, False, False, True, True),
    (64, 128, 64, True, True, True, False), (33, 9, 32, True, False, False, True), (130, 20, 256, False, True, False, True),
    (1021, 5, 128, True, True, True, True), (300, 64, 64, False, True, True, True), (19, 1000, 64, False, True, True, False),
    (2, 0, 64, False, True, True, True)])
def test_append(T, N, page, fp8, norm, interleaved, latent):
    c = Case(T, N, page, fp8, norm, seed=T * 7 + N)
    if T > 4:
        c.slots[::3] = -1
        c.slots[1] = c.cache.shape[0] * page            # past the cache: padding too
    before = c.cache.clone()
    q_out = torch.full((T, max(N, 1), ROPE), 7.0, dtype=torch.bfloat16, device="cuda")
    lat = torch.full((T, DQK + 16), 7.0, dtype=torch.bfloat16, device="cuda") if latent else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache,
                         q_pe=c.q[..., 128:] if N else None, q_pe_out=q_out if N else None, norm_weight=c.weight,
                         interleaved=interleaved, kv_scale=c.kv_scale,
                         latent_out=lat[:, :DQK] if latent else None, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    ref = c.rows(interleaved)
    mag = c.magnitude(ref)
    flat, old = f64(c.cache.float()).reshape(-1, DQK), f64(before.float()).reshape(-1, DQK)
    slots = c.slots.cpu().numpy()
    kept = (slots >= 0) & (slots < flat.shape[0])
    if fp8:
        near(flat[slots[kept]] * np.float32(c.kv_scale), ref[kept], mag[kept], 2.0 ** -4, floor=2.0 ** -10 * c.kv_scale)
    else:
        near(flat[slots[kept]], ref[kept], mag[kept], 2.0 ** -8)
    rest = np.ones(flat.shape[0], bool)
    rest[slots[kept]] = False
    assert np.array_equal(flat[rest], old[rest])
    if latent:
        near(f64(lat[:, :DQK]), ref, mag, 2.0 ** -8)
        assert torch.all(lat[:, DQK:] == 7.0)
    if N:
        t = f64(c.table)[c.positions.cpu().numpy()][:, None]
        q = f64(c.q[..., 128:])
        rq = prompt_ref.rotate(q, t[..., :32], t[..., 32:], interleaved)
        near(f64(q_out), rq, np.abs(q).max(axis=-1, keepdims=True) * 2, 2.0 ** -8)
    else:
        assert torch.all(q_out == 7.0)


def test_append_in_place_and_head_major_strides():
    """The query rotated where it lies (columns 128.. of [T, N, 192]), the
    latent rows written over their own inputs, a head-major query."""
    c = Case(41, 6, 64, False, True, seed=3, wide=False)
    ref = c.rows(True)
    q0 = c.q.clone()
    lat = torch.empty(41, DQK, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty(41, 6, ROPE, dtype=torch.bfloat16, device="cuda")
    mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache, q_pe=c.q[..., 128:], q_pe_out=q_out,
                         norm_weight=c.weight, latent_out=lat)
    assert torch.equal(c.q, q0)
    head_major = c.q[..., 128:].transpose(0, 1).contiguous().transpose(0, 1)
    cache1 = c.cache.clone()
    mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache, q_pe=head_major, q_pe_out=head_major,
                         norm_weight=c.weight, latent_out=None)
    assert torch.equal(head_major, q_out)
    mla.rope_cache_write(c.down[:, :LKV], c.down[:, LKV:], c.positions, c.table, c.slots, c.cache,
                         q_pe=c.q[..., 128:], q_pe_out=c.q[..., 128:], norm_weight=c.weight, latent_out=c.down)
    torch.cuda.synchronize()
    assert torch.equal(c.q[..., 128:], q_out) and torch.equal(c.q[..., :128], q0[..., :128])
    assert torch.equal(c.down, lat) and torch.equal(c.cache, cache1)
    near(f64(lat), ref, c.magnitude(ref), 2.0 ** -8)


def test_append_without_norm_is_the_plain_write():
    """Unnormalised rows at position 0 (cos 1, sin 0) are the plain cache
    write's, bit for bit, in both cache types."""
    for fp8 in (False, True):
        c = Case(50, 2, 64, fp8, False, seed=5, wide=False)
        c.positions.zero_()
        other = c.cache.clone()
        mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache, kv_scale=c.kv_scale)
        mla.cache_write(c.kv_c.contiguous(), c.k_pe.contiguous(), c.slots, other, c.kv_scale)
        torch.cuda.synchronize()
        assert torch.equal(c.cache.view(torch.uint8), other.view(torch.uint8))


def test_append_bad_positions_are_flagged_and_skipped():
    c = Case(9, 4, 64, False, True, seed=6)
    c.positions[2], c.positions[7] = -1, 5000
    before, lat = c.cache.clone(), torch.full((9, DQK), 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.full((9, 4, ROPE), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.full((1,), 2, dtype=torch.int32, device="cuda")
    mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache, q_pe=c.q[..., 128:], q_pe_out=q_out,
                         norm_weight=c.weight, latent_out=lat, status=status)
    torch.cuda.synchronize()
    assert status.item() == (2 | mla.DEVERR_BAD_POSITION)
    for t in (2, 7):
        s = int(c.slots[t])
        assert torch.equal(c.cache.view(-1, DQK)[s], before.view(-1, DQK)[s])
        assert torch.all(lat[t] == 7.0) and torch.all(q_out[t] == 7.0)
    assert not torch.any(q_out[0] == 7.0) and not torch.any(lat[8] == 7.0)


def test_append_non_finite_values_stay_in_their_token():
    """A NaN or an infinity spoils its own row's norm and nothing else; an
    e4m3 cache stores NaN as NaN and saturates an infinity."""
    c = Case(6, 1, 64, True, False, seed=8, wide=False)
    c.down[1, 5], c.down[2, 9] = float("nan"), float("inf")
    mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache, kv_scale=c.kv_scale)
    torch.cuda.synchronize()
    rows = c.cache.view(-1, DQK)[c.slots].float()
    assert torch.isnan(rows[1, 5]) and rows[2, 9] == 448
    assert torch.isfinite(rows).sum() == rows.numel() - 1
    c = Case(6, 1, 64, False, True, seed=8, wide=False)
    c.down[1, 5] = float("nan")
    mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache, norm_weight=c.weight)
    torch.cuda.synchronize()
    rows = c.cache.view(-1, DQK)[c.slots].float()
    assert torch.isnan(rows[1, :LKV]).all() and torch.isfinite(rows[1, LKV:]).all()
    assert torch.isfinite(rows[[0, 2, 3, 4, 5]]).all()


def test_append_zero_tokens_and_captured_replay():
    c = Case(16, 8, 64, False, True, seed=9, wide=False)
    e = torch.empty
    mla.rope_cache_write(e(0, 512, dtype=torch.bfloat16, device="cuda"), e(0, 64, dtype=torch.bfloat16, device="cuda"),
                         e(0, dtype=torch.int64, device="cuda"), c.table, e(0, dtype=torch.int64, device="cuda"), c.cache)
    q_out = torch.empty(16, 8, ROPE, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, c.cache, q_pe=c.q[..., 128:],
                             q_pe_out=q_out, norm_weight=c.weight, stream=stream)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    c.down.copy_(torch.randn_like(c.down.float()))
    c.positions.add_(1).remainder_(5000)
    g.replay()
    torch.cuda.synchronize()
    again, cache = q_out.clone(), c.cache.clone()
    side = torch.cuda.Stream()
    c.cache.zero_()
    q_out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert torch.equal(q_out, again)
    assert torch.equal(c.cache.view(-1, DQK)[c.slots], cache.view(-1, DQK)[c.slots])
    ref = c.rows(True)
    near(f64(c.cache).reshape(-1, DQK)[c.slots.cpu().numpy()], ref, c.magnitude(ref), 2.0 ** -8)


def test_append_from_one_fused_projection():
    """Queries and latent rows as column ranges of the same rows, the query
    rotated where it lies; nothing else of the rows changes."""
    T, N = 37, 4
    c = Case(T, N, 64, False, True, seed=12, wide=False)
    fused = torch.empty(T, N * 192 + DQK, dtype=torch.bfloat16, device="cuda")
    q = fused.as_strided((T, N, 192), (fused.stride(0), 192, 1))
    q.copy_(c.q)
    fused[:, N * 192:] = c.down
    before = fused.clone()
    want_q = torch.empty(T, N, ROPE, dtype=torch.bfloat16, device="cuda")
    other = c.cache.clone()
    mla.rope_cache_write(c.kv_c, c.k_pe, c.positions, c.table, c.slots, other, q_pe=c.q[..., 128:], q_pe_out=want_q,
                         norm_weight=c.weight)
    mla.rope_cache_write(fused[:, N * 192:N * 192 + LKV], fused[:, N * 192 + LKV:], c.positions, c.table, c.slots, c.cache,
                         q_pe=q[..., 128:], q_pe_out=q[..., 128:], norm_weight=c.weight)
    torch.cuda.synchronize()
    assert torch.equal(c.cache, other) and torch.equal(q[..., 128:], want_q)
    assert torch.equal(q[..., :128], c.q[..., :128]) and torch.equal(fused[:, N * 192:], before[:, N * 192:])
