"""GPU tests of the latent-to-heads projection against float64 products of the
same bf16 inputs.

Tolerance: one bf16 rounding of the float32 sum (2^-8 of the value) plus the
accumulation's own error: 512 products summed in float32, each addition off by
at most 2^-23 of the running magnitude (the tensor cores may truncate), so by
512 * 2^-23 = 2^-14 of the sum of the magnitudes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla


def data(T, N, D, seed, wide):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lat = torch.randn((T, 576 if wide else 512), generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn((N, D, 512), generator=g, device="cuda") / 512 ** 0.5).to(torch.bfloat16)
    return lat, w


def check(kv, lat, w):
    x, y = lat[:, :512].double(), w.double().reshape(-1, 512)
    ref, mag = (x @ y.t()).view(kv.shape), (x.abs() @ y.abs().t()).view(kv.shape)
    err, bound = (kv.double() - ref).abs(), 2.0 ** -8 * ref.abs() + 2.0 ** -14 * mag
    assert torch.isfinite(kv).all()
    assert (err <= bound).all(), f"worst excess {(err - bound).max().item():.3g}"
    assert mla.proj_status() == 0


@pytest.mark.parametrize("T,N,D,wide", [
    (1, 1, 256, True), (1, 128, 256, False), (15, 16, 256, True), (16, 3, 8, False), (37, 5, 72, True),
    (64, 128, 256, True), (127, 7, 256, False), (128, 2, 256, True), (129, 2, 256, True), (255, 9, 256, False),
    (256, 16, 256, True), (257, 1, 136, False), (513, 20, 256, True), (1021, 40, 256, False), (2048, 128, 256, True),
    (4099, 17, 256, True), (300, 1, 2048, False), (700, 1024, 8, True)])
def test_kv_up_proj(T, N, D, wide):
    lat, w = data(T, N, D, T + N + D, wide)
    buf = torch.full((T + 1, N, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[T:] = 7.0
    mla.kv_up_proj(lat[:, :512], w, buf[:T])
    torch.cuda.synchronize()
    check(buf[:T], lat, w)
    assert torch.all(buf[T:] == 7.0)


def test_kv_up_proj_rows_do_not_touch_each_other():
    """A NaN token or weight row spoils its own outputs only."""
    for T in (20, 400):
        lat, w = data(T, 3, 256, T, True)
        lat[T - 1, 511] = float("nan")
        w[1, 200, 0] = float("nan")
        kv = torch.empty(T, 3, 256, dtype=torch.bfloat16, device="cuda")
        mla.kv_up_proj(lat[:, :512], w, kv)
        torch.cuda.synchronize()
        bad = torch.isnan(kv)
        assert bad[T - 1].all() and bad[:, 1, 200].all()
        bad[T - 1], bad[:, 1, 200] = False, False
        assert not bad.any()


def test_kv_up_proj_empty_captured_and_on_another_stream():
    lat, w = data(333, 4, 256, 1, True)
    kv = torch.empty(333, 4, 256, dtype=torch.bfloat16, device="cuda")
    mla.kv_up_proj(lat[:0, :512], w, kv[:0])
    mla.kv_up_proj(lat[:, :512], w, kv)
    torch.cuda.synchronize()
    first = kv.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.kv_up_proj(lat[:, :512], w, kv)
    kv.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(kv, first)
    side = torch.cuda.Stream()
    kv.zero_()
    side.wait_stream(torch.cuda.current_stream())
    mla.kv_up_proj(lat[:, :512], w, kv, stream=side)
    side.synchronize()
    assert torch.equal(kv, first)


def test_kv_up_proj_splits_into_key_and_value_weights():
    """The projection's halves are q_absorb's and v_up_proj's weights: k_nope
    is latent . W_UK and v is latent . W_UV, v also by v_up_proj."""
    lat, w = data(70, 6, 256, 4, False)
    kv = torch.empty(70, 6, 256, dtype=torch.bfloat16, device="cuda")
    mla.kv_up_proj(lat, w, kv)
    v = torch.empty(70, 6, 128, dtype=torch.bfloat16, device="cuda")
    mla.v_up_proj(lat[:, None].expand(-1, 6, -1).contiguous(), w[:, 128:].transpose(1, 2).contiguous(), v)
    torch.cuda.synchronize()
    assert mla.proj_status() == 0
    x = lat.double()
    mag = torch.einsum("tl,ndl->tnd", x.abs(), w[:, 128:].double().abs())
    ref = torch.einsum("tl,ndl->tnd", x, w[:, 128:].double())
    assert ((kv[..., 128:].double() - v.double()).abs() <= 2 * (2.0 ** -8 * ref.abs() + 2.0 ** -14 * mag)).all()
    check(kv, lat, w)


@pytest.mark.parametrize("T,N,D", [(1021, 20, 256), (1021, 40, 256), (300, 40, 256), (2048, 20, 256), (2050, 39, 264),
                                   (37, 19, 256), (128, 5, 40), (128, 20, 256), (200, 64, 256), (1021, 64, 256)])
def test_kv_up_proj_tile_widths(T, N, D):
    """Sizes that take each of the tile widths, more than one tile a pair, three
    times with other operands: no tile's stores meet the next one's."""
    for seed in range(3):
        lat, w = data(T, N, D, 7 * T + N + seed, True)
        kv = torch.full((T, N, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        mla.kv_up_proj(lat[:, :512], w, kv)
        torch.cuda.synchronize()
        check(kv, lat, w)
