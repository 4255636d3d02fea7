"""GPU tests of the prompt-side operators where offsets pass 2^31 elements and
2^32 bytes, and of the one-launch prefill replayed over other lengths.
Tolerances are those of the operators' own tests (bf16 2^-8 of the value, the
projection's 2^-14 of its magnitudes, the attention's 2^-8 + 6.6e-4 + 2^-18 of
the mean magnitude it averages)."""
import math

import pytest
import torch

import prompt_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla

SCALE = 1.0 / math.sqrt(192)


def rnd(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def test_projection_and_prefill_past_32_bit_offsets():
    heads, keys, new = 128, 70001, 40                     # kv: 2.3e9 values
    lat, w = rnd(keys, 576, seed=1), rnd(heads, 256, 512, seed=2) / 512 ** 0.5
    kv = torch.empty(keys, heads, 256, dtype=torch.bfloat16, device="cuda")
    mla.kv_up_proj(lat[:, :512], w, kv)
    rows = torch.cat([torch.arange(0, 50), torch.arange(65400, 65700), torch.arange(keys - 300, keys)]).cuda()
    x, y = lat[rows, :512].double(), w.double().view(-1, 512)
    ref, mag = x @ y.t(), x.abs() @ y.abs().t()
    assert ((kv[rows].double().view(len(rows), -1) - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * mag).all()

    q = rnd(new, heads, 192, seed=3)
    cu_q = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    cu_kv = torch.tensor([0, keys], dtype=torch.int32, device="cuda")
    out = torch.empty(new, heads, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(new, heads, device="cuda")
    kv[keys - 1, 127, 200] = float("inf")                 # the last row's alone: the others are computed again
    for splits in (0, 1):
        ws = torch.empty(mla.prefill_workspace_size(1, new, heads, splits), dtype=torch.uint8, device="cuda")
        mla.prefill(q, kv, lat[:, 512:], cu_q, cu_kv, out, ws, scale=SCALE, lse=lse, num_splits=splits)
        assert mla.prefill_status(ws) == 0
        bad = ~torch.isfinite(out)
        assert bad.sum() == 1 and bad[new - 1, 127, 72]
        for h in (0, 127):
            part = kv[:, h:h + 1].clone()
            part[keys - 1, 0, 200] = 0
            want, l, m = prompt_ref.prefill_torch(q[:, h:h + 1], part, lat[:, 512:], [0, new], [0, keys], SCALE, True)
            err = (out[:, h:h + 1].double() - want).abs()
            bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 6.6e-4 + 2.0 ** -18) * m
            assert (err <= bound)[~bad[:, h:h + 1]].all()
            assert ((lse[:, h:h + 1].double() - l).abs() <= 3.3e-4 + 2.0 ** -20 * l.abs()).all()


def test_append_past_32_bit_offsets():
    pages, page, T = 58500, 64, 70                        # 2.16e9 codes
    cache = torch.zeros(pages, page, 576, dtype=torch.uint8, device="cuda")
    slots = torch.arange(T, device="cuda") * ((pages * page - 1) // (T - 1))
    slots[-1] = pages * page - 1
    down = rnd(T, 576, seed=4)
    q = torch.empty_strided((T, 2, 64), (2 ** 25, 64, 1), dtype=torch.bfloat16, device="cuda")   # rows up to 2^31.1
    q.copy_(rnd(T, 2, 64, seed=5))
    table = torch.zeros(10, 64, device="cuda")
    table[:, :32] = 1.0                                   # no turn: the rows are what they were
    pos = torch.arange(T, device="cuda") % 10
    got = torch.empty(T, 2, 64, dtype=torch.bfloat16, device="cuda")
    mla.rope_cache_write(down[:, :512], down[:, 512:], pos, table, slots, cache, q_pe=q, q_pe_out=got, kv_scale=0.5)
    torch.cuda.synchronize()
    want = (down.float() / 0.5).clamp(-448, 448).to(torch.float8_e4m3fn)
    flat = cache.view(-1, 576)
    assert torch.equal(flat[slots].view(torch.float8_e4m3fn).float(), want.float())
    assert torch.equal(got, q)
    assert int((flat != 0).any(1).sum()) == T             # and no other row


def test_prefill_of_one_launch_replayed_over_other_lengths():
    heads, Tq, Tk = 5, 260, 500
    q, kv, pe = rnd(Tq, heads, 192, seed=6), rnd(Tk, heads, 256, seed=7), rnd(Tk, 64, seed=8)
    cu_q, cu_kv = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.empty(Tq, heads, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(Tq, heads, device="cuda")
    ws = torch.empty(mla.prefill_workspace_size(3, Tq, heads), dtype=torch.uint8, device="cuda")

    def call():
        mla.prefill(q, kv, pe, cu_q, cu_kv, out, ws, scale=SCALE, lse=lse)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for at_q, at_kv in (([0, 0, 0, 0], [0, 0, 0, 0]), ([0, 1, 1, 260], [0, 77, 80, 500]), ([3, 260, 260, 260], [9, 490, 490, 500]),
                        ([0, 90, 80, 260], [0, 100, 200, 300]), ([0, 20, 120, 259], [0, 20, 120, 259])):
        cu_q.copy_(torch.tensor(at_q, dtype=torch.int32))
        cu_kv.copy_(torch.tensor(at_kv, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        sound = at_q == sorted(at_q)
        assert mla.prefill_status(ws) == (0 if sound else mla.DEVERR_BAD_QSL)
        inside = torch.zeros(Tq, dtype=torch.bool, device="cuda")
        if sound:
            inside[at_q[0]:at_q[-1]] = True
        assert (out[~inside] == 7.0).all() and (lse[~inside] == 7.0).all()
        if not sound:
            continue
        want, l, m = prompt_ref.prefill_torch(q, kv, pe, at_q, at_kv, SCALE, True)
        err = (out.double() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 6.6e-4 + 2.0 ** -18) * m)[inside].all()
        seen = inside[:, None] & ~l.isinf()
        assert ((lse.double() - l).abs() <= 3.3e-4 + 2.0 ** -20 * l.abs())[seen].all()
        assert (lse[inside[:, None] & l.isinf()] == -math.inf).all()


@pytest.mark.parametrize("extra,heads", [(0, 5), (40, 5), (0, 200)])
def test_prefill_replayed_over_other_lengths_with_cut_items(extra, heads):
    """The same where items are cut and joined: spans found by the pairs, by a
    plan (more than 32 sequences), and a list of many items."""
    Tq, Tk = 700, 4000
    q, kv, pe = rnd(Tq, heads, 192, seed=9), rnd(Tk, heads, 256, seed=10), rnd(Tk, 64, seed=11)
    n = 3 + extra
    cu_q, cu_kv = torch.zeros(n + 1, dtype=torch.int32, device="cuda"), torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    out = torch.empty(Tq, heads, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(Tq, heads, device="cuda")
    ws = torch.full((mla.prefill_workspace_size(n, Tq, heads),), 0xEE, dtype=torch.uint8, device="cuda")

    def call():
        mla.prefill(q, kv, pe, cu_q, cu_kv, out, ws, scale=SCALE, lse=lse)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for at_q, at_kv in (([0, 1, 2, 3], [0, 3999, 4000, 4000]), ([0, 0, 0, 0], [0, 1000, 2000, 4000]),
                        ([0, 600, 601, 700], [0, 700, 3000, 4000]), ([5, 6, 6, 6], [9, 3990, 3990, 3990]),
                        ([0, 300, 500, 700], [0, 5000, 5000, 5000]), ([0, 300, 200, 700], [0, 1000, 2000, 3000]),
                        ([0, 256, 512, 700], [0, 100, 200, 300]), ([0, 700, 700, 700], [0, 4000, 4000, 4000])):
        cu_q.copy_(torch.tensor(at_q + [at_q[-1]] * extra, dtype=torch.int32))
        cu_kv.copy_(torch.tensor(at_kv + [at_kv[-1]] * extra, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        want_bits = (0 if at_q == sorted(at_q) else mla.DEVERR_BAD_QSL) | (0 if at_kv[-1] <= Tk else mla.DEVERR_BAD_SEQ_LEN)
        assert mla.prefill_status(ws) == want_bits
        inside = torch.zeros(Tq, dtype=torch.bool, device="cuda")
        if want_bits == 0:
            inside[at_q[0]:at_q[-1]] = True
        assert (out[~inside] == 7.0).all() and (lse[~inside] == 7.0).all()
        if want_bits:
            continue
        for h in (0, heads - 1):
            want, l, m = prompt_ref.prefill_torch(q[:, h:h + 1], kv[:, h:h + 1], pe, at_q, at_kv, SCALE, True)
            err = (out[:, h:h + 1].double() - want).abs()
            assert (err <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 6.6e-4 + 2.0 ** -18) * m)[inside].all()
            seen = inside[:, None] & ~l.isinf()
            assert ((lse[:, h:h + 1].double() - l).abs() <= 3.3e-4 + 2.0 ** -20 * l.abs())[seen].all()
            assert (lse[:, h:h + 1][inside[:, None] & l.isinf()] == -math.inf).all()
