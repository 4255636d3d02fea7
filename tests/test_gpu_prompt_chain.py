"""The prompt-side operators together, as a serving step uses them: new tokens
are normalised, rotated and appended (rope_cache_write), the cached context is
gathered, both are expanded (kv_up_proj), the new tokens attend to themselves
(prefill, causal) and to the context (prefill, all keys), and the two results
are merged.

Every stage is checked against float64 on its own inputs, with the tolerances
of its own tests.  The whole is checked against float64 from the cached rows:
rounding a key to bf16 moves a score by at most d = 2^-8 * scale * sum |q||k|
(the sum bounded from the data), which moves an output by at most 2 d of the
mean magnitude of its values; rounding the values and the probabilities adds
2^-8 each, the partial results and the merged one 2^-8 each of the magnitude;
the float32 arithmetic 2^-10.
"""
import math

import numpy as np
import pytest
import torch

import prompt_ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mla_latent_kv_15_gb300 as mla

SCALE = 1 / math.sqrt(192)


class Chain:
    def __init__(self, new, context, heads, fp8, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

        self.new, self.context, self.heads, self.kv_scale = new, context, heads, (0.02 if fp8 else 1.0)
        T, B = sum(new), len(new)
        self.total = [n + c for n, c in zip(new, context)]
        pages = [-(-t // page) for t in self.total]
        perm = torch.randperm(sum(pages) + 5, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((B, max(max(pages), 1)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cache = rnd(sum(pages) + 5, page, 576)
        if fp8:
            self.cache = (self.cache.float() / self.kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
        self.down, self.weight = rnd(T, 576), (1 + 0.1 * rnd(512)).to(torch.bfloat16)
        self.q = rnd(T, heads, 192)
        self.w = rnd(heads, 256, 512, scale=512 ** -0.5)
        ang = np.arange(8192)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64.0)
        self.cos_sin = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
        pos = np.concatenate([np.arange(c, c + n) for n, c in zip(new, context)]).astype(np.int64)
        self.positions = torch.from_numpy(pos).cuda()
        seq = torch.from_numpy(np.repeat(np.arange(B), new)).cuda()
        self.slots = self.table[seq, self.positions // page].long() * page + self.positions % page

        def cu(n):
            return torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device="cuda")

        self.cu_q, self.cu_ctx, self.cu_all = cu(new), cu(context), cu(self.total)
        e = torch.empty
        C = sum(context)
        self.latent = e(T, 576, dtype=torch.bfloat16, device="cuda")
        self.ctx_rows = e(C, 576, dtype=torch.bfloat16, device="cuda")
        self.kv_new, self.kv_ctx = (e(n, heads, 256, dtype=torch.bfloat16, device="cuda") for n in (T, C))
        self.o_new, self.o_ctx, self.out = (e(T, heads, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        self.l_new, self.l_ctx, self.lse = (e(T, heads, device="cuda") for _ in range(3))
        self.ws = [e(mla.prefill_workspace_size(B, T, heads), dtype=torch.uint8, device="cuda") for _ in range(2)]

    def run(self):
        mla.rope_cache_write(self.down[:, :512], self.down[:, 512:], self.positions, self.cos_sin, self.slots, self.cache,
                             q_pe=self.q[..., 128:], q_pe_out=self.q_rot[..., 128:], norm_weight=self.weight,
                             kv_scale=self.kv_scale, latent_out=self.latent)
        mla.gather_cache(self.cache, self.table, self.cu_ctx, self.ctx_rows, kv_scale=self.kv_scale)
        mla.kv_up_proj(self.latent[:, :512], self.w, self.kv_new)
        mla.kv_up_proj(self.ctx_rows[:, :512], self.w, self.kv_ctx)
        mla.prefill(self.q_rot, self.kv_new, self.latent[:, 512:], self.cu_q, self.cu_q, self.o_new, self.ws[0],
                    scale=SCALE, lse=self.l_new)
        mla.prefill(self.q_rot, self.kv_ctx, self.ctx_rows[:, 512:], self.cu_q, self.cu_ctx, self.o_ctx, self.ws[1],
                    scale=SCALE, causal=False, lse=self.l_ctx)
        rows = self.o_new.shape[0] * self.heads
        mla.merge_states(self.o_ctx.view(rows, 128), self.l_ctx.view(rows), self.o_new.view(rows, 128),
                         self.l_new.view(rows), self.out.view(rows, 128), self.lse.view(rows))

    def prepare(self):
        self.q_rot = self.q.clone()
        return self


@pytest.mark.parametrize("new,context,heads,fp8", [([70, 1, 300], [500, 129, 0], 4, False), ([33, 600], [1000, 200], 16, True),
                                                   ([5, 0, 1], [0, 40, 3000], 3, False)])
def test_chunked_prompt(new, context, heads, fp8):
    c = Chain(new, context, heads, fp8, seed=sum(new)).prepare()
    c.run()
    torch.cuda.synchronize()
    assert mla.proj_status() == 0 and all(mla.prefill_status(w) == 0 for w in c.ws)
    first = c.out.clone()
    # captured and replayed, into outputs that hold something else
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for t in (c.out, c.lse, c.latent, c.kv_new, c.kv_ctx, c.q_rot[..., 128:]):
        t.fill_(3.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, first)

    # stage by stage
    for lat, kv in ((c.latent, c.kv_new), (c.ctx_rows, c.kv_ctx)):
        x, y = lat[:, :512].double(), c.w.double().reshape(-1, 512)
        ref, mag = (x @ y.t()).view(kv.shape), (x.abs() @ y.abs().t()).view(kv.shape)
        assert ((kv.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * mag).all()
    at_q, at_c = [0] + list(np.cumsum(new)), [0] + list(np.cumsum(context))
    for kv, pe, at, causal, o, l in ((c.kv_new, c.latent, at_q, True, c.o_new, c.l_new),
                                     (c.kv_ctx, c.ctx_rows, at_c, False, c.o_ctx, c.l_ctx)):
        ref, lse, mag = prompt_ref.prefill_torch(c.q_rot, kv, pe[:, 512:], at_q, at, SCALE, causal)
        assert ((o.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 6.6e-4 + 2.0 ** -18) * mag).all()
        some = ~lse.isinf()
        assert torch.equal(l.isinf(), ~some)
        assert ((l.double() - lse).abs()[some] <= 3.3e-4 + 2.0 ** -20 * lse.abs()[some]).all()

    # the whole: one causal attention over context and new tokens, from the cached rows in 64 bits
    rows, at_all = [], [0] + list(np.cumsum(c.total))
    for b in range(len(new)):
        rows += [c.ctx_rows[at_c[b]:at_c[b + 1]], c.latent[at_q[b]:at_q[b + 1]]]
    rows = torch.cat(rows).double()
    kv = torch.einsum("tl,ndl->tnd", rows[:, :512], c.w.double())
    ref, lse, mag = prompt_ref.prefill_torch(c.q_rot, kv, rows[:, 512:], at_q, at_all, SCALE, True)
    qa = c.q_rot[..., :128].double().abs()
    worst = max(float(torch.einsum("nd,jnd->nj", qa[i], kv[..., :128].abs()).max()) for i in range(qa.shape[0])) if len(qa) else 0
    d = 2.0 ** -8 * SCALE * worst
    assert ((c.out.double() - ref).abs() <= (2 * d + 5 * 2.0 ** -8 + 2.0 ** -10) * mag).all()
    assert ((c.lse.double() - lse).abs() <= d + 2.0 ** -10).all()


def test_prompt_agrees_with_the_absorbed_decode():
    """The last tokens of the prompt by the expanded operators and by the
    absorbed decode over the cache the append has written: the same attention
    in its two forms.  Each is within its bound of the float64 result: the
    expanded one as above; the absorbed one rounds the absorbed query (2^-8 of
    sum |q_abs||kv_c|) and its latent output (2^-8, and 2^-8 for the
    probabilities, of the latent magnitudes, through |W_UV|)."""
    new, context, heads = [4, 3], [700, 260], 16
    c = Chain(new, context, heads, False, seed=9).prepare()
    c.run()
    w_uk, w_uv = c.w[:, :128], c.w[:, 128:]
    T = sum(new)
    q_abs = torch.empty(T, heads, 512, dtype=torch.bfloat16, device="cuda")
    mla.q_absorb(c.q_rot[..., :128], w_uk.contiguous(), q_abs)
    o_lat = torch.empty(T, heads, 512, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, heads, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, heads, device="cuda")
    ws = torch.empty(mla.decode_workspace_size(2, T, heads), dtype=torch.uint8, device="cuda")
    mla.decode(q_abs, c.q_rot[..., 128:].contiguous(), c.cache, c.table, torch.tensor(c.total, dtype=torch.int32, device="cuda"),
               o_lat, ws, scale=SCALE, query_start_loc=c.cu_q, lse=lse)
    mla.v_up_proj(o_lat, w_uv.transpose(1, 2).contiguous(), out)
    torch.cuda.synchronize()
    assert mla.decode_status(ws) == 0 and mla.proj_status() == 0
    kv_c = torch.cat([c.ctx_rows, c.latent])[:, :512].double().abs()
    worst = float(torch.einsum("tnl,jl->tnj", q_abs.double().abs(), kv_c).max())
    qa = c.q_rot[..., :128].double().abs()
    kv = torch.cat([c.kv_ctx, c.kv_new]).double().abs()
    worst2 = float(torch.einsum("tnd,jnd->tnj", qa, kv[..., :128]).max())
    d = 2.0 ** -8 * SCALE * (worst + worst2)
    assert ((lse - c.lse).abs() <= d + 2.0 ** -9).all()
    v_max = kv[..., 128:].amax(dim=0)                                        # [heads, 128]
    lat_max = torch.einsum("l,ndl->nd", kv_c.amax(dim=0), w_uv.double().abs())
    bound = (2 * d + 5 * 2.0 ** -8 + 2.0 ** -10) * v_max + (3 * 2.0 ** -8) * lat_max
    assert ((out.double() - c.out.double()).abs() <= bound).all()
