"""The prompt-side operators of latent attention, as cases to be measured.

Three operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as a user's call of the framework:

* ``append``: the step's latent rows normalised, their shared key rotated by
  the token's position, written into the paged cache, with every head's
  rotated query part beside it (``rope_cache_write``);
* ``expand``: latent rows to every head's key and value (``kv_up_proj``);
* ``prefill``: attention of packed sequences over the expanded keys and
  values, with the log-sum-exp (``prefill``).
"""
import math

import torch

own = False

LKV, ROPE, NOPE, VDIM = 512, 64, 128, 128
DQK = LKV + ROPE              # a latent row [kv_c | k_pe]
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
EPS = 1e-6
MAX_POS = 32768
HEADS = (1, 2, 3, 5, 8, 10, 16, 20, 32, 40, 64, 100, 128)


def listed():
    return [
        # one request's decode step on a 16-head shard: the smallest append, latency alone
        dict(name="append_decode_1", op="append", tokens=1, heads=16, page=64, fp8=False, norm=True, pairs=True, latent=False),
        # the decode step of a batch of 64 with 128 heads into an e4m3 cache
        dict(name="append_decode_64_e4m3", op="append", tokens=64, heads=128, page=64, fp8=True, norm=True, pairs=True, latent=False),
        # an odd-sized prompt chunk, halves rotated together, rows normalised by the caller, small pages
        dict(name="append_chunk_1021_e4m3", op="append", tokens=1021, heads=20, page=16, fp8=True, norm=False, pairs=False, latent=True),
        # the prompts of a full scheduling step
        dict(name="append_prompt_8192", op="append", tokens=8192, heads=128, page=64, fp8=False, norm=True, pairs=True, latent=True),
        # a short chunk of one request on a 16-head shard: the weights are all the work
        dict(name="expand_37", op="expand", tokens=37, heads=16, wide=True),
        # an odd-sized chunk with 20 heads
        dict(name="expand_1021", op="expand", tokens=1021, heads=20, wide=True),
        # the prompts of a full scheduling step with 128 heads
        dict(name="expand_8192", op="expand", tokens=8192, heads=128, wide=False),
        # a short question on a 16-head shard: latency
        dict(name="prefill_short_37", op="prefill", heads=16, causal=True, q="37", kv="37"),
        # single new tokens over ragged contexts, an empty one among them: few rows, long keys
        dict(name="prefill_single_tokens", op="prefill", heads=16, causal=True, q="1,1,1,1,1,1,1,1", kv="8191,4097,1,777,6000,129,8000,0"),
        # a mixed batch: prompts, chunks that extend a cached context, single tokens, a request without tokens
        dict(name="prefill_mixed_batch", op="prefill", heads=128, causal=True, q="1021,64,1,512,0,333,128,2000", kv="1021,2500,777,4096,100,333,129,2000"),
        # a context chunk under the new tokens of one request: every key is visible
        dict(name="prefill_context_16384", op="prefill", heads=128, causal=False, q="512", kv="16384"),
        # one long prompt
        dict(name="prefill_prompt_8192", op="prefill", heads=128, causal=True, q="8192", kv="8192"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "expand", "prefill", "prefill"))
    heads = rng.choice(HEADS)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=heads, page=rng.choice((16, 32, 64, 128, 256)), fp8=rng.random() < 0.5,
                    norm=rng.random() < 0.7, pairs=rng.random() < 0.7, latent=rng.random() < 0.5)
    if op == "expand":
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=heads, wide=rng.random() < 0.5)
    causal = rng.random() < 0.7
    batch = _log(rng, 1, 24)
    q, kv, pairs = [], [], 0
    for _ in range(batch):
        kind = rng.choice(("prompt", "extend", "single", "context"))
        a = 1 if kind == "single" else _log(rng, 1, 4096)
        b = a if kind == "prompt" else a + _log(rng, 1, 16384)
        if batch > 1 and rng.random() < 0.04:
            a = 0
        if rng.random() < 0.04:
            b = 0
        # no more score pairs than the largest listed case has, in all sequences together
        left = 8192 * 8192 * 128 // 2 // heads - pairs
        b = min(b, max(left // max(a, 1), 0))
        q.append(a)
        kv.append(b)
        pairs += a * b
    return dict(op=op, heads=heads, causal=causal, q=",".join(map(str, q)), kv=",".join(map(str, kv)))


def _lengths(case):
    return [int(x) for x in case["q"].split(",")], [int(x) for x in case["kv"].split(",")]


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _visible(case):
    """(query, key) pairs that the mask leaves."""
    n = 0
    for a, b in zip(*_lengths(case)):
        if not case["causal"]:
            n += a * b
        else:                          # row i sees b - a + 1 + i keys
            full = min(a, b)           # the rows that see any
            n += full * b - full * (full - 1) // 2
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    st = dict(case=case)
    if case["op"] == "append":
        t, n, page = case["tokens"], case["heads"], case["page"]
        # the fused down-projection's output, whose columns the call reads as they lie
        st["down"] = normal(t, DQK)
        st["q"] = normal(t, n, NOPE + ROPE)
        st["q_out"] = torch.empty(t, n, ROPE, dtype=torch.bfloat16, device="cuda")
        st["positions"] = torch.randint(0, MAX_POS, (t,), generator=g, device="cuda")
        freq = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
        angle = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * freq
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        blocks = -(-t // page) + 8
        st["cache"] = normal(blocks, page, DQK)
        st["slots"] = torch.randperm(blocks * page, generator=g, device="cuda")[:t].contiguous()
        if t > 4:
            st["slots"][::97] = -1     # padding tokens of a captured batch: nothing of theirs is written
        st["kv_scale"] = 1.0
        if case["fp8"]:
            st["kv_scale"] = 6.0 / 448.0
            st["cache"] = (st["cache"].float() / st["kv_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        st["weight"] = (1.0 + 0.1 * torch.randn(LKV, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        st["latent"] = torch.empty(t, DQK, dtype=torch.bfloat16, device="cuda") if case["latent"] else None
    elif case["op"] == "expand":
        t, n = case["tokens"], case["heads"]
        # wide: rows as a context gather leaves them, [kv_c | k_pe]
        st["latent"] = normal(t, DQK if case["wide"] else LKV)[:, :LKV]
        st["weight"] = normal(n, NOPE + VDIM, LKV, scale=LKV ** -0.5)
        st["kv"] = torch.empty(t, n, NOPE + VDIM, dtype=torch.bfloat16, device="cuda")
    else:
        n = case["heads"]
        lq, lk = _lengths(case)
        st["at_q"], st["at_kv"] = _starts(lq), _starts(lk)
        tq, tk = st["at_q"][-1], st["at_kv"][-1]
        st["q"] = normal(tq, n, NOPE + ROPE)
        st["kv"] = normal(tk, n, NOPE + VDIM)
        st["k_pe"] = normal(tk, DQK)[:, LKV:]
        st["cu_q"] = torch.tensor(st["at_q"], dtype=torch.int32, device="cuda")
        st["cu_kv"] = torch.tensor(st["at_kv"], dtype=torch.int32, device="cuda")
        st["out"] = torch.empty(tq, n, VDIM, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.empty(tq, n, dtype=torch.float32, device="cuda")
        if own:
            import mla_latent_kv_15_gb300 as mla
            st["workspace"] = torch.empty(mla.prefill_workspace_size(len(lq), tq, n), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms


def _rotate(x, cos, sin, pairs):
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :ROPE // 2], x[..., ROPE // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    return torch.stack([ra, rb], dim=-1).flatten(-2) if pairs else torch.cat([ra, rb], dim=-1)


def _plain_append(st):
    case = st["case"]
    kv_c, k_pe = st["down"][:, :LKV].float(), st["down"][:, LKV:].float()
    if case["norm"]:
        kv_c = kv_c * torch.rsqrt((kv_c * kv_c).mean(dim=1, keepdim=True) + EPS) * st["weight"].float()
    row = st["cos_sin"][st["positions"]]
    cos, sin = row[:, :ROPE // 2], row[:, ROPE // 2:]
    rows = torch.cat([kv_c, _rotate(k_pe, cos, sin, case["pairs"])], dim=1)
    kept = st["slots"] >= 0
    flat = st["cache"].view(-1, DQK)
    if case["fp8"]:
        codes = (rows / st["kv_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn)
        flat.view(torch.uint8)[st["slots"][kept]] = codes.view(torch.uint8)[kept]
    else:
        flat[st["slots"][kept]] = rows.to(torch.bfloat16)[kept]
    q = _rotate(st["q"][..., NOPE:].float(), cos[:, None], sin[:, None], case["pairs"]).to(torch.bfloat16)
    out = dict(cache=st["cache"], q_pe=q)
    if case["latent"]:
        out["latent"] = rows.to(torch.bfloat16)
    return out


def _plain_expand(st):
    w = st["weight"]
    kv = st["latent"].float() @ w.reshape(-1, LKV).float().t()
    return kv.to(torch.bfloat16).view(-1, w.shape[0], w.shape[1])


def _plain_prefill(st):
    causal = st["case"]["causal"]
    out, lse = st["out"], st["lse"]
    for b in range(len(st["at_q"]) - 1):
        q0, q1, k0, k1 = st["at_q"][b], st["at_q"][b + 1], st["at_kv"][b], st["at_kv"][b + 1]
        if q1 == q0:
            continue
        kv = st["kv"][k0:k1].float().transpose(0, 1)
        k = torch.cat([kv[..., :NOPE], st["k_pe"][k0:k1].float().expand(kv.shape[0], -1, -1)], dim=-1)
        s = (st["q"][q0:q1].float() * SCALE).transpose(0, 1) @ k.transpose(1, 2)
        if causal:
            i = torch.arange(q1 - q0, device=s.device)[:, None] + (k1 - k0) - (q1 - q0)
            s.masked_fill_(torch.arange(k1 - k0, device=s.device)[None] > i, -math.inf)
        m = s.amax(dim=-1, keepdim=True) if k1 > k0 else s.new_full((*s.shape[:2], 1), -math.inf)
        s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
        total = s.sum(dim=-1, keepdim=True)
        o = (s @ kv[..., NOPE:]) / torch.where(total == 0, 1.0, total)
        out[q0:q1] = o.transpose(0, 1).to(torch.bfloat16)
        lse[q0:q1] = (m + total.log()).squeeze(-1).t()
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ the calls


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"append": _plain_append, "expand": _plain_expand, "prefill": _plain_prefill}[op](st)
    import mla_latent_kv_15_gb300 as mla
    if op == "append":
        down = st["down"]
        mla.rope_cache_write(down[:, :LKV], down[:, LKV:], st["positions"], st["cos_sin"], st["slots"], st["cache"],
                             q_pe=st["q"][..., NOPE:], q_pe_out=st["q_out"], norm_weight=st["weight"], norm_eps=EPS,
                             interleaved=st["case"]["pairs"], kv_scale=st["kv_scale"], latent_out=st["latent"])
        out = dict(cache=st["cache"], q_pe=st["q_out"])
        if st["latent"] is not None:
            out["latent"] = st["latent"]
        return out
    if op == "expand":
        mla.kv_up_proj(st["latent"], st["weight"], st["kv"])
        return st["kv"]
    mla.prefill(st["q"], st["kv"], st["k_pe"], st["cu_q"], st["cu_kv"], st["out"], st["workspace"], scale=SCALE,
                causal=st["case"]["causal"], lse=st["lse"])
    return dict(out=st["out"], lse=st["lse"])


def work(case):
    """Each input read once, each output written once; a cache row is 576 values, a table row 64 floats."""
    if case["op"] == "append":
        t, n = case["tokens"], case["heads"]
        row = DQK * 2 + DQK * (1 if case["fp8"] else 2) + (DQK * 2 if case["latent"] else 0) + ROPE * 4 + 8 + 8
        return {"bytes": t * (row + 2 * n * ROPE * 2) + (LKV * 2 if case["norm"] else 0),
                "flops": t * (4 * LKV * case["norm"] + 3 * ROPE * (n + 1))}
    if case["op"] == "expand":
        t, cols = case["tokens"], case["heads"] * (NOPE + VDIM)
        return {"bytes": 2 * (t * LKV + cols * LKV + t * cols), "flops": 2 * t * cols * LKV}
    n = case["heads"]
    lq, lk = _lengths(case)
    tq, tk = sum(lq), sum(lk)
    return {"bytes": tq * n * (2 * (NOPE + ROPE) + 2 * VDIM + 4) + tk * (2 * n * (NOPE + VDIM) + 2 * ROPE) + 8 * (len(lq) + 1),
            "flops": 2 * (NOPE + ROPE + VDIM) * n * _visible(case)}


# --------------------------------------------------------------- in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "append":
        x = st["down"].to(f64)
        c = x[:, :LKV]
        if case["norm"]:
            c = c / ((c ** 2).sum(1, keepdim=True) / LKV + EPS).sqrt() * st["weight"].to(f64)
        # a rotation as a product of complex numbers
        turn = torch.complex(*st["cos_sin"].to(f64)[st["positions"]].split(ROPE // 2, dim=1))

        def rotated(v, turn):
            if case["pairs"]:
                return torch.view_as_real(torch.view_as_complex(v.contiguous().unflatten(-1, (-1, 2))) * turn).flatten(-2)
            z = torch.complex(v[..., :ROPE // 2].contiguous(), v[..., ROPE // 2:].contiguous()) * turn
            return torch.cat([z.real, z.imag], dim=-1)

        rows = torch.cat([c, rotated(x[:, LKV:], turn)], dim=1)
        cache = st["cache"].to(f64).view(-1, DQK)
        kept = (st["slots"] >= 0).nonzero().squeeze(1)
        cache[st["slots"][kept]] = (rows[kept] / st["kv_scale"]).clamp(-448, 448) if case["fp8"] else rows[kept]
        out = dict(cache=cache.view(st["cache"].shape), q_pe=rotated(st["q"][..., NOPE:].to(f64), turn[:, None]))
        if case["latent"]:
            out["latent"] = rows
        return out
    if case["op"] == "expand":
        if 2 * case["tokens"] * case["heads"] * (NOPE + VDIM) * LKV > 6e12:
            return None
        return torch.einsum("tl,ndl->tnd", st["latent"].to(f64), st["weight"].to(f64))
    lq, lk = _lengths(case)
    if 2 * (NOPE + ROPE + VDIM) * case["heads"] * sum(a * b for a, b in zip(lq, lk)) > 8e12:
        return None
    n = case["heads"]
    out = torch.zeros(sum(lq), n, VDIM, dtype=f64, device="cuda")
    lse = torch.full((sum(lq), n), -math.inf, dtype=f64, device="cuda")
    for b, (a, c) in enumerate(zip(lq, lk)):
        if a == 0 or c == 0:
            continue
        q, kv = st["q"][st["at_q"][b]:st["at_q"][b + 1]], st["kv"][st["at_kv"][b]:st["at_kv"][b + 1]]
        pe = st["k_pe"][st["at_kv"][b]:st["at_kv"][b + 1]].to(f64)
        for h in range(n):
            for r in range(0, a, 2048):
                e = min(r + 2048, a)
                seen = min(c, max(0, c - a + e)) if case["causal"] else c     # keys of the last row
                if seen == 0:
                    continue
                s = q[r:e, h, :NOPE].to(f64) @ kv[:seen, h, :NOPE].to(f64).t() + q[r:e, h, NOPE:].to(f64) @ pe[:seen].t()
                s = s / math.sqrt(NOPE + ROPE)
                if case["causal"]:
                    s = torch.where(torch.ones_like(s, dtype=torch.bool).tril(c - a + r), s, -math.inf)
                l = torch.logsumexp(s, dim=1)
                p = torch.exp(s - torch.where(l.isinf(), 0.0, l)[:, None])
                rows = slice(st["at_q"][b] + r, st["at_q"][b] + e)
                out[rows, h] = p @ kv[:seen, h, NOPE:].to(f64)
                lse[rows, h] = l
    return dict(out=out, lse=lse)
