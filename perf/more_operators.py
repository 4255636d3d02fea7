"""Long contexts over the latent cache, as cases to be measured: a prefix that a
batch shares, and keeping a cache small by what attention made of its keys.

Four operators, each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) and as a user's call of the framework:

* ``shared``: absorbed decode of requests behind shared prefixes, each prefix
  stored once and read once for all its requests (``decode_shared``);
* ``weights``: the attention weight that every cached key of a request gets
  from all query rows, accumulated over steps (``key_weights``);
* ``select``: the keys a request keeps: its first ones, its last ones and, of
  the others, those of the largest weight (``evict_select``);
* ``compact``: the kept rows moved to the front of the request's pages, their
  accumulated weights with them (``cache_compact``).
"""
import math
import random

import torch

own = False

LKV, ROPE = 512, 64
DQK = LKV + ROPE                     # a cache row [kv_c | k_pe]
SCALE = 1.0 / math.sqrt(192)
HEADS = (1, 2, 3, 5, 8, 10, 16, 20, 32, 40, 64, 100, 128)
PAGES = (16, 32, 64, 128, 256)


def listed():
    return [
        # four chats behind one system prompt on a 16-head shard: latency alone
        dict(name="shared_chats_4", op="shared", heads=16, batch=4, prefix="512", lo=1, hi=64, sq=1, page=64, fp8=False),
        # parallel agents over one document, all 128 heads
        dict(name="shared_agents_64", op="shared", heads=128, batch=64, prefix="8192", lo=64, hi=1024, sq=1, page=64, fp8=False),
        # two prompts of odd lengths, two verified tokens a request, small pages, e4m3 rows
        dict(name="shared_two_prompts_e4m3", op="shared", heads=40, batch=33, prefix="4097,1500", lo=2, hi=777, sq=2, page=16, fp8=True),
        # many samples of one long context on a 16-head shard
        dict(name="shared_samples_128", op="shared", heads=16, batch=128, prefix="32768", lo=512, hi=2048, sq=1, page=64, fp8=False),
        # one request's step on a 16-head shard
        dict(name="weights_one_777", op="weights", heads=16, batch=1, lo=777, hi=777, sq=1, page=64, fp8=False, decay=1.0),
        # a decode batch of contexts of 1k to 8k, all 128 heads
        dict(name="weights_64", op="weights", heads=128, batch=64, lo=1024, hi=8192, sq=1, page=64, fp8=False, decay=1.0),
        # four verified tokens a request over longer contexts, e4m3 rows, older steps counting less
        dict(name="weights_verify_32_e4m3", op="weights", heads=128, batch=32, lo=2048, hi=16384, sq=4, page=64, fp8=True, decay=0.9),
        # one request over its budget
        dict(name="select_one_4096", op="select", batch=1, lo=4096, hi=4096, budget=1024, sinks=4, recent=64, ties=False),
        # a batch of long contexts, a quarter of whose keys was never attended to
        dict(name="select_128", op="select", batch=128, lo=8192, hi=32768, budget=4096, sinks=4, recent=512, ties=True),
        # one request: the latency of an eviction
        dict(name="compact_one_8192", op="compact", batch=1, lo=8192, hi=8192, budget=2048, page=64, fp8=False, weights=True),
        # small pages of e4m3 rows, an odd budget
        dict(name="compact_64_e4m3", op="compact", batch=64, lo=1024, hi=8192, budget=1021, page=16, fp8=True, weights=False),
        # a batch of long contexts cut to an eighth to a half
        dict(name="compact_128", op="compact", batch=128, lo=8192, hi=32768, budget=4096, page=64, fp8=False, weights=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("shared", "shared", "weights", "weights", "select", "compact"))
    batch = _log(rng, 1, 128)
    salt = rng.randrange(1 << 20)    # other lengths of the same range
    page, fp8, sq, heads = rng.choice(PAGES), rng.random() < 0.4, rng.choice((1, 1, 1, 2, 4)), rng.choice(HEADS)
    if op == "shared":
        groups = min(batch, rng.choice((1, 1, 1, 2, 3, 7)))
        lo = _log(rng, sq, 1024)
        hi = _log(rng, lo, max(lo, 2048))
        # no more score pairs than the largest listed case has
        left = 8192 * 9216 // (batch * heads * sq)
        prefix = [min(_log(rng, 1, 32768), max(left, 16)) if rng.random() > 0.05 else 0 for _ in range(groups)]
        return dict(op=op, heads=heads, batch=batch, prefix=",".join(map(str, prefix)), lo=lo, hi=hi, sq=sq, page=page, fp8=fp8, salt=salt)
    if op == "weights":
        # no more score pairs and rows than the largest listed cases have
        top = min(32768, 32 * 512 * 9216 // (batch * heads * sq), 32 * 9216 * 2 // batch)
        lo = _log(rng, sq, max(top, sq))
        return dict(op=op, heads=heads, batch=batch, lo=lo, hi=_log(rng, lo, max(top, lo)), sq=sq, page=page, fp8=fp8,
                    decay=rng.choice((0.0, 0.5, 1.0)), salt=salt)
    lo = _log(rng, 1, 32768)
    hi = _log(rng, lo, 32768)
    budget = _log(rng, 1, 4096)
    if op == "select":
        sinks = rng.randrange(0, min(budget, 8) + 1)
        return dict(op=op, batch=batch, lo=lo, hi=hi, budget=budget, sinks=sinks, recent=rng.randrange(0, budget - sinks + 1),
                    ties=rng.random() < 0.5, salt=salt)
    return dict(op=op, batch=batch, lo=lo, hi=hi, budget=budget, page=page, fp8=fp8, weights=rng.random() < 0.5, salt=salt)


def _lengths(case):
    rng = random.Random("%d %d %d %d" % (case["batch"], case["lo"], case["hi"], case.get("salt", 0)))
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _prefixes(case):
    """Prefix lengths, and the first request behind each (and behind the last)."""
    p = [int(x) for x in case["prefix"].split(",")]
    return p, [case["batch"] * i // len(p) for i in range(len(p) + 1)]


def _pages(lengths, page):
    return [-(-n // page) for n in lengths]


# ---------------------------------------------------------------- the inputs


def _tables(lengths, page, g, total_pages):
    """[len(lengths), most] pages drawn from the pool, none twice, -1 behind a row's last."""
    counts = torch.tensor(_pages(lengths, page), device="cuda")
    most = max(int(max(_pages(lengths, page))), 1)
    at = torch.arange(most, device="cuda")[None]
    start = counts.cumsum(0) - counts
    perm = torch.randperm(total_pages, generator=g, device="cuda").to(torch.int32)
    index = (start[:, None] + at).clamp(max=total_pages - 1)
    return torch.where(at < counts[:, None], perm[index], -1).contiguous()


def _cache(pages, page, fp8, g):
    flat = torch.randn(pages * page, DQK, generator=g, device="cuda", dtype=torch.bfloat16)
    if not fp8:
        return flat.view(pages, page, DQK), 1.0
    kv_scale = 6.0 / 448.0
    codes = torch.empty(flat.shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in range(0, flat.shape[0], 1 << 17):            # in parts: 32-bit copies of a large pool are larger still
        codes[part:part + (1 << 17)] = (flat[part:part + (1 << 17)].float() / kv_scale).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(pages, page, DQK), kv_scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, lens = case["op"], _lengths(case)
    batch = case["batch"]
    st = dict(case=case, seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if op in ("shared", "weights"):
        heads, sq, page = case["heads"], case["sq"], case["page"]
        prefix, begin = _prefixes(case) if op == "shared" else ([], [])
        total = sum(_pages(prefix + lens, page)) + 8
        table = _tables(prefix + lens, page, g, total)
        st["cache"], st["kv_scale"] = _cache(total, page, case["fp8"], g)
        st["block_table"] = table[len(prefix):, :max(_pages(lens, page))].contiguous()
        st["most"] = max(lens)
        t = batch * sq
        st["q_abs"] = torch.randn(t, heads, LKV, generator=g, device="cuda", dtype=torch.bfloat16)
        st["q_pe"] = torch.randn(t, heads, ROPE, generator=g, device="cuda", dtype=torch.bfloat16)
        st["query_start_loc"] = torch.arange(0, t + 1, sq, dtype=torch.int32, device="cuda") if sq > 1 else None
        if op == "shared":
            st["most_prefix"] = max(1, *prefix)
            st["prefix_table"] = table[:len(prefix), :max(1, *_pages(prefix, page))].contiguous()
            st["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
            st["prefix_requests"] = torch.tensor(begin, dtype=torch.int32, device="cuda")
            st["begin"] = begin
            st["out"] = torch.empty(t, heads, LKV, dtype=torch.bfloat16, device="cuda")
            st["lse"] = torch.empty(t, heads, dtype=torch.float32, device="cuda")
            if own:
                import mla_latent_kv_15_gb300 as mla
                st["workspace"] = torch.empty(mla.decode_shared_workspace_size(batch, len(prefix), t, heads), dtype=torch.uint8, device="cuda")
        else:
            # scores of normal rows are normal, of |q| times the scale: the sum of n such exponentials
            size = st["q_abs"].float().square().sum(-1) + st["q_pe"].float().square().sum(-1)
            seen = (st["seq_lens"][:, None] - sq + 1 + torch.arange(sq, device="cuda")).clamp(min=1).reshape(-1, 1)
            st["lse"] = (seen.float().log() + 0.5 * SCALE * SCALE * size).contiguous()
            st["weights"] = torch.rand(batch, max(lens), generator=g, device="cuda") * heads
        return st
    most = max(lens)
    weights = torch.exp(2.0 * torch.randn(batch, most, generator=g, device="cuda"))
    if op == "select":
        if case["ties"]:             # keys whose weights underflowed, and weights of few values
            weights = torch.where(weights < 0.25, 0.0, weights.to(torch.bfloat16).float())
        st["weights"] = weights
        st["keep"] = torch.empty(batch, case["budget"], dtype=torch.int32, device="cuda")
        st["keep_lens"] = torch.empty(batch, dtype=torch.int32, device="cuda")
        return st
    total = sum(_pages(lens, case["page"])) + 8
    st["block_table"] = _tables(lens, case["page"], g, total)
    st["cache"], _ = _cache(total, case["page"], case["fp8"], g)
    st["keep"], st["keep_lens"] = _kept(weights, st["seq_lens"], case["budget"], min(4, case["budget"]), 0)
    st["weights"] = weights if case["weights"] else None
    return st


# ---------------------------------------------------------------- plain forms


def _rows(st, table, lens, most):
    """[requests, most, 576] rows in 32 bits, and which of them there are."""
    cache = st["cache"]
    page = cache.shape[1]
    at = torch.arange(most, device="cuda")
    there = at[None] < lens[:, None]
    blocks = table[:, at // page].clamp(min=0).long()
    rows = cache.view(-1, DQK)[blocks * page + at % page].float()
    return (rows * st["kv_scale"] if st["case"]["fp8"] else rows), there


def _queries(st):
    """[requests, tokens * heads, 576] in 32 bits."""
    q = torch.cat([st["q_abs"].float(), st["q_pe"].float()], dim=-1)
    return q.view(st["case"]["batch"], -1, DQK)


def _own_scores(st, q, rows, there):
    """Scores of each request's rows over its own keys; a token sees the keys up to its own."""
    case, n = st["case"], rows.shape[1]
    s = (q * SCALE) @ rows.transpose(1, 2)
    token = torch.arange(case["sq"], device="cuda").repeat_interleave(case["heads"])
    seen = st["seq_lens"][:, None, None] - case["sq"] + 1 + token[None, :, None]
    at = torch.arange(n, device="cuda")[None, None]
    return s.masked_fill_(~((at < seen) & there[:, None]), -math.inf)


def _plain_shared(st):
    case = st["case"]
    q = _queries(st)
    rows, there = _rows(st, st["block_table"], st["seq_lens"], st["most"])
    s = _own_scores(st, q, rows, there)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total, o = p.sum(dim=-1, keepdim=True), p @ rows[..., :LKV]
    del s, p
    # a prefix's rows once for all its requests' query rows
    begin = st["begin"]
    pre, there = _rows(st, st["prefix_table"], st["prefix_lens"], st["most_prefix"])
    of = torch.cat([torch.full((b - a,), i, device="cuda") for i, (a, b) in enumerate(zip(begin, begin[1:]))])
    width = max(b - a for a, b in zip(begin, begin[1:]))
    place = torch.arange(case["batch"], device="cuda") - st["prefix_requests"].long()[of]
    packed = q.new_zeros(len(begin) - 1, width, *q.shape[1:])
    packed[of, place] = q * SCALE
    s = packed.flatten(1, 2) @ pre.transpose(1, 2)
    s.masked_fill_(~there[:, None], -math.inf)
    m2 = s.amax(dim=-1, keepdim=True)
    p = s.sub_(torch.where(m2 == -math.inf, 0.0, m2)).exp_()
    total2, o2 = p.sum(dim=-1, keepdim=True), p @ pre[..., :LKV]
    m2, total2, o2 = (x.view(len(begin) - 1, width, q.shape[1], -1)[of, place] for x in (m2, total2, o2))
    top = torch.maximum(m, m2)
    top = torch.where(top == -math.inf, 0.0, top)
    a, b = torch.exp(m - top), torch.exp(m2 - top)
    total = a * total + b * total2
    o = (a * o + b * o2) / torch.where(total == 0, 1.0, total)
    st["out"].copy_(o.view(st["out"].shape))
    st["lse"].copy_((top + total.log()).view(st["lse"].shape))
    return dict(out=st["out"], lse=st["lse"])


def _plain_weights(st):
    case, w = st["case"], st["weights"]
    rows, there = _rows(st, st["block_table"], st["seq_lens"], st["most"])
    s = _own_scores(st, _queries(st), rows, there)
    del rows
    got = torch.exp(s.sub_(st["lse"].view(case["batch"], -1, 1))).sum(dim=1)
    old = w * case["decay"] if case["decay"] else torch.zeros_like(w)
    w.copy_(torch.where(there, old + got, w))
    return w


def _kept(weights, seq_lens, budget, sinks, recent):
    """(indices kept, ascending, -1 behind the last; how many) of each row."""
    at = torch.arange(weights.shape[1], device="cuda")[None]
    n = seq_lens[:, None]
    key = weights.masked_fill((at < sinks) | (at >= n - recent), math.inf).masked_fill(at >= n, -math.inf)
    order = key.sort(dim=1, descending=True, stable=True).indices[:, :budget]
    lens = seq_lens.clamp(max=budget)
    place = torch.arange(order.shape[1], device="cuda")[None]
    order = order.masked_fill(place >= lens[:, None], weights.shape[1]).sort(dim=1).values
    keep = torch.full((weights.shape[0], budget), -1, dtype=torch.int32, device="cuda")
    keep[:, :order.shape[1]] = torch.where(place < lens[:, None], order, -1).to(torch.int32)
    return keep, lens


def _plain_select(st):
    case = st["case"]
    keep, lens = _kept(st["weights"], st["seq_lens"], case["budget"], case["sinks"], case["recent"])
    st["keep"].copy_(keep)
    st["keep_lens"].copy_(lens)
    return dict(keep=st["keep"], keep_lens=st["keep_lens"])


def _plain_compact(st):
    cache, keep, weights = st["cache"], st["keep"].long(), st["weights"]
    page = cache.shape[1]
    to = torch.arange(keep.shape[1], device="cuda")[None].expand_as(keep)
    live = to < st["keep_lens"][:, None]
    row = torch.arange(keep.shape[0], device="cuda")[:, None].expand_as(keep)
    row, to, src = row[live], to[live], keep[live]
    flat = cache.view(-1, DQK)
    flat = flat.view(torch.uint8) if st["case"]["fp8"] else flat
    table = st["block_table"].long()
    flat[table[row, to // page] * page + to % page] = flat[table[row, src // page] * page + src % page]
    out = dict(cache=cache)
    if weights is not None:
        weights[row, to] = weights[row, src]
        out["weights"] = weights
    return out


# ------------------------------------------------------------------ the calls


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"shared": _plain_shared, "weights": _plain_weights, "select": _plain_select, "compact": _plain_compact}[op](st)
    import mla_latent_kv_15_gb300 as mla
    if op == "shared":
        mla.decode_shared(st["q_abs"], st["q_pe"], st["cache"], st["prefix_table"], st["prefix_lens"], st["prefix_requests"],
                          st["block_table"], st["seq_lens"], st["out"], st["workspace"], scale=SCALE,
                          query_start_loc=st["query_start_loc"], lse=st["lse"], kv_scale=st["kv_scale"])
        return dict(out=st["out"], lse=st["lse"])
    if op == "weights":
        mla.key_weights(st["q_abs"], st["q_pe"], st["cache"], st["block_table"], st["seq_lens"], st["lse"], st["weights"],
                        scale=SCALE, query_start_loc=st["query_start_loc"], decay=case["decay"], kv_scale=st["kv_scale"])
        return st["weights"]
    if op == "select":
        mla.evict_select(st["weights"], st["seq_lens"], st["keep"], st["keep_lens"], sinks=case["sinks"], recent=case["recent"])
        return dict(keep=st["keep"], keep_lens=st["keep_lens"])
    mla.cache_compact(st["cache"], st["block_table"], st["keep"], st["keep_lens"], weights=st["weights"])
    out = dict(cache=st["cache"])
    if st["weights"] is not None:
        out["weights"] = st["weights"]
    return out


def work(case):
    """Each input read once and each output written once."""
    op, lens = case["op"], _lengths(case)
    if op in ("shared", "weights"):
        rows = case["batch"] * case["sq"] * case["heads"]
        a_row = DQK * (1 if case["fp8"] else 2)
        pairs = case["heads"] * sum(case["sq"] * n - case["sq"] * (case["sq"] - 1) // 2 for n in lens)
        if op == "weights":
            return {"bytes": rows * (2 * DQK + 4) + sum(lens) * (a_row + 4 + 4 * bool(case["decay"])), "flops": 2 * DQK * pairs}
        prefix, begin = _prefixes(case)
        pairs += case["heads"] * case["sq"] * sum(p * (b - a) for p, a, b in zip(prefix, begin, begin[1:]))
        return {"bytes": rows * (2 * DQK + 2 * LKV + 4) + (sum(lens) + sum(prefix)) * a_row, "flops": 2 * (DQK + LKV) * pairs}
    kept = sum(min(n, case["budget"]) for n in lens)
    if op == "select":
        return {"bytes": 4 * sum(lens) + 4 * case["batch"] * case["budget"], "flops": sum(lens)}
    return {"bytes": kept * (2 * DQK * (1 if case["fp8"] else 2) + 4 + 8 * case["weights"]), "flops": 0}


# --------------------------------------------------------------- in 64 bits


def _exact_rows(st, pages, n):
    page, at = st["cache"].shape[1], torch.arange(n, device="cuda")
    rows = st["cache"][pages[at // page].long(), at % page].to(torch.float64)
    return rows * st["kv_scale"] if st["case"]["fp8"] else rows


def exact(case, seed):
    st = prepare(case, seed)
    op, lens = case["op"], _lengths(case)
    f64 = torch.float64
    if op in ("shared", "weights"):
        if work(case)["flops"] > 8e12:
            return None
        sq, heads = case["sq"], case["heads"]
        if op == "shared":
            out, lse = torch.zeros(st["out"].shape, dtype=f64, device="cuda"), torch.zeros(st["lse"].shape, dtype=f64, device="cuda")
            prefix, begin = _prefixes(case)
        else:
            w = st["weights"].to(f64)
        for b, n in enumerate(lens):
            keys = _exact_rows(st, st["block_table"][b], n)
            first = 0
            if op == "shared":
                g = max(i for i in range(len(prefix)) if begin[i] <= b and begin[i + 1] > begin[i])
                keys = torch.cat([_exact_rows(st, st["prefix_table"][g], prefix[g]), keys])
                first = prefix[g]
            got = torch.zeros(n, dtype=f64, device="cuda")
            for t in range(sq):
                token, seen = b * sq + t, first + max(0, n - sq + 1 + t)
                q = torch.cat([st["q_abs"][token].to(f64), st["q_pe"][token].to(f64)], dim=1)
                s = q @ keys[:seen].t() / math.sqrt(192)
                if op == "shared":
                    lse[token] = torch.logsumexp(s, dim=1)
                    out[token] = torch.exp(s - lse[token][:, None]) @ keys[:seen, :LKV]
                else:
                    got[:seen] += torch.exp(s - st["lse"][token].to(f64)[:, None]).sum(0)
            if op == "weights":
                w[b, :n] = w[b, :n] * case["decay"] + got
        return dict(out=out, lse=lse) if op == "shared" else w
    if op == "select":
        return None                  # whole numbers
    cache = st["cache"].to(f64)
    weights = st["weights"].to(f64) if st["weights"] is not None else None
    page = case["page"]
    for b, kept in enumerate(st["keep_lens"].tolist()):
        src, to, pages = st["keep"][b, :kept].long(), torch.arange(kept, device="cuda"), st["block_table"][b].long()
        cache[pages[to // page], to % page] = cache[pages[src // page], src % page]
        if weights is not None:
            weights[b, :kept] = weights[b, src]
    out = dict(cache=cache)
    if weights is not None:
        out["weights"] = weights
    return out
