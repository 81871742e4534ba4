"""Timed cases of the paged-cache operators beyond plain decode.

Three operators that make up one serving step on the device:

* ``tables``: block tables, context lengths and the slot map of a step's new
  tokens from the requests' lengths (``binding.tables_step``);
* ``prefix``: decode attention of a batch whose sequences share a long prefix,
  the prefix attended once for all of them (``binding.decode_prefix``);
* ``mod``: decode attention with modified scores: a tanh cap, a bias that
  falls with distance, a sliding window, a first visible token (document
  mask) and a prefix that every query sees (``binding.decode_mod``,
  ``binding.decode_fp8_mod``).

``run`` computes them with elementary torch operations in 32 bits, or, when
``own`` is true, through this package.  ``exact`` states them once more, one
sequence at a time, in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"


# ---- cases ---------------------------------------------------------------------


def _mod(name, **kw):
    case = dict(op="mod", dtype="bf16", seqs=1, queries=1, heads=32, kv_heads=8, head=128, block=16, ctx_lo=1,
                ctx_hi=1024, cap=0.0, alibi=False, window=0, docs=False, prefix=0)
    case.update(kw)
    return dict(case, name=name) if name else case


def _prefix(name, **kw):
    case = dict(op="prefix", seqs=1, queries=1, heads=32, kv_heads=8, head=128, block=16, prefix=1024, own_lo=1,
                own_hi=512)
    case.update(kw)
    return dict(case, name=name) if name else case


def _tables(name, **kw):
    case = dict(op="tables", seqs=1, block=16, ctx=4096, chunk=1, prefill=0.0, leave=0.0, prefix_blocks=0)
    case.update(kw)
    return dict(case, name=name) if name else case


def listed():
    return [
        # One decode step of a mid-sized batch: a token for every sequence.
        _tables("tables decode 64", seqs=64, ctx=4096),
        # Continuous batching: decodes, prompt chunks, requests that leave and
        # requests that start behind a shared prefix, in one step.
        _tables("tables mixed 517", seqs=517, ctx=8192, chunk=700, prefill=0.12, leave=0.05, prefix_blocks=64),
        # The largest: thousands of sequences, half a million new tokens.
        _tables("tables prompt 4096", seqs=4096, ctx=8192, chunk=1024, prefill=0.125, leave=0.03,
                prefix_blocks=16),
        # A few chat requests behind a short system prompt: latency.
        _prefix("prefix 5 on 1k", seqs=5, prefix=1024, own_lo=1, own_hi=300),
        # A serving batch behind a long system prompt.
        _prefix("prefix 64 on 4k", seqs=64, prefix=4096, own_lo=16, own_hi=1024),
        # Verification of 4 drafted tokens behind a document that few requests share.
        _prefix("prefix 9x4 on 32k", seqs=9, queries=4, heads=64, kv_heads=8, prefix=32768, own_lo=5,
                own_hi=777, block=32),
        # The largest: many samples of one long prompt.
        _prefix("prefix 256 on 16k", seqs=256, prefix=16384, own_lo=1, own_hi=2048),
        # The smallest batch in 32 bits: one short sequence, capped scores.
        _mod("mod f32 cap 1", dtype="f32", heads=8, kv_heads=8, head=64, ctx_lo=200, ctx_hi=200, cap=30.0),
        # Capped scores with a sliding window, the ordinary serving batch.
        _mod("mod cap window 64", seqs=64, ctx_lo=512, ctx_hi=8192, cap=50.0, window=4096),
        # Distance bias over long contexts, one KV head per query head.
        _mod("mod alibi 4 on 32k", seqs=4, heads=16, kv_heads=16, ctx_lo=30000, ctx_hi=32768, alibi=True),
        # Drafted tokens verified over an FP8 pool: cap, window and 128 tokens kept in sight.
        _mod("mod fp8 verify 48x4", dtype="fp8", seqs=48, queries=4, ctx_lo=300, ctx_hi=12000, cap=50.0, window=2048,
             prefix=128),
        # Packed documents with a bidirectional prefix, several queries each.
        _mod("mod documents 96x3", seqs=96, queries=3, heads=24, kv_heads=4, head=64, block=8, ctx_lo=40,
             ctx_hi=5000, docs=True, prefix=700, alibi=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "prefix", "mod", "mod"])
    if op == "tables":
        return _tables(None, seqs=_log(rng, 1, 4096), block=rng.choice([8, 16, 32, 64]), ctx=_log(rng, 64, 8192),
                       chunk=_log(rng, 1, 1024), prefill=round(rng.uniform(0.0, 0.125), 3),
                       leave=round(rng.uniform(0.0, 0.1), 3), prefix_blocks=rng.choice([0, 0, 1, 7, 64]))
    group, kv = rng.randint(1, 8), rng.choice([1, 2, 4, 8])
    head = rng.choice([64, 128, 128])
    queries = rng.choice([1, 1, 1, 2, 3, 4])
    if op == "prefix":
        block = rng.choice([8, 16, 32, 64])
        while True:
            seqs, prefix, own_hi = _log(rng, 1, 256), _log(rng, 128, 32768), _log(rng, 8, 2048)
            prefix = -(-prefix // block) * block
            if seqs * queries * group * kv * head * prefix <= 256 * 32 * 128 * 16384:
                break
        return _prefix(None, seqs=seqs, queries=queries, heads=group * kv, kv_heads=kv, head=head, block=block,
                       prefix=prefix, own_lo=queries, own_hi=own_hi + queries)
    dtype = rng.choice(["bf16", "bf16", "fp8", "f32"])
    if dtype == "fp8" and head == 64:
        kv = max(2, kv)
    queries = 1 if dtype == "f32" else min(queries, 32 // group)
    while True:
        seqs, hi = _log(rng, 1, 128), _log(rng, 16, 32768)
        if seqs * hi * kv * head <= 64 * 8192 * 8 * 128:
            break
    return _mod(None, dtype=dtype, seqs=seqs, queries=queries, heads=group * kv, kv_heads=kv, head=head,
                block=rng.choice([8, 16, 24, 32, 64]), ctx_lo=max(queries, hi // rng.choice([1, 3, 20])),
                ctx_hi=hi + queries, cap=rng.choice([0.0, 20.0, 50.0]), alibi=rng.random() < 0.4,
                window=rng.choice([0, 1, _log(rng, 2, hi), _log(rng, 2, hi)]), docs=rng.random() < 0.3,
                prefix=rng.choice([0, 0, _log(rng, 1, hi)]))


# ---- inputs --------------------------------------------------------------------


def _spaced(lo, hi, n, gen):
    """n whole numbers evenly over [lo, hi], in an order of the seed's."""
    x = torch.arange(n, device=DEV) * (hi - lo + 1) // n + lo
    return x[torch.randperm(n, generator=gen, device=DEV)]


def _rows(counts, width, pool_order):
    """[S, width] int32: counts[s] entries from pool_order, one after another, then -1."""
    ends = torch.cumsum(counts, 0)
    j = torch.arange(width, device=DEV)
    at = (ends - counts)[:, None] + j[None, :]
    some = j[None, :] < counts[:, None]
    return torch.where(some, pool_order[torch.where(some, at, 0)], -1).to(torch.int32).contiguous()


def _pools(blocks, block, kv_heads, head, dtype, gen):
    """K and V pools of N(0, 1) values (E4M3 codes of scaled values for fp8)."""
    shape = (blocks, block, kv_heads, head)
    if dtype == "fp8":
        return [(torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).float() / s).clamp(-448, 448)
                .to(torch.float8_e4m3fn).view(torch.uint8) for s in (0.02, 0.015)]
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    return [torch.randn(shape, generator=gen, device=DEV, dtype=t) for _ in range(2)]


def _ceil(a, b):
    return -(-a // b)


def _budget(case):
    """Slots of a step's token buffer: what the scheduler grants at most."""
    return case["seqs"] + int(case["prefill"] * case["seqs"]) * case["chunk"]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    S, bs = c["seqs"], c["block"]
    if c["op"] == "tables":
        np_ = c["prefix_blocks"]
        kinds = torch.randperm(S, generator=gen, device=DEV)
        starts, leaves = int(c["prefill"] * S), int(c["leave"] * S)
        ctx = _spaced(1, c["ctx"], S, gen) + np_ * bs
        new = torch.ones(S, dtype=torch.int64, device=DEV)
        chunks = torch.randint(1, c["chunk"] + 1, (S,), generator=gen, device=DEV)
        new = torch.where(kinds < starts, chunks, new)
        # Half of the prompts are new requests, the others go on with theirs.
        ctx = torch.where(kinds < starts // 2, 0, ctx)
        new = torch.where(kinds >= S - leaves, -1, new)
        width = np_ + _ceil(c["ctx"] + c["chunk"], bs) + 1
        held = _ceil_t(ctx, bs)
        pool = np_ + S * (_ceil(c["ctx"], bs) // 2 + 2) + _ceil(_budget(c), bs) + S
        order = torch.randperm(pool, generator=gen, device=DEV)
        own_held = (held - np_).clamp(min=0)
        tables = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
        tables[:, np_:] = _rows(own_held, width - np_, order[np_:])
        prefix = order[:np_].to(torch.int32)
        tables[:, :np_] = torch.where((ctx > 0)[:, None], prefix[None, :], -1)
        used = np_ + int(own_held.sum())
        free = torch.zeros(pool, dtype=torch.int32, device=DEV)
        free[: pool - used] = order[used:].to(torch.int32)
        return dict(case=c, block_tables=tables, context_lens=ctx.to(torch.int32), new_lens=new.to(torch.int32),
                    free_blocks=free, free_count=torch.tensor([pool - used], dtype=torch.int32, device=DEV),
                    prefix_table=prefix if np_ else None,
                    context_lens_out=torch.empty(S, dtype=torch.int32, device=DEV),
                    free_count_out=torch.empty(1, dtype=torch.int32, device=DEV),
                    seq_starts=torch.empty(S + 1, dtype=torch.int32, device=DEV),
                    slot_mapping=torch.empty(_budget(c), dtype=torch.int64, device=DEV))
    Q, H, Hk, D = c["queries"], c["heads"], c["kv_heads"], c["head"]
    dtype = c.get("dtype", "bf16")
    if c["op"] == "prefix":
        shared = c["prefix"] // bs
        ctx = _spaced(c["own_lo"], c["own_hi"], S, gen) + c["prefix"]
    else:
        shared = 0
        ctx = _spaced(c["ctx_lo"], c["ctx_hi"], S, gen)
    counts = _ceil_t(ctx, bs) - shared
    total = shared + int(counts.sum())
    blocks = total + total // 10 + 1
    order = torch.randperm(blocks, generator=gen, device=DEV)
    width = _ceil(c["own_hi"], bs) if shared else _ceil(c["ctx_hi"], bs)
    tables = _rows(counts, width, order[shared:])
    k, v = _pools(blocks, bs, Hk, D, dtype, gen)
    q = torch.randn((S, Q, H, D) if Q > 1 else (S, H, D), generator=gen, device=DEV)
    q = q if dtype == "f32" else q.to(torch.bfloat16)
    state = dict(case=c, q=q, k_cache=k, v_cache=v, context_lens=ctx.to(torch.int32), scale=1.0 / math.sqrt(D))
    if c["op"] == "prefix":
        prefix = order[:shared].to(torch.int32)
        state.update(prefix_table=prefix, block_tables=torch.cat([prefix[None, :].expand(S, -1), tables], 1).contiguous())
        return state
    state["block_tables"] = tables
    state["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H).float() if c["alibi"] else None
    part = torch.rand(S, generator=gen, device=DEV)
    # Documents: the queries' own one starts anywhere in the first half.
    state["first"] = (ctx * part * 0.5).to(torch.int32) if c["docs"] else None
    state["prefix_lens"] = torch.minimum(_spaced(1, c["prefix"], S, gen), ctx).to(torch.int32) if c["prefix"] else None
    state["scales"] = (0.02, 0.015) if dtype == "fp8" else None
    return state


def _ceil_t(x, b):
    return (x + b - 1) // b


# ---- one pass --------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "tables":
        return _plain_tables(state)
    return _plain_prefix(state) if op == "prefix" else _plain_mod(state)


def _run_own(st, op):
    from paged_kv_cache_292_gb300 import binding

    c = st["case"]
    if op == "tables":
        binding.tables_step(st["block_tables"], st["context_lens"], st["new_lens"], st["free_blocks"],
                            st["free_count"], c["block"], st["slot_mapping"], prefix_table=st["prefix_table"],
                            context_lens_out=st["context_lens_out"], free_count_out=st["free_count_out"],
                            seq_starts=st["seq_starts"])
        return {k: st[k] for k in ("block_tables", "context_lens_out", "free_blocks", "free_count_out", "seq_starts",
                                   "slot_mapping")}
    if op == "prefix":
        return binding.decode_prefix(st["q"], st["k_cache"], st["v_cache"], st["prefix_table"], st["block_tables"],
                                     st["context_lens"], st["scale"])
    mods = dict(softcap=c["cap"], alibi_slopes=st["slopes"], window=c["window"], first_tokens=st["first"],
                prefix_lens=st["prefix_lens"])
    if c["dtype"] == "fp8":
        return binding.decode_fp8_mod(st["q"], st["k_cache"], st["v_cache"], st["block_tables"], st["context_lens"],
                                      st["scale"], *st["scales"], **mods)
    return binding.decode_mod(st["q"], st["k_cache"], st["v_cache"], st["block_tables"], st["context_lens"],
                              st["scale"], **mods)


def _plain_tables(st):
    c = st["case"]
    bs, np_ = c["block"], c["prefix_blocks"]
    tables, free = st["block_tables"], st["free_blocks"]
    width, pool, budget = tables.shape[1], free.numel(), st["slot_mapping"].numel()
    ctx, new = st["context_lens"].long(), st["new_lens"].long()
    count = st["free_count"].long()
    # Requests that leave give their own blocks back, in table order.
    gone = new == -1
    back = torch.where(gone, (_ceil_t(ctx, bs) - np_).clamp(min=0), 0)
    back_end = torch.cumsum(back, 0)
    k = torch.arange(pool, device=DEV)
    s = torch.searchsorted(back_end, k, right=True).clamp(max=ctx.numel() - 1)
    given = k < back_end[-1]
    entry = torch.where(given, np_ + k - (back_end - back)[s], 0)
    at = torch.where(given, count + k, pool)
    stack = torch.cat([free, free.new_zeros(1)])
    stack.scatter_(0, at, tables[s, entry])
    free.copy_(stack[:pool])
    top = count + back_end[-1]
    # Requests that grow take blocks from the top of the stack, in order.
    begin = (ctx == 0) & (new > 0)
    base = torch.where(begin, np_ * bs, ctx)
    grow = new.clamp(min=0)
    fits = _ceil_t(base + grow, bs) <= width
    grow = torch.where(fits, grow, 0)
    need = torch.where(grow > 0, _ceil_t(base + grow, bs) - _ceil_t(base, bs), 0)
    served = (torch.cumsum(need, 0) <= top) & (torch.cumsum(grow, 0) <= budget)
    grow, need = torch.where(served, grow, 0), torch.where(served, need, 0)
    need_end, grow_end = torch.cumsum(need, 0), torch.cumsum(grow, 0)
    s = torch.searchsorted(need_end, k, right=True).clamp(max=ctx.numel() - 1)
    taken = k < need_end[-1]
    cell = s * width + _ceil_t(base, bs)[s] + k - (need_end - need)[s]
    cells = torch.cat([tables.reshape(-1), tables.new_zeros(1)])
    cells.scatter_(0, torch.where(taken, cell, cells.numel() - 1), free[torch.where(taken, top - 1 - k, 0)])
    tables.copy_(cells[:-1].view_as(tables))
    if np_:
        fresh = (begin & (grow > 0))[:, None]
        tables[:, :np_] = torch.where(fresh, st["prefix_table"][None, :], tables[:, :np_])
    # Slots of the new tokens, back to back; -1 behind the last.
    i = torch.arange(budget, device=DEV)
    s = torch.searchsorted(grow_end, i, right=True).clamp(max=ctx.numel() - 1)
    real = i < grow_end[-1]
    pos = torch.where(real, base[s] + i - (grow_end - grow)[s], 0)
    slots = torch.where(real, tables[s, pos // bs].long() * bs + pos % bs, -1)
    ctx = torch.where(gone, 0, torch.where(grow > 0, base + grow, ctx))
    starts = torch.cat([grow_end.new_zeros(1), grow_end])
    return dict(block_tables=tables, context_lens_out=ctx.to(torch.int32), free_blocks=free,
                free_count_out=(top - need_end[-1]).to(torch.int32), seq_starts=starts.to(torch.int32),
                slot_mapping=slots)


def _attend(scores, values, allowed):
    """softmax(scores) @ values over the last axis, zero where nothing is allowed."""
    scores = scores.masked_fill(~allowed, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, values) / torch.where(total > 0, total, 1.0)


def _gather(pool, tables, scale=None):
    """[S, Hk, T, D] in 32 bits: the pool's rows in the order of the tables."""
    x = pool[tables.long().clamp(min=0)]
    S, B, bs, Hk, D = x.shape
    x = x.view(S, B * bs, Hk, D).transpose(1, 2)
    return x.float() if scale is None else x.view(torch.float8_e4m3fn).float() * scale


def _plain_prefix(st):
    c = st["case"]
    Hk, D, P = c["kv_heads"], c["head"], c["prefix"]
    S, Q = c["seqs"], c["queries"]
    G = c["heads"] // Hk
    ctx = st["context_lens"].long()
    # [S, Hk, G * Q rows, D]; row g * Q + i is query i of group head g.
    q = st["q"].float().view(S, Q, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * Q, D) * st["scale"]
    shared = [_gather(x, st["prefix_table"][None, :])[0] for x in (st["k_cache"], st["v_cache"])]
    rest = st["block_tables"][:, P // c["block"]:]
    rest = [_gather(x, rest) for x in (st["k_cache"], st["v_cache"])]
    rows = q.transpose(0, 1).reshape(Hk, S * G * Q, D)
    s_shared = torch.matmul(rows, shared[0].transpose(1, 2))
    s_shared = s_shared.view(Hk, S, G * Q, P).transpose(0, 1)
    s_rest = torch.matmul(q, rest[0].transpose(2, 3))
    pos = (ctx[:, None] - Q + torch.arange(Q, device=DEV)).repeat(1, G)[:, None, :, None]
    t = P + torch.arange(s_rest.shape[-1], device=DEV)
    s_rest = s_rest.masked_fill(t > pos, -math.inf)
    top = torch.maximum(s_shared.amax(-1, keepdim=True), s_rest.amax(-1, keepdim=True))
    p_shared, p_rest = torch.exp(s_shared - top), torch.exp(s_rest - top)
    total = p_shared.sum(-1, keepdim=True) + p_rest.sum(-1, keepdim=True)
    # Rows of the table behind a context hold no token: their weight is zero,
    # their value any block's.
    out = torch.matmul(p_rest, rest[1])
    out = out + torch.matmul(p_shared.transpose(0, 1).reshape(Hk, S * G * Q, P), shared[1]).view(Hk, S, G * Q, D).transpose(0, 1)
    out = out / total
    out = out.view(S, Hk, G, Q, D).permute(0, 3, 1, 2, 4).reshape(st["q"].shape)
    return out.to(st["q"].dtype)


def _plain_mod(st):
    c = st["case"]
    S, Q, Hk, D = c["seqs"], c["queries"], c["kv_heads"], c["head"]
    G = c["heads"] // Hk
    ctx = st["context_lens"].long()
    ks, vs = st["scales"] or (None, None)
    k, v = _gather(st["k_cache"], st["block_tables"], ks), _gather(st["v_cache"], st["block_tables"], vs)
    q = st["q"].float().view(S, Q, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * Q, D)
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    t = torch.arange(s.shape[-1], device=DEV)[None, None, None, :]
    pos = (ctx[:, None] - Q + torch.arange(Q, device=DEV)).repeat(1, G)[:, None, :, None]
    if st["slopes"] is not None:
        slope = st["slopes"].view(1, Hk, G, 1).expand(-1, -1, -1, Q).reshape(1, Hk, G * Q, 1)
        s = s - slope * (pos - t).abs().float()
    seen = t <= pos
    if c["window"]:
        seen = seen & (pos - t < c["window"])
    if st["prefix_lens"] is not None:
        seen = seen | (t < st["prefix_lens"].long().view(S, 1, 1, 1))
    seen = seen & (t < ctx.view(S, 1, 1, 1)) & (pos >= 0)
    if st["first"] is not None:
        seen = seen & (t >= st["first"].long().view(S, 1, 1, 1))
    out = _attend(s, v, seen)
    out = out.view(S, Hk, G, Q, D).permute(0, 3, 1, 2, 4).reshape(st["q"].shape)
    return out.to(st["q"].dtype)


# ---- what a pass cannot do without -------------------------------------------------


def _lens(lo, hi, n):
    return [i * (hi - lo + 1) // n + lo for i in range(n)]


def work(case):
    c = case
    S, bs = c["seqs"], c["block"]
    if c["op"] == "tables":
        starts, leaves = int(c["prefill"] * S), int(c["leave"] * S)
        grown = (S - starts - leaves) / bs + starts * (0.5 + (c["chunk"] + 1) / 2 / bs)
        back = leaves * (c["ctx"] / 2 / bs + 0.5)
        tokens = _budget(c)
        # Lengths in and out, starts, slots; a taken block is read from the
        # free list and entered in a table, a returned one the other way.
        return {"bytes": 16 * S + 8 * tokens + 8 * (grown + back) + 4 * c["prefix_blocks"] * (1 + starts // 2),
                "flops": 0}
    Q, H, Hk, D = c["queries"], c["heads"], c["kv_heads"], c["head"]
    elt = {"f32": 4, "fp8": 1}.get(c.get("dtype", "bf16"), 2)
    qelt = 4 if c.get("dtype") == "f32" else 2
    rows = 2 * S * Q * H * D * qelt
    if c["op"] == "prefix":
        lens = _lens(c["own_lo"], c["own_hi"], S)
        keys = c["prefix"] + sum(lens)
        pairs = S * Q * c["prefix"] + Q * sum(lens)
        table = 4 * sum(_ceil(n, bs) for n in lens) + 4 * c["prefix"] // bs
        return {"bytes": keys * Hk * D * 2 * elt + rows + table + 4 * S, "flops": 4 * pairs * H * D}
    keys = 0.0
    for n in _lens(c["ctx_lo"], c["ctx_hi"], S):
        pre = min(n, (c["prefix"] + 1) / 2) if c["prefix"] else 0
        first = n / 4 if c["docs"] else 0
        low = max(first, n - Q + 1 - c["window"] if c["window"] else 0)
        keys += max(0, min(pre, low) - first) + n - low
    return {"bytes": keys * Hk * D * 2 * elt + rows + 4 * keys / bs + 8 * S, "flops": 4 * keys * Q * H * D}


# ---- the definition, in 64 bits -----------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(st)
    c = case
    bs, Hk = c["block"], c["kv_heads"]
    G = c["heads"] // Hk
    q = st["q"].double().view(c["seqs"], c["queries"], c["heads"], c["head"])
    out = torch.zeros_like(q)
    lens, tables = st["context_lens"].tolist(), st["block_tables"]
    first = st["first"].tolist() if st.get("first") is not None else None
    prefix = st["prefix_lens"].tolist() if st.get("prefix_lens") is not None else None
    ks, vs = st.get("scales") or (None, None)

    def tokens(pool, ids, n, scale):
        x = pool[ids]
        x = x.view(torch.float8_e4m3fn).float().double() * scale if scale else x.double()
        return x.reshape(-1, Hk, c["head"])[:n].repeat_interleave(G, 1)

    for s, n in enumerate(lens):
        ids = tables[s, : _ceil(n, bs)].long()
        k, v = tokens(st["k_cache"], ids, n, ks), tokens(st["v_cache"], ids, n, vs)
        at = torch.arange(n, device=DEV)
        for i in range(c["queries"]):
            pos = n - c["queries"] + i
            if pos < 0:
                continue
            score = torch.einsum("hd,thd->ht", q[s, i], k) / math.sqrt(c["head"])
            if c.get("cap"):
                score = torch.tanh(score / c["cap"]) * c["cap"]
            if c.get("alibi"):
                score = score - st["slopes"].double()[:, None] * (at - pos).abs().double()
            ok = at <= pos
            if c.get("window"):
                ok &= at > pos - c["window"]
            if prefix is not None:
                ok |= at < prefix[s]
            if first is not None:
                ok &= at >= first[s]
            if bool(ok.any()):
                out[s, i] = torch.einsum("ht,thd->hd", torch.softmax(score[:, ok], -1), v[ok])
    return out.view(st["q"].shape)


def _exact_tables(st):
    c = st["case"]
    bs, np_ = c["block"], c["prefix_blocks"]
    tables = [row for row in st["block_tables"].cpu().numpy()]
    lens, new = st["context_lens"].tolist(), st["new_lens"].tolist()
    n_free = int(st["free_count"])
    stack = st["free_blocks"].tolist()
    prefix = st["prefix_table"].tolist() if np_ else []
    budget, width = st["slot_mapping"].numel(), len(tables[0])
    for s, n in enumerate(new):
        if n == -1:
            for j in range(np_, _ceil(lens[s], bs)):
                stack[n_free] = int(tables[s][j])
                n_free += 1
            lens[s] = 0
    slots, starts, short = [], [0], False
    for s, n in enumerate(new):
        if n > 0:
            base = lens[s] or np_ * bs
            end = _ceil(base + n, bs)
            need = end - _ceil(base, bs)
            if end <= width:
                short = short or need > n_free or len(slots) + n > budget
                if not short:
                    if lens[s] == 0:
                        tables[s][:np_] = prefix
                    for j in range(end - need, end):
                        n_free -= 1
                        tables[s][j] = stack[n_free]
                    slots += [int(tables[s][p // bs]) * bs + p % bs for p in range(base, base + n)]
                    lens[s] = base + n
        starts.append(len(slots))
    slots += [-1] * (budget - len(slots))
    i32 = torch.int32
    return dict(block_tables=torch.stack([torch.from_numpy(r) for r in tables]),
                context_lens_out=torch.tensor(lens, dtype=i32), free_blocks=torch.tensor(stack, dtype=i32),
                free_count_out=torch.tensor([n_free], dtype=i32), seq_starts=torch.tensor(starts, dtype=i32),
                slot_mapping=torch.tensor(slots, dtype=torch.int64))
