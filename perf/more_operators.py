"""Timed cases of a step's chunk attention and of the 8-bit integer cache.

What a serving step does beside plain decode, over the paged pools:

* ``attend``: causal attention of a ragged batch of new tokens, from one token
  to a long prompt chunk per sequence, over bf16 or f32 pools
  (``binding.prefill``) or over int8 pools with a scale for every token and KV
  head (``binding.prefill_int8``; one token each: ``binding.decode_int8``);
* ``store``: new K/V rows quantised into the int8 pools as they are written, and
  read back (``binding.write_cache_int8``, ``binding.read_cache_int8``);
* ``load``: whole contexts read back from the int8 pools.

``run`` computes them with elementary torch operations in 32 bits (64 where a
quotient may lie next to a rounding border), or, when ``own`` is true, through
this package.  ``exact`` states them once more, one sequence at a time, in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------


def _attend_case(name, **kw):
    case = dict(op="attend", pool="bf16", form="ragged", seqs=1, ones=0, idle=0, new_lo=1, new_hi=512, old_lo=0,
                old_hi=0, heads=32, kv_heads=8, head=128, block=16, tail=0)
    case.update(kw)
    return dict(case, name=name) if name else case


def _cache_case(name, op, **kw):
    case = dict(op=op, dtype="bf16", seqs=1, new_lo=1, new_hi=1, old_lo=0, old_hi=0, kv_heads=8, head=128, block=16)
    case.update(kw)
    return dict(case, name=name) if name else case


def listed():
    return [
        # The next 16 tokens of one chat request (a tool's answer, say): latency.
        _attend_case("16 on 1k", new_lo=16, new_hi=16, old_lo=1024, old_hi=1024),
        # Prompts that arrive together, none with a context yet, in a token
        # buffer with a few rows to spare.
        _attend_case("prompts 7", seqs=7, new_lo=33, new_hi=2047, tail=19),
        # Continuous batching: mostly decodes, three prompt chunks and two idle rows.
        _attend_case("mixed 24", seqs=24, ones=19, idle=2, new_lo=200, new_hi=256, old_lo=100, old_hi=4096),
        # The largest: a chunk of a long document.
        _attend_case("4k on 12k", new_lo=4096, new_hi=4096, old_lo=12288, old_hi=12288),
        # Eight query heads a KV head, blocks of 32, ragged chunks on ragged contexts.
        _attend_case("chunks 5 group 8", seqs=5, new_lo=100, new_hi=1021, old_lo=1, old_hi=6000, heads=64, block=32),
        # Prompts in 32 bits, one KV head per query head.
        _attend_case("f32 3", pool="f32", seqs=3, new_lo=5, new_hi=200, old_lo=0, old_hi=300, heads=8, kv_heads=8,
                     head=64),
        # A decode step of an ordinary serving batch over the int8 cache.
        _attend_case("int8 decode 64", pool="int8", form="decode", seqs=64, new_lo=1, new_hi=1, old_lo=511, old_hi=4095),
        # Few long contexts over the int8 cache.
        _attend_case("int8 decode 8 on 32k", pool="int8", form="decode", seqs=8, new_lo=1, new_hi=1, old_lo=32000,
                     old_hi=32767),
        # Prompt chunks over the int8 cache, beside decodes.
        _attend_case("int8 chunks 6", pool="int8", seqs=6, ones=2, new_lo=300, new_hi=1024, old_lo=1000, old_hi=7000),
        # One decode step's new rows: latency.
        _cache_case("store 64", "store", seqs=64, old_lo=500, old_hi=4000),
        # The rows of a long prompt.
        _cache_case("store prompt f32", "store", dtype="f32", seqs=4, new_lo=1000, new_hi=4099),
        # Whole contexts read back, as for an engine that attends over plain rows.
        _cache_case("load 64", "load", seqs=64, new_lo=512, new_hi=4096),
    ]


#: Scores that the largest listed case has: what a drawn one is held to.
MOST = 32 * 4096 * 16384


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "store", "load"])
    block = rng.choice([8, 16, 16, 24, 32, 64])
    head = rng.choice([64, 128, 128])
    if op != "attend":
        kv = rng.choice([1, 2, 4, 8])
        while True:
            seqs, hi = _log(rng, 1, 256), _log(rng, 1, 8192)
            if seqs * hi * kv * head <= 64 * 4096 * 8 * 128:
                break
        return _cache_case(None, op, dtype=rng.choice(["bf16", "bf16", "f32"]), seqs=seqs,
                           new_lo=max(1, hi // rng.choice([1, 3, 20])), new_hi=hi,
                           old_hi=_log(rng, 1, 2048) if op == "store" else 0, kv_heads=kv, head=head, block=block)
    pool = rng.choice(["bf16", "bf16", "int8", "int8", "f32"])
    group, kv = rng.randint(1, 8), rng.choice([1, 2, 4, 8])
    form = rng.choice(["ragged", "decode"]) if pool == "int8" else "ragged"
    while True:
        seqs, old = _log(rng, 1, 64), _log(rng, 1, 32768)
        new = 1 if form == "decode" else _log(rng, 1, 4096)
        # Plain scores of the padded batch, the work of a pass, and the pools.
        if seqs * new * (new + old) * group * kv > MOST or seqs * (new + old) * kv * head > 64 * 8192 * 8 * 128:
            continue
        if seqs * new * (new / 2 + old) * group * kv * head <= MOST * 64 // (8 if pool == "f32" else 1):
            break
    ones = rng.randint(0, seqs - 1) if form == "ragged" else 0
    return _attend_case(None, pool=pool, form=form, seqs=seqs, ones=ones,
                        idle=rng.randint(0, (seqs - ones - 1) // 2) if form == "ragged" else 0,
                        new_lo=max(1, new // rng.choice([1, 3, 20])), new_hi=new,
                        old_lo=rng.choice([0, 0, old // 2]), old_hi=old, heads=group * kv, kv_heads=kv, head=head,
                        block=block, tail=rng.choice([0, 0, 1, 57]) if form == "ragged" else 0)


# ---- inputs --------------------------------------------------------------------


def _ceil(a, b):
    return -(-a // b)


def _spaced(lo, hi, n):
    return [i * (hi - lo + 1) // n + lo for i in range(n)]


def _lens(c):
    """[(new tokens, tokens before them)] of the batch: chunks, single tokens, idle sequences."""
    ones, idle = c.get("ones", 0), c.get("idle", 0)
    new = _spaced(c["new_lo"], c["new_hi"], c["seqs"] - ones - idle) + [1] * ones + [0] * idle
    old = _spaced(c["old_lo"], c["old_hi"], c["seqs"])
    step = next(k for k in (7, 5, 3, 2, 1) if math.gcd(k, c["seqs"]) == 1 or k == 1)
    return [(n, old[(i * step) % c["seqs"]]) for i, n in enumerate(new)]


def _quantise(x):
    """Codes (int8) and scales of rows [..., D]: the largest magnitude becomes 127."""
    x = x.double()
    scale = (x.abs().amax(-1) / 127).float()
    code = torch.round(x / torch.where(scale > 0, scale, 1.0).double()[..., None])
    return code.clamp(-127, 127).to(torch.int8), scale


def _rows(tokens, kv_heads, head, gen):
    """K or V rows in 32 bits: N(0, 1) by a size of each token and head, with a few strong channels."""
    x = torch.randn(tokens, kv_heads, head, generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn(tokens, kv_heads, 1, generator=gen, device=DEV))
    return x * torch.where(torch.rand(1, kv_heads, head, generator=gen, device=DEV) < 0.02, 4.0, 1.0)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    S, bs, Hk, D = c["seqs"], c["block"], c["kv_heads"], c["head"]
    lens = torch.tensor(_lens(c), device=DEV)[torch.randperm(S, generator=gen, device=DEV)]
    new, ctx = lens[:, 0], lens.sum(1)
    starts = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    counts = _ceil_t(ctx, bs)
    total = int(counts.sum())
    blocks = total + total // 10 + 1
    order = torch.randperm(blocks, generator=gen, device=DEV)
    width = max(1, int(counts.max()))
    j = torch.arange(width, device=DEV)
    at = (torch.cumsum(counts, 0) - counts)[:, None] + j
    tables = torch.where(j < counts[:, None], order[at.clamp(max=blocks - 1)], -1).to(torch.int32).contiguous()
    st = dict(case=c, block_tables=tables, context_lens=ctx.to(torch.int32), seq_starts=starts.to(torch.int32),
              scale=1.0 / math.sqrt(D))
    T = int(starts[-1])
    shape = (blocks, bs, Hk, D)
    if c["op"] == "store":
        st["k_new"], st["v_new"] = (_rows(T, Hk, D, gen).to(TYPES[c["dtype"]]) for _ in range(2))
        row = torch.arange(T, device=DEV)
        seq = torch.searchsorted(starts, row, right=True) - 1
        pos = (ctx - new)[seq] + row - starts[seq]
        st["slots"] = tables[seq, pos // bs].long() * bs + pos % bs
        st["k_cache"], st["v_cache"] = (torch.zeros(shape, dtype=torch.int8, device=DEV) for _ in range(2))
        st["k_scales"], st["v_scales"] = (torch.zeros(blocks, Hk, bs, device=DEV) for _ in range(2))
        st["first"] = (ctx - new).to(torch.int32)
    elif c["op"] == "load" or c["pool"] == "int8":
        for x in "kv":
            code, scale = _quantise(_rows(blocks * bs, Hk, D, gen))
            st[x + "_cache"] = code.view(shape)
            st[x + "_scales"] = scale.view(blocks, bs, Hk).transpose(1, 2).contiguous()
        st["first"] = None
    else:
        for x in "kv":
            st[x + "_cache"] = torch.randn(shape, generator=gen, device=DEV, dtype=TYPES[c["pool"]])
    if c["op"] == "attend":
        q = torch.randn(T + c["tail"], c["heads"], D, generator=gen, device=DEV)
        st["q"] = q if c["pool"] == "f32" else q.to(torch.bfloat16)
        st["out"] = torch.zeros_like(st["q"])
    else:
        st["k_out"], st["v_out"] = (torch.empty(T, Hk, D, dtype=TYPES[c["dtype"]], device=DEV) for _ in range(2))
    return st


def _ceil_t(x, b):
    return (x + b - 1) // b


# ---- one pass --------------------------------------------------------------------


def run(state):
    if own:
        return _run_own(state)
    return {"attend": _plain_attend, "store": _plain_store, "load": _plain_load}[state["case"]["op"]](state)


def _run_own(st):
    from paged_kv_cache_292_gb300 import binding

    c = st["case"]
    if c["op"] == "attend":
        where = (st["block_tables"], st["context_lens"])
        if c["pool"] != "int8":
            return binding.prefill(st["q"], st["k_cache"], st["v_cache"], *where, st["seq_starts"], st["scale"],
                                   out=st["out"])
        pools = (st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"])
        if c["form"] == "decode":
            return binding.decode_int8(st["q"], *pools, *where, st["scale"], out=st["out"])
        return binding.prefill_int8(st["q"], *pools, *where, st["seq_starts"], st["scale"], out=st["out"])
    pools = (st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"])
    if c["op"] == "store":
        binding.write_cache_int8(st["k_new"], st["v_new"], st["slots"], *pools)
    binding.read_cache_int8(*pools, st["block_tables"], st["seq_starts"], st["k_out"], st["v_out"],
                            first_tokens=st["first"])
    if c["op"] == "load":
        return {"k": st["k_out"], "v": st["v_out"]}
    return {"k": st["k_out"], "v": st["v_out"], "k_scales": st["k_scales"], "v_scales": st["v_scales"]}


def _tokens(st, x):
    """[S, Hk, T, D] in 32 bits: the rows of a pool in the order of the tables."""
    ids = st["block_tables"].long().clamp(min=0)
    rows = st[x + "_cache"][ids].float()
    if x + "_scales" in st:
        rows = rows * st[x + "_scales"][ids].transpose(2, 3)[..., None]
    S, B, bs, Hk, D = rows.shape
    return rows.view(S, B * bs, Hk, D).transpose(1, 2)


def _plain_attend(st):
    c = st["case"]
    S, Hk, D = c["seqs"], c["kv_heads"], c["head"]
    G, most = c["heads"] // Hk, c["new_hi"]
    starts, ctx = st["seq_starts"].long(), st["context_lens"].long()
    new = starts[1:] - starts[:-1]
    i = torch.arange(most, device=DEV)
    row = (starts[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][row].float().view(S, most, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hk, G * most, D)
    s = torch.matmul(q, _tokens(st, "k").transpose(2, 3)) * st["scale"]
    pos = (ctx - new)[:, None] + i
    unseen = (torch.arange(s.shape[-1], device=DEV) > pos[..., None]) | (i >= new[:, None])[..., None]
    s = s.view(S, Hk, G, most, -1).masked_fill_(unseen[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    # Rows of a block behind a context's end hold no token: their weight is zero.
    out = torch.matmul(p.view(S, Hk, G * most, -1), _tokens(st, "v")).view(S, Hk, G, most, D)
    out = (out / torch.where(total > 0, total, 1.0)).permute(0, 3, 1, 2, 4).reshape(S, most, c["heads"], D)
    # Back to the token buffer; rows behind the last sequence stay.
    row = torch.arange(st["q"].shape[0], device=DEV)
    seq = (torch.searchsorted(starts, row, right=True) - 1).clamp(max=S - 1)
    real = (row < starts[-1])[:, None, None]
    out = out[seq, (row - starts[seq]).clamp(max=most - 1)]
    return torch.where(real, out, st["out"].float()).to(st["q"].dtype)


def _plain_store(st):
    c = st["case"]
    bs = c["block"]
    for x in "kv":
        code, scale = _quantise(st[x + "_new"])
        st[x + "_cache"].view(-1, c["kv_heads"], c["head"])[st["slots"]] = code
        st[x + "_scales"][st["slots"] // bs, :, st["slots"] % bs] = scale
    return dict(_plain_load(st), k_scales=st["k_scales"], v_scales=st["v_scales"])


def _plain_load(st):
    bs = st["case"]["block"]
    starts = st["seq_starts"].long()
    row = torch.arange(st["k_out"].shape[0], device=DEV)
    seq = torch.searchsorted(starts, row, right=True) - 1
    pos = row - starts[seq]
    if st["first"] is not None:
        pos = pos + st["first"].long()[seq]
    block = st["block_tables"][seq, pos // bs].long()
    for x in "kv":
        value = st[x + "_cache"][block, pos % bs].float() * st[x + "_scales"][block, :, pos % bs][..., None]
        st[x + "_out"].copy_(value)
    return {"k": st["k_out"], "v": st["v_out"]}


# ---- what a pass cannot do without -------------------------------------------------


def work(case):
    c = case
    Hk, D = c["kv_heads"], c["head"]
    lens = _lens(c)
    tokens = sum(n for n, _ in lens)
    if c["op"] != "attend":
        elt = 4 if c["dtype"] == "f32" else 2
        # A value and its code, both ways for what is stored and read back; scales, slots, tables.
        ways = 2 if c["op"] == "store" else 1
        return {"bytes": tokens * Hk * 2 * ways * (D * (elt + 1) + 4) + 8 * tokens * (ways - 1)
                + 4 * sum(_ceil(n + o, c["block"]) for n, o in lens), "flops": 0}
    row = {"bf16": 4 * D, "f32": 8 * D, "int8": 2 * D + 8}[c["pool"]]
    keys = sum(n + o for n, o in lens if n)
    pairs = sum(n * o + n * (n + 1) // 2 for n, o in lens)
    return {"bytes": keys * Hk * row + 2 * tokens * c["heads"] * D * (4 if c["pool"] == "f32" else 2)
            + 4 * keys // c["block"] + 8 * c["seqs"], "flops": 4 * pairs * c["heads"] * D}


# ---- the definition, in 64 bits -----------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    bs, Hk, D = c["block"], c["kv_heads"], c["head"]
    starts, lens = st["seq_starts"].tolist(), st["context_lens"].tolist()

    def held(x, s, first, last):
        """Tokens first .. last - 1 of sequence s in pool x: [tokens, Hk, D]."""
        t = torch.arange(first, last, device=DEV)
        ids = st["block_tables"][s, t // bs].long()
        value = st[x + "_cache"][ids, t % bs].double()
        if x + "_scales" in st:
            value = value * st[x + "_scales"][ids, :, t % bs].double().unsqueeze(-1)
        return value

    if c["op"] == "load":
        return {x: torch.cat([held(x, s, 0, n) for s, n in enumerate(lens)]) for x in "kv"}
    if c["op"] == "store":
        result = {}
        for x in "kv":
            rows = st[x + "_new"].double()
            scale = (rows.abs().max(-1).values / 127.0).float().double()
            steps = rows / scale.unsqueeze(-1)
            low = steps.floor()
            part = steps - low
            # Halves go to the even neighbour.
            up = (part > 0.5) | ((part == 0.5) & (low % 2 != 0))
            result[x] = (low + up.double()).clamp(-127, 127) * scale.unsqueeze(-1)
            scales = st[x + "_scales"].double()
            for t, slot in enumerate(st["slots"].tolist()):
                scales[slot // bs, :, slot % bs] = scale[t]
            result[x + "_scales"] = scales
        return result
    G = c["heads"] // Hk
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for s, n in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        if a == b:
            continue
        k, v = held("k", s, 0, n), held("v", s, 0, n)
        hidden = torch.arange(n, device=DEV)[None, :] > torch.arange(n - (b - a), n, device=DEV)[:, None]
        for h in range(c["heads"]):
            score = st["q"][a:b, h].double() @ k[:, h // G].T / math.sqrt(D)
            out[a:b, h] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v[:, h // G]
    return out
