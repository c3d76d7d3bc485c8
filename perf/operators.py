"""What the attention and cache operators are measured on.

Three operators: ``attn_prompt`` (attention over packed prompts), ``attn_decode``
(one new token over a paged cache) and the pages of that cache (``kv_extend``,
``kv_write``, ``kv_fork``, ``kv_free``, ``kv_compact``, ``kv_copy_pages``).  With ``own`` false, ``run``
computes them from elementary torch operations; with ``own`` true it makes the
library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
NEG = float("-inf")


# ------------------------------------------------------------------- cases

def listed():
    return [
        # three chat turns that arrive together: latency counts
        dict(name="prompt_short", op="prompt", ranks=1, heads=8, kv_heads=2, dim=96, lens="17,1,40",
             shard=-1, causal=True, dtype="bf16"),
        # a prefill batch packed without padding, one rank with all heads
        dict(name="prompt_packed", op="prompt", ranks=1, heads=32, kv_heads=8, dim=128,
             lens="1531,700,64,2048,1,999,333,1200", shard=-1, causal=True, dtype="bf16"),
        # one long document, the 8192 tokens x 32 heads x 128 of the attention merge
        dict(name="prompt_long", op="prompt", ranks=1, heads=32, kv_heads=8, dim=128, lens="8192",
             shard=-1, causal=True, dtype="bf16"),
        # context parallel: the queries of shard 5 against the key shards of 8 ranks, partial
        # outputs for the merge (shards 0-4 whole, 5 on the diagonal, 6 and 7 with no key visible)
        dict(name="prompt_context", op="prompt", ranks=8, heads=16, kv_heads=4, dim=64,
             lens="900,131", shard=5, causal=True, dtype="fp16"),
        # one user, one short cache, the heads of one of 8 tensor-parallel ranks: latency counts
        dict(name="decode_one", op="decode", ranks=1, heads=8, kv_heads=1, dim=128, lens="777",
             page=16, dtype="bf16"),
        # a serving batch with caches of all ages
        dict(name="decode_batch", op="decode", ranks=1, heads=32, kv_heads=8, dim=128,
             lens=_lens(64, 1, 4096, 7), page=16, dtype="bf16"),
        # two long documents: few rows, so the work has to be split over the length
        dict(name="decode_long", op="decode", ranks=1, heads=32, kv_heads=8, dim=128,
             lens="131072,100001", page=64, dtype="bf16"),
        # context parallel decode: each of 8 ranks holds a part of every cache, some of them none
        dict(name="decode_context", op="decode", ranks=8, heads=16, kv_heads=4, dim=64,
             lens=_lens(15, 1, 2000, 9) + ",0", page=32, dtype="fp16"),
        # a small beam search: latency counts
        dict(name="fork_few", op="fork", entries=4, seqs=2, tokens=300, layers=2, pages=256, page=16,
             heads=2, dim=64, dtype="bf16"),
        # parallel sampling: 128 continuations of 64 prompts, 8 layers
        dict(name="fork_many", op="fork", entries=128, seqs=64, tokens=700, layers=8, pages=4096,
             page=16, heads=8, dim=128, dtype="bf16"),
        # a fragmented cache squeezed together before it shrinks
        dict(name="compact", op="compact", live=1600, seqs=64, layers=8, pages=4096, page=16,
             heads=8, dim=128, dtype="bf16"),
        # the keys and values of a packed prefill go to fresh pages
        dict(name="write", op="write", lens=_lens(9, 1, 2048, 5), before=37, pages=2048, page=16,
             heads=8, dim=128, dtype="bf16"),
    ]


def _lens(n, lo, hi, seed):
    """n lengths from lo to hi, as text, the same for the same arguments."""
    x, got = seed * 2654435761 % (1 << 32), []
    for _ in range(n):
        x = (x * 1664525 + 1013904223) % (1 << 32)
        got.append(lo + x * (hi - lo + 1) // (1 << 32))
    return ",".join(map(str, got))


def _ints(text):
    return [int(x) for x in text.split(",")]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "fork", "compact", "write"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    if op == "prompt":
        ranks = rng.choice([1, 1, 2, 4])
        group = rng.choice([1, 2, 4, 5, 8])
        group = max(1, min(group, 32 // (kv * ranks)))
        causal = rng.random() < 0.8
        n = rng.choice([1, 2, 3, 5, 9])
        pairs = 5.4e11 / (4 * ranks * kv * group * dim) * (2 if causal else 1)   # of the largest listed case
        longest = _log(rng, 3, int(min(8192, math.sqrt(pairs / n))))
        lens = [longest] + [_log(rng, 1, longest) for _ in range(n - 1)]
        rng.shuffle(lens)
        shard = rng.choice([-1, -1, 0, ranks - 1])
        return dict(op=op, ranks=ranks, heads=kv * group, kv_heads=kv, dim=dim,
                    lens=",".join(map(str, lens)), shard=shard, causal=causal, dtype=dtype)
    if op == "decode":
        ranks = rng.choice([1, 1, 2, 8])
        group = rng.choice([1, 2, 3, 4, 8, 16, 20])
        batch = _log(rng, 1, 96)
        top = max(2, min(131072, 200_000_000 // (ranks * kv * dim * batch)))
        longest = _log(rng, 1, top)
        lens = [longest] + [rng.randint(0, longest) for _ in range(batch - 1)]
        return dict(op=op, ranks=ranks, heads=kv * group, kv_heads=kv, dim=dim,
                    lens=",".join(map(str, lens)), page=rng.choice([1, 8, 16, 20, 32, 64, 128]),
                    dtype=dtype)
    page = rng.choice([8, 16, 20, 64])
    layers = rng.choice([1, 2, 4, 7])
    pages = _log(rng, 128, min(4096, 500_000_000 // (page * kv * dim * 2 * layers)))
    if op == "fork":
        seqs = rng.randint(1, max(1, pages // 64))
        return dict(op=op, entries=_log(rng, 1, pages // 8), seqs=seqs,
                    tokens=_log(rng, 1, page * (pages // 2) // seqs), layers=layers, pages=pages,
                    page=page, heads=kv, dim=dim, dtype=dtype)
    if op == "compact":
        return dict(op=op, live=rng.randint(pages // 16, pages - 1), seqs=rng.randint(1, 40),
                    layers=layers, pages=pages, page=page, heads=kv, dim=dim, dtype=dtype)
    n = rng.choice([1, 2, 7, 30])
    before = rng.randint(0, 3 * page)
    top = (pages // n - 5) * page
    while top < 1:
        n //= 2
        top = (pages // n - 5) * page
    return dict(op=op, lens=",".join(str(_log(rng, 1, top)) for _ in range(n)), before=before,
                pages=pages, page=page, heads=kv, dim=dim, dtype=dtype)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def prepare(case, seed):
    return {"prompt": _prepare_prompt, "decode": _prepare_decode, "fork": _prepare_fork,
            "compact": _prepare_compact, "write": _prepare_write}[case["op"]](case, seed)


def _prepare_prompt(c, seed):
    """Queries, keys and values are the three parts of a fused projection's output."""
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    R, H, KV, D, lens = c["ranks"], c["heads"], c["kv_heads"], c["dim"], _ints(c["lens"])
    T = sum(lens)
    s = dict(case=c, q=[], k=[], v=[], o=[], lse=[], starts=[], diag=None)
    for r in range(R):
        qkv = _normal(g, (T, H + 2 * KV, D), dt)
        s["q"].append(qkv[:, :H])
        s["k"].append(qkv[:, H:H + KV])
        s["v"].append(qkv[:, H + KV:])
        s["o"].append(torch.empty((T, H, D), dtype=dt, device="cuda"))
        s["lse"].append(torch.empty((T, H), dtype=torch.float32, device="cuda"))
        s["starts"].append(_i32(_starts(lens)))
    if c["shard"] >= 0:
        s["diag"] = [_i32([(c["shard"] - r) * n for n in lens]) for r in range(R)]
    return s


def _prepare_decode(c, seed):
    """Pages are scattered over the pool, as after a while of serving."""
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    R, H, KV, D, P, lens = c["ranks"], c["heads"], c["kv_heads"], c["dim"], c["page"], _ints(c["lens"])
    B, width = len(lens), max(1, -(-max(lens) // P))
    need = sum(-(-n // P) for n in lens)
    N = need + need // 8 + 1
    s = dict(case=c, q=[], k=[], v=[], o=[], lse=[], table=[], lens=[])
    have = torch.arange(width)[None] < torch.tensor([-(-n // P) for n in lens])[:, None]
    for r in range(R):
        s["q"].append(_normal(g, (B, H, D), dt))
        s["k"].append(_normal(g, (N, P, KV, D), dt))
        s["v"].append(_normal(g, (N, P, KV, D), dt))
        s["o"].append(torch.empty((B, H, D), dtype=dt, device="cuda"))
        s["lse"].append(torch.empty((B, H), dtype=torch.float32, device="cuda"))
        perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        table[have.cuda()] = perm[:need]
        s["table"].append(table)
        s["lens"].append(_i32(lens))
    return s


def _pools(g, c, layers):
    shape = (layers, c["pages"], c["page"], c["heads"], c["dim"])
    return [_normal(g, shape, DTYPES[c["dtype"]]) for _ in range(2)]


def _prepare_fork(c, seed):
    """Prompts of about the same length fill scattered pages; rows of the table wait for forks."""
    g = _gen(seed)
    S, n, P, N = c["seqs"], c["entries"], c["page"], c["pages"]
    lens = [max(1, c["tokens"] - (7 * b) % (c["tokens"] // 2 + 1)) for b in range(S)]
    width = max(-(-x // P) for x in lens) + 1
    have = torch.arange(width)[None] < torch.tensor([-(-x // P) for x in lens])[:, None]
    table = torch.full((S + n, width), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    used = perm[:int(have.sum())]
    table[:S][have.cuda()] = used
    ref = torch.zeros(N, dtype=torch.int32, device="cuda")
    ref[used.long()] = 1
    src = torch.randint(0, S, (n,), generator=g, device="cuda").to(torch.int32)
    return dict(case=c, pools=_pools(g, c, c["layers"]), table=table, lens=_i32(lens + [0] * n), ref=ref,
                src=src, dst=_i32(list(range(S, S + n))),
                moves=torch.empty((n, 2), dtype=torch.int32, device="cuda"),
                count=torch.empty(1, dtype=torch.int32, device="cuda"),
                status=torch.empty(n, dtype=torch.int32, device="cuda"))


def _prepare_compact(c, seed):
    """`live` pages at random places, dealt to the sequences; what was there before is kept so
    that every pass starts from the same fragmented cache."""
    g = _gen(seed)
    S, N, live = c["seqs"], c["pages"], c["live"]
    width = -(-live // S)
    perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    table.view(-1)[:live] = perm[:live]
    ref = torch.zeros(N, dtype=torch.int32, device="cuda")
    ref[perm[:live].long()] = 1
    return dict(case=c, pools=_pools(g, c, c["layers"]), table0=table, ref0=ref,
                table=table.clone(), ref=ref.clone(),
                moves=torch.empty((max(1, N // 2), 2), dtype=torch.int32, device="cuda"),
                count=torch.empty(1, dtype=torch.int32, device="cuda"))


def _prepare_write(c, seed):
    """Sequences with `before` tokens in the cache get the rows of a packed projection."""
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    lens, P, N, KV, D = _ints(c["lens"]), c["page"], c["pages"], c["heads"], c["dim"]
    S = len(lens)
    first = -(-c["before"] // P)
    width = -(-(c["before"] + max(lens)) // P)
    perm = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    table[:, :first] = perm[:S * first].view(S, first)
    ref = torch.zeros(N, dtype=torch.int32, device="cuda")
    ref[perm[:S * first].long()] = 1
    kv = _normal(g, (sum(lens), 2 * KV, D), dt)
    k_pool, v_pool = (p[0] for p in _pools(g, c, 1))
    len0 = _i32([c["before"]] * S)
    return dict(case=c, k=kv[:, :KV], v=kv[:, KV:], k_pool=k_pool, v_pool=v_pool, table0=table, ref0=ref,
                len0=len0, table=table.clone(), ref=ref.clone(), lens=len0.clone(),
                starts=_i32(_starts(lens)), seqs=_i32(list(range(S))), add=_i32(lens),
                status=torch.empty(S, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "decode": _own_decode, "fork": _own_fork,
                "compact": _own_compact, "write": _own_write}[op](state)
    return {"prompt": _plain_prompt, "decode": _plain_decode, "fork": _plain_fork,
            "compact": _plain_compact, "write": _plain_write}[op](state)


def _bits(t):
    return t.view(torch.int16)


def _own_prompt(s):
    from collective_communication_amd import coll
    if "plan" not in s:
        s["plan"] = coll.prepare(coll.attn_prompt, s["q"], s["k"], s["v"], s["o"], s["starts"], s["starts"],
                                 lses=s["lse"], diags=s["diag"], causal=s["case"]["causal"])
    s["plan"]()
    return {"o": s["o"], "lse": s["lse"]}


def _own_decode(s):
    from collective_communication_amd import coll
    if "plan" not in s:
        c = s["case"]
        need = coll.attn_decode_workspace_bytes(c["ranks"], s["q"][0].shape[0],
                                                s["table"][0].shape[1] * c["page"], c["heads"],
                                                c["kv_heads"], c["dim"])
        work = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        s["plan"] = coll.prepare(coll.attn_decode, s["q"], s["k"], s["v"], s["table"], s["lens"], s["o"],
                                 work, lses=s["lse"])
    s["plan"]()
    return {"o": s["o"], "lse": s["lse"]}


def _own_fork(s):
    from collective_communication_amd import coll
    P = s["case"]["page"]
    if "plans" not in s:
        s["plans"] = [
            coll.prepare(coll.kv_free, s["table"], s["lens"], s["ref"], s["dst"]),
            coll.prepare(coll.kv_fork, s["table"], s["lens"], s["ref"], s["src"], s["dst"], P, s["moves"],
                         s["count"], s["status"]),
            coll.prepare(coll.kv_copy_pages, s["pools"], s["moves"], s["count"], layered=True)]
    for plan in s["plans"]:
        plan()
    return dict(k=_bits(s["pools"][0]), v=_bits(s["pools"][1]), table=s["table"], lens=s["lens"], ref=s["ref"],
                moves=s["moves"], count=s["count"], status=s["status"])


def _own_compact(s):
    from collective_communication_amd import coll
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    if "plans" not in s:
        work = torch.empty(coll.kv_compact_workspace_bytes(s["ref"].numel()), dtype=torch.uint8, device="cuda")
        s["plans"] = [
            coll.prepare(coll.kv_compact, s["table"], s["ref"], s["moves"], s["count"], work),
            coll.prepare(coll.kv_copy_pages, s["pools"], s["moves"], s["count"], layered=True)]
    for plan in s["plans"]:
        plan()
    return dict(k=_bits(s["pools"][0]), v=_bits(s["pools"][1]), table=s["table"], ref=s["ref"],
                moves=s["moves"], count=s["count"])


def _own_write(s):
    from collective_communication_amd import coll
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    s["lens"].copy_(s["len0"])
    if "plans" not in s:
        s["plans"] = [
            coll.prepare(coll.kv_extend, s["table"], s["lens"], s["ref"], s["seqs"], s["add"],
                         s["case"]["page"], s["status"]),
            coll.prepare(coll.kv_write, [s["k"]], [s["v"]], [s["k_pool"]], [s["v_pool"]], [s["table"]],
                         [s["lens"]], [s["starts"]])]
    for plan in s["plans"]:
        plan()
    return dict(k=_bits(s["k_pool"]), v=_bits(s["v_pool"]), table=s["table"], lens=s["lens"], ref=s["ref"],
                status=s["status"])


# ------------------------------------------------------------- plain forms

def _softmax_parts(s):
    """exp(s - max), its sum and the log-sum-exp over the last axis; a row of -inf gives 0, 0, -inf."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == NEG, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return p, l, m.squeeze(-1) + torch.log(l.squeeze(-1))


def _plain_prompt(s):
    """The packed rows are laid out by sequence, padded to the longest one."""
    c = s["case"]
    R, H, KV, D, lens = c["ranks"], c["heads"], c["kv_heads"], c["dim"], _ints(c["lens"])
    n, L, G, T = len(lens), max(lens), H // KV, sum(lens)
    starts = torch.stack(s["starts"])[0].long()
    at = torch.arange(L, device="cuda")
    size = starts[1:] - starts[:-1]
    inside = at[None] < size[:, None]
    rows = torch.where(inside, starts[:-1, None] + at[None], 0)                  # [n, L]
    q, k, v = (torch.stack(s[x]).float()[:, rows] for x in "qkv")                # [R, n, L, heads, D]
    q = q.view(R, n, L, KV, G, D).permute(0, 1, 3, 4, 2, 5).reshape(R * n * KV, G * L, D)
    k = k.permute(0, 1, 3, 4, 2).reshape(R * n * KV, D, L)
    v = v.permute(0, 1, 3, 2, 4).reshape(R * n * KV, L, D)
    sc = torch.bmm(q, k).mul_(1.0 / math.sqrt(D)).view(R, n, KV, G, L, L)
    see = inside[None, :, None, :].expand(R, n, L, L)
    if c["causal"]:
        diag = torch.stack(s["diag"]).long() if s["diag"] is not None else torch.zeros((R, n), device="cuda")
        see = see & (at[None, None, None, :] <= at[None, None, :, None] + diag[:, :, None, None])
    sc.masked_fill_(~see[:, :, None, None], NEG)
    p, l, lse = _softmax_parts(sc)
    o = torch.bmm(p.view(R * n * KV, G * L, L), v).view(R, n, KV, G, L, D)
    o = torch.where(l == 0, 0.0, o / l)
    o = o.permute(0, 1, 4, 2, 3, 5).reshape(R, n * L, H, D)
    lse = lse.permute(0, 1, 4, 2, 3).reshape(R, n * L, H)
    back = torch.where(inside, rows, T).view(-1)                                 # padding goes to a row of its own
    oo = torch.empty((R, T + 1, H, D), dtype=DTYPES[c["dtype"]], device="cuda")
    ll = torch.empty((R, T + 1, H), dtype=torch.float32, device="cuda")
    oo[:, back] = o.to(oo.dtype)
    ll[:, back] = lse
    return {"o": list(oo[:, :T]), "lse": list(ll[:, :T])}


def _plain_decode(s):
    """Every cache is gathered from its pages, padded to the longest one."""
    c = s["case"]
    R, H, KV, D, P = c["ranks"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    q, table, lens = torch.stack(s["q"]), torch.stack(s["table"]).long(), torch.stack(s["lens"]).long()
    B, L, G = q.shape[1], table.shape[2] * P, H // KV
    at = torch.arange(L, device="cuda")
    inside = at < lens[..., None]                                                # [R, B, L]
    row = torch.where(inside, table[:, :, at // P] * P + at % P, 0)
    k, v = (torch.stack([p.reshape(-1, KV, D)[i] for p, i in zip(s[x], row)]).float() for x in "kv")
    q = q.float().view(R * B * KV, G, D)
    k = k.permute(0, 1, 3, 4, 2).reshape(R * B * KV, D, L)
    v = v.permute(0, 1, 3, 2, 4).reshape(R * B * KV, L, D)
    sc = torch.bmm(q, k).mul_(1.0 / math.sqrt(D)).view(R, B, KV, G, L)
    sc.masked_fill_(~inside[:, :, None, None], NEG)
    p, l, lse = _softmax_parts(sc)
    o = torch.bmm(p.view(R * B * KV, G, L), v).view(R, B, KV, G, D)
    o = torch.where(l == 0, 0.0, o / l).view(R, B, H, D)
    return {"o": list(o.to(DTYPES[c["dtype"]])), "lse": list(lse.view(R, B, H))}


def _plain_free(table, lens, ref, seqs):
    rows = table[seqs]
    ref.index_put_((rows[rows >= 0].long(),), torch.tensor(-1, dtype=torch.int32, device="cuda"), accumulate=True)
    table[seqs] = -1
    lens[seqs] = 0


def _plain_fork(s):
    """All entries name rows that exist and destinations that are empty and distinct."""
    P, table, lens, ref = s["case"]["page"], s["table"], s["lens"], s["ref"]
    src, dst, n = s["src"].long(), s["dst"].long(), s["src"].numel()
    _plain_free(table, lens, ref, dst)
    full, part = lens[src] // P, lens[src] % P > 0
    upto = torch.cumsum(part.int(), 0)
    free = torch.sort((ref != 0).int(), stable=True).indices
    served = upto <= (ref == 0).sum()
    fresh = free[torch.clamp(upto - 1, 0, free.numel() - 1).long()].int()
    col = torch.arange(table.shape[1], device="cuda")[None]
    rows = torch.where(col < full[:, None], table[src],
                       torch.where((col == full[:, None]) & part[:, None], fresh[:, None], -1))
    last = torch.gather(table[src], 1, torch.clamp(full, max=table.shape[1] - 1).long()[:, None])[:, 0]
    table[dst] = torch.where(served[:, None], rows, table[dst])
    lens[dst] = torch.where(served, lens[src], 0)
    gained = rows[served]
    ref.index_put_((gained[gained >= 0].long(),), torch.tensor(1, dtype=torch.int32, device="cuda"), accumulate=True)
    need = served & part
    moves = torch.full((n, 2), -1, dtype=torch.int32, device="cuda")
    pairs = torch.stack([last, fresh], 1)[need]
    moves[:pairs.shape[0]] = pairs
    for pool in s["pools"]:
        pool[:, pairs[:, 1].long()] = pool[:, pairs[:, 0].long()]
    return dict(k=_bits(s["pools"][0]), v=_bits(s["pools"][1]), table=table, lens=lens, ref=ref, moves=moves,
                count=need.sum().int()[None], status=torch.where(served, 0, -2).int())


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    table, ref = s["table"], s["ref"]
    at = torch.arange(ref.numel(), device="cuda")
    live = ref > 0
    n = live.sum()
    hole, high = (~live & (at < n)).nonzero()[:, 0], (live & (at >= n)).nonzero()[:, 0]
    to = at.clone()
    to[high] = hole
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    ref[hole] = ref[high]
    ref[high] = 0
    moves = torch.full_like(s["moves"], -1)
    moves[:hole.numel()] = torch.stack([high, hole], 1).int()
    for pool in s["pools"]:
        pool[:, hole] = pool[:, high]
    return dict(k=_bits(s["pools"][0]), v=_bits(s["pools"][1]), table=table, ref=ref, moves=moves,
                count=torch.full((1,), hole.numel(), dtype=torch.int32, device="cuda"))


def _plain_write(s):
    """All entries name distinct rows, and there are pages for all of them."""
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    s["lens"].copy_(s["len0"])
    P, table, lens, ref, seqs = s["case"]["page"], s["table"], s["lens"], s["ref"], s["seqs"].long()
    have = (lens[seqs] + P - 1) // P
    need = (lens[seqs] + s["add"] + P - 1) // P - have
    upto = torch.cumsum(need, 0)
    free = torch.sort((ref != 0).int(), stable=True).indices
    col = torch.arange(table.shape[1], device="cuda")[None]
    k = (upto - need)[:, None] + col - have[:, None]
    new = (col >= have[:, None]) & (col < (have + need)[:, None])
    table[seqs] = torch.where(new, free[k.clamp(0, free.numel() - 1)].int(), table[seqs])
    ref[free[:int(upto[-1])]] = 1
    lens[seqs] += s["add"]
    starts = s["starts"].long()
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(starts, t, right=True) - 1
    pos = lens[b] - (starts[b + 1] - t)
    page, slot = table[b, pos // P].long(), pos % P
    s["k_pool"][page, slot] = s["k"]
    s["v_pool"][page, slot] = s["v"]
    return dict(k=_bits(s["k_pool"]), v=_bits(s["v_pool"]), table=table, lens=lens, ref=ref,
                status=torch.zeros_like(s["status"]))


# -------------------------------------------------------------------- work

def _pairs(c):
    """Visible (query, key) pairs of all ranks and sequences."""
    total = 0
    for r in range(c["ranks"]):
        for n in _ints(c["lens"]):
            d = (c["shard"] - r) * n if c["shard"] >= 0 else 0
            if not c["causal"] or d >= n - 1:
                total += n * n
            elif d > -n:                 # row i sees min(n, max(0, i + d + 1)) keys
                lo, hi = max(0, d + 1), min(n, n + d)
                rising = hi - lo + 1
                total += (lo + hi) * rising // 2 + n * (n - max(0, -d) - rising)
    return total


def work(case):
    c = case
    if c["op"] == "prompt":
        T, R = sum(_ints(c["lens"])), c["ranks"]
        return {"bytes": R * T * (2 * c["dim"] * (2 * c["heads"] + 2 * c["kv_heads"]) + 4 * c["heads"]),
                "flops": 4 * c["dim"] * c["heads"] * _pairs(c)}
    if c["op"] == "decode":
        T, R, B = sum(_ints(c["lens"])), c["ranks"], len(_ints(c["lens"]))
        return {"bytes": R * (T * c["kv_heads"] * c["dim"] * 4 + B * c["heads"] * (4 * c["dim"] + 4)),
                "flops": R * 4 * c["dim"] * c["heads"] * T}
    row = c["heads"] * c["dim"] * 2
    if c["op"] == "write":
        T = sum(_ints(c["lens"]))
        return {"bytes": 4 * T * row + 8 * c["pages"], "flops": 0}
    if c["op"] == "fork":
        P = c["page"]
        lens = [max(1, c["tokens"] - (7 * b) % (c["tokens"] // 2 + 1)) for b in range(c["seqs"])]
        ragged = sum(1 for x in lens if x % P) / len(lens)       # an entry's parent is any of them
        shared = sum(x // P for x in lens) / len(lens)
        return {"bytes": c["entries"] * (4 * ragged * c["layers"] * P * row + 16 * shared) + 4 * c["pages"],
                "flops": 0}
    moved = c["live"] * (c["pages"] - c["live"]) / c["pages"]    # live pages at or above the live count
    return {"bytes": 4 * moved * c["layers"] * c["page"] * row + 8 * c["pages"] + 8 * c["live"], "flops": 0}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    c = case
    if c["op"] == "prompt":
        return _exact_prompt(c, prepare(c, seed))
    if c["op"] == "decode":
        return _exact_decode(c, prepare(c, seed))
    return None                          # whole numbers: the plain form is exact


def _exact_rows(q, k, v, see):
    """One head: softmax(q k^T / sqrt(D)) v and its log-sum-exp in 64 bits; `see` marks the keys of a row."""
    s = (q.double() @ k.double().t().contiguous()) / math.sqrt(q.shape[1])
    s = s.masked_fill(~see, NEG)
    lse = torch.logsumexp(s, 1)
    w = torch.exp(s - lse[:, None])
    w = torch.where(see & (lse[:, None] > NEG), w, 0.0)
    return w @ v.double(), lse


def _exact_prompt(c, s):
    lens = _ints(c["lens"])
    out = {"o": [], "lse": []}
    for r in range(c["ranks"]):
        o = torch.zeros(s["o"][r].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["lse"][r].shape, dtype=torch.float64, device="cuda")
        a = 0
        for n in lens:
            d = (c["shard"] - r) * n if c["shard"] >= 0 else 0
            see = torch.ones((n, n), dtype=torch.bool, device="cuda")
            if c["causal"]:
                see = see.tril(d)
            for h in range(c["heads"]):
                kh = h // (c["heads"] // c["kv_heads"])
                o[a:a + n, h], lse[a:a + n, h] = _exact_rows(s["q"][r][a:a + n, h], s["k"][r][a:a + n, kh],
                                                             s["v"][r][a:a + n, kh], see)
            a += n
        out["o"].append(o)
        out["lse"].append(lse)
    return out


def _exact_decode(c, s):
    lens, P, G = _ints(c["lens"]), c["page"], c["heads"] // c["kv_heads"]
    out = {"o": [], "lse": []}
    for r in range(c["ranks"]):
        o = torch.zeros(s["o"][r].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"][r].shape, NEG, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pages = s["table"][r][b, :-(-n // P)].long()
            k = s["k"][r][pages].flatten(0, 1)[:n]
            v = s["v"][r][pages].flatten(0, 1)[:n]
            see = torch.ones((G, n), dtype=torch.bool, device="cuda")
            for h in range(c["kv_heads"]):
                rows = slice(h * G, h * G + G)
                o[b, rows], lse[b, rows] = _exact_rows(s["q"][r][b, rows], k[:, h], v[:, h], see)
        out["o"].append(o)
        out["lse"].append(lse)
    return out
