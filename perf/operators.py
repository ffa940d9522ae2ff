"""Measured cases of the shared-prefix paged cache: block tables and slot maps, the append of new tokens' rows and the attention
of a batch that shares a prefix.

A case names its operator in "op":

tables  one scheduling step of a continuous batch: every request's pages and the slots of its new tokens from its lengths
append  the new tokens' K and V rows into the pages
attn    attention of the batch's new tokens over the shared prefix and over each request's own tokens

Keys and queries are clustered as the package's synthetic workloads are (centres N(0, 1), spread 0.3), values N(0, 1).
"""
import math
import random
import zlib

import torch

own = False

D = 128  # head dimension of the library
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of a small batch: 16 requests, a token each
        dict(name="tables_decode_16", op="tables", requests=16, page=16, longest=2048, new=1, mix="decode"),
        # continuous batching: most requests decode, some prefill a chunk, some are done, some drop rejected draft tokens
        dict(name="tables_mixed_256", op="tables", requests=256, page=16, longest=8192, new=512, mix="mixed"),
        # many short prompts at once, odd page size
        dict(name="tables_prefill_4096", op="tables", requests=4096, page=24, longest=1000, new=499, mix="prefill"),
        # a decode step's rows of one layer
        dict(name="append_decode_64", op="append", tokens=64, kv_heads=8, page=16, dtype="bf16"),
        # a long prompt's rows of one layer
        dict(name="append_prefill_32k", op="append", tokens=32768, kv_heads=8, page=32, dtype="bf16"),
        # 32-bit rows, odd count and page size
        dict(name="append_f32_5001", op="append", tokens=5001, kv_heads=4, page=12, dtype="f32"),
        # one question on a short prompt: latency
        dict(name="attn_one_4k", op="attn", requests=1, kv_heads=8, group=4, page=16, prefix=4096, suffix=100, query=1, dtype="bf16"),
        # parallel samples of a 36k-token document
        dict(name="attn_16_36k", op="attn", requests=16, kv_heads=8, group=4, page=16, prefix=36864, suffix=500, query=1, dtype="bf16"),
        # batched serving on a 32k-token shared prompt, ragged own parts
        dict(name="attn_256_32k", op="attn", requests=256, kv_heads=8, group=4, page=32, prefix=32768, suffix=2047, query=1, dtype="bf16"),
        # questions of up to 1021 tokens prefilled on an 8k-token document
        dict(name="attn_chunk_8k", op="attn", requests=7, kv_heads=8, group=4, page=16, prefix=8191, suffix=300, query=1021, dtype="bf16"),
        # few requests on a 250k-token context, two draft tokens each at most
        dict(name="attn_4_250k", op="attn", requests=4, kv_heads=8, group=4, page=16, prefix=250000, suffix=1000, query=2, dtype="bf16"),
        # 32-bit rows: one KV head, two query heads
        dict(name="attn_f32_4k", op="attn", requests=24, kv_heads=1, group=2, page=16, prefix=4096, suffix=777, query=1, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn"])
    page = rng.choice([8, 16, 16, 32, 64, 12, 24, 5])
    if op == "tables":
        mix = rng.choice(["decode", "mixed", "prefill"])
        return dict(op=op, requests=_log(rng, 1, 4096), page=page, longest=_log(rng, 16, 4096),
                    new=1 if mix == "decode" else _log(rng, 2, 400), mix=mix)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 16384), kv_heads=rng.choice([1, 2, 4, 8]), page=page,
                    dtype=rng.choice(["bf16", "f32"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    query = rng.choice([1, 1, 1, _log(rng, 2, 700)])
    if dtype == "f32":
        return dict(op=op, requests=_log(rng, 1, 16), kv_heads=min(4, kv_heads), group=group, page=page, prefix=_log(rng, 1, 4096),
                    suffix=_log(rng, 1, 500), query=min(query, 64), dtype=dtype)
    requests = _log(rng, 1, 128) if query == 1 else _log(rng, 1, 8)
    return dict(op=op, requests=requests, kv_heads=kv_heads, group=group, page=page, prefix=_log(rng, 1, 40000 if query == 1 else 8000),
                suffix=_log(rng, 1, 2000 if query == 1 else 300), query=query, dtype=dtype)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _uniform(g, lo, hi, n):
    """n whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64)


def _lengths(c):
    """The case's requests as (tokens before, new tokens), the same for every seed; a seed sets their order."""
    rng = random.Random(zlib.crc32(repr(sorted((k, v) for k, v in c.items() if k != "name")).encode()))
    found = []
    for _ in range(c["requests"]):
        if c["op"] == "attn":
            found.append((rng.randint(0, c["suffix"]), rng.randint(1, c["query"])))
            continue
        old, new = rng.randint(1, c["longest"]), rng.randint(1, c["new"])
        if c["mix"] == "prefill" and rng.randrange(8):  # a new request; one in eight continues
            old = 0
        if c["mix"] == "mixed":
            kind = rng.randrange(20)
            if kind == 1:  # the end of a request
                new = -old
            elif kind == 2:  # rejected draft tokens
                new = -min(old, rng.randint(1, 4))
            elif kind:  # a decode step; else a chunk of a prompt
                new = 1
        found.append((old, new))
    return found


def _shuffled_lengths(c, g):
    x = torch.tensor(_lengths(c), dtype=torch.int64, device="cuda")[torch.randperm(c["requests"], generator=g, device="cuda")]
    return x[:, 0].contiguous(), x[:, 1].contiguous()


def _prepare_tables(c, g):
    B, P = c["requests"], c["page"]
    old, add = _shuffled_lengths(c, g)
    columns = (c["longest"] + c["new"] + P - 1) // P
    have = (old + P - 1) // P
    first = torch.cumsum(have, 0) - have
    total = int(have.sum())
    n_pages = total + int(((old + add + P - 1) // P - have).clamp(min=0).sum()) + 37
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    col = torch.arange(columns, device="cuda")
    at = torch.where(col[None] < have[:, None], first[:, None] + col[None], torch.zeros_like(col)[None])
    block_table = torch.where(col[None] < have[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
    # the ring has run for a while: its head is somewhere
    head = int(_uniform(g, 0, 10 ** 6, 1))
    free_pages = torch.empty(n_pages, dtype=torch.int32, device="cuda")
    where = (head + torch.arange(n_pages, device="cuda")) % n_pages
    free_pages[where[: n_pages - total]] = order[total:]
    free_pages[where[n_pages - total:]] = -1
    slots = (int(add.clamp(min=0).sum()) + 63) // 64 * 64  # padded, as a captured batch is
    s = dict(case=c, P=P, n_pages=n_pages, slots=slots, seq_len=old.int(), n_new=add.int(), block_table=block_table, free_pages=free_pages,
             free_state=torch.tensor([head, head + n_pages - total], dtype=torch.int64, device="cuda"))
    if own:
        from semantic_paged_kv_head_gb300 import ice
        s["cache"] = ice.PagedCache(n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=n_pages, max_requests=B, max_blocks=columns,
                                    max_tokens=1)
    return s


def _prepare_append(c, g):
    n, H, P, t = c["tokens"], c["kv_heads"], c["page"], TYPES[c["dtype"]]
    n_pages = n // P + 17
    k, v = (torch.randn((n, H, D), generator=g, device="cuda").to(t) for _ in range(2))
    k_pages, v_pages = (torch.randn((n_pages, H, P, D), generator=g, device="cuda").to(t) for _ in range(2))
    # whole runs of a page's slots, pages in any order, the last three rows padding where there are that many
    page = torch.randperm(n_pages, generator=g, device="cuda")
    i = torch.arange(n, device="cuda") + int(_uniform(g, 0, P - 1, 1))
    slot_map = page[i // P] * P + i % P
    if n > 8:
        slot_map[-3:] = -1
    s = dict(case=c, P=P, k=k, v=v, k_pages=k_pages, v_pages=v_pages, slot_map=slot_map)
    if own:
        from semantic_paged_kv_head_gb300 import ice
        s["cache"] = ice.PagedCache(n_kv_heads=H, n_q_heads=H, page_size=P, n_pages=n_pages, max_requests=1, max_blocks=1, max_tokens=1,
                                    dtype=t)
    return s


def _prepare_attn(c, g):
    B, H, G, P, L, t = c["requests"], c["kv_heads"], c["group"], c["page"], c["prefix"], TYPES[c["dtype"]]
    before, nq = _shuffled_lengths(c, g)
    seq_len = before + nq
    columns = (c["query"] + c["suffix"] + P - 1) // P
    have = (seq_len + P - 1) // P
    first = torch.cumsum(have, 0) - have
    prefix_pages = (L + P - 1) // P
    n_pages = prefix_pages + int(have.sum())
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    col = torch.arange(columns, device="cuda")
    at = torch.where(col[None] < have[:, None], prefix_pages + first[:, None] + col[None], torch.zeros_like(col)[None])
    block_table = torch.where(col[None] < have[:, None], order[at], torch.full_like(order[at], -1)).contiguous()
    T = int(nq.sum())
    centres = torch.randn((H, 64, D), generator=g, device="cuda")
    head = torch.arange(H, device="cuda")

    def near(shape, dim):  # rows around their head's centres; `dim`: the head's place in `shape`
        pick = torch.randint(0, 64, shape, generator=g, device="cuda")
        which = head.view([-1 if k == dim else 1 for k in range(len(shape))])
        return (centres[which, pick] + 0.3 * torch.randn((*shape, D), generator=g, device="cuda")).to(t)

    k_pages = near((n_pages, H, P), 1)
    v_pages = torch.randn((n_pages, H, P, D), generator=g, device="cuda").to(t)
    pick = torch.randint(0, 64, (T, H, 1), generator=g, device="cuda")  # a group's query heads look at one centre
    q = (centres[head[None, :, None], pick] + 0.3 * torch.randn((T, H, G, D), generator=g, device="cuda")).to(t).view(T, H * G, D)
    q_start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    q_start[1:] = torch.cumsum(nq, 0)
    s = dict(case=c, P=P, q=q, q_start=q_start, seq_len=seq_len.int(), block_table=block_table, prefix_table=order[:prefix_pages].contiguous(),
             prefix_len=L, k_pages=k_pages, v_pages=v_pages)
    if own:
        from semantic_paged_kv_head_gb300 import ice
        s["cache"] = ice.PagedCache(n_kv_heads=H, n_q_heads=H * G, page_size=P, n_pages=n_pages, max_requests=B, max_blocks=columns,
                                    max_tokens=B * c["query"], dtype=t)
    return s


def prepare(case, seed):
    g = _generator(seed)
    return {"tables": _prepare_tables, "append": _prepare_append, "attn": _prepare_attn}[case["op"]](case, g)


def _plain_tables(s):
    P, n_pages, slots = s["P"], s["n_pages"], s["slots"]
    old, add = s["seq_len"].long(), s["n_new"].long()
    table, ring, head, tail = s["block_table"], s["free_pages"], s["free_state"][0], s["free_state"][1]
    new = old + add
    had, has = (old + P - 1) // P, (new + P - 1) // P
    col = torch.arange(table.shape[1], device="cuda")
    grow, shrink = (has - had).clamp(min=0), (had - has).clamp(min=0)
    given = torch.cumsum(shrink, 0) - shrink
    taken = torch.cumsum(grow, 0) - grow
    gone = (col[None] >= has[:, None]) & (col[None] < had[:, None])
    ring[((tail + given[:, None] + col[None] - has[:, None]) % n_pages)[gone]] = table[gone]
    fresh = (col[None] >= had[:, None]) & (col[None] < has[:, None])
    table[fresh] = ring[((head + taken[:, None] + col[None] - had[:, None]) % n_pages)[fresh]]
    q_start = torch.zeros(len(old) + 1, dtype=torch.int64, device="cuda")
    q_start[1:] = torch.cumsum(add.clamp(min=0), 0)
    i = torch.arange(slots, device="cuda")
    r = (torch.searchsorted(q_start, i, right=True) - 1).clamp(max=len(old) - 1)
    used = i < q_start[-1]
    at = torch.where(used, old[r] + i - q_start[r], torch.zeros_like(i))
    slot_map = torch.where(used, table[r, at // P].long() * P + at % P, torch.full_like(i, -1))
    state = torch.stack([head + grow.sum(), tail + shrink.sum()])
    return dict(seq_len=new.int(), free_state=state, q_start=q_start.int(), slot_map=slot_map, positions=at.int(), block_table=table,
                free_pages=ring)


def _plain_append(s):
    slot = s["slot_map"]
    used = slot >= 0
    page, off = slot[used] // s["P"], slot[used] % s["P"]
    s["k_pages"][page, :, off] = s["k"][used]
    s["v_pages"][page, :, off] = s["v"][used]
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"])


def _plain_attn(s):
    c, q = s["case"], s["q"]
    B, H, G, P, L = c["requests"], c["kv_heads"], c["group"], c["page"], s["prefix_len"]
    T, scale = q.shape[0], 1.0 / math.sqrt(D)
    start, length = s["q_start"].long(), s["seq_len"].long()
    nq = start[1:] - start[:-1]
    rows = q.float().view(T, H, G, D) * scale
    # the prefix: all rows of a KV head against its keys
    kp, vp = (x[s["prefix_table"].long()].transpose(0, 1).reshape(H, -1, D)[:, :L].float() for x in (s["k_pages"], s["v_pages"]))
    w1 = rows.transpose(0, 1).reshape(H, T * G, D) @ kp.transpose(1, 2)
    # the requests' own tokens: queries padded to the longest
    Q = c["query"]
    i = torch.arange(Q, device="cuda")
    tok = (start[:-1, None] + i[None]).clamp(max=T - 1)  # [B, Q]
    page = s["block_table"].long().clamp(min=0)
    ks, vs = (x[page].transpose(1, 2).reshape(B, H, -1, D).float() for x in (s["k_pages"], s["v_pages"]))
    w2 = rows[tok].permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D) @ ks.transpose(2, 3)
    t = torch.arange(ks.shape[2], device="cuda")
    seen = t[None, None] <= (length - nq)[:, None, None] + i[None, :, None]  # [B, Q, S]
    w2 = torch.where(seen[:, None, :, None], w2.view(B, H, Q, G, -1), torch.full((), -math.inf, device="cuda")).view(B, H, Q * G, -1)
    # back to one row a token: r its request, j its place among that request's new tokens
    r = torch.searchsorted(start, torch.arange(T, device="cuda"), right=True) - 1
    j = torch.arange(T, device="cuda") - start[r]
    per_token = lambda x: x.view(B, H, Q, G, -1)[r, :, j].transpose(0, 1).reshape(H, T * G, -1)  # noqa: E731
    m2 = w2.amax(-1, keepdim=True)
    p2 = torch.exp(w2 - m2)
    l2, o2 = p2.sum(-1, keepdim=True), p2 @ vs
    m1 = w1.amax(-1, keepdim=True)
    m2, l2, o2 = per_token(m2), per_token(l2), per_token(o2)
    m = torch.maximum(m1, m2)
    p1 = torch.exp(w1 - m)
    f = torch.exp(m2 - m)
    out = (p1 @ vp + f * o2) / (p1.sum(-1, keepdim=True) + f * l2)
    return out.view(H, T, G, D).transpose(0, 1).reshape(T, H * G, D).to(q.dtype)


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tables": _plain_tables, "append": _plain_append, "attn": _plain_attn}[op](s)
    cache = s["cache"]
    if op == "tables":
        seq_len, free_state, q_start, slot_map, positions = cache.tables(s["seq_len"], s["n_new"], s["block_table"], s["free_pages"],
                                                                         s["free_state"], s["slots"])
        return dict(seq_len=seq_len, free_state=free_state, q_start=q_start, slot_map=slot_map, positions=positions,
                    block_table=s["block_table"], free_pages=s["free_pages"])
    if op == "append":
        cache.append(s["k"], s["v"], s["slot_map"], s["k_pages"], s["v_pages"])
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"])
    return cache.attn(s["q"], s["q_start"], s["seq_len"], s["block_table"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_len"])


def work(case):
    op = case["op"]
    if op == "append":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["tokens"] * (8 + 4 * case["kv_heads"] * D * es), "flops": 0}
    lengths, P = _lengths(case), case["page"]
    if op == "tables":
        # 8 B read and 8 B written a request, 4 B read and 4 B written a page moved, 12 B written a slot
        slots = sum(max(0, n) for _, n in lengths)
        moved = sum(abs((o + n + P - 1) // P - (o + P - 1) // P) for o, n in lengths)
        return {"bytes": 16 * len(lengths) + 8 * moved + 12 * slots, "flops": 0}
    es = 2 if case["dtype"] == "bf16" else 4
    H, G, L = case["kv_heads"], case["group"], case["prefix"]
    T, keys = sum(n for _, n in lengths), sum(o + n for o, n in lengths)
    pairs = T * L + sum(n * o + n * (n + 1) // 2 for o, n in lengths)
    return {"bytes": 2 * es * D * H * (L + keys) + 2 * es * D * H * G * T, "flops": 4 * D * H * G * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers only
    P = case["page"]
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            # the pages as rows [page * P + offset][head]
            pool = s[name + "_pages"].double().permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], D).clone()
            for n in range(0, case["tokens"], 4096):
                slot = s["slot_map"][n:n + 4096]
                pool[slot[slot != -1]] = s[name][n:n + 4096][slot != -1].double()
            out[name + "_pages"] = pool.view(-1, P, case["kv_heads"], D).permute(0, 2, 1, 3).contiguous()
        return out
    H, G, L = case["kv_heads"], case["group"], s["prefix_len"]
    start, length = s["q_start"].tolist(), s["seq_len"].tolist()
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")

    def tokens(pool, table, n):  # [H, n, D] of the first n tokens of a page list
        table = table[: (n + P - 1) // P].long()
        return pool[table].permute(1, 0, 2, 3).reshape(H, -1, D)[:, :n].double()

    pk, pv = (tokens(s[x], s["prefix_table"], L) for x in ("k_pages", "v_pages"))
    for b in range(case["requests"]):
        n, S = start[b + 1] - start[b], length[b]
        sk, sv = (tokens(s[x], s["block_table"][b], S) for x in ("k_pages", "v_pages"))
        for a in range(0, n, 128):
            e = min(n, a + 128)
            qb = s["q"][start[b] + a:start[b] + e].double().view(e - a, H, G, D).permute(1, 0, 2, 3).reshape(H, -1, D)
            far = torch.arange(S, device="cuda")[None] > S - n + torch.arange(a, e, device="cuda")[:, None]
            own_part = (qb @ sk.transpose(1, 2)).view(H, e - a, G, S).masked_fill(far[None, :, None], -math.inf).view(H, -1, S)
            p = torch.softmax(torch.cat([qb @ pk.transpose(1, 2), own_part], 2) / math.sqrt(D), dim=2)
            o = p[:, :, :L] @ pv + p[:, :, L:] @ sv
            out[start[b] + a:start[b] + e] = o.view(H, e - a, G, D).permute(1, 0, 2, 3).reshape(e - a, H * G, D)
    return out
