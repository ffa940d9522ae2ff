"""Measured cases of a serving step around the paged cache: rotary positions with several axes on the way into the pages,
requests that share pages (forking, copy on write, ending), compaction of the pool, and verification of drafted tokens.

A case names its operator in "op":

rope     new tokens' queries and keys rotated by their positions on one or several axes, keys and values written into the pages
fork     the life of parallel samples: requests are forked, every one takes the slots of its new tokens (what is shared is copied
         on write, in every layer), and the forked ones end
compact  the pool's pages in use moved to its front: block tables, reference counts, ring of free pages, the pages of every layer
verify   drafted tokens against the target's probabilities (with given random numbers) or its logits (greedy)
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
        # a decode step's rows of one layer: 64 requests, a token each, positions of time, height and width
        dict(name="rope_decode_64", op="rope", tokens=64, kv_heads=8, group=4, page=16, axes=3, pairs=64, interleaved=False, dtype="bf16"),
        # a long prompt of text, images and video of one layer
        dict(name="rope_prefill_32k", op="rope", tokens=32768, kv_heads=8, group=4, page=32, axes=3, pairs=64, interleaved=False, dtype="bf16"),
        # 32-bit rows, neighbouring elements as pairs, a quarter of the head not rotated, odd count and page size
        dict(name="rope_f32_5001", op="rope", tokens=5001, kv_heads=4, group=2, page=12, axes=2, pairs=48, interleaved=True, dtype="f32"),
        # 16 samples of one 36k-token document
        dict(name="fork_16_36k", op="fork", parents=1, children=15, longest=36864, new=1, kv_heads=8, page=16, layers=4, dtype="bf16"),
        # 64 requests of up to 2047 tokens as four beams each, a token and up to four drafts a step
        dict(name="fork_256_2k", op="fork", parents=64, children=3, longest=2047, new=5, kv_heads=8, page=16, layers=4, dtype="bf16"),
        # many short prompts, eight samples each, odd page size, 32-bit rows
        dict(name="fork_4096_500", op="fork", parents=512, children=7, longest=500, new=1, kv_heads=2, page=24, layers=1, dtype="f32"),
        # a small pool after some requests have ended
        dict(name="compact_1k", op="compact", pages=1000, requests=16, kv_heads=8, page=16, layers=4, dtype="bf16"),
        # a pool of 2 GB a layer, half in use by 256 requests
        dict(name="compact_32k", op="compact", pages=32768, requests=256, kv_heads=8, page=16, layers=1, dtype="bf16"),
        # one request, four drafts: latency
        dict(name="verify_one", op="verify", requests=1, drafts=4, vocab=128000, mode="sample", dtype="f32"),
        # a batch with up to seven drafts a request
        dict(name="verify_64", op="verify", requests=64, drafts=7, vocab=128000, mode="sample", dtype="f32"),
        # drafts looked up in the prompt: the draft has no probabilities; bf16, odd vocabulary
        dict(name="verify_lookup_256", op="verify", requests=256, drafts=3, vocab=50001, mode="lookup", dtype="bf16"),
        # greedy decoding on logits, odd vocabulary
        dict(name="verify_greedy_128", op="verify", requests=128, drafts=4, vocab=150001, mode="greedy", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "fork", "compact", "verify", "verify"])
    page, dtype, kv_heads = rng.choice([8, 16, 16, 32, 64, 12, 24, 5]), rng.choice(["bf16", "bf16", "f32"]), rng.choice([1, 2, 4, 8])
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 12000), kv_heads=kv_heads, group=rng.choice([1, 2, 4, 8]), page=page, axes=rng.choice([1, 2, 3, 3, 4]),
                    pairs=rng.choice([64, 64, 8, 16, 32, 48]), interleaved=rng.random() < 0.3, dtype=dtype)
    if op == "fork":
        children = _log(rng, 1, 31)
        return dict(op=op, parents=_log(rng, 1, 512 // (children + 1)), children=children, longest=_log(rng, 1, 3000), new=_log(rng, 1, 40),
                    kv_heads=kv_heads, page=page, layers=rng.choice([1, 2, 4]), dtype=dtype)
    if op == "compact":
        return dict(op=op, pages=_log(rng, 40, 8000), requests=_log(rng, 1, 300), kv_heads=min(4, kv_heads), page=page,
                    layers=rng.choice([1, 2]), dtype=dtype)
    return dict(op=op, requests=_log(rng, 1, 100), drafts=_log(rng, 1, 7), vocab=_log(rng, 30, 130000),
                mode=rng.choice(["sample", "sample", "lookup", "greedy"]), dtype=dtype)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rng(c):
    return random.Random(zlib.crc32(repr(sorted((k, v) for k, v in c.items() if k != "name")).encode()))


def _randn(g, shape, t):
    return torch.randn(shape, generator=g, device="cuda", dtype=t)


def _whole(g, lo, hi, n):
    """n whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64)


# ---- rope ---------------------------------------------------------------------------------

def _sections(c):
    """Frequency and axis of each pair: one geometric series over all pairs, cut into a section an axis."""
    n, axes = c["pairs"], c["axes"]
    freq = [500000.0 ** (-i / n) for i in range(n)]
    return freq, [0 if axes == 1 else min(axes - 1, i * axes // n) for i in range(n)]


def _prepare_rope(c, g):
    T, H, G, P, t = c["tokens"], c["kv_heads"], c["group"], c["page"], TYPES[c["dtype"]]
    rows = _randn(g, (T, (G + 2) * H * D), t)  # the output of a fused projection
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split([G * H * D, H * D, H * D], 1))
    n_pages = T // P + 17
    k_pages, v_pages = (_randn(g, (n_pages, H, P, D), t) for _ in range(2))
    page = torch.randperm(n_pages, generator=g, device="cuda")
    i = torch.arange(T, device="cuda") + int(_whole(g, 0, P - 1, 1))
    slot_map = page[i // P] * P + i % P
    if T > 8:  # padding, as a captured batch has it
        slot_map[-3:] = -1
    # text counts on all axes alike; frames of 14 x 18 patches stand still in time and count in height and width
    if T <= 256:  # requests at positions of their own
        positions = _whole(g, 0, 120000, T)[None].repeat(c["axes"], 1)
        positions[1:] -= _whole(g, 0, 500, T)[None]
    else:
        at = torch.arange(T, device="cuda")
        film = (at // 1024) % 2 == 1
        patch = at % 252
        axes = [torch.where(film, x, at) for x in (at // 252, at - patch + patch // 18, at - patch + patch % 18)]
        positions = torch.stack((axes + [at])[: c["axes"]]) + _whole(g, 0, 50000, 1)
    freq, axis = _sections(c)
    s = dict(case=c, P=P, q=q, k=k, v=v, positions=positions.int().contiguous(), offset=int(_whole(g, 0, 40000, 1)), slot_map=slot_map,
             k_pages=k_pages, v_pages=v_pages, q_out=torch.zeros((T, G * H, D), dtype=t, device="cuda"))
    if own:
        from semantic_paged_kv_head_gb300 import ice
        s["rope"] = ice.Rope(freq, axis, interleaved=c["interleaved"])
        s["cache"] = ice.PagedCache(n_kv_heads=H, n_q_heads=H * G, page_size=P, n_pages=n_pages, max_requests=1, max_blocks=1, max_tokens=1,
                                    dtype=t)
    else:
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        s["axis"] = torch.tensor(axis, device="cuda")
    return s


def _plain_rope(s):
    c, used = s["case"], s["slot_map"] >= 0
    n = c["pairs"]
    angle = (s["positions"].long() + s["offset"]).double()[s["axis"]].T * s["freq"]  # [tokens, pairs]
    cos, sin = (x.float()[:, None] for x in (torch.cos(angle), torch.sin(angle)))

    def turn(x):
        y = x.float().clone()
        if c["interleaved"]:
            a, b = y[..., 0:2 * n:2].clone(), y[..., 1:2 * n:2].clone()
            y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., :n].clone(), y[..., n:2 * n].clone()
            y[..., :n], y[..., n:2 * n] = a * cos - b * sin, b * cos + a * sin
        return y.to(x.dtype)

    s["q_out"][used] = turn(s["q"])[used]
    page, off = s["slot_map"][used] // s["P"], s["slot_map"][used] % s["P"]
    s["k_pages"][page, :, off] = turn(s["k"])[used]
    s["v_pages"][page, :, off] = s["v"][used]
    return dict(q=s["q_out"], k_pages=s["k_pages"], v_pages=s["v_pages"])


def _own_rope(s):
    s["cache"].rope_append(s["q"], s["k"], s["v"], s["positions"], s["rope"], s["slot_map"], s["k_pages"], s["v_pages"],
                           pos_offset=s["offset"], q_out=s["q_out"])
    return dict(q=s["q_out"], k_pages=s["k_pages"], v_pages=s["v_pages"])


def _exact_rope(c, s):
    T, H, P = c["tokens"], c["kv_heads"], c["page"]
    freq, axis = _sections(c)
    out = {name: s[name].double() for name in ("k_pages", "v_pages")}
    out["q"] = s["q_out"].double()
    unit = torch.ones((T, c["pairs"]), dtype=torch.complex128, device="cuda")
    for i, (f, a) in enumerate(zip(freq, axis)):
        unit[:, i] = torch.exp(1j * ((s["positions"][a].double() + s["offset"]) * f))
    live = torch.nonzero(s["slot_map"] >= 0).view(-1)
    at = s["slot_map"][live]
    for name, x in (("q", s["q"]), ("k_pages", s["k"]), ("v_pages", s["v"])):
        x = x.double().contiguous()
        if name != "v_pages":
            head = x[..., : 2 * c["pairs"]]
            pairs = head.unflatten(2, (-1, 2)) if c["interleaved"] else head.unflatten(2, (2, -1)).transpose(2, 3)
            pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit[:, None])
            x = torch.cat([(pairs if c["interleaved"] else pairs.transpose(2, 3)).flatten(2), x[..., 2 * c["pairs"]:]], 2)
        if name == "q":
            out["q"][live] = x[live]
        else:
            flat = out[name].permute(0, 2, 1, 3).reshape(-1, H, D)
            flat[at] = x[live]
            out[name] = flat.view(-1, P, H, D).permute(0, 2, 1, 3).contiguous()
    return dict(q=out["q"], k_pages=out["k_pages"], v_pages=out["v_pages"])


# ---- fork ---------------------------------------------------------------------------------

def _lengths(c):
    """The parents' tokens and every request's new ones (parents first), the same for every seed; a seed sets the order."""
    rng = _rng(c)
    some = c["longest"] if c["parents"] == 1 else None
    return ([some or rng.randint(1, c["longest"]) for _ in range(c["parents"])],
            [rng.randint(1, c["new"]) for _ in range(c["parents"] * (c["children"] + 1))])


def _prepare_fork(c, g):
    P, B0, t = c["page"], c["parents"], TYPES[c["dtype"]]
    n = B0 * (c["children"] + 1)
    length, new = (torch.tensor(x, device="cuda") for x in _lengths(c))
    if B0 == 1:  # the document's end lies inside a page
        length -= _whole(g, 1, max(1, min(P - 1, c["longest"] - 1)), 1) if c["longest"] > 1 else 0
    length, new = length[torch.randperm(B0, generator=g, device="cuda")], new[torch.randperm(n, generator=g, device="cuda")]
    columns = (c["longest"] + c["new"] + P - 1) // P
    have = (length + P - 1) // P
    first = torch.cumsum(have, 0) - have
    total = int(have.sum())
    n_pages = total + n * ((c["new"] + P - 1) // P + 1) + 5
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    col = torch.arange(columns, device="cuda")
    row = torch.randperm(n, generator=g, device="cuda")  # whose row is whose
    parent, child = row[:B0], row[B0:]
    block_table = torch.full((n, columns), -1, dtype=torch.int32, device="cuda")
    at = torch.where(col[None] < have[:, None], first[:, None] + col[None], torch.zeros_like(col)[None])
    block_table[parent] = torch.where(col[None] < have[:, None], order[at], torch.full_like(order[at], -1))
    page_refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    page_refs[order[:total].long()] = 1
    head = int(_whole(g, 0, 10 ** 6, 1))
    free_pages = torch.empty(n_pages, dtype=torch.int32, device="cuda")
    where = (head + torch.arange(n_pages, device="cuda")) % n_pages
    free_pages[where[: n_pages - total]] = order[total:]
    free_pages[where[n_pages - total:]] = -1
    seq_len = torch.zeros(n, dtype=torch.int64, device="cuda")
    seq_len[parent] = length
    src = parent.repeat(c["children"])
    forked = torch.zeros(n, dtype=torch.bool, device="cuda")
    forked[child] = True
    after = seq_len.clone()
    after[child] = seq_len[src]
    k_pages, v_pages = (_randn(g, (c["layers"], n_pages, c["kv_heads"], P, D), t) for _ in range(2))
    s = dict(case=c, P=P, n_pages=n_pages, slots=(int(new.sum()) + 63) // 64 * 64, seq_len=seq_len.int(), src=src.int(), dst=child.int(),
             n_new=new.int(), n_end=torch.where(forked, -(after + new), -new).int(), block_table=block_table, page_refs=page_refs,
             free_pages=free_pages, free_state=torch.tensor([head, head + n_pages - total], dtype=torch.int64, device="cuda"),
             k_pages=k_pages, v_pages=v_pages)
    if own:
        from semantic_paged_kv_head_gb300 import ice
        s["cache"] = ice.PagedCache(n_kv_heads=c["kv_heads"], n_q_heads=c["kv_heads"], page_size=P, n_pages=n_pages, max_requests=n,
                                    max_blocks=columns, max_tokens=1, dtype=t)
    return s


def _plain_step(s, seq_len, n_new, slots):
    """Block tables, counts and ring of one step of requests that share pages, in place; what the step gives besides."""
    P, n_pages, table, ring, refs = s["P"], s["n_pages"], s["block_table"], s["free_pages"], s["page_refs"]
    old, add = seq_len.long(), n_new.long()
    head, tail = s["free_state"][0], s["free_state"][1]
    new, r = old + add, torch.arange(len(old), device="cuda")
    had, has = (old + P - 1) // P, (new + P - 1) // P
    col = torch.arange(table.shape[1], device="cuda")
    # holders let go: of pages that they no longer touch, and (if anybody else holds it) of the page that they grow in
    gone = (col[None] >= has[:, None]) & (col[None] < had[:, None])
    grower = (add > 0) & (old % P > 0)
    mine = table.gather(1, (old // P).clamp(max=table.shape[1] - 1)[:, None])[:, 0].long().clamp(min=0)
    pages = torch.cat([table[gone].long(), mine[grower]])
    left = refs - torch.bincount(pages, minlength=n_pages).int()
    big = 1 << 20
    who = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
    who.scatter_reduce_(0, pages, torch.cat([(r + 1)[:, None].expand_as(gone)[gone], (r + 1 + big)[grower]]), "amax")
    keeps = grower & (left[mine] == 0) & (who[mine] == r + 1 + big)
    copies = grower & ~keeps
    at = table.long().clamp(min=0)
    freed = gone & (left[at] == 0) & (who[at] == r[:, None] + 1)
    grow = (has - had).clamp(min=0)
    takes = grow + copies
    taken = torch.cumsum(takes, 0) - takes
    back = table[freed]
    ring[(tail + torch.arange(len(back), device="cuda")) % n_pages] = back
    fresh = (col[None] >= had[:, None]) & (col[None] < has[:, None])
    got = ring[((head + (taken + copies)[:, None] + col[None] - had[:, None]) % n_pages)[fresh]]
    copy_to = ring[(head + taken) % n_pages]
    none = torch.full_like(copy_to, -1)
    copy_src, copy_dst = torch.where(copies, mine.int(), none), torch.where(copies, copy_to, none)
    table[fresh] = got
    table[r[copies], (old // P)[copies]] = copy_to[copies]
    refs.copy_(left)
    refs[torch.cat([got, copy_to[copies], mine[keeps].int()]).long()] = 1
    q_start = torch.zeros(len(old) + 1, dtype=torch.int64, device="cuda")
    q_start[1:] = torch.cumsum(add.clamp(min=0), 0)
    i = torch.arange(slots, device="cuda")
    whose = (torch.searchsorted(q_start, i, right=True) - 1).clamp(max=len(old) - 1)
    used = i < q_start[-1]
    place = torch.where(used, old[whose] + i - q_start[whose], torch.zeros_like(i))
    slot_map = torch.where(used, table[whose, place // P].long() * P + place % P, torch.full_like(i, -1))
    s["free_state"].copy_(torch.stack([head + takes.sum(), tail + freed.sum()]))
    return new.int(), q_start.int(), slot_map, place.int(), copy_src, copy_dst


def _plain_copy(s, src, dst):
    live = dst >= 0
    src, dst = src[live].long(), dst[live].long()
    s["k_pages"][:, dst] = s["k_pages"][:, src]
    s["v_pages"][:, dst] = s["v_pages"][:, src]


def _fork_outputs(s, step, end):
    new, q_start, slot_map, positions, copy_src, copy_dst = step
    return dict(seq_len=new, q_start=q_start, slot_map=slot_map, positions=positions, copy_src=copy_src, copy_dst=copy_dst, end_len=end,
                **{x: s[x] for x in ("block_table", "page_refs", "free_pages", "free_state", "k_pages", "v_pages")})


def _plain_fork(s):
    P, seq_len, src, dst = s["P"], s["seq_len"].clone(), s["src"].long(), s["dst"].long()
    table = s["block_table"]
    length = seq_len[src]
    col = torch.arange(table.shape[1], device="cuda")
    shared = col[None] < ((length + P - 1) // P)[:, None]
    table[dst] = torch.where(shared, table[src], table[dst])
    s["page_refs"] += torch.bincount(table[src][shared].long(), minlength=s["n_pages"]).int()
    seq_len[dst] = length
    step = _plain_step(s, seq_len, s["n_new"], s["slots"])
    _plain_copy(s, step[4], step[5])
    end = _plain_step(s, step[0], s["n_end"], 0)
    return _fork_outputs(s, step, end[0])


def _own_fork(s):
    cache, table, refs, ring, state = s["cache"], s["block_table"], s["page_refs"], s["free_pages"], s["free_state"]
    seq_len = cache.fork(s["src"], s["dst"], s["seq_len"], table, refs)
    new, _, q_start, slot_map, positions, copy_src, copy_dst = cache.tables_shared(seq_len, s["n_new"], table, ring, state, refs, s["slots"],
                                                                                   free_state_out=state)
    cache.copy(copy_src, copy_dst, s["k_pages"], s["v_pages"])
    end = cache.tables_shared(new, s["n_end"], table, ring, state, refs, 0, free_state_out=state)
    return _fork_outputs(s, (new, q_start, slot_map, positions, copy_src, copy_dst), end[0])


# ---- compact ------------------------------------------------------------------------------

def _in_use(c):
    """Pages of each request and how many of them it shares with the one before, the same for every seed."""
    rng = _rng(c)
    most, found, used = c["pages"] // 2, [], 0
    for r in range(c["requests"]):
        n = min(most - used, rng.randint(1, max(1, c["pages"] // c["requests"])))
        share = rng.randint(0, min(3, found[-1][0])) if found and n > 0 else 0
        found.append((n + share, share))
        used += n
    return found


def _prepare_compact(c, g):
    P, n_pages, t = c["page"], c["pages"], TYPES[c["dtype"]]
    have = _in_use(c)
    columns = max(max(n for n, _ in have), 1)
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    rows, at, before = [], 0, []
    for n, share in have:
        own_pages = list(range(at, at + n - share))
        at += n - share
        before = before[:share] + own_pages
        rows.append(before + [-1] * (columns - n))
    rows = torch.tensor(rows, device="cuda")
    table = torch.where(rows >= 0, order[rows.clamp(min=0)], torch.full_like(order[rows.clamp(min=0)], -1)).contiguous()
    prefix = order[at:at + min(16, n_pages - at)].contiguous()  # the batch's shared prefix
    refs = torch.bincount(torch.cat([table[table >= 0], prefix]).long(), minlength=n_pages).int()
    seq_len = torch.tensor([n * P for n, _ in have], device="cuda") - _whole(g, 0, P - 1, len(have))
    k_pages, v_pages = (_randn(g, (c["layers"], n_pages, c["kv_heads"], P, D), t) for _ in range(2))
    s = dict(case=c, P=P, n_pages=n_pages, seq_len=seq_len.clamp(min=0).int(), block_table=table, page_refs=refs, prefix=prefix,
             free_pages=torch.full((n_pages,), -1, dtype=torch.int32, device="cuda"), k_pages=k_pages, v_pages=v_pages,
             free_state=torch.zeros(2, dtype=torch.int64, device="cuda"), table_out=torch.full_like(table, -1),
             refs_out=torch.empty_like(refs), prefix_out=torch.empty_like(prefix))
    if own:
        from semantic_paged_kv_head_gb300 import ice
        s["cache"] = ice.PagedCache(n_kv_heads=c["kv_heads"], n_q_heads=c["kv_heads"], page_size=P, n_pages=n_pages,
                                    max_requests=c["requests"], max_blocks=columns, max_tokens=1, dtype=t)
    return s


def _compact_outputs(s, move_src, move_dst):
    return dict(move_src=move_src, move_dst=move_dst, **{x: s[x] for x in ("table_out", "refs_out", "prefix_out", "free_pages", "free_state",
                                                                            "k_pages", "v_pages")})


def _plain_compact(s):
    n_pages, refs, P = s["n_pages"], s["page_refs"], s["P"]
    live, page = refs > 0, torch.arange(n_pages, device="cuda")
    n_live = live.sum()
    src, dst = page[live & (page >= n_live)], page[~live & (page < n_live)]
    goes = page.clone()
    goes[src] = dst
    move_src, move_dst = (torch.full((n_pages // 2,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    move_src[: len(src)], move_dst[: len(src)] = src.int(), dst.int()
    held = torch.arange(s["block_table"].shape[1], device="cuda")[None] < ((s["seq_len"] + P - 1) // P)[:, None]
    s["table_out"][held] = goes[s["block_table"][held].long()].int()
    s["prefix_out"].copy_(goes[s["prefix"].long()])
    s["refs_out"].zero_()
    s["refs_out"][goes[live]] = refs[live]
    rest = page[page >= n_live]
    s["free_pages"][: len(rest)] = rest.int()
    s["free_state"].copy_(torch.stack([n_live * 0, n_pages - n_live]))
    _plain_copy(s, move_src, move_dst)
    return _compact_outputs(s, move_src, move_dst)


def _own_compact(s):
    cache = s["cache"]
    move_src, move_dst = cache.compact(s["seq_len"], s["block_table"], s["page_refs"], s["free_pages"], s["free_state"],
                                       extra_pages=s["prefix"], block_table_out=s["table_out"], page_refs_out=s["refs_out"],
                                       extra_pages_out=s["prefix_out"])[:2]
    cache.copy(move_src, move_dst, s["k_pages"], s["v_pages"])
    return _compact_outputs(s, move_src, move_dst)


# ---- verify -------------------------------------------------------------------------------

def _drafted(c):
    """Drafts and accepted ones of each request, the same for every seed; a seed sets their order."""
    rng = _rng(c)
    found = []
    for _ in range(c["requests"]):
        n = c["drafts"] if rng.randrange(3) else rng.randint(0, c["drafts"])
        a = 0
        while a < n and rng.random() < 0.7:
            a += 1
        found.append((n, a))
    return found


def _prepare_verify(c, g):
    n, K, V, t = c["requests"], c["drafts"], c["vocab"], TYPES[c["dtype"]]
    have = torch.tensor(_drafted(c), device="cuda")[torch.randperm(n, generator=g, device="cuda")]
    n_draft, accepted = have[:, 0].contiguous(), have[:, 1].contiguous()
    base = 2.5 * _randn(g, (n, K + 1, V), torch.float32)
    i = torch.arange(K, device="cuda")
    taken = i[None] < accepted[:, None]
    s = dict(case=c, n_draft=n_draft.int(), draft=None, uniform=None)
    if c["mode"] == "greedy":
        s["target"] = base.to(t)  # logits
        best = s["target"].float()
        lowest = torch.where(best == best.amax(-1, keepdim=True), torch.arange(V, device="cuda"), torch.full((), V, device="cuda")).amin(-1)[:, :K]
        other = (lowest + 1 + torch.randint(0, V - 1, (n, K), generator=g, device="cuda")) % V
        tokens = torch.where(taken, lowest, other)
    else:
        s["target"] = torch.softmax(base, -1).to(t)
        if c["mode"] == "sample":  # a draft model that is near the target
            s["draft"] = torch.softmax(base[:, :K] + 0.7 * _randn(g, (n, K, V), torch.float32), -1).to(t)
            p, q = s["target"][:, :K].float(), s["draft"].float()
            weight = torch.where(taken[..., None], torch.minimum(p, q), (q - p).clamp(min=0))
        else:  # the drafted token is one that the target would, or would not, have taken
            weight = s["target"][:, :K].float()
        race = torch.empty((n, K, V), device="cuda").exponential_(generator=g)
        tokens = (weight / race).argmax(-1)
        pick = lambda x: x[:, :K].float().gather(2, tokens[..., None])[..., 0]  # noqa: E731
        ratio = (pick(s["target"]) / (pick(s["draft"]) if s["draft"] is not None else 1.0)).clamp(max=1.0)
        u = torch.rand((n, K), generator=g, device="cuda")
        u = torch.where(taken, u * ratio * 0.999, (ratio + u * (1 - ratio)).clamp(max=1 - 2.0 ** -24))
        s["uniform"] = torch.cat([u, torch.rand((n, 1), generator=g, device="cuda")], 1).contiguous()
    s["tokens"] = tokens.int()
    if own:
        from semantic_paged_kv_head_gb300 import ice
        s["cache"] = ice.PagedCache(n_kv_heads=1, n_q_heads=1, page_size=16, n_pages=1, max_requests=n, max_blocks=1, max_tokens=1)
    return s


def _plain_verify(s):
    c, target, tokens, n_draft, u = s["case"], s["target"], s["tokens"].long(), s["n_draft"].long(), s["uniform"]
    n, K, V = c["requests"], c["drafts"], c["vocab"]
    i = torch.arange(K, device="cuda")
    places, r = torch.arange(V, device="cuda"), torch.arange(n, device="cuda")
    if u is None:
        x = target.float()
        best = torch.where(x == x.amax(-1, keepdim=True), places, torch.full((), V, device="cuda")).amin(-1)
        good = tokens == best[:, :K]
    else:
        p = target[:, :K].gather(2, tokens[..., None])[..., 0].double()
        q = s["draft"].gather(2, tokens[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(p)
        good = u[:, :K].double() * q < p
    good &= i[None] < n_draft[:, None]
    accepted = torch.cumprod(good.long(), 1).sum(1)
    if u is None:
        last = best[r, accepted]
    else:
        # what the target has above the draft, or all of it behind the last draft; 64 bits: a place next to a border
        weight = target[r, accepted].double()
        at = accepted.clamp(max=K - 1)
        below = s["draft"][r, at].double() if s["draft"] is not None else (places[None] == tokens[r, at][:, None]).double()
        above = (weight - below).clamp(min=0)
        residual = (accepted < n_draft) & (above.sum(1) > 0)
        sums = torch.cumsum(torch.where(residual[:, None], above, weight), 1)
        last = torch.searchsorted(sums, (u[:, K].double() * sums[:, -1])[:, None], right=True)[:, 0].clamp(max=V - 1)
    out = torch.where(i[None] < accepted[:, None], tokens, torch.full_like(tokens, -1))
    out = torch.cat([out, torch.full_like(out[:, :1], -1)], 1)
    out[r, accepted] = last
    return dict(tokens=out.int(), accepted=accepted.int(), n_new=(accepted - n_draft).int())


def _own_verify(s):
    tokens, accepted, n_new = s["cache"].verify(s["tokens"], s["n_draft"], s["target"], s["draft"], s["uniform"])
    return dict(tokens=tokens, accepted=accepted, n_new=n_new)


def _exact_verify(c, s):
    K, V = c["drafts"], c["vocab"]
    tokens, accepted, n_new = [], [], []
    for r, (n, drafted) in enumerate(zip(s["n_draft"].tolist(), s["tokens"].tolist())):
        row, a, last = [-1] * (K + 1), 0, None
        while last is None:
            p = s["target"][r, a].double()
            if s["uniform"] is None:
                token = int(torch.nonzero(p == p.max())[0])
                if a < n and drafted[a] == token:
                    row[a] = token
                    a += 1
                    continue
                last = token
                break
            q = None
            if a < n:
                q = s["draft"][r, a].double() if s["draft"] is not None else torch.zeros(V, dtype=torch.float64, device="cuda")
                if s["draft"] is None:
                    q[drafted[a]] = 1.0
                if float(s["uniform"][r, a]) * float(q[drafted[a]]) < float(p[drafted[a]]):
                    row[a] = drafted[a]
                    a += 1
                    continue
                rest = torch.relu(p - q)
                p = rest if float(rest.sum()) > 0 else p
            reached = torch.cumsum(p, 0)
            beyond = torch.nonzero(reached > float(s["uniform"][r, K]) * float(reached[-1]))
            last = int(beyond[0]) if len(beyond) else V - 1
        row[a] = last
        tokens.append(row)
        accepted.append(a)
        n_new.append(a - n)
    return {k: torch.tensor(x, dtype=torch.int32, device="cuda") for k, x in (("tokens", tokens), ("accepted", accepted), ("n_new", n_new))}


# ---- the cases' functions -------------------------------------------------------------------

def prepare(case, seed):
    g = _generator(seed)
    return {"rope": _prepare_rope, "fork": _prepare_fork, "compact": _prepare_compact, "verify": _prepare_verify}[case["op"]](case, g)


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "fork": _own_fork, "compact": _own_compact, "verify": _own_verify}[op](s)
    return {"rope": _plain_rope, "fork": _plain_fork, "compact": _plain_compact, "verify": _plain_verify}[op](s)


def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "rope":
        T, H, G = case["tokens"], case["kv_heads"], case["group"]
        return {"bytes": T * (2 * (G + 2) * H * D * es + 8 + 4 * case["axes"]), "flops": T * (G + 1) * H * 6 * case["pairs"]}
    if op == "verify":
        # the accepted drafts' probabilities, then the rows that decide the last token; greedy: every row up to the first wrong draft
        K, V, n_bytes = case["drafts"], case["vocab"], 0
        for n, a in _drafted(case):
            rows = a + 1 if case["mode"] == "greedy" else 2 if case["mode"] == "sample" and a < n else 1
            n_bytes += rows * V * es + 4 * (K + 5)
        return {"bytes": n_bytes, "flops": 0}
    page = case["kv_heads"] * case["page"] * D * es
    P = case["page"]
    if op == "fork":
        length, new = _lengths(case)
        c = case["children"]
        pages = sum((x + P - 1) // P for x in length)
        # tables: entries copied and counts raised, the same dropped, slots and lengths; pages: the copies of those whose end is shared
        copies = sum(c for x in length if case["parents"] == 1 or x % P)
        return {"bytes": pages * c * 16 + sum(new) * 12 + len(new) * 32 + copies * case["layers"] * 4 * page, "flops": 0}
    have = _in_use(case)
    entries, live = sum(n for n, _ in have), sum(n - share for n, share in have)
    live += min(16, case["pages"] - live)
    moved = live * (case["pages"] - live) // case["pages"]  # pages in any order: as many of them lie behind the front
    return {"bytes": 8 * entries + 12 * case["pages"] + moved * case["layers"] * 4 * page, "flops": 0}


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers and copies of the inputs
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_verify(case, s)
