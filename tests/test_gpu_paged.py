"""The plain paged cache on the GPU against its definition in 64 bits: block tables and slot
maps, the append by slot map, the attention over a shared prefix and own tokens; refusals,
streams, graphs, and a run of all three as a decode loop uses them."""
import ctypes
import random

import pytest
import torch

from tests.paged_helpers import D, pages_of, plain_attn, plain_tables

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ice():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from semantic_paged_kv_head_gb300 import build
    build.build_lib()
    from semantic_paged_kv_head_gb300 import ice as m
    return m


def _cache(ice, **over):
    p = dict(n_kv_heads=2, n_q_heads=8, page_size=16, n_pages=64, max_requests=8, max_blocks=8, max_tokens=64)
    p.update(over)
    return ice.PagedCache(**p)


# ---- block tables and slot maps ----------------------------------------------------------

def _table_state(seed, n, P, cols, spare, kinds):
    """Lists: lengths, changes, table, ring, state of a pool that has run for a while."""
    rng = random.Random(seed)
    lens = [rng.randint(0, cols * P // 2) for _ in range(n)]
    new = []
    for a in lens:
        k = rng.choice(kinds)
        new.append({"one": 1, "none": 0, "end": -a, "drop": -min(a, rng.randint(1, 2 * P)),
                    "chunk": rng.randint(0, cols * P - a), "fill": cols * P - a}[k])
    used = sum(pages_of(a, P) for a in lens)
    need = sum(max(0, pages_of(a + b, P) - pages_of(a, P)) for a, b in zip(lens, new))
    n_pages = used + need + spare
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, at = [], 0
    for a in lens:
        k = pages_of(a, P)
        table.append(ids[at:at + k] + [-1] * (cols - k))
        at += k
    head = rng.randint(0, 5 * n_pages)
    ring = [-1] * n_pages
    for i, x in enumerate(ids[at:]):
        ring[(head + i) % n_pages] = x
    return lens, new, table, ring, [head, head + n_pages - used], n_pages


def _run_tables(ice, pc, lens, new, table, ring, state, n_slots, in_place=False):
    t = lambda x, d=torch.int32: torch.tensor(x, dtype=d, device="cuda")  # noqa: E731
    s, tb, rg, st = t(lens), t(table), t(ring), t(state, torch.int64)
    kw = dict(seq_len_out=s, free_state_out=st) if in_place else {}
    got = pc.tables(s, t(new), tb, rg, st, n_slots, **kw)
    code = pc.get_error()
    if not in_place:
        assert s.tolist() == lens and st.tolist() == state  # inputs stay
    return (code, *(x.tolist() for x in got), tb.tolist(), rg.tolist())


@pytest.mark.parametrize("n,P,cols,kinds", [
    (1, 16, 8, ["one"]), (1, 1, 5, ["end"]), (3, 64, 4, ["none"]), (16, 16, 8, ["one"]),
    (33, 16, 12, ["one", "none", "end", "drop", "chunk"]), (257, 5, 40, ["one", "end", "drop", "chunk", "fill"]),
    (1025, 12, 9, ["one", "none", "end", "drop", "chunk"]), (8192, 24, 6, ["one", "end", "chunk"]),
    (40, 3, 700, ["chunk", "fill", "end"])])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables(ice, n, P, cols, kinds, in_place):
    lens, new, table, ring, state, n_pages = _table_state(n + P, n, P, cols, 3, kinds)
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=n_pages, max_requests=n, max_blocks=cols, max_tokens=1)
    total = sum(max(0, x) for x in new)
    for n_slots in (total, total + 70):
        ref = plain_tables(lens, new, table, ring, state, n_slots, P)
        assert ref[0] == 0
        assert _run_tables(ice, pc, lens, new, table, ring, state, n_slots, in_place) == ref


@pytest.mark.parametrize("n,P,cols,kinds", [(256, 16, 30, ["one", "end", "drop", "chunk"]), (200, 16, 100, ["fill"])])
def test_tables_few_requests(ice, n, P, cols, kinds):
    """As many requests as the small blocks take, and fewer with more slots than those take."""
    test_tables(ice, n, P, cols, kinds, False)


@pytest.mark.parametrize("fault", ["pages", "columns", "slots", "negative", "too_long", "below_zero", "ring_backwards",
                                   "ring_too_full", "given_twice"])
def test_tables_all_or_nothing(ice, fault):
    P, cols = 4, 6
    lens, new, table, ring, state, n_pages = _table_state(5, 9, P, cols, 2, ["one", "chunk"])
    lens[2], new[2] = 9, 0
    table[2] = [0, 0, 0, -1, -1, -1]  # its ids do not matter here
    n_slots = sum(max(0, x) for x in new) + 3
    if fault == "pages":
        state = [state[0], state[0]]
        new = [x + P if lens[i] + x + P <= cols * P else x for i, x in enumerate(new)]
        n_slots += 9 * P
    elif fault == "columns":
        new[2] = cols * P - 9 + 1
        n_slots += cols * P
    elif fault == "slots":
        n_slots -= 4
    elif fault == "negative":
        lens[2] = -1
    elif fault == "too_long":
        lens[2] = cols * P + 1
    elif fault == "below_zero":
        new[2] = -10
    elif fault == "ring_backwards":
        state = [state[1] + 1, state[1]]
    elif fault == "ring_too_full":
        state = [state[0], state[0] + n_pages + 1]
    elif fault == "given_twice":
        state = [state[0], state[0] + n_pages]
        new = [0] * 9
        new[2] = -9
    ref = plain_tables(lens, new, table, ring, state, n_slots, P)
    assert ref[0] != 0
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=n_pages, max_requests=9, max_blocks=cols, max_tokens=1)
    assert _run_tables(ice, pc, lens, new, table, ring, state, n_slots) == ref
    assert pc.get_error() == 0  # cleared


# ---- append ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,H,P", [(1, 1, 1), (5, 2, 16), (64, 8, 16), (301, 3, 12), (2000, 8, 64)])
@pytest.mark.parametrize("strided", [False, True])
def test_append(ice, dtype, n, H, P, strided):
    n_pages = pages_of(n, P) + 3
    pc = _cache(ice, n_kv_heads=H, n_q_heads=H, page_size=P, n_pages=n_pages, dtype=dtype)
    g = torch.Generator().manual_seed(n)
    if strided:  # slices of one fused projection
        x = torch.randn((n, 3 * H, D), generator=g).to(dtype).cuda()
        k, v = x[:, H:2 * H], x[:, 2 * H:]
    else:
        k, v = (torch.randn((n, H, D), generator=g).to(dtype).cuda() for _ in range(2))
    slots = torch.randperm(n_pages * P, generator=g)[:n]
    slots[n // 2::7] = -1
    kp, vp = (torch.randn((n_pages, H, P, D), generator=g).to(dtype) for _ in range(2))
    kc, vc = kp.cuda(), vp.cuda()
    pc.append(k, v, slots.cuda(), kc, vc)
    assert pc.get_error() == 0
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            kp[s // P, :, s % P], vp[s // P, :, s % P] = k[i].cpu(), v[i].cpu()
    assert torch.equal(kc.cpu(), kp) and torch.equal(vc.cpu(), vp)


def test_append_reports_bad_slots(ice):
    pc = _cache(ice, n_pages=4)
    k = torch.ones((4, 2, D), dtype=BF16, device="cuda")
    kp, vp = (torch.zeros((4, 2, 16, D), dtype=BF16, device="cuda") for _ in range(2))
    pc.append(k, k, torch.tensor([3, 64, -2, 1 << 40], device="cuda"), kp, vp)
    assert pc.get_error() == ice.ICE_ERR_BOUNDS
    assert float(kp.float().sum()) == 2 * D and float(vp.float().sum()) == 2 * D and float(kp[0, :, 3].float().min()) == 1.0


# ---- attention ---------------------------------------------------------------------------

def _attn_case(seed, dtype, H, G, P, L, reqs, scale=1.0, stale=float("nan"), spare_rows=0, cols=None):
    """Everything an attention call takes; reqs: (new tokens, own tokens) of each request. Slots that
    hold no token are filled with `stale`."""
    g = torch.Generator().manual_seed(seed)
    T, B = sum(a for a, _ in reqs), len(reqs)
    cols = cols or max([1] + [pages_of(s, P) for _, s in reqs])
    n_pre = pages_of(L, P)
    n_pages = n_pre + sum(pages_of(s, P) for _, s in reqs) + 2
    ids = torch.randperm(n_pages, generator=g).int()
    kp, vp = (torch.randn((n_pages, H, P, D), generator=g) for _ in range(2))
    table = torch.full((B, cols), -1, dtype=torch.int32)
    at = n_pre
    lists = [(ids[:n_pre], L)]
    for b, (_, s) in enumerate(reqs):
        k = pages_of(s, P)
        table[b, :k] = ids[at:at + k]
        lists.append((ids[at:at + k], s))
        at += k
    used = torch.zeros((n_pages, P), dtype=torch.bool)
    for pages, n in lists:
        for j, p in enumerate(pages.tolist()):
            used[p, :min(P, n - j * P)] = True
    for x in (kp, vp):
        x.masked_fill_(~used[:, None, :, None], stale)
    q = scale * torch.randn((T + spare_rows, H * G, D), generator=g)
    q_start = torch.tensor([0] + [a for a, _ in reqs]).cumsum(0).int()
    seq_len = torch.tensor([s for _, s in reqs], dtype=torch.int32)
    return dict(q=q.to(dtype), q_start=q_start, seq_len=seq_len, table=table, k=kp.to(dtype), v=vp.to(dtype),
                prefix=ids[:n_pre].clone(), L=L, H=H, G=G, P=P, n_pages=n_pages)


def _attn_run(ice, c, pc=None, out=None, q=None, **over):
    x = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in {**c, **over}.items()}
    if pc is None:
        pc = _cache(ice, n_kv_heads=c["H"], n_q_heads=c["H"] * c["G"], page_size=c["P"], n_pages=c["n_pages"],
                    max_requests=len(c["seq_len"]), max_blocks=c["table"].shape[1], max_tokens=max(1, c["q"].shape[0]),
                    dtype=c["q"].dtype)
    got = pc.attn(x["q"] if q is None else q, x["q_start"], x["seq_len"], x["table"], x["k"], x["v"], x["prefix"], x["L"],
                  out=out)
    return got, pc


def _attn_check(ice, c, **kw):
    got, pc = _attn_run(ice, c, **kw)
    assert pc.get_error() == 0
    ref, tol = plain_attn(c["q"], c["q_start"], c["seq_len"], c["table"], c["k"], c["v"], c["prefix"], c["L"])
    n = int(c["q_start"][-1])
    err = (got.cpu().double()[:n] - ref[:n]).abs()
    assert bool((err <= tol[:n]).all()), float((err / tol[:n]).max())
    return got


# (new tokens, own tokens) of each request
DECODE = [(1, 1), (1, 16), (1, 17), (1, 300)]
MIXED = [(0, 40), (1, 40), (3, 3), (70, 90), (0, 0), (2, 129), (129, 400)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,G,P,L,reqs", [
    (1, 1, 16, 0, [(1, 1)]), (1, 1, 16, 1, [(1, 1)]), (1, 8, 16, 127, [(1, 5)]), (2, 4, 16, 128, DECODE),
    (2, 4, 16, 129, DECODE), (3, 2, 16, 0, DECODE), (2, 4, 12, 1000, DECODE), (1, 4, 5, 333, DECODE), (1, 2, 1, 150, DECODE),
    (2, 8, 64, 700, DECODE), (2, 1, 32, 515, MIXED), (2, 4, 16, 0, MIXED), (1, 8, 16, 260, MIXED), (2, 4, 24, 1, MIXED),
    (1, 4, 16, 500, [(1, 0), (2, 1), (4, 2)]),  # new tokens that no own token belongs to see the prefix only
    (1, 4, 16, 0, [(1, 0), (2, 1), (4, 2)]),    # or nothing: zeros
    (8, 4, 16, 4000, [(1, 60)]), (1, 1, 16, 90, [(300, 300)]), (1, 4, 16, 2000, [(1, 3000), (1, 2), (1, 700)]),
    (1, 2, 16, 64, [(0, 5), (0, 0)]),           # nothing to do
    (1, 4, 3, 200, DECODE), (2, 4, 48, 300, DECODE), (5, 1, 63, 257, DECODE),  # pages that fill no tile
    (1, 8, 16, 3000, [(1, 40), (2, 2500), (1, 129)]),  # one KV head: a range's halves side by side
    (8, 4, 16, 130, [(700, 700), (650, 900), (1, 5), (40, 60)]),  # long requests, whole and in parts
    (8, 4, 16, 0, [(1300, 1300)]), (4, 8, 32, 1000, [(17, 20), (16, 300), (33, 33)]),
    (1, 4, 16, 320, [(1, 1 + i % 37) for i in range(150)])])
def test_attn(ice, dtype, H, G, P, L, reqs):
    _attn_check(ice, _attn_case(H * 1000 + L, dtype, H, G, P, L, reqs))


@pytest.mark.parametrize("H,G,L,reqs", [
    (1, 2, 4096, [(1, 30)] * 24), (1, 1, 700, [(1, 9)] * 40), (2, 8, 200, [(3, 20), (2, 2), (1, 70)]), (4, 4, 3000, [(1, 5)] * 16),
    (1, 1, 9000, [(16, 16), (1, 1)]), (1, 2, 300, [(9, 9), (8, 30), (16, 200), (33, 40)]), (1, 8, 0, [(90, 150), (2, 40), (4, 4)]),
    (1, 4, 64, [(200, 300)])])
def test_attn_f32_row_blocks(ice, H, G, L, reqs):
    """Blocks of 16, 32 and 64 rows, full and not, and requests on both sides of a block's tokens."""
    _attn_check(ice, _attn_case(L + G, F32, H, G, 16, L, reqs))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,G,extra", [(1, 1, []), (2, 2, [(70, 90), (200, 200)])])
def test_attn_thousands_of_requests(ice, dtype, H, G, extra):
    """More requests than the kernels keep the lengths of in shared memory."""
    _attn_check(ice, _attn_case(21, dtype, H, G, 16, 70, [(1 if i % 5 else 0, 1 + i % 3) for i in range(2500)] + extra))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_most_requests(ice, dtype):
    _attn_check(ice, _attn_case(24, dtype, 1, 1, 16, 70, [(1 if i % 3 else 0, 1 + i % 3) for i in range(8190)] + [(150, 160), (3, 40)]))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,G", [(4096, 1), (512, 8)])
def test_attn_most_heads(ice, dtype, H, G):
    _attn_check(ice, _attn_case(25, dtype, H, G, 4, 9, [(1, 5), (0, 3), (2, 2)]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_most_tokens(ice, dtype):
    """2^20 tokens of 8192 requests and 16 heads: 2^31 elements of queries and of outputs, more of parts."""
    B, nq, H, P, L, s = 8192, 128, 16, 16, 100, 130
    g = torch.Generator().manual_seed(26)
    n, cols = 60, pages_of(s, P)
    k, v = (torch.randn((n, H, P, D), generator=g).to(dtype) for _ in range(2))
    table = torch.randint(0, n, (B, cols), generator=g).int()
    prefix = torch.randperm(n, generator=g)[:pages_of(L, P)].int()
    q_start, lens = torch.arange(B + 1, dtype=torch.int32) * nq, torch.full((B,), s, dtype=torch.int32)
    q = torch.randn((B * nq, H, D), generator=torch.Generator(device="cuda").manual_seed(27), device="cuda", dtype=dtype)
    pc = _cache(ice, n_kv_heads=H, n_q_heads=H, page_size=P, n_pages=n, max_requests=B, max_blocks=cols, max_tokens=B * nq, dtype=dtype)
    got = pc.attn(q, q_start.cuda(), lens.cuda(), table.cuda(), k.cuda(), v.cuda(), prefix.cuda(), L)
    assert pc.get_error() == 0
    for r in (0, 1, 4099, B - 1):
        rows = slice(r * nq, (r + 1) * nq)
        ref, tol = plain_attn(q[rows].cpu(), torch.tensor([0, nq]), lens[r:r + 1], table[r:r + 1], k, v, prefix, L)
        err = (got[rows].cpu().double() - ref).abs()
        assert bool((err <= tol).all()), (r, float((err / tol).max()))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0, 0.01, 30.0])
def test_attn_score_ranges(ice, dtype, scale):
    """Equal scores, near-equal ones, and ones so far apart that a key has nearly all the weight."""
    _attn_check(ice, _attn_case(3, dtype, 2, 4, 16, 700, MIXED, scale=scale))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_rising_scores(ice, dtype):
    """Keys grow along the context, so that every tile raises the maximum."""
    c = _attn_case(4, dtype, 1, 4, 16, 1500, [(1, 600), (5, 300)], stale=0.0)
    c["q"] = c["q"].abs()
    for j, p in enumerate(c["prefix"].tolist()):
        c["k"][p] = c["k"][p].abs() * (0.02 * j)
    _attn_check(ice, c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("stale", [float("inf"), float("-inf"), 3e38])
def test_attn_stale_slots(ice, dtype, stale):
    _attn_check(ice, _attn_case(5, dtype, 2, 4, 16, 133, MIXED, stale=stale))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("L,reqs", [(300, MIXED), (0, MIXED), (300, [(1, 0), (3, 0)]), (5000, [(1, 0), (3, 0)])])
def test_attn_rows_behind_the_last(ice, dtype, L, reqs):
    """Rows of a padded batch stay as they were."""
    c = _attn_case(6, dtype, 2, 4, 16, L, reqs, spare_rows=75)
    out = torch.full(c["q"].shape, 7.0, dtype=dtype, device="cuda")
    _attn_check(ice, c, out=out)
    assert bool((out[int(c["q_start"][-1]):] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_strided_q(ice, dtype):
    c = _attn_case(7, dtype, 2, 4, 16, 200, MIXED)
    wide = torch.randn((c["q"].shape[0], 8 + 4, D)).to(dtype).cuda()
    wide[:, 2:10] = c["q"].cuda()
    a = _attn_check(ice, c)
    assert torch.equal(_attn_check(ice, c, q=wide[:, 2:10]), a)


def test_attn_repeats_bit_for_bit(ice):
    c = _attn_case(8, BF16, 2, 4, 16, 900, MIXED + DECODE)
    a, pc = _attn_run(ice, c)
    for _ in range(3):
        assert torch.equal(_attn_run(ice, c, pc=pc)[0], a)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_shapes_share_a_handle(ice, dtype):
    """Calls of other sizes before and after do not show in a result: scratch and counters are left as found."""
    big = _attn_case(22, dtype, 2, 4, 16, 900, MIXED + DECODE)
    small = [_attn_case(23 + i, dtype, 2, 4, 16, L, reqs) for i, (L, reqs) in enumerate(
        [(0, [(1, 1)]), (5000, [(1, 3)]), (17, [(0, 0), (3, 2)]), (300, [(130, 200)])])]
    pc = _cache(ice, n_kv_heads=2, n_q_heads=8, page_size=16, n_pages=max(c["n_pages"] for c in [big] + small), dtype=dtype,
                max_requests=len(big["seq_len"]), max_blocks=max(c["table"].shape[1] for c in [big] + small),
                max_tokens=big["q"].shape[0])
    n_pages, cols = pc.params.n_pages, pc.params.max_blocks
    for c in [big] + small:  # one handle: pools and tables of its sizes
        for x in ("k", "v"):
            c[x] = torch.cat([c[x], torch.zeros((n_pages - c[x].shape[0], *c[x].shape[1:]), dtype=dtype)])
        c["table"] = torch.cat([c["table"], torch.full((c["table"].shape[0], cols - c["table"].shape[1]), -1, dtype=torch.int32)], 1)
    first = [_attn_check(ice, c, pc=pc) for c in [big] + small]
    for k in (2, 0, 4, 1, 3, 0):
        assert torch.equal(_attn_run(ice, ([big] + small)[k], pc=pc)[0], first[k])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_graphs_share_a_handle(ice, dtype):
    """Two captured graphs of one handle, replayed in turn on one stream, on buffers whose contents change."""
    cs = [_attn_case(31, dtype, 2, 4, 16, 200, MIXED), _attn_case(32, dtype, 2, 4, 16, 200, MIXED)]
    _, pc = _attn_run(ice, cs[0])
    x = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in cs[0].items()}
    graphs, outs = [], []
    for L in (200, 0):
        out = torch.empty_like(x["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pc.attn(x["q"], x["q_start"], x["seq_len"], x["table"], x["k"], x["v"], x["prefix"], L, out=out)
        graphs.append(g)
        outs.append(out)
    for c in (cs[1], cs[0], cs[1]):
        for k, v in x.items():
            if isinstance(v, torch.Tensor):
                v.copy_(c[k])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert pc.get_error() == 0
        for out, L in zip(outs, (200, 0)):
            ref, tol = plain_attn(c["q"], c["q_start"], c["seq_len"], c["table"], c["k"], c["v"], c["prefix"], L)
            assert bool(((out.cpu().double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_bad_pages(ice, dtype):
    """A page id outside the pool reads as zeros; other requests are untouched."""
    c = _attn_case(9, dtype, 1, 4, 16, 100, [(1, 40), (1, 50)], stale=0.0)
    good, pc = _attn_run(ice, c)
    bad = c["table"].clone()
    bad[0, 1], bad[0, 2] = -1, c["n_pages"]
    got, _ = _attn_run(ice, c, pc=pc, table=bad)
    assert pc.get_error() == ice.ICE_ERR_BOUNDS
    assert torch.equal(got[1], good[1])
    z = {**c, "k": c["k"].clone(), "v": c["v"].clone()}
    for j in (1, 2):
        z["k"][c["table"][0, j]], z["v"][c["table"][0, j]] = 0, 0
    assert torch.equal(_attn_run(ice, z, pc=pc)[0][0], got[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("which,at,value", [("q_start", 0, 1), ("q_start", 1, -1), ("q_start", 2, 9), ("q_start", 1, 3),
                                            ("seq_len", 0, -1), ("seq_len", 1, 65)])
def test_attn_bad_lengths_leave_out(ice, dtype, which, at, value):
    c = _attn_case(10, dtype, 1, 4, 16, 100, [(1, 40), (1, 50)])
    out = torch.full(c["q"].shape, 7.0, dtype=dtype, device="cuda")
    x = c[which].clone()
    x[at] = value
    _, pc = _attn_run(ice, c, out=out, **{which: x})
    assert pc.get_error() == ice.ICE_ERR_BOUNDS
    assert bool((out == 7.0).all())


def _long_prefix_call(ice, dtype, H, G, P, nq, L, table, k, v, q):
    """One request of nq new tokens that see the prefix only."""
    pc = _cache(ice, n_kv_heads=H, n_q_heads=H * G, page_size=P, n_pages=k.shape[0], max_requests=1, max_blocks=1, max_tokens=nq,
                dtype=dtype)
    out = pc.attn(q.cuda(), torch.tensor([0, nq], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                  torch.zeros((1, 1), dtype=torch.int32, device="cuda"), k.cuda(), v.cuda(), table.cuda(), L)
    assert pc.get_error() == 0
    return out.cpu()


def test_attn_equal_weights_of_millions_of_keys(ice):
    """Sums of one sign over 2^22 keys in one pass: q = 0, so that every weight is 1 and only sums round.

    Tolerance: the output's rounding, 2^-8; O's additions between two folds, 8192 x 2^-23 = 2^-10 of the mean of |v|; the
    sums of the folds and l, 1024 tiles and 32 folds a 2^-24 each, twice: 2^-12."""
    P, L, nq = 64, 1 << 22, 152 * 32  # a block of rows for every SM: none is cut into ranges
    g = torch.Generator().manual_seed(41)
    k = torch.randn((2, 1, P, D), generator=g).to(BF16)
    v = (1 + torch.rand((2, 1, P, D), generator=g)).to(BF16)
    table = torch.tensor([0, 1], dtype=torch.int32).repeat(L // P // 2)
    got = _long_prefix_call(ice, BF16, 1, 8, P, nq, L, table, k, v, torch.zeros((nq, 8, D), dtype=BF16)).double()
    mean = v.double().mean((0, 1, 2))
    err = (got / mean - 1).abs().max()
    assert float(err) <= 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12


def test_attn_items_longer_than_a_wait(ice):
    """2^25 keys in one pass: an item takes twice as long as a wait may without progress, and the last block's second
    stream has no rows and waits all that time. The tolerance as above, with 256 folds."""
    P, L, nq = 64, 1 << 25, 152 * 32 - 16
    g = torch.Generator().manual_seed(45)
    k = torch.randn((2, 1, P, D), generator=g).to(BF16)
    v = (1 + torch.rand((2, 1, P, D), generator=g)).to(BF16)
    table = torch.tensor([0, 1], dtype=torch.int32).repeat(L // P // 2)
    got = _long_prefix_call(ice, BF16, 1, 8, P, nq, L, table, k, v, torch.zeros((nq, 8, D), dtype=BF16)).double()
    mean = v.double().mean((0, 1, 2))
    assert float((got / mean - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12


def test_attn_f32_equal_weights_of_a_million_keys(ice):
    """The same for fp32: a prefix under blocks of 64 rows, and own tokens under blocks of 8.

    Tolerance: the sums of a tile's 64 products, and 16 more roundings (carried sums, joining of lanes, warps and parts,
    division, output): 80 x 2^-24 of the mean of |v|."""
    P, L, nq = 64, 1 << 20, 152 * 8
    g = torch.Generator().manual_seed(44)
    k, v = torch.randn((2, 1, P, D), generator=g), 1 + torch.rand((2, 1, P, D), generator=g)
    mean = v.double().mean((0, 1, 2))
    got = _long_prefix_call(ice, F32, 1, 8, P, nq, L, torch.tensor([0, 1], dtype=torch.int32).repeat(L // P // 2), k, v,
                            torch.zeros((nq, 8, D))).double()
    assert float((got / mean - 1).abs().max()) <= 80 * 2.0 ** -24
    # so many rows that the scratch holds three parts a row: the first request's own tokens are three long ranges
    reqs = [(1, L)] + [(8, 8)] * 1400
    table = torch.zeros((len(reqs), L // P), dtype=torch.int32)
    table[0, 1::2] = 1
    q_start = torch.tensor([0] + [x for x, _ in reqs]).cumsum(0).int()
    c = dict(q=torch.zeros((int(q_start[-1]), 8, D)), q_start=q_start, seq_len=torch.tensor([s for _, s in reqs], dtype=torch.int32),
             table=table, k=k, v=v, prefix=None, L=0, P=P, H=1, G=8, n_pages=2)
    got, pc = _attn_run(ice, c)
    assert pc.get_error() == 0
    assert float((got[0].cpu().double() / mean - 1).abs().max()) <= 80 * 2.0 ** -24


@pytest.mark.parametrize("dtype,tol", [(BF16, 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12), (F32, 80 * 2.0 ** -24)])
def test_attn_one_token_on_millions_of_keys(ice, dtype, tol):
    """The same for a decode step, whose few rows take the prefix in 64 parts of thousands of tiles. The tolerances as above."""
    P, L = 64, 1 << 24
    g = torch.Generator().manual_seed(46)
    k, v = torch.randn((2, 1, P, D), generator=g).to(dtype), (1 + torch.rand((2, 1, P, D), generator=g)).to(dtype)
    table = torch.tensor([0, 1], dtype=torch.int32).repeat(L // P // 2)
    got = _long_prefix_call(ice, dtype, 1, 8, P, 1, L, table, k, v, torch.zeros((1, 8, D), dtype=dtype)).double()
    assert float((got / v.double().mean((0, 1, 2)) - 1).abs().max()) <= tol


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rise", [0.0, 1.0])
def test_attn_long_passes(ice, dtype, rise):
    """Several thousand tiles in one pass, scores that rise along the context among them."""
    H, G, P, L, nq = 2, 4, 64, 2 * 131072 + 5000, 76 * 64
    n = pages_of(L, P)
    g = torch.Generator().manual_seed(42)
    k, v = (torch.randn((n, H, P, D), generator=g) for _ in range(2))
    q = torch.randn((nq, H * G, D), generator=g)
    if rise:
        k, q = k.abs() * (torch.arange(n) / n * rise).view(-1, 1, 1, 1), q.abs()
    k, v, q = (x.to(dtype) for x in (k, v, q))
    table = torch.randperm(n, generator=g).int() if not rise else torch.arange(n, dtype=torch.int32)
    got = _long_prefix_call(ice, dtype, H, G, P, nq, L, table, k, v, q).double()
    some = [0, 33, 64, 2000, nq - 1]
    ref, tol = plain_attn(q[some], torch.tensor([0, len(some)]), torch.zeros(1), torch.zeros((1, 1), dtype=torch.int32), k, v, table, L)
    err = (got[some] - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,G", [(1, 8), (2, 4)])
def test_attn_long_parts_are_joined(ice, dtype, H, G):
    """So many rows that the scratch holds one part of the prefix and two of own tokens, both of over a thousand tiles."""
    P, L, TS = 64, 150000, 128 // G
    reqs = [(2, 290000), (1, 50), (2, 300)] + [(TS, TS + 3)] * (89600 // (H * G) // TS)
    g = torch.Generator().manual_seed(43)
    n = pages_of(L, P)
    k, v = (torch.randn((n, H, P, D), generator=g).to(dtype) for _ in range(2))
    table = torch.randint(0, n, (len(reqs), pages_of(290000, P)), generator=g).int()  # pages may serve several requests
    prefix = torch.randperm(n, generator=g).int()
    q_start = torch.tensor([0] + [x for x, _ in reqs]).cumsum(0).int()
    lens = torch.tensor([s for _, s in reqs], dtype=torch.int32)
    q = torch.randn((int(q_start[-1]), H * G, D), generator=g).to(dtype)
    c = dict(q=q, q_start=q_start, seq_len=lens, table=table, k=k, v=v, prefix=prefix, L=L, P=P, H=H, G=G, n_pages=n)
    got, pc = _attn_run(ice, c)
    assert pc.get_error() == 0
    ref, tol = plain_attn(q[:5], q_start[:4], lens[:3], table, k, v, prefix, L)
    err = (got[:5].cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def test_attn_long_own_part_in_a_large_pool(ice):
    """Offsets past 2^31 elements: the last pages of a pool of 20 GB in all."""
    P, H = 64, 8
    n_pages = (1 << 31) // (P * H * D) + 100  # K alone has more than 2^31 elements
    pc = _cache(ice, n_kv_heads=H, n_q_heads=H * 4, page_size=P, n_pages=n_pages, max_requests=2, max_blocks=4, max_tokens=4)
    kp, vp = pc.new_pages()
    g = torch.Generator().manual_seed(1)
    ids = torch.tensor([[n_pages - 1, n_pages - 7, 0, -1], [n_pages - 2, n_pages - 60, n_pages - 3, -1]], dtype=torch.int32)
    small_k, small_v = (torch.randn((8, H, P, D), generator=g).to(BF16) for _ in range(2))
    flat = ids[:, :3].reshape(-1).long()
    pre = torch.tensor([n_pages - 50, n_pages - 51], dtype=torch.int32)
    where = torch.cat([flat, pre.long()])
    slots = (where[:, None] * P + torch.arange(P)[None]).reshape(-1).cuda()
    rows = [x.permute(0, 2, 1, 3).reshape(-1, H, D).contiguous().cuda() for x in (small_k, small_v)]
    pc.append(*rows, slots, kp, vp)
    q = torch.randn((3, H * 4, D), generator=g).to(BF16)
    q_start, lens = torch.tensor([0, 1, 3], dtype=torch.int32), torch.tensor([150, 192], dtype=torch.int32)
    got = pc.attn(q.cuda(), q_start.cuda(), lens.cuda(), ids.cuda(), kp, vp, pre.cuda(), 100)
    assert pc.get_error() == 0
    local = torch.tensor([[0, 1, 2, -1], [3, 4, 5, -1]], dtype=torch.int32)
    ref, tol = plain_attn(q, q_start, lens, local, small_k, small_v, torch.tensor([6, 7], dtype=torch.int32), 100)
    assert bool(((got.cpu().double() - ref).abs() <= tol).all())


# ---- the bounded waits ---------------------------------------------------------------------

@pytest.mark.parametrize("H,G,L,reqs", [
    (2, 4, 3000, [(1, 20)] * 100),     # two row tiles on one key tile
    (2, 4, 60000, [(1, 20)] * 3),      # two parts of the prefix side by side
    (2, 4, 0, [(1, 2500), (2, 700)]),  # two heads side by side
    (1, 4, 0, [(1, 2500), (1, 1)]),    # two halves of one head's range
    (3, 2, 0, [(1, 100)]),             # one tile
    (2, 4, 1000, [(300, 400), (1, 5)])])  # a request of its own
def test_forced_timeout_reports_and_recovers(ice, H, G, L, reqs):
    """A copy that never completes: the call ends with ICE_ERR_TIMEOUT, and the handle's next calls are exact."""
    c = _attn_case(51, BF16, H, G, 16, L, reqs)
    good, pc = _attn_run(ice, c)
    assert pc.get_error() == 0
    pc.debug_set_flags(ice.DEBUG_STALL_ATTN)
    _attn_run(ice, c, pc=pc)
    assert pc.get_error() == ice.ICE_ERR_TIMEOUT
    assert pc.get_error() == 0
    pc.debug_set_flags(0)
    for _ in range(3):
        got, _ = _attn_run(ice, c, pc=pc)
        assert pc.get_error() == 0
        assert torch.equal(got, good)
    with pytest.raises(ice.IceError):
        pc.debug_set_flags(1 << 5)


# ---- refusals ----------------------------------------------------------------------------

def test_refusals_on_a_live_handle(ice):
    raw, E = ice.raw_library(), ice.ICE_ERR_INVALID_ARG
    c = _attn_case(11, BF16, 2, 4, 16, 100, [(1, 40), (1, 50)])
    good, pc = _attn_run(ice, c)
    x = {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}
    out = torch.empty_like(x["q"])
    s = torch.cuda.current_stream().cuda_stream
    host = torch.zeros(4096, dtype=torch.int64)
    pinned = torch.zeros(4096, dtype=torch.int64).pin_memory()

    def attn(n_req=2, n_tok=2, q=x["q"].data_ptr(), stride=1024, q0=x["q_start"].data_ptr(), lens=x["seq_len"].data_ptr(),
             table=x["table"].data_ptr(), pre=x["prefix"].data_ptr(), L=100, k=x["k"].data_ptr(), v=x["v"].data_ptr(),
             o=out.data_ptr()):
        return raw.ice_paged_attn(pc._h, n_req, n_tok, q, stride, q0, lens, table, pre, L, k, v, o, s)

    assert attn() == ice.ICE_OK
    for over in (dict(n_req=0), dict(n_req=3), dict(n_tok=-1), dict(n_tok=3), dict(q=None), dict(q=x["q"].data_ptr() + 2),
                 dict(stride=1023), dict(stride=1028), dict(stride=512), dict(q0=None), dict(lens=None), dict(table=None),
                 dict(pre=None), dict(L=-1), dict(L=(1 << 30) + 1), dict(k=None), dict(v=x["v"].data_ptr() + 8), dict(o=None),
                 dict(o=out.data_ptr() + 4), dict(o=x["q"].data_ptr()), dict(o=x["q"].data_ptr() + 2048),
                 dict(lens=host.data_ptr()), dict(table=pinned.data_ptr()), dict(o=host.data_ptr())):
        assert attn(**over) == E, over
    assert attn(n_tok=0, q=None) == ice.ICE_OK  # nothing to do
    kv = torch.zeros((2, 2, D), dtype=BF16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")

    def append(n=2, k=kv.data_ptr(), ks=256, v=kv.data_ptr(), vs=256, sl=slots.data_ptr(), kp=x["k"].data_ptr(), vp=x["v"].data_ptr()):
        return raw.ice_paged_append(pc._h, n, k, ks, v, vs, sl, kp, vp, s)

    for over in (dict(n=-1), dict(k=None), dict(k=kv.data_ptr() + 2), dict(ks=255), dict(vs=128), dict(vs=260), dict(sl=None),
                 dict(sl=host.data_ptr()), dict(kp=None), dict(vp=pinned.data_ptr())):
        assert append(**over) == E, over
    ints = torch.zeros(64, dtype=torch.int64, device="cuda").data_ptr()

    def tables(n=2, args=None, n_slots=2):
        a = [ints] * 10 if args is None else args
        return raw.ice_paged_tables(pc._h, n, *a, n_slots, s)

    assert tables(n=0) == E and tables(n=3) == E and tables(n_slots=-1) == E
    for k in range(9):  # positions, the last, may be NULL
        a = [ints] * 10
        a[k] = None
        assert tables(args=a) == E, k
        a[k] = ints + 2
        assert tables(args=a) == E, k
        a[k] = host.data_ptr()
        assert tables(args=a) == E, k
    torch.cuda.synchronize()
    assert pc.get_error() == 0
    assert torch.equal(_attn_run(ice, c, pc=pc)[0], good)  # nothing was launched by the refused calls


def test_binding_refusals(ice):
    c = _attn_case(12, BF16, 2, 4, 16, 100, [(1, 40), (1, 50)])
    _, pc = _attn_run(ice, c)
    x = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    kv = torch.zeros((2, 2, D), dtype=BF16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    for over in (dict(q=x["q"].float()), dict(q=x["q"][:, :4]), dict(q=x["q"].cpu()), dict(q=x["q"].transpose(0, 1)),
                 dict(q_start=x["q_start"].long()), dict(q_start=x["q_start"][:2]), dict(table=x["table"][:, :1]),
                 dict(k=x["k"][1:]), dict(v=x["v"].float()), dict(prefix=None), dict(prefix=x["prefix"][:2]),
                 dict(seq_len=x["seq_len"].cpu())):
        y = {**x, **over}
        with pytest.raises(ValueError):
            pc.attn(y["q"], y["q_start"], y["seq_len"], y["table"], y["k"], y["v"], y["prefix"], y["L"])
    with pytest.raises(ValueError):
        pc.attn(x["q"], x["q_start"], x["seq_len"], x["table"], x["k"], x["v"], x["prefix"], x["L"], out=x["q"][:1].clone())
    for args in ((kv.float(), kv, slots), (kv[:, :1], kv, slots), (kv, kv[:1], slots), (kv, kv, slots.int()), (kv, kv, slots.cpu())):
        with pytest.raises(ValueError):
            pc.append(*args, x["k"], x["v"])
    lens, table, ring, state = pc.new_tables(2)
    for a in ((lens.long(), lens, table, ring, state), (lens, lens[:1], table, ring, state), (lens, lens, table[:1], ring, state),
              (lens, lens, table, ring[1:], state), (lens, lens, table, ring, state.int())):
        with pytest.raises(ValueError):
            pc.tables(*a, 4)


def test_failed_launches_leave_no_error_behind(ice):
    """Launches into a capture that has become invalid (by a wait for its stream) fail; the status says so, and the
    runtime's last error, which the caller's next check would take for its own, is clear."""
    c = _attn_case(12, BF16, 2, 4, 16, 100, [(1, 40), (1, 50)])
    good, pc = _attn_run(ice, c)
    x = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    kv, slots = torch.zeros((2, 2, D), dtype=BF16, device="cuda"), torch.full((2,), -1, dtype=torch.int64, device="cuda")
    lens, table, ring, state = pc.new_tables(2)
    outs = pc.tables(lens, lens, table, ring, state, 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    rt, s = ctypes.CDLL("libcudart.so.13"), ctypes.c_void_p(side.cuda_stream)
    codes, left = [], []
    assert rt.cudaStreamBeginCapture(s, 0) == 0
    try:
        assert rt.cudaStreamSynchronize(s) != 0
        rt.cudaGetLastError()
        for call in (lambda: pc.attn(x["q"], x["q_start"], x["seq_len"], x["table"], x["k"], x["v"], x["prefix"], x["L"],
                                     out=good, stream=side),
                     lambda: pc.append(kv, kv, slots, x["k"], x["v"], stream=side),
                     lambda: pc.tables(lens, lens, table, ring, state, 2, *outs, stream=side)):
            try:
                call()
                codes.append(0)
            except ice.IceError as e:
                codes.append(e.code)
            left.append(rt.cudaGetLastError())
    finally:
        graph = ctypes.c_void_p()
        assert rt.cudaStreamEndCapture(s, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
    assert codes == [ice.ICE_ERR_CUDA] * 3 and left == [0, 0, 0]
    assert torch.equal(_attn_run(ice, c, pc=pc)[0], good) and pc.get_error() == 0


@pytest.mark.parametrize("wrong", [None, 3, [1, 2], "number"])
def test_binding_refuses_what_is_no_tensor(ice, wrong):
    """Every tensor argument in turn: ValueError, as for a tensor of the wrong kind ("number": a tensor of no dimension)."""
    wrong = torch.tensor(1, dtype=torch.int32, device="cuda") if wrong == "number" else wrong
    c = _attn_case(12, BF16, 2, 4, 16, 100, [(1, 40), (1, 50)])
    good, pc = _attn_run(ice, c)
    x = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    kv, slots = torch.zeros((2, 2, D), dtype=BF16, device="cuda"), torch.full((2,), -1, dtype=torch.int64, device="cuda")
    lens, table, ring, state = pc.new_tables(2)
    calls = [(pc.attn, [x["q"], x["q_start"], x["seq_len"], x["table"], x["k"], x["v"], x["prefix"], x["L"], good.clone()], (7, )),
             (pc.append, [kv, kv, slots, x["k"], x["v"]], ()),
             (pc.tables, [lens, lens, table, ring, state, 2] + [t.clone() for t in (lens, state)]
              + [torch.zeros(n, dtype=t, device="cuda") for n, t in ((3, torch.int32), (2, torch.int64), (2, torch.int32))], (5, ))]
    for call, args, numbers in calls:
        call(*args)
        for i in range(len(args)):
            # outputs may be None: they are then made by the call
            if i in numbers or (wrong is None and i > {pc.attn: 7, pc.append: 9, pc.tables: 5}[call]):
                continue
            with pytest.raises(ValueError):
                call(*args[:i], wrong, *args[i + 1:])
    torch.cuda.synchronize()
    assert pc.get_error() == 0


# ---- streams, graphs, and the three calls together ------------------------------------------

def test_outputs_belong_to_the_given_stream(ice):
    """Memory that was freed while the current stream still writes to it is not what a call on another
    stream gets for its outputs."""
    c = _attn_case(13, BF16, 2, 4, 16, 100, [(1, 40), (1, 50)])
    good, pc = _attn_run(ice, c)
    x = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    lens, table, ring, state = pc.new_tables(2)
    new = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    plain = [t.tolist() for t in pc.tables(lens, new, table.clone(), ring.clone(), state, 8)]
    table2, ring2 = table.clone(), ring.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.empty_like(good)] + [torch.empty(n, dtype=d, device="cuda") for n, d in
                                       ((2, torch.int32), (2, torch.int64), (3, torch.int32), (8, torch.int64), (8, torch.int32))]
    torch.cuda._sleep(100_000_000)  # about 50 ms
    for t in late:
        t.fill_(77)
    del late, t
    out = pc.attn(x["q"], x["q_start"], x["seq_len"], x["table"], x["k"], x["v"], x["prefix"], x["L"], stream=side)
    got = pc.tables(lens, new, table2, ring2, state, 8, stream=side)
    torch.cuda.synchronize()
    assert pc.get_error() == 0
    assert torch.equal(out, good)
    assert [t.tolist() for t in got] == plain


def _steps(seed, n_steps, B):
    """Changes of the lengths over a serving loop: prompts, decode steps, rejected drafts, an end and a new
    request in its place."""
    rng = random.Random(seed)
    lens = [0] * B
    steps = []
    for t in range(n_steps):
        new = []
        for b in range(B):
            if lens[b] == 0:
                x = rng.randint(1, 40)
            elif t % 7 == 3 and b % 3 == 0:
                x = -lens[b]
            elif t % 5 == 2 and b % 2:
                x = -min(lens[b], rng.randint(1, 20))
            else:
                x = rng.choice([1, 1, 1, 0, 3])
            new.append(x)
            lens[b] += x
        steps.append(new)
    return steps


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(ice, dtype, graph):
    """Tables, append and attention of two layers over a loop, with fixed buffers (eagerly on a stream of its own,
    or captured once and replayed), against a plain cache that keeps every request's rows."""
    B, H, G, P, L, layers, cap = 5, 2, 4, 16, 75, 2, 256
    pc = _cache(ice, n_kv_heads=H, n_q_heads=H * G, page_size=P, n_pages=40, max_requests=B + 1, max_blocks=8, max_tokens=cap,
                dtype=dtype)
    g = torch.Generator().manual_seed(2)
    side = torch.cuda.Stream()
    pools = [pc.new_pages() for _ in range(layers)]
    for k, v in pools:  # what nobody wrote must not matter
        k.fill_(float("nan"))
        v.fill_(float("nan"))
    # the prefix is a request of its own, in its own row of a table
    lens, table, ring, state = pc.new_tables(B)
    one, pre_row = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1, 8), -1, dtype=torch.int32, device="cuda")
    _, state, _, slots, _ = pc.tables(one, one + L, pre_row, ring, state, L)
    pre_kv = [[torch.randn((L, H, D), generator=g).to(dtype) for _ in range(2)] for _ in range(layers)]
    for (kp, vp), (k, v) in zip(pools, pre_kv):
        pc.append(k.cuda(), v.cuda(), slots, kp, vp)
    prefix = pre_row[0, :pages_of(L, P)].contiguous()
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.zeros((layers, cap, H * G, D), dtype=dtype, device="cuda")
    kn, vn = (torch.zeros((layers, cap, H, D), dtype=dtype, device="cuda") for _ in range(2))
    q_start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slot_map = torch.zeros(cap, dtype=torch.int64, device="cuda")
    pos = torch.zeros(cap, dtype=torch.int32, device="cuda")
    out = torch.zeros((layers, cap, H * G, D), dtype=dtype, device="cuda")

    def step():
        pc.tables(lens, new, table, ring, state, cap, lens, state, q_start, slot_map, pos)
        for y in range(layers):
            pc.append(kn[y], vn[y], slot_map, *pools[y])
            pc.attn(q[y], q_start, lens, table, *pools[y], prefix, L, out=out[y])

    torch.cuda.synchronize()
    replay = None
    if graph:
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay):
            step()
    plain = [[[torch.zeros((0, H, D), dtype=dtype)] * 2 for _ in range(B)] for _ in range(layers)]
    for t, change in enumerate(_steps(3, 24, B)):
        n = sum(max(0, x) for x in change)
        new.copy_(torch.tensor(change, dtype=torch.int32))
        for x in (q, kn, vn):
            x.copy_(torch.randn(x.shape, generator=g).to(dtype))
        out.fill_(5.0)
        torch.cuda.synchronize()
        if graph:
            replay.replay()
        else:
            with torch.cuda.stream(side):
                step()
        torch.cuda.synchronize()
        assert pc.get_error() == 0, t
        for y in range(layers):
            at = 0
            for b, x in enumerate(change):
                for j, src in enumerate((kn, vn)):
                    old = plain[y][b][j]
                    plain[y][b] = list(plain[y][b])
                    plain[y][b][j] = torch.cat([old, src[y, at:at + x].cpu()]) if x > 0 else old[:old.shape[0] + x]
                at += max(0, x)
            # the plain cache as one page a request
            rows = [(pre_kv[y][0], pre_kv[y][1])] + [tuple(r) for r in plain[y]]
            S = max(r[0].shape[0] for r in rows)
            kf, vf = (torch.zeros((B + 1, H, S, D), dtype=dtype) for _ in range(2))
            for i, (k, v) in enumerate(rows):
                kf[i, :, :k.shape[0]], vf[i, :, :v.shape[0]] = k.transpose(0, 1), v.transpose(0, 1)
            assert lens.tolist() == [r[0].shape[0] for r in rows[1:]], t
            ref, tol = plain_attn(q[y, :n].cpu(), q_start.cpu(), lens.cpu(), torch.arange(1, B + 1, dtype=torch.int32)[:, None],
                                  kf, vf, torch.tensor([0], dtype=torch.int32), L)
            err = (out[y, :n].cpu().double() - ref).abs()
            assert bool((err <= tol).all()), (t, y, float((err / tol).max()))
            assert bool((out[y, n:] == 5.0).all())
    held = int((state[1] - state[0]).item()) + sum(pages_of(x, P) for x in lens.tolist()) + pages_of(L, P)
    assert held == 40  # no page was lost
