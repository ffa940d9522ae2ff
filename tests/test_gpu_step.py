"""What surrounds the paged cache's attention in a serving step, on the GPU against its definition in 64 bits: rotating append,
requests that share pages, copies of pages, compaction, verification of drafted tokens; refusals, streams, graphs, and a run
of all of them as a loop of speculative decoding uses them."""
import ctypes
import math
import random
from fractions import Fraction

import pytest
import torch

from tests.step_helpers import D, pages_of, plain_compact, plain_fork, plain_rope, plain_tables_shared, plain_verify

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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- rotating append ------------------------------------------------------------------------

FREQ = [10000.0 ** (-i / 64) for i in range(64)]


def _rope_case(seed, dtype, n, H, G, P, pairs, axes, strided=False, most=100000):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn((n, (G + 2) * H * D + (64 if strided else 0)), generator=g).to(dtype)
    if strided:  # slices of one fused projection
        q, k, v = (rows[:, a:b].unflatten(1, (-1, D)) for a, b in ((0, G * H * D), (G * H * D, (G + 1) * H * D),
                                                                   ((G + 1) * H * D, (G + 2) * H * D)))
    else:
        q, k, v = (x.contiguous().unflatten(1, (-1, D)) for x in rows.split([G * H * D, H * D, H * D], 1))
    n_pages = pages_of(n, P) + 3
    slots = torch.randperm(n_pages * P, generator=g)[:n]
    pos = torch.randint(0, most, (axes, n), generator=g, dtype=torch.int32)
    axis = [min(axes - 1, i * axes // pairs) for i in range(pairs)]
    return dict(q=q, k=k, v=v, slots=slots, pos=pos, freq=[10000.0 ** (-i / pairs) for i in range(pairs)], axis=axis, n_pages=n_pages,
                H=H, G=G, P=P, dtype=dtype)


def _gpu(x):
    """On the GPU with the strides that it has."""
    if x.is_contiguous():
        return x.cuda()
    base = torch.zeros(x.untyped_storage().size() // x.element_size(), dtype=x.dtype)
    base = torch.as_strided(x, (base.numel(),), (1,), 0).cuda()
    return torch.as_strided(base, x.shape, x.stride(), x.storage_offset())


def _rope_run(ice, c, interleaved=False, offset=0, in_place=False, with_q=True):
    pc = _cache(ice, n_kv_heads=c["H"], n_q_heads=c["H"] * c["G"], page_size=c["P"], n_pages=c["n_pages"], dtype=c["dtype"])
    kp, vp = pc.new_pages()
    kp.fill_(7.0)
    vp.fill_(7.0)
    q = _gpu(c["q"])
    out = q if in_place else torch.full(q.shape, 7.0, dtype=c["dtype"], device="cuda")
    rope = ice.Rope(c["freq"], c["axis"], interleaved)
    got = pc.rope_append(q if with_q else None, _gpu(c["k"]), _gpu(c["v"]), _gpu(c["pos"]), rope, c["slots"].cuda(), kp, vp, offset,
                         out if with_q else None)
    assert (got is out) if with_q else got is None
    return pc, out.cpu(), kp.cpu(), vp.cpu()


def _rope_check(c, interleaved, offset, out, kp, vp):
    H, P = c["H"], c["P"]
    live = c["slots"] >= 0
    want = {}
    for name, x in (("q", c["q"]), ("k", c["k"])):
        want[name] = plain_rope(x, c["pos"], offset, c["freq"], c["axis"], interleaved)
    if out is not None:
        y, tol = want["q"]
        bad = ((out.double() - y).abs() > tol)[live]
        assert not bool(bad.any())
        assert bool((out[~live] == 7.0).all())
    rest = torch.ones(kp.shape[0] * P, dtype=torch.bool)
    rest[c["slots"][live]] = False
    flat = [x.transpose(1, 2).reshape(-1, H, D) for x in (kp, vp)]
    y, tol = want["k"]
    assert bool(((flat[0][c["slots"][live]].double() - y[live]).abs() <= tol[live]).all())
    assert torch.equal(flat[1][c["slots"][live]], c["v"][live])
    for x in flat:
        assert bool((x[rest] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,H,G,P,pairs,axes", [
    (1, 1, 1, 1, 64, 1), (1, 8, 4, 16, 64, 3), (3, 2, 4, 5, 8, 2), (64, 8, 4, 16, 64, 3), (301, 3, 8, 12, 48, 4), (2431, 1, 1, 64, 32, 3),
    (2500, 4, 2, 16, 56, 2)])
def test_rope(ice, dtype, interleaved, n, H, G, P, pairs, axes):
    c = _rope_case(n, dtype, n, H, G, P, pairs, axes)
    pc, *got = _rope_run(ice, c, interleaved, 1234)
    assert pc.get_error() == 0
    _rope_check(c, interleaved, 1234, *got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_most_heads(ice, dtype, in_place):
    c = _rope_case(4, dtype, 2, 512, 8, 1, 64, 2)
    pc, *got = _rope_run(ice, c, in_place=in_place)
    assert pc.get_error() == 0
    _rope_check(c, False, 0, *got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_strided(ice, dtype, in_place):
    c = _rope_case(3, dtype, 130, 2, 4, 16, 64, 3, strided=True)
    c["pos"] = torch.cat([c["pos"], c["pos"]], 1)[:, :130]  # rows further apart than the tokens
    c["pos"] = torch.as_strided(torch.cat([c["pos"], torch.zeros((3, 7), dtype=torch.int32)], 1).contiguous(), (3, 130), (137, 1))
    pc, *got = _rope_run(ice, c, in_place=in_place)
    assert pc.get_error() == 0
    _rope_check(c, False, 0, *got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("n", [1, 2, 65])
def test_rope_columns_of_one_buffer(ice, dtype, first, n):
    """Queries and rotated queries as columns of one buffer, in either order: rows of one stride that share no memory."""
    c = _rope_case(12, dtype, n, 2, 4, 16, 64, 1)
    width, gap = 8 * D, 16
    buf = torch.full((n, 2 * width + gap), 7.0, dtype=dtype, device="cuda")
    a, b = (x.unflatten(1, (8, D)) for x in (buf[:, :width], buf[:, width:2 * width]))
    q, out = (b, a) if first else (a, b)
    q.copy_(c["q"])
    pc = _cache(ice, n_pages=c["n_pages"], dtype=dtype)
    kp, vp = pc.new_pages()
    kp.fill_(7.0)
    vp.fill_(7.0)
    rest = (c["k"].cuda(), c["v"].cuda(), c["pos"].cuda(), ice.Rope(c["freq"]), c["slots"].cuda(), kp, vp)
    assert pc.rope_append(q, *rest, q_out=out) is out
    assert pc.get_error() == 0
    _rope_check(c, False, 0, out.cpu(), kp.cpu(), vp.cpu())
    assert torch.equal(q.cpu(), c["q"]) and bool((buf[:, 2 * width:] == 7.0).all())
    # a part of a row, or of the row before or behind, in common: refused
    step = 2 * width + gap
    base = torch.zeros((2 * n + 2) * step, dtype=dtype, device="cuda")
    at = lambda x: torch.as_strided(base, (n, 8, D), (step, D, 1), x)  # noqa: E731
    for x, y, fine in ((width - 8, 0, False), (0, width - 8, False), (width + gap + 8, 0, n == 1), (0, width + gap + 8, n == 1),
                       (step, 0, n == 1), (0, (n - 1) * step + width - 8, False), (0, (n - 1) * step + width, True),
                       ((n - 1) * step + width, 0, True), (width, 0, True), (width + gap, 0, True), (0, width + gap, True)):
        if fine:
            pc.rope_append(at(x), *rest, q_out=at(y))
            continue
        with pytest.raises(ice.IceError) as e:
            pc.rope_append(at(x), *rest, q_out=at(y))
        assert e.value.code == ice.ICE_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert pc.get_error() == 0


@pytest.mark.parametrize("pos,offset", [(0, 0), (2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, 0), (-2 ** 31, -2 ** 31), (-3, 3),
                                        (2 ** 24 + 1, 0)])
def test_rope_far_positions(ice, pos, offset):
    c = _rope_case(5, F32, 33, 2, 2, 16, 64, 1)
    c["pos"].fill_(pos)
    c["freq"] = [1.0, 0.5, -0.25, 3.0, 6.5, 0.0, 1e-9, math.pi] + c["freq"][8:]
    pc, *got = _rope_run(ice, c, offset=offset)
    assert pc.get_error() == 0
    _rope_check(c, False, offset, *got)
    if pos + offset == 0:  # no turn: as it was
        assert torch.equal(got[0], c["q"])


TURN = Fraction("6.2831853071795864769252867665590057683943387987502116419498891846156")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pos,offset", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, -2 ** 31), (1234567891, 7), (120001, 40000)])
def test_rope_far_angles_to_the_last_bits(ice, dtype, pos, offset):
    """Angles in exact fractions: no part of the tolerance grows with the position."""
    c = _rope_case(9, dtype, 3, 2, 2, 16, 64, 1)
    c["pos"].fill_(pos)
    c["freq"] = [1.0, 0.5, -0.25, 3.0, 6.5, 0.0, 1e-9, math.pi, 1e-3, -1e-5, 0.1, 1e6, -1e15, 1e300, 2.0 ** -60, 5e-324] + c["freq"][16:]
    pc, *got = _rope_run(ice, c, offset=offset)
    assert pc.get_error() == 0
    # more than two turns a position have no use: those pairs only have to stay turns
    known = torch.tensor([abs(f) < 10 for f in c["freq"]])
    near = torch.tensor([float(Fraction(f) * (pos + offset) % TURN) for f in c["freq"]], dtype=torch.float64)
    keys = got[1].transpose(1, 2).reshape(-1, 2, D)[c["slots"]]
    for have, x in ((got[0], c["q"]), (keys, c["k"])):
        a, b = x.double()[..., :64], x.double()[..., 64:]
        want = torch.cat([a * near.cos() - b * near.sin(), b * near.cos() + a * near.sin()], 2)
        u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
        # the fraction of a turn in 32 bits and in fp32, the functions, two products and their sum, the output; the
        # frequency in 2^-64 turns, 2^-63 of a turn over 2^32 positions at most: 2 pi 2^-31
        err = 2 * math.pi * (2.0 ** -33 + 2.0 ** -31) + math.pi * 2.0 ** -25 + 2.0 ** -22 + 2 * 2.0 ** -24
        tol = err * (a.abs() + b.abs()).repeat(1, 1, 2) + u * want.abs()
        assert bool((((have.double() - want).abs() <= tol) | ~known.repeat(2)).all())
        size, size0 = torch.hypot(have.double()[..., :64], have.double()[..., 64:]), torch.hypot(a, b)
        assert bool(((size - size0).abs() <= 4 * (err + u) * size0).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pos,offset", [(1, 0), (1000003, 0), (-77, 50), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_rope_near_the_axes(ice, pos, offset, interleaved):
    """Angles near quarters of a turn, where the sine or the cosine is small, in exact fractions. Rows (0, 1) come out as (-sin, cos)
    with no rounding of their own.

    The angle: its fraction of a turn in 32 bits, 2 pi 2^-33, and the frequency's 2^-65 turns a position; what is left of it in fp32 is exact below
    2^24 / 2^32 of a turn from an axis. The functions: two steps of the result, 2^-22 of it."""
    c = _rope_case(13, F32, 5, 2, 2, 16, 64, 1)
    c["pos"].fill_(pos)
    p, rng = pos + offset, random.Random(pos)
    c["freq"] = [(math.pi / 2 * rng.randint(-9, 9) + rng.choice([1, -1]) * 10.0 ** -rng.uniform(1.7, 9)) / p for _ in range(64)]
    first, second = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, 64), slice(64, D))
    for name in ("q", "k"):
        c[name][..., first], c[name][..., second] = 0.0, 1.0
    pc, out, kp, _ = _rope_run(ice, c, interleaved, offset)
    assert pc.get_error() == 0
    near = torch.tensor([float((Fraction(f) * p + TURN / 2) % TURN - TURN / 2) for f in c["freq"]], dtype=torch.float64)
    axis = torch.tensor([float((Fraction(f) * p + TURN / 8) % (TURN / 4) - TURN / 8) for f in c["freq"]], dtype=torch.float64)
    assert bool((axis.abs() < 2 * math.pi * 2.0 ** -8).all())
    angle = 2 * math.pi * (2.0 ** -33 + abs(p) * 2.0 ** -65)
    for have in (out, kp.transpose(1, 2).reshape(-1, 2, D)[c["slots"]]):
        for got, want in ((have[..., first], -near.sin()), (have[..., second], near.cos())):
            assert bool(((got.double() - want).abs() <= 1.01 * angle + 2.0 ** -22 * want.abs()).all())


def test_rope_keys_alone(ice):
    c = _rope_case(6, BF16, 77, 4, 2, 16, 64, 2)
    pc, _, kp, vp = _rope_run(ice, c, with_q=False)
    assert pc.get_error() == 0
    _rope_check(c, False, 0, None, kp, vp)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_leaves_the_rest(ice, dtype, interleaved):
    """Elements behind the pairs, values, and rows of padded tokens keep their bits, whatever they hold."""
    c = _rope_case(7, dtype, 40, 2, 4, 16, 24, 2)
    special = torch.tensor([math.nan, math.inf, -math.inf, -0.0]).to(dtype)
    for x in ("q", "k"):
        c[x][:, :, 48:52] = special
    c["v"][:, :, :4] = special
    c["slots"][::7] = -1
    c["pos"][:, 3] = 5
    pc, out, kp, vp = _rope_run(ice, c, interleaved)
    assert pc.get_error() == 0
    live = c["slots"] >= 0
    bits = torch.int16 if dtype == BF16 else torch.int32
    flat = [x.transpose(1, 2).reshape(-1, 2, D) for x in (kp, vp)]
    assert torch.equal(out[live][..., 48:].contiguous().view(bits), c["q"][live][..., 48:].contiguous().view(bits))
    assert torch.equal(flat[0][c["slots"][live]][..., 48:].contiguous().view(bits), c["k"][live][..., 48:].contiguous().view(bits))
    assert torch.equal(flat[1][c["slots"][live]].view(bits), c["v"][live].contiguous().view(bits))
    assert bool((out[~live] == 7.0).all())


def test_rope_bad_slots(ice):
    c = _rope_case(8, BF16, 20, 2, 4, 16, 64, 1)
    c["slots"][4], c["slots"][9] = c["n_pages"] * 16, -2
    pc, *got = _rope_run(ice, c)
    assert pc.get_error() == ice.ICE_ERR_BOUNDS and pc.get_error() == 0
    c["slots"][4] = c["slots"][9] = -1  # skipped as those are
    _rope_check(c, False, 0, *got)


def test_rope_in_a_large_pool(ice):
    """Rows whose offsets in the pages pass 2^32 elements, and rows of q, k and v that far apart."""
    n_pages, stride = 131500, 1 << 30
    pc = _cache(ice, n_kv_heads=4, n_q_heads=4, page_size=64, n_pages=n_pages)
    kp, vp = pc.new_pages()
    c = _rope_case(1, BF16, 6, 4, 1, 64, 64, 1)
    c["slots"] = torch.tensor([n_pages * 64 - 1, 0, 131072 * 64 + 5, -1, 7, 9])
    rows = torch.empty(5 * stride + 3 * 512, dtype=BF16, device="cuda")
    q, k, v = (torch.as_strided(rows, (6, 4, D), (stride, D, 1), i * 512) for i in range(3))
    for name, x in (("q", q), ("k", k), ("v", v)):
        x.copy_(c[name])
    assert pc.rope_append(q, k, v, c["pos"].cuda(), ice.Rope(c["freq"]), c["slots"].cuda(), kp, vp, q_out=q) is q
    assert pc.get_error() == 0
    for i, slot in enumerate(c["slots"].tolist()):
        for x, name, pool in ((q, "q", None), (k, "k", kp), (v, "v", vp)):
            got = x[i] if pool is None else pool[slot // 64, :, slot % 64]
            if slot < 0:
                assert torch.equal(x[i].cpu(), c[name][i])  # as it was
                continue
            want, tol = plain_rope(c[name][i:i + 1], c["pos"][:, i:i + 1], 0, c["freq"], c["axis"], False)
            assert torch.equal(got.cpu(), c[name][i]) if name == "v" else bool(((got.cpu().double() - want[0]).abs() <= tol[0]).all())


def test_rope_without_turns_is_append(ice):
    c = _rope_case(9, BF16, 100, 8, 4, 16, 64, 1)
    c["freq"] = [0.0] * 64
    _, _, kp, vp = _rope_run(ice, c)
    pc = _cache(ice, n_kv_heads=8, n_q_heads=32, n_pages=c["n_pages"])
    k2, v2 = (torch.full(kp.shape, 7.0, dtype=BF16, device="cuda") for _ in range(2))
    pc.append(c["k"].cuda(), c["v"].cuda(), c["slots"].cuda(), k2, v2)
    assert torch.equal(kp, k2.cpu()) and torch.equal(vp, v2.cpu())


# ---- shared pages ---------------------------------------------------------------------------

class Pool:
    """Requests that share pages, as lists, moved on by the definitions."""

    def __init__(self, seed, n, P, cols, n_pages):
        self.rng = random.Random(seed)
        self.P, self.cols, self.n_pages = P, cols, n_pages
        self.lens, self.table, self.refs = [0] * n, [[-1] * cols for _ in range(n)], [0] * n_pages
        ids = list(range(n_pages))
        self.rng.shuffle(ids)
        head = self.rng.randint(0, 3 * n_pages)
        self.ring = [0] * n_pages
        for i, p in enumerate(ids):
            self.ring[(head + i) % n_pages] = p
        self.state = [head, head + n_pages]

    def change(self, kinds=("one", "none", "end", "drop", "chunk", "some")):
        rng, free = self.rng, self.state[1] - self.state[0]
        new = []
        for a in self.lens:
            k = rng.choice(kinds) if a else rng.choice(["none", "start"])
            x = {"one": 1, "none": 0, "end": -a, "drop": -min(a, rng.randint(1, 2 * self.P)), "start": rng.randint(1, self.cols * self.P // 2),
                 "chunk": rng.randint(0, self.cols * self.P - a), "some": rng.randint(1, 5)}[k]
            if a + x > self.cols * self.P:
                x = 0
            need = max(0, pages_of(a + x, self.P) - pages_of(a, self.P)) + 1 if x > 0 else 0
            if need > free:
                x = 0
            else:
                free -= need
            new.append(x)
        return new

    def forks(self):
        full = [r for r, a in enumerate(self.lens) if a]
        empty = [r for r, a in enumerate(self.lens) if not a]
        self.rng.shuffle(empty)
        if not full or not empty:
            return [], [], []
        dst = empty[:self.rng.randint(1, len(empty))]
        src = [self.rng.choice(full) for _ in dst]
        return src, dst, [self.rng.choice([self.lens[s], self.rng.randint(0, self.lens[s])]) for s in src]

    def check(self):
        """Counts are those of the tables; every page is free or held, never both, none lost."""
        held = [0] * self.n_pages
        for r, a in enumerate(self.lens):
            for p in self.table[r][:pages_of(a, self.P)]:
                held[p] += 1
        assert held == self.refs
        free = [self.ring[i % self.n_pages] for i in range(*self.state)]
        assert len(set(free)) == len(free) and not any(held[p] for p in free)
        assert len(free) + sum(x > 0 for x in held) == self.n_pages


class Shared:
    """The same on the GPU."""

    def __init__(self, pool, **over):
        self.pc = over["pc"]
        self.lens, self.table, self.ring, self.refs = _i32(pool.lens), _i32(pool.table), _i32(pool.ring), _i32(pool.refs)
        self.state = torch.tensor(pool.state, dtype=torch.int64, device="cuda")

    def lists(self):
        return (self.lens.tolist(), self.table.tolist(), self.ring.tolist(), self.state.tolist(), self.refs.tolist())


def _pool_lists(p):
    return p.lens, p.table, p.ring, p.state, p.refs


@pytest.mark.parametrize("n,P,cols,n_pages,rounds", [
    (3, 4, 6, 20, 30), (9, 1, 12, 60, 25), (40, 16, 10, 160, 20), (128, 5, 12, 700, 10), (129, 16, 10, 500, 10), (300, 3, 40, 5000, 6),
    (20, 2, 4000, 30000, 5), (140, 2, 4000, 60000, 4), (1100, 4, 20, 9000, 4), (10, 2, 4000, 20000, 5), (70, 4, 300, 5000, 6)])
@pytest.mark.parametrize("in_place", [False, True])
def test_shared_tables_and_forks(ice, n, P, cols, n_pages, rounds, in_place):
    """A loop of forks and steps, moved on by the kernels and by the definition."""
    pool = Pool(n + P, n, P, cols, n_pages)
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=n_pages, max_requests=n, max_blocks=cols, max_tokens=1)
    gpu = Shared(pool, pc=pc)
    copied = kept = 0
    for t in range(rounds):
        src, dst, lens = pool.forks() if t % 2 else ([], [], [])
        whole = self_len = [pool.lens[s] for s in src]
        use = None if t % 4 == 1 else lens
        ref = plain_fork(src, dst, use, *_pool_lists(pool)[:2], pool.refs, P)
        assert ref[0] == 0 and whole == self_len
        got = pc.fork(_i32(src), _i32(dst), gpu.lens, gpu.table, gpu.refs, None if use is None else _i32(use),
                      gpu.lens if in_place else None)
        if not in_place:
            assert gpu.lens.tolist() == pool.lens
        gpu.lens = got
        pool.lens, pool.table, pool.refs = ref[1:]
        assert gpu.lists() == _pool_lists(pool), t
        pool.check()
        new = pool.change()
        total = sum(max(0, x) for x in new)
        n_slots = total + (t % 3) * 37
        ref = plain_tables_shared(pool.lens, new, pool.table, pool.ring, pool.state, pool.refs, n_slots, P)
        assert ref[0] == 0
        before = _pool_lists(pool)
        outs = pc.tables_shared(gpu.lens, _i32(new), gpu.table, gpu.ring, gpu.state, gpu.refs, n_slots,
                                gpu.lens if in_place else None, gpu.state if in_place else None)
        assert pc.get_error() == 0
        if not in_place:
            assert gpu.lens.tolist() == before[0] and gpu.state.tolist() == before[3]
        gpu.lens, gpu.state = outs[:2]
        _, pool.lens, pool.state, q_start, slots, pos, csrc, cdst, pool.table, pool.ring, pool.refs = ref
        assert [x.tolist() for x in outs[2:]] == [q_start, slots, pos, csrc, cdst], t
        assert gpu.lists() == _pool_lists(pool), t
        pool.check()
        copied += sum(x >= 0 for x in csrc)
        kept += sum(x > 0 for x in new) - sum(x >= 0 for x in csrc)
        if t % 5 == 4:
            _compact_step(ice, pool, gpu, in_place)
    assert kept and (copied or P == 1)


def _compact_step(ice, pool, gpu, in_place):
    pc, L = gpu.pc, sum(x > 0 for x in pool.refs)
    moves = sum(x > 0 for x in pool.refs[L:])
    for room in ([None] if in_place else [moves, None]):
        m = pool.n_pages // 2 if room is None else room
        ref = plain_compact(pool.lens, pool.table, [], pool.refs, pool.ring, pool.state, m, pool.P)
        assert ref[0] == 0
        ring, state = (gpu.ring, gpu.state) if in_place else (gpu.ring.clone(), gpu.state.clone())
        table, refs = (None, None) if in_place else (gpu.table.clone(), torch.full_like(gpu.refs, 77))
        got = pc.compact(gpu.lens, gpu.table, gpu.refs, ring, state, n_moves=room, block_table_out=table, page_refs_out=refs)
        assert pc.get_error() == 0
        assert [x.tolist() for x in got[:4]] == [ref[1], ref[2], ref[3], ref[5]]
        assert ring.tolist() == ref[6] and state.tolist() == ref[7]
    _, _, _, gpu.table, gpu.refs = *(None,) * 3, got[2], got[3]
    gpu.ring, gpu.state = ring, state
    _, _, _, pool.table, _, pool.refs, pool.ring, pool.state = ref
    pool.check()


def test_shared_tables_most_requests(ice):
    n, P, cols = 8192, 16, 4
    pool = Pool(5, n, P, cols, 30000)
    pool.lens = [pool.rng.choice([0, 5, 16, 17, 33]) for _ in range(n)]
    ids, at = list(range(30000)), 0
    for r, a in enumerate(pool.lens):
        k = pages_of(a, P)
        pool.table[r][:k] = ids[at:at + k]
        at += k
    pool.refs = [int(p < at) for p in ids]
    pool.ring, pool.state = ids[at:] + [-1] * at, [0, 30000 - at]
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=30000, max_requests=n, max_blocks=cols, max_tokens=1)
    gpu = Shared(pool, pc=pc)
    src, dst, lens = pool.forks()
    ref = plain_fork(src, dst, lens, pool.lens, pool.table, pool.refs, P)
    gpu.lens = pc.fork(_i32(src), _i32(dst), gpu.lens, gpu.table, gpu.refs, _i32(lens))
    pool.lens, pool.table, pool.refs = ref[1:]
    assert ref[0] == 0 and gpu.lists() == _pool_lists(pool)
    new = pool.change(("one", "end", "drop"))
    ref = plain_tables_shared(pool.lens, new, pool.table, pool.ring, pool.state, pool.refs, 8192 * 40, P)
    assert ref[0] == 0
    outs = pc.tables_shared(gpu.lens, _i32(new), gpu.table, gpu.ring, gpu.state, gpu.refs, 8192 * 40)
    assert pc.get_error() == 0
    assert [x.tolist() for x in outs] == [ref[1], ref[2], *ref[3:8]]
    assert [gpu.table.tolist(), gpu.ring.tolist(), gpu.refs.tolist()] == list(ref[8:])


def _three_holders(P=4):
    """Requests 0, 1, 2 hold page 5 (full) and page 2 (incomplete); 3 holds page 0; 4 nothing."""
    table = [[5, 2, -1], [5, 2, -1], [5, 2, -1], [0, -1, -1], [-1, -1, -1]]
    return [6, 6, 5, 2, 0], table, [1, 3, 4, 6, 7, -1, -1, -1], [0, 5], [1, 0, 3, 0, 0, 3, 0, 0]


@pytest.mark.parametrize("new", [
    [1, 1, 1, 0, 0], [1, 0, 0, 0, 0], [0, 0, 1, 1, 0], [1, -6, -5, 0, 0], [-6, -6, -5, -2, 0], [-6, 1, -5, 0, 0], [1, 1, -5, 0, 3],
    [-2, -2, -1, 0, 0], [-3, -2, -1, 0, 0], [6, 6, 0, 0, 0], [-6, -6, 0, 0, 0], [0, 0, 0, 0, 0], [-2, 1, 1, 0, 0]])
@pytest.mark.parametrize("many", [False, True])
def test_shared_tables_by_hand(ice, new, many):
    """Every way of letting go of a page that three hold; many: the same with the three launches."""
    P = 4
    lens, table, ring, state, refs = _three_holders(P)
    if many:
        lens, new, table = lens + [0] * 1100, new + [0] * 1100, table + [[-1] * 3 for _ in range(1100)]
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=8, max_requests=len(lens), max_blocks=3, max_tokens=1)
    ref = plain_tables_shared(lens, new, table, ring, state, refs, 20, P)
    assert ref[0] == 0
    t = [_i32(x) for x in (lens, new, table, ring)]
    st, rf = torch.tensor(state, dtype=torch.int64, device="cuda"), _i32(refs)
    outs = pc.tables_shared(*t, st, rf, 20)
    assert pc.get_error() == 0
    assert [x.tolist() for x in outs] == list(ref[1:8])
    assert [t[2].tolist(), t[3].tolist(), rf.tolist()] == list(ref[8:])


@pytest.mark.parametrize("fault", ["pages", "columns", "slots", "negative", "too_long", "below_zero", "ring_backwards", "ring_too_full",
                                   "count_too_low", "bad_page", "bad_tail_page", "given_twice"])
@pytest.mark.parametrize("many", [False, True])
def test_shared_tables_all_or_nothing(ice, fault, many):
    P = 4
    lens, table, ring, state, refs = _three_holders(P)
    new, n_slots = [1, 7, -5, -2, 4], 40
    if fault == "pages":
        state = [0, 2]
    elif fault == "columns":
        new[1] = 7
        new[0] = 3 * P - 6 + 1
    elif fault == "slots":
        n_slots = 3
    elif fault == "negative":
        lens[4] = -1
    elif fault == "too_long":
        lens[4] = 3 * P + 1
    elif fault == "below_zero":
        new[3] = -3
    elif fault == "ring_backwards":
        state = [6, 5]
    elif fault == "ring_too_full":
        state = [0, 9]
    elif fault == "count_too_low":
        refs[2] = 2
    elif fault == "bad_page":
        table[0][1] = 8
    elif fault == "bad_tail_page":
        table[2][1] = -1
    elif fault == "given_twice":
        state = [0, 8]
        new = [0, 0, 0, -2, 0]
    if many:
        lens, new, table = lens + [0] * 1100, new + [0] * 1100, table + [[-1] * 3 for _ in range(1100)]
    ref = plain_tables_shared(lens, new, table, ring, state, refs, n_slots, P)
    assert ref[0] != 0
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=8, max_requests=len(lens), max_blocks=3, max_tokens=1)
    t = [_i32(x) for x in (lens, new, table, ring)]
    st, rf = torch.tensor(state, dtype=torch.int64, device="cuda"), _i32(refs)
    outs = pc.tables_shared(*t, st, rf, n_slots)
    assert pc.get_error() == ref[0] and pc.get_error() == 0
    assert [x.tolist() for x in outs] == list(ref[1:8])
    assert [t[2].tolist(), t[3].tolist(), rf.tolist()] == list(ref[8:])
    # the handle's scratch is as before: a good call after it
    lens, table, ring, state, refs = _three_holders(P)
    new = [1, 1, 1, 0, 0]
    if many:
        lens, new, table = lens + [0] * 1100, new + [0] * 1100, table + [[-1] * 3 for _ in range(1100)]
    ref = plain_tables_shared(lens, new, table, ring, state, refs, 20, P)
    t = [_i32(x) for x in (lens, new, table, ring)]
    st, rf = torch.tensor(state, dtype=torch.int64, device="cuda"), _i32(refs)
    outs = pc.tables_shared(*t, st, rf, 20)
    assert pc.get_error() == 0 and [x.tolist() for x in outs] == list(ref[1:8]) and rf.tolist() == ref[10]


@pytest.mark.parametrize("bad", [-1, 8, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("place", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("many", [False, True])
def test_shared_tables_bad_ring(ice, bad, place, many):
    """An id in the ring that is no page's: a step that would take it changes nothing, one that takes only those before it is carried
    out. Of the requests here 0 copies, 1 keeps its page and takes another, 4 takes one: three pages."""
    P = 4
    lens, table, ring, state, refs = _three_holders(P)
    new = [1, 3, -5, 0, 2]
    head = 8 * 5 + 6  # the ring's free part runs over its end
    ring = [ring[(i - head) % 8] for i in range(8)]
    state = [head, head + 5]
    if many:
        lens, new, table = lens + [0] * 1100, new + [0] * 1100, table + [[-1] * 3 for _ in range(1100)]
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=8, max_requests=len(lens), max_blocks=3, max_tokens=1)
    ref = plain_tables_shared(lens, new, table, ring, state, refs, 20, P)
    assert ref[0] == 0 and ref[2][0] - head == 3
    ring[(head + place) % 8] = bad
    for in_place in (False, True):
        t = [_i32(x) for x in (lens, new, table, ring)]
        st, rf = torch.tensor(state, dtype=torch.int64, device="cuda"), _i32(refs)
        outs = pc.tables_shared(*t, st, rf, 20, t[0] if in_place else None, st if in_place else None)
        if place < 3:
            n = len(lens)
            assert pc.get_error() == ice.ICE_ERR_BOUNDS and pc.get_error() == 0
            assert [x.tolist() for x in outs] == [lens, state, [0] * (n + 1), [-1] * 20, [0] * 20, [-1] * n, [-1] * n]
            assert [t[2].tolist(), t[3].tolist(), rf.tolist()] == [table, ring, refs]
        else:
            assert pc.get_error() == 0
            assert [x.tolist() for x in outs] == list(ref[1:8])
            want = list(ref[9])
            want[(head + place) % 8] = bad
            assert [t[2].tolist(), t[3].tolist(), rf.tolist()] == [ref[8], want, ref[10]]


@pytest.mark.parametrize("src,dst,lens", [
    ([0], [5], None), ([-1], [4], None), ([5], [4], None), ([0], [-1], None), ([0], [3], None), ([0, 1], [4, 4], None), ([0], [4], [7]),
    ([0], [4], [-1]), ([4], [4], None), ([0, 4], [4, 3], None)])
def test_fork_all_or_nothing(ice, src, dst, lens):
    P = 4
    have, table, _, _, refs = _three_holders(P)
    ref = plain_fork(src, dst, lens, have, table, refs, P)
    assert ref[0] == -5
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=8, max_requests=5, max_blocks=3, max_tokens=1)
    a, t, rf = _i32(have), _i32(table), _i32(refs)
    out = pc.fork(_i32(src), _i32(dst), a, t, rf, None if lens is None else _i32(lens))
    assert pc.get_error() == ice.ICE_ERR_BOUNDS and pc.get_error() == 0
    assert [out.tolist(), t.tolist(), rf.tolist()] == list(ref[1:])
    same = pc.fork(_i32(src), _i32(dst), a, t, rf, None if lens is None else _i32(lens), a)
    assert pc.get_error() == ice.ICE_ERR_BOUNDS and same is a and a.tolist() == have


def test_fork_of_a_source_length_out_of_range(ice):
    have, table, _, _, refs = _three_holders(4)
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=4, n_pages=8, max_requests=5, max_blocks=3, max_tokens=1)
    for bad in (-1, 13):
        have[0] = bad
        a, t, rf = _i32(have), _i32(table), _i32(refs)
        out = pc.fork(_i32([0]), _i32([4]), a, t, rf)
        assert pc.get_error() == ice.ICE_ERR_BOUNDS
        assert out.tolist() == have and t.tolist() == table and rf.tolist() == refs


def test_fork_reports_bad_pages(ice):
    have, table, _, _, refs = _three_holders(4)
    table[0][1] = 99
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=4, n_pages=8, max_requests=5, max_blocks=3, max_tokens=1)
    a, t, rf = _i32(have), _i32(table), _i32(refs)
    out = pc.fork(_i32([0]), _i32([4]), a, t, rf)
    assert pc.get_error() == ice.ICE_ERR_BOUNDS
    assert out.tolist() == [6, 6, 5, 2, 6] and t[4].tolist() == [5, 99, -1] and rf.tolist() == [1, 0, 3, 0, 0, 4, 0, 0]


@pytest.mark.parametrize("fault", ["moves", "count", "page", "unused", "length", "extra", "extra_unused"])
def test_compact_all_or_nothing(ice, fault):
    P = 4
    lens, table, ring, state, refs = _three_holders(P)
    extra, room = [5], 4
    refs[5] += 1
    if fault == "moves":
        room = 0
    elif fault == "count":
        refs[7] = -1
    elif fault == "page":
        table[3][0] = 8
    elif fault == "unused":
        table[3][0] = 7
    elif fault == "length":
        lens[4] = 13
    elif fault == "extra":
        extra = [-1]
    elif fault == "extra_unused":
        extra = [1]
    ref = plain_compact(lens, table, extra, refs, ring, state, room, P)
    assert ref[0] != 0
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=8, max_requests=5, max_blocks=3, max_tokens=1)
    for in_place in (False, True):
        t, x, rf, rg = _i32(table), _i32(extra), _i32(refs), _i32(ring)
        st = torch.tensor(state, dtype=torch.int64, device="cuda")
        kw = {} if in_place else dict(block_table_out=t.clone(), page_refs_out=torch.zeros_like(rf), extra_pages_out=torch.zeros_like(x))
        got = pc.compact(_i32(lens), t, rf, rg, st, x, room, **kw)
        assert pc.get_error() == ref[0] and pc.get_error() == 0
        assert [y.tolist() for y in got] == [ref[1], ref[2], ref[3], ref[5], ref[4]]
        assert rg.tolist() == ring and st.tolist() == state


@pytest.mark.parametrize("length", [-1, 13, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("wide", [False, True])
def test_compact_tables_of_a_refused_call(ice, length, wide):
    """A call that changes nothing gives the tables that it was given: each request's entries, and the whole row of one whose length is
    impossible. One cluster, and three launches."""
    P, cols, n_pages = 4, 3, 20000 if wide else 8
    table = [[5, 2, -1], [7, -9, 3], [0, 1, 4]]
    refs = [1] * 8 + [0] * (n_pages - 8)
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=n_pages, max_requests=3, max_blocks=cols, max_tokens=1)
    t, rf, ring = _i32(table), _i32(refs), _i32([-3] * n_pages)
    st = torch.tensor([4, 5], dtype=torch.int64, device="cuda")
    out = torch.full_like(t, 99)
    src, dst, to, ro, _ = pc.compact(_i32([6, length, 12]), t, rf, ring, st, block_table_out=out, page_refs_out=torch.zeros_like(rf))
    assert pc.get_error() == ice.ICE_ERR_BOUNDS and pc.get_error() == 0
    assert to.tolist() == [[5, 2, 99], table[1], table[2]] and ro.tolist() == refs and t.tolist() == table
    assert set(src.tolist() + dst.tolist()) == {-1} and st.tolist() == [4, 5] and set(ring.tolist()) == {-3}


@pytest.mark.parametrize("n_pages,fill,n,cols", [
    (1, 0, 37, 50), (1, 1, 37, 50), (1023, 0.5, 37, 50), (4096, 0.3, 37, 50), (4097, 1.0, 37, 50), (5000, 0.02, 37, 50), (200000, 0.4, 37, 50),
    (1, 1, 300, 3600), (1025, 0.9, 300, 3600), (30000, 0.5, 300, 3600), (1100000, 0.3, 37, 50)])
def test_compact_pools(ice, n_pages, fill, n, cols):
    """Pools of one and of many chunks, empty and full, with a list of the caller's own; one cluster and three launches."""
    rng = random.Random(n_pages)
    P = 2
    used = rng.sample(range(n_pages), int(n_pages * fill))
    refs = [0] * n_pages
    for p in used:
        refs[p] = rng.randint(1, 3)
    lens, table = [], []
    for r in range(n):
        k = rng.randint(0, min(cols, len(used)))
        lens.append(max(0, k * P - rng.randint(0, 1)))
        row = rng.sample(used, k)
        table.append(row + [-7] * (cols - k))
    extra = rng.sample(used, min(len(used), 300))
    ring, state = [-3] * n_pages, [11, 12]
    ref = plain_compact(lens, table, extra, refs, ring, state, n_pages // 2, P)
    assert ref[0] == 0
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=n_pages, max_requests=n, max_blocks=cols, max_tokens=1)
    for in_place in (False, True):
        t, x, rf, rg = _i32(table), _i32(extra), _i32(refs), _i32(ring)
        st = torch.tensor(state, dtype=torch.int64, device="cuda")
        kw = {} if in_place else dict(block_table_out=t.clone(), page_refs_out=torch.full_like(rf, 99), extra_pages_out=torch.zeros_like(x))
        got = pc.compact(_i32(lens), t, rf, rg, st, x, **kw)
        assert pc.get_error() == 0
        assert [y.tolist() for y in got] == [ref[1], ref[2], ref[3], ref[5], ref[4]]
        assert rg.tolist() == ref[6] and st.tolist() == ref[7]


# ---- copies of pages ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H,P,n_pages,n,layers,gap", [
    (1, 1, 9, 3, 1, 0), (2, 16, 40, 11, 3, 0), (8, 16, 300, 140, 2, 1), (3, 5, 5000, 2400, 1, 0), (1, 3, 4000, 1900, 2, 3), (8, 64, 10, 1, 4, 0)])
def test_copy(ice, dtype, H, P, n_pages, n, layers, gap):
    pc = _cache(ice, n_kv_heads=H, n_q_heads=H, page_size=P, n_pages=n_pages, dtype=dtype)
    g = torch.Generator().manual_seed(n)
    ids = torch.randperm(n_pages, generator=g)
    src, dst = ids[torch.randint(0, n_pages - n, (n,), generator=g)], ids[n_pages - n:]  # sources more than once
    src, dst = src.clone(), dst.clone()
    src[1::3], dst[2::5] = -1, -1
    pools = [torch.randn((layers, n_pages + gap, H, P, D), generator=g).to(dtype) for _ in range(2)]
    gpu = [x.cuda()[:, :n_pages] for x in pools]
    live = (src >= 0) & (dst >= 0)
    pc.copy(_i32(src.tolist()), _i32(dst.tolist()), *(x[0] if layers == 1 and n % 2 else x for x in gpu))
    assert pc.get_error() == 0
    for x, y in zip(pools, gpu):
        x[:, dst[live]] = x[:, src[live]]
        assert torch.equal(x[:, :n_pages], y.cpu())


def test_copy_bad_pages(ice):
    pc = _cache(ice, n_pages=6)
    kp, vp = (torch.randn((6, 2, 16, D), device="cuda").to(BF16) for _ in range(2))
    for s, d in ((6, 0), (-2, 0), (0, 6), (0, -2)):
        k2, v2 = kp.clone(), vp.clone()
        pc.copy(_i32([1, s]), _i32([2, d]), k2, v2)
        assert pc.get_error() == ice.ICE_ERR_BOUNDS and pc.get_error() == 0
        want = kp.clone()
        want[2] = kp[1]
        assert torch.equal(k2, want)
        want = vp.clone()
        want[2] = vp[1]
        assert torch.equal(v2, want)


def test_copy_in_a_large_pool(ice):
    """Pages whose offsets pass 2^32 bytes and 2^31 elements, and a second layer behind them."""
    n_pages = 130000
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=64, n_pages=n_pages)
    pool = torch.zeros((4, n_pages, 1, 64, D), dtype=BF16, device="cuda")
    pool[:, 3], pool[:, n_pages - 1] = 1.0, 2.0
    pool[3, 3] = 5.0
    pc.copy(_i32([3, n_pages - 1]), _i32([n_pages - 2, 0]), pool[:2], pool[2:])
    assert pc.get_error() == 0
    assert [float(pool[y, p, 0, 17, 5]) for y in range(4) for p in (0, n_pages - 2)] == [2, 1, 2, 1, 2, 1, 2, 5]
    pool[:, [0, 3, n_pages - 2, n_pages - 1]] = 0
    assert not bool(pool.any())


# ---- verification of drafts -----------------------------------------------------------------

def _verify_case(seed, mode, dtype, n, K, V, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    base = sharp * torch.randn((n, K + 1, V), generator=g)
    target = (base if mode == "greedy" else torch.softmax(base, -1)).to(dtype)
    draft = torch.softmax(base[:, :K] + 0.5 * torch.randn((n, K, V), generator=g), -1).to(dtype) if mode == "sample" else None
    n_draft = torch.randint(-1, K + 1, (n,), generator=g, dtype=torch.int32)
    if mode == "greedy":
        tokens = target[:, :K].float().argmax(-1)
        wrong = torch.rand((n, K), generator=g) < 0.3
        tokens = torch.where(wrong, torch.randint(0, V, (n, K), generator=g), tokens)
        uniform = None
    else:
        like = draft if mode == "sample" else target[:, :K]
        tokens = torch.multinomial(like.float().reshape(-1, V), 1, generator=g).view(n, K) if K else torch.zeros((n, 0), dtype=torch.int64)
        uniform = torch.rand((n, K + 1), generator=g)
        if mode == "lookup":
            uniform[:, :K] *= 0.1 * uniform[:, :K]
    return [tokens.to(torch.int32), n_draft, target, draft, uniform]


def _verify_run(ice, c, pc=None):
    pc = pc or _cache(ice, n_kv_heads=1, n_q_heads=1, n_pages=1, max_requests=len(c[1]), max_blocks=1, max_tokens=1)
    got = pc.verify(*[None if x is None else _gpu(x) if x.dim() == 3 else x.cuda() for x in c])
    return pc, [x.cpu() for x in got]


def _verify_check(ice, c, got, code):
    tokens, accepted, n_new = got
    K = c[0].shape[1]
    answers = plain_verify(*c)
    assert code == (ice.ICE_ERR_BOUNDS if any(a[0] for a in answers) else 0)
    for r, (_, kept, check) in enumerate(answers):
        n = int(c[1][r])
        takes_part = 0 <= n <= K
        assert int(accepted[r]) == kept, r
        assert int(n_new[r]) == (kept - n if takes_part else 0), r
        row = tokens[r].tolist()
        assert row[:kept] == c[0][r, :kept].tolist(), r
        assert check(row[kept]), (r, row, kept)
        assert row[kept + 1:] == [-1] * (K - kept), r


@pytest.mark.parametrize("mode", ["sample", "lookup", "greedy"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,K,V", [
    (1, 0, 1), (3, 2, 1), (5, 4, 2), (40, 3, 30), (9, 1, 1023), (9, 5, 1024), (9, 2, 1025), (17, 4, 5001), (300, 2, 2049), (2, 63, 3001),
    (6, 4, 50001), (3, 7, 128000), (2, 1, 150001), (1, 4, 150002), (100, 1, 66001), (200, 1, 66001), (1300, 1, 1025)])
def test_verify(ice, mode, dtype, n, K, V):
    c = _verify_case(n + K + V, mode, dtype, n, K, V)
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())


@pytest.mark.parametrize("mode", ["sample", "greedy"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_verify_largest_vocabulary(ice, mode, dtype):
    c = _verify_case(1, mode, dtype, 2, 1, 1 << 22, sharp=0.5)
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_verify_most_requests(ice, dtype):
    c = _verify_case(2, "sample", dtype, 8192, 1, 40)
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())


@pytest.mark.parametrize("mode", ["sample", "lookup", "greedy"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 5, 7])
def test_verify_strided(ice, mode, dtype, shift):
    """Rows at any element, requests and rows further apart than the vocabulary."""
    n, K, V = 7, 3, 4500
    c = _verify_case(shift, mode, dtype, n, K, V)

    def spread(x, row, req):
        if x is None:
            return None
        base = torch.full((n * req + shift + 16,), math.nan, dtype=x.dtype)
        y = torch.as_strided(base, x.shape, (req, row, 1), shift)
        y.copy_(x)
        return y

    c[2], c[3] = spread(c[2], V + 3, (K + 1) * (V + 3) + 1), spread(c[3], V + 1, K * (V + 1) + 2)
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())


@pytest.mark.parametrize("mode", ["sample", "greedy"])
def test_verify_rows_far_apart(ice, mode):
    """Rows whose offsets pass 2^32 elements."""
    n, K, V = 2, 1, 3001
    c = _verify_case(9, mode, BF16, n, K, V)
    c[1][:] = 1
    big = torch.empty((1 << 32) + (1 << 30) + 4 * V, dtype=BF16, device="cuda")
    far = torch.as_strided(big, (n, K + 1, V), (1 << 32, (1 << 30) + 1, 1), 3)
    far.copy_(c[2])
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, n_pages=1, max_requests=n, max_blocks=1, max_tokens=1)
    got = pc.verify(c[0].cuda(), c[1].cuda(), far, None if c[3] is None else c[3].cuda(), None if c[4] is None else c[4].cuda())
    _verify_check(ice, c, [x.cpu() for x in got], pc.get_error())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [5, 3000, 130000])
def test_verify_borders(ice, dtype, V):
    """Equal weights, whose borders are known: token floor(u V), at the ends and beyond them."""
    us = [0.0, -1.0, math.nan, 2.0 ** -149, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 1.0, math.inf, 1 / 3, 0.999]
    target = torch.full((len(us), 1, V), 2.0 ** -10).to(dtype)
    c = [torch.zeros((len(us), 0), dtype=torch.int32), torch.zeros(len(us), dtype=torch.int32), target, None,
         torch.tensor(us, dtype=torch.float32)[:, None]]
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())
    assert got[0][:4, 0].tolist() == [0, 0, 0, 0]
    assert got[0][5, 0] == V // 2 and got[0][7, 0] == V - 1 and got[0][9, 0] == V - 1


@pytest.mark.parametrize("dtype,V", [(F32, 1 << 19), (F32, 300001), (BF16, 1 << 20)])
@pytest.mark.parametrize("spread", [3.0, 8.0])
def test_verify_weight_before_empty_tiles(ice, dtype, V, spread):
    """Half of the weight near the row's beginning and as much far behind, a long row of nothing after each: half the sum is the border
    between the two, up to the sums' last bits, and what the first half's tiles hold in one order of addition may lie on either side of what
    they hold in another. A token is drawn all the same, one with weight next to the border."""
    n, tile = 64, 512 if dtype == F32 else 1024
    g = torch.Generator().manual_seed(V)
    target = torch.zeros((n, 1, V))
    for r in range(n):
        x = torch.exp(spread * torch.randn(4 * tile, generator=g))
        target[r, 0, :4 * tile], target[r, 0, V // 2:V // 2 + 4 * tile] = x, x[torch.randperm(4 * tile, generator=g)]
    c = [torch.zeros((n, 0), dtype=torch.int32), torch.zeros(n, dtype=torch.int32), target.to(dtype), None, torch.full((n, 1), 0.5)]
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("at", [0, 1023, 1024, 2500, 4999])
def test_verify_one_entry_alone(ice, dtype, at):
    """All the weight, or all that the target has above the draft, in one place; everything else is nothing."""
    V, us = 5000, [0.0, 0.5, 1 - 2.0 ** -24]
    target = torch.zeros((3, 2, V))
    target[..., at] = 1.0
    target[..., (at + 7) % V], target[..., (at + 9) % V], target[..., (at + 11) % V] = math.nan, -1.0, math.inf
    draft = torch.zeros((3, 1, V))
    draft[..., at], draft[..., (at + 1) % V] = 0.5, 0.5
    tokens = torch.full((3, 1), (at + 1) % V, dtype=torch.int32)
    u = torch.tensor([[0.5, x] for x in us])
    for d, n in ((draft, 1), (None, 1), (None, 0)):
        c = [tokens, torch.full((3,), n, dtype=torch.int32), target.to(dtype), None if d is None else d.to(dtype), u]
        pc, got = _verify_run(ice, c)
        _verify_check(ice, c, got, pc.get_error())
        assert got[0].tolist() == [[at, -1]] * 3 and got[1].tolist() == [0, 0, 0]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mode", ["alone", "draft", "lookup"])
@pytest.mark.parametrize("V", [700, 9001])
def test_verify_entries_of_every_size(ice, dtype, mode, V):
    """Entries below the normal numbers, of 2^100, of both in one row, and tiles whose largest entry is far below the row's."""
    g = torch.Generator().manual_seed(V)
    j, some = torch.arange(V), lambda: torch.rand((V,), generator=g, dtype=torch.float64) + 0.01
    least = 2.0 ** (-149 if dtype == F32 else -133)
    rows = [torch.ceil(100 * some()) * least, torch.exp2(torch.floor(some() * 225 - 128)) * (1 + some()), torch.full((V,), 2.0 ** 100, dtype=torch.float64),
            torch.exp2(-j / 50.0), torch.where(j < V // 2, some() * 2.0 ** -120, some()), torch.where(j % 512 < 3, 1.0 + some(), some() * 2.0 ** -30),
            3.0 * some()]
    target = torch.stack(rows).to(dtype).repeat(6, 1)[:, None].repeat(1, 2, 1)
    n = len(target)
    draft = None
    if mode == "draft":
        draft = (target[:, :1].double() * (0.25 + 1.5 * torch.rand((n, 1, V), generator=g, dtype=torch.float64))).to(dtype)
    u = torch.rand((n, 2), generator=g)
    u[:, 0] = 1.0
    tokens = torch.randint(0, V, (n, 1), generator=g, dtype=torch.int32)
    c = [tokens, torch.full((n,), 0 if mode == "alone" else 1, dtype=torch.int32), target, draft, u]
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())


@pytest.mark.parametrize("mode", ["alone", "draft", "lookup"])
@pytest.mark.parametrize("V", [8, 601, 5000])
def test_verify_sums_of_the_least_numbers(ice, mode, V):
    """Weights of a few times 2^-149, as they are left where two models nearly agree: the border u W lies between two numbers."""
    us = [i / 40 for i in range(40)] + [2.0 ** -30, 1 - 2.0 ** -24]
    n = len(us)
    least = 2.0 ** -149
    w = (1 + torch.arange(V) % 3).double() * least
    target, draft = w.float().expand(n, 2, V).contiguous(), None
    u = torch.tensor([[1.0, x] for x in us])
    if mode == "draft":  # every weight is what the target has above the draft
        draft = (torch.arange(V) % 5).double() * least
        target = (w + draft).float().expand(n, 2, V).contiguous()
        draft = draft.float().expand(n, 1, V).contiguous()
        target[:, 0, 5], u[:, 0] = 0.0, 1.0  # the draft itself is rejected
    tokens = torch.full((n, 1), 5, dtype=torch.int32)
    c = [tokens, torch.full((n,), 0 if mode == "alone" else 1, dtype=torch.int32), target, draft, u]
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())


def test_verify_same_rows_for_all(ice):
    """Rows that are one row of memory (strides of 0)."""
    V = 3001
    g = torch.Generator().manual_seed(3)
    row = torch.softmax(2 * torch.randn((V,), generator=g), 0)
    c = [torch.randint(0, V, (7, 3), generator=g, dtype=torch.int32), torch.full((7,), 3, dtype=torch.int32), row.expand(7, 4, V),
         row.expand(7, 3, V), torch.rand((7, 4), generator=g)]
    for d in (c[3], None):
        pc = _cache(ice, n_kv_heads=1, n_q_heads=1, n_pages=1, max_requests=7, max_blocks=1, max_tokens=1)
        one = row.cuda()
        got = pc.verify(c[0].cuda(), c[1].cuda(), one.expand(7, 4, V), None if d is None else one.expand(7, 3, V), c[4].cuda())
        _verify_check(ice, [c[0], c[1], c[2], d, c[4]], [x.cpu() for x in got], pc.get_error())


def test_verify_nothing_above_the_draft(ice):
    """A rejected draft whose target is nowhere above the draft model's: a token of the target's own; without any, -1."""
    V = 3000
    target = torch.full((4, 3, V), 1.0 / V)
    draft = torch.full((4, 2, V), 2.0 / V)
    target[1] = 0.0
    target[2] = math.nan
    target[3], draft[3] = 0.0, 0.0
    target[3, 0, 77] = 2.0 ** 101  # counts as 0
    c = [torch.full((4, 2), 5, dtype=torch.int32), torch.full((4,), 2, dtype=torch.int32), target, draft, torch.full((4, 3), 0.7)]
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())
    assert got[0][:, 0].tolist()[1:] == [-1, -1, -1] and got[1].tolist() == [0, 0, 0, 0] and got[2].tolist() == [-2] * 4


def test_verify_differences_that_cancel(ice):
    """The target a last bit above the draft in every place: what the subtraction cuts off counts."""
    V = 70000
    g = torch.Generator().manual_seed(1)
    draft = (torch.rand((6, 1, V), generator=g) + 0.5) / V
    target = torch.cat([torch.nextafter(draft, torch.full_like(draft, 1.0)), draft], 1)
    target[:, 0] += (torch.rand((6, V), generator=g) < 0.3) * 2.0 ** -40
    c = [torch.full((6, 1), 3, dtype=torch.int32), torch.ones(6, dtype=torch.int32), target, draft,
         torch.cat([torch.full((6, 1), 1.0), torch.rand((6, 1), generator=g)], 1)]
    target[:, 0, 3] = 0.0  # the draft itself is rejected
    pc, got = _verify_run(ice, c)
    _verify_check(ice, c, got, pc.get_error())
    assert got[1].tolist() == [0] * 6


def test_verify_bad_drafts(ice):
    for mode in ("sample", "lookup", "greedy"):
        c = _verify_case(4, mode, F32, 6, 3, 2000)
        c[1][:] = torch.tensor([3, 3, -2, 4, 2, 3])
        c[0][0, 1], c[0][1, 0], c[0][4, 1] = 2000, -1, -2 ** 31
        pc, got = _verify_run(ice, c)
        _verify_check(ice, c, got, pc.get_error())
        assert got[0][2].tolist() == [-1] * 4 and got[0][3].tolist() == [-1] * 4 and got[2][2:4].tolist() == [0, 0]
        assert pc.get_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [70, 1024, 9001])
def test_verify_greedy_ties(ice, dtype, V):
    """Of equal entries the lowest index; both zeros are equal; NaN is passed over; a row of infinities, of NaN."""
    rows = torch.full((7, 1, V), -3.0)
    rows[0, 0, 69] = rows[0, 0, 13] = 4.0
    rows[1, 0] = -0.0
    rows[1, 0, 41:] = 0.0
    rows[2, 0], rows[2, 0, 50] = math.nan, -1e30
    rows[3] = -math.inf
    rows[4] = math.nan
    rows[5, 0, 60], rows[5, 0, 65] = math.inf, math.inf
    rows[6, 0, ::2] = math.nan
    c = [torch.zeros((7, 0), dtype=torch.int32), torch.zeros(7, dtype=torch.int32), rows.to(dtype), None, None]
    pc, got = _verify_run(ice, c)
    assert pc.get_error() == ice.ICE_ERR_BOUNDS
    assert got[0][:, 0].tolist() == [13, 0, 50, 0, -1, 60, 1]
    _verify_check(ice, c, got, ice.ICE_ERR_BOUNDS)


def test_verify_repeats(ice):
    c = _verify_case(5, "sample", F32, 33, 5, 40001)
    pc, a = _verify_run(ice, c)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, _verify_run(ice, c, pc)[1]))


def test_verify_draws_by_the_target(ice):
    """Draws over many random numbers come as often as the weights say: chi-square of 40 cells below its mean plus ten of its
    standard deviations (39 + 10 sqrt(78))."""
    V, n = 40, 8192
    g = torch.Generator().manual_seed(3)
    p, q = (torch.softmax(torch.randn(V, generator=g), 0) for _ in range(2))
    drafts = torch.multinomial(q, n, True, generator=g).to(torch.int32)[:, None]
    c = [drafts, torch.ones(n, dtype=torch.int32), p.expand(n, 2, V).contiguous(), q.expand(n, 1, V).contiguous(),
         torch.rand((n, 2), generator=g)]
    pc, got = _verify_run(ice, c)
    assert pc.get_error() == 0
    # the first token of each request is distributed as the target's, whatever the draft model
    count = torch.bincount(got[0][:, 0].long(), minlength=V).double()
    want = n * p.double() / p.double().sum()
    assert float(((count - want) ** 2 / want).sum()) < 39 + 10 * math.sqrt(78)
    assert 0 < int(got[1].sum()) < n
