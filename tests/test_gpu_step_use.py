"""The calls around the paged cache's attention as a program uses them: refusals on a live handle, streams, graphs, and a loop of
speculative decoding over requests that share pages."""
import ctypes
import os
import random
import re

import pytest
import torch

from tests.paged_helpers import plain_attn
from tests.step_helpers import D, pages_of, plain_rope, plain_verify
from tests.test_gpu_step import BF16, F32, Pool, Shared, _cache, _i32, _pool_lists, _rope_case, _rope_check, _verify_case, ice  # noqa: F401

pytestmark = pytest.mark.gpu


class Calls:
    """A small valid call of each entry, as C arguments that a test can replace."""

    def __init__(self, ice):
        self.ice, self.raw = ice, ice.raw_library()
        self.pc = _cache(ice, max_requests=4, max_blocks=4)
        self.host = torch.zeros(4096, dtype=torch.int64)
        self.pinned = torch.zeros(4096, dtype=torch.int64, pin_memory=True)
        self.ints = torch.zeros(4096, dtype=torch.int64, device="cuda")
        self.kp, self.vp = self.pc.new_pages()
        self.kp.zero_()
        self.vp.zero_()
        self.q, self.qo = (torch.zeros((3, 8, D), dtype=BF16, device="cuda") for _ in range(2))
        self.kv = torch.zeros((3, 2, D), dtype=BF16, device="cuda")
        self.rope = ice.Rope([1.0] * 64, [0] * 32 + [1] * 32)
        self.slots = torch.full((3,), -1, dtype=torch.int64, device="cuda")
        self.probs = torch.zeros(4096, device="cuda")
        self.s = torch.cuda.current_stream().cuda_stream
        i = self.ints.data_ptr()
        kp, vp, kv, q = self.kp.data_ptr(), self.vp.data_ptr(), self.kv.data_ptr(), self.q.data_ptr()
        p = self.probs.data_ptr()
        # scratch buffers of the outputs do not overlap the inputs
        self.args = {
            "rope_append": dict(n=3, rope=self.rope._ref, pos=i, pos_stride=3, offset=0, q=q, qs=1024, qo=self.qo.data_ptr(), qos=1024, k=kv,
                                ks=256, v=kv, vs=256, slots=self.slots.data_ptr(), kp=kp, vp=vp),
            "fork": dict(n=0, src=i, dst=i, len=None, n_req=2, lens=i, table=i + 512, refs=i + 1024, out=i + 2048),
            "tables_shared": dict(n_req=2, lens=i, new=i, table=i + 512, ring=i + 1024, state=i + 2048, refs=i + 2560, out=i + 3328,
                                  state_out=i + 3584, q0=i + 4096, slots=i + 4608, pos=i + 5120, n_slots=2, src=i + 5632, dst=i + 6144),
            "copy": dict(n=2, src=i + 8192, dst=i + 8192, layers=1, stride=0, kp=kp, vp=vp),
            "compact": dict(n_req=2, lens=i, table=i + 512, n_extra=0, extra=None, refs=i + 1024, ring=i + 8192, state=i + 10240, n_moves=2,
                            src=i + 11264, dst=i + 12288, table_out=i + 512, extra_out=None, refs_out=i + 1024),
            "verify": dict(n_req=2, k=2, vocab=5, dtype=ice.ICE_F32, tokens=i, n_draft=i, target=p, ts=15, tr=5, draft=p, ds=10, dr=5,
                           uniform=p, out=i + 8192, acc=i + 10240, new=i + 12288)}
        self.ints[1024:1034] = -1  # copy: nothing

    def __call__(self, name, **over):
        a = self.args[name]
        assert set(over) <= set(a), over
        return getattr(self.raw, "ice_paged_" + name)(self.pc._h, *{**a, **over}.values(), self.s)


NUMBERS = {  # arguments that are no device buffers, with values that are refused
    "rope_append": dict(n=[-1], rope=[None], pos_stride=[2, 0, -3, (1 << 40) + 1], offset=[1 << 31, -(1 << 31) - 1], qs=[1023, 1028, 512],
                        qos=[1023, 512], ks=[255, 128, 260], vs=[128, (1 << 30) + 8]),
    "fork": dict(n=[-1, 3], n_req=[0, 5]),
    "tables_shared": dict(n_req=[0, 5], n_slots=[-1, (1 << 30) + 1]),
    "copy": dict(n=[-1], layers=[0, -1, 4097], stride=[]),
    "compact": dict(n_req=[0, 5], n_extra=[-1], n_moves=[-1]),
    "verify": dict(n_req=[0, 5], k=[-1], vocab=[0], dtype=[2, -1], ts=[-1], tr=[-1, 1 << 46], ds=[-1], dr=[-1]),
}
MAY_BE_NULL = {"fork": {"len"}, "tables_shared": {"pos"}, "verify": {"draft", "uniform"}}
ALIGNED = dict(q=16, qo=16, k=16, v=16, kp=16, vp=16, state=8, state_out=8, slots=8)


@pytest.mark.parametrize("name", list(NUMBERS))
def test_refusals_on_a_live_handle(ice, name):
    c = Calls(ice)
    E = ice.ICE_ERR_INVALID_ARG
    live = dict(n=1) if name == "fork" else dict(n_extra=1, extra=c.ints.data_ptr() + 30000, extra_out=c.ints.data_ptr() + 31000) \
        if name == "compact" else {}
    assert c(name) == ice.ICE_OK
    for arg, values in NUMBERS[name].items():
        for v in values:
            assert c(name, **{arg: v}) == E, (arg, v)
    buffers = [a for a in c.args[name] if a not in NUMBERS[name]]
    for arg in buffers:
        ok = {**c.args[name], **live}[arg]
        if arg not in MAY_BE_NULL.get(name, ()) and not (name == "rope_append" and arg in ("q", "qo")):
            assert c(name, **{**live, arg: None}) == E, arg
        base = ok or c.ints.data_ptr()
        assert c(name, **{**live, arg: base + ALIGNED.get(arg, 4) // 2}) == E, arg
        for t in (c.host, c.pinned):
            assert c(name, **{**live, arg: t.data_ptr()}) == E, arg
    if name == "rope_append":
        assert c(name, q=None) == E and c(name, qo=None) == E and c(name, q=None, qo=None) == ice.ICE_OK
        assert c(name, qo=c.q.data_ptr() + 2048) == E and c(name, qo=c.q.data_ptr(), qos=2048) == E
        assert c(name, qo=c.q.data_ptr()) == ice.ICE_OK
        assert c(name, n=0, k=None) == ice.ICE_OK  # nothing to do
        for field, value in (("n_axes", 0), ("n_axes", 5), ("n_axes", 1), ("n_pairs", 0), ("n_pairs", 12), ("n_pairs", 72), ("interleaved", 2),
                             ("reserved", 1)):
            p = ice.ice_rope.from_buffer_copy(c.rope.params)
            setattr(p, field, value)
            assert c(name, rope=ctypes.byref(p)) == E, field
        for k, value in ((63, float("nan")), (0, float("inf"))):
            p = ice.ice_rope.from_buffer_copy(c.rope.params)
            p.freq[k] = value
            assert c(name, rope=ctypes.byref(p)) == E
    if name == "copy":
        layer = 64 * 2 * 16 * D
        assert c(name, layers=2, stride=layer - 8) == E and c(name, layers=2, stride=layer + 4) == E and c(name, n=0, kp=None) == ice.ICE_OK
    if name == "verify":
        assert c(name, k=64) == ice.ICE_ERR_UNSUPPORTED and c(name, vocab=(1 << 22) + 1) == ice.ICE_ERR_UNSUPPORTED
        assert c(name, k=0, tokens=None, draft=None) == ice.ICE_OK
    torch.cuda.synchronize()
    c.pc.get_error()


def test_scratch_is_not_made_in_a_capture(ice):
    """A capture's first call on shared pages is refused and leaves the capture whole; after one eager call it is taken."""
    pc = _cache(ice)
    lens, table, ring, state = pc.new_tables(2)
    refs, none = pc.new_refs(), torch.empty(0, dtype=torch.int32, device="cuda")
    out = lens.clone()
    codes = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            try:
                pc.fork(none, none, lens, table, refs, seq_len_out=out)
                codes.append(0)
            except ice.IceError as e:
                codes.append(e.code)
        pc.fork(none, none, lens, table, refs, seq_len_out=out)
    assert codes == [ice.ICE_ERR_INVALID_ARG, 0]
    torch.cuda.synchronize()
    assert pc.get_error() == 0


def test_failed_launches_leave_no_error_behind(ice):
    """Launches into a capture that has become invalid fail; the status says so, and the runtime's last error is clear."""
    c = Calls(ice)
    for name in c.args:
        assert c(name) == ice.ICE_OK
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    rt, s = ctypes.CDLL("libcudart.so.13"), ctypes.c_void_p(side.cuda_stream)
    codes, left = [], []
    assert rt.cudaStreamBeginCapture(s, 0) == 0
    try:
        assert rt.cudaStreamSynchronize(s) != 0
        rt.cudaGetLastError()
        c.s = side.cuda_stream
        for name in c.args:
            codes.append(c(name))
            left.append(rt.cudaGetLastError())
    finally:
        graph = ctypes.c_void_p()
        assert rt.cudaStreamEndCapture(s, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
    assert codes == [ice.ICE_ERR_CUDA] * 6 and left == [0] * 6
    c.s = torch.cuda.current_stream().cuda_stream
    for name in c.args:
        assert c(name) == ice.ICE_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("wrong", [None, 3, [1, 2], "number", "cpu", "type", "shape"])
def test_binding_refusals(ice, wrong):
    """Every tensor argument in turn."""
    pc = _cache(ice)
    lens, table, ring, state = pc.new_tables(3)
    refs, e = pc.new_refs(), torch.empty(0, dtype=torch.int32, device="cuda")
    kp, vp = pc.new_pages()
    q, kv = torch.zeros((5, 8, D), dtype=BF16, device="cuda"), torch.zeros((5, 2, D), dtype=BF16, device="cuda")
    slots, pos = torch.full((5,), -1, dtype=torch.int64, device="cuda"), torch.zeros((1, 5), dtype=torch.int32, device="cuda")
    probs = torch.rand((3, 3, 7), device="cuda")
    rope = ice.Rope([1.0] * 64)
    outs = pc.tables_shared(lens, lens, table, ring, state, refs, 4)
    moves = pc.compact(lens, table, refs, ring.clone(), state.clone(), e)
    ver = pc.verify(outs[6].view(3, 1).expand(3, 2).contiguous(), lens, probs, probs[:, :2].contiguous(), probs[:, 0, :3].contiguous())
    calls = [  # arguments; those that are no tensors; those that may be None
        (pc.rope_append, [q, kv, kv, pos, rope, slots, kp, vp, 0, q.clone()], {4, 8}, {0, 9}),
        (pc.fork, [e, e, lens, table, refs, e, lens.clone()], set(), {5, 6}),
        (pc.tables_shared, [lens, lens, table, ring, state, refs, 4, *[t.clone() for t in outs]], {6}, set(range(7, 14))),
        (pc.copy, [outs[5], outs[6], kp, vp], set(), set()),
        (pc.compact, [lens, table, refs, ring.clone(), state.clone(), e, 4, table.clone(), refs.clone(), e.clone(), moves[0][:4].clone(),
                      moves[1][:4].clone()], {6}, {5, 7, 8, 9, 10, 11}),
        (pc.verify, [outs[6].view(3, 1).expand(3, 2).contiguous(), lens, probs, probs[:, :2].contiguous(), probs[:, 0, :3].contiguous(),
                     *[t.clone() for t in ver]], set(), {3, 4, 5, 6, 7})]
    for call, args, numbers, optional in calls:
        call(*args)
        for i in range(len(args)):
            if i in numbers or (wrong is None and i in optional):
                continue
            bad = wrong
            if wrong == "number":
                bad = torch.tensor(1, dtype=torch.int32, device="cuda")
            elif wrong == "cpu":
                bad = args[i].cpu()
            elif wrong == "type":
                bad = args[i].to(torch.float16)
            elif wrong == "shape":
                bad = torch.cat([args[i], args[i][-1:] if args[i].numel() else torch.zeros(1, dtype=args[i].dtype, device="cuda")])
            with pytest.raises(ValueError):
                call(*args[:i], bad, *args[i + 1:])
    torch.cuda.synchronize()
    assert pc.get_error() == 0


def test_binding_refuses_layers_and_strides(ice):
    pc = _cache(ice, n_pages=4)
    none = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    pool = torch.zeros((3, 5, 2, 16, D), dtype=BF16, device="cuda")
    good = pool[:, :4]
    pc.copy(none, none, good, pool.clone()[:, :4])
    for k, v in ((pool, pool), (good, good[:2]), (good, good.contiguous()), (good, good[0]), (good[:0], good[:0]),
                 (good.transpose(2, 3), good), (good.float(), good), (good[..., :64], good), (good, good.cpu())):
        with pytest.raises(ValueError):
            pc.copy(none, none, k, v)
    kv, q = torch.zeros((4, 2, D), dtype=BF16, device="cuda"), torch.zeros((4, 8, D), dtype=BF16, device="cuda")
    slots, pos = torch.full((4,), -1, dtype=torch.int64, device="cuda"), torch.zeros((2, 8), dtype=torch.int32, device="cuda")
    rope = ice.Rope([1.0] * 8, [0, 1] * 4)
    kp, vp = pc.new_pages()
    pc.rope_append(q, kv, kv, pos[:, :4], rope, slots, kp, vp)
    for p in (pos, pos[0, :4], pos[:, ::2], pos[:1, :4], pos[:1, :4].expand(2, 4), pos.T[:4].T.contiguous().T):
        with pytest.raises(ValueError):
            pc.rope_append(q, kv, kv, p, rope, slots, kp, vp)
    with pytest.raises(ValueError):
        pc.rope_append(None, kv, kv, pos[:, :4], rope, slots, kp, vp, q_out=q)
    with pytest.raises(ValueError, match="pos_offset"):
        pc.rope_append(q, kv, kv, pos[:, :4], rope, slots, kp, vp, 1 << 32)
    odd = torch.as_strided(torch.zeros(5000, dtype=BF16, device="cuda"), (4, 8, D), (1028, D, 1))  # rows not 16 bytes apart
    with pytest.raises(ice.IceError):
        pc.rope_append(q, kv, kv, pos[:, :4], rope, slots, kp, vp, 0, odd)


def test_outputs_belong_to_the_given_stream(ice):
    """Memory that was freed while the current stream still writes to it is not what a call on another stream gets for its
    outputs."""
    pc = _cache(ice)
    lens, table, ring, state = pc.new_tables(3)
    refs = pc.new_refs()
    new = _i32([3, 5, 0])
    c = _verify_case(1, "sample", F32, 3, 2, 500)
    c = [x.cuda() for x in c]
    plain = [t.tolist() for t in pc.tables_shared(lens, new, table.clone(), ring.clone(), state, refs.clone(), 8)]
    ref = [t.tolist() for t in pc.verify(*c)]
    f = [_i32([0]), _i32([2]), _i32([7, 0, 0])]
    forked = pc.fork(f[0], f[1], f[2], table.clone().zero_(), refs.clone()).tolist()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late = [torch.empty(n, dtype=d, device="cuda") for n, d in ((3, torch.int32), (2, torch.int64), (4, torch.int32), (8, torch.int64),
                                                                (8, torch.int32), (9, torch.int32), (3, torch.int32), (3, torch.int32))]
    t2, r2, rf2, tz, rz = table.clone(), ring.clone(), refs.clone(), table.clone().zero_(), refs.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    for t in late:
        t.fill_(77)
    del late, t
    got = pc.tables_shared(lens, new, t2, r2, state, rf2, 8, stream=side)
    out = pc.verify(*c, stream=side)
    fk = pc.fork(f[0], f[1], f[2], tz, rz, stream=side)
    torch.cuda.synchronize()
    assert pc.get_error() == 0
    assert [t.tolist() for t in got] == plain and [t.tolist() for t in out] == ref and fk.tolist() == forked


def test_outputs_without_the_short_allocation(ice, monkeypatch):
    """Outputs are allocated by a short way where PyTorch has it, else by torch.empty: the same tensors, and calls give the same."""
    shapes = [((5,), torch.int32), ((0,), torch.int32), ((2,), torch.int64), ((3, 4), torch.int32), ((1, 1), torch.float32), ((3, 1), torch.int32)]

    def outputs():
        pc = _cache(ice)
        made = [ice._empty(shape, t, pc.device) for shape, t in shapes]
        lens, table, ring, state = pc.new_tables(3)
        refs = pc.new_refs()
        step = pc.tables_shared(lens, _i32([3, 17, 0]), table, ring, state, refs, 24)
        forked = pc.fork(_i32([1]), _i32([2]), step[0], table, refs)
        moves = pc.compact(forked, table, refs, ring, state)
        ver = pc.verify(*[None if x is None else x.cuda() for x in _verify_case(1, "sample", F32, 3, 2, 500)])
        assert pc.get_error() == 0
        return [(x.shape, x.stride(), x.dtype, x.device) for x in made], [x.tolist() for x in (*step, forked, *moves[:4], refs, *ver)]

    first = outputs()
    monkeypatch.setattr(ice, "_empty_strided", None)
    second = outputs()
    assert first == second
    assert first[0] == [(x.shape, x.stride(), x.dtype, x.device) for x in (torch.empty(s, dtype=t, device="cuda") for s, t in shapes)]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rope_and_verify_in_graphs(ice, dtype):
    """Captured once, replayed on other inputs; two captured calls share a handle."""
    c = [_rope_case(s, dtype, 70, 2, 4, 16, 64, 3) for s in (1, 2)]
    pc = _cache(ice, n_kv_heads=2, n_q_heads=8, n_pages=c[0]["n_pages"], dtype=dtype, max_requests=16)
    v = {m: [_verify_case(s, m, dtype, 16, 3, 3001) for s in (3, 4)] for m in ("sample", "greedy")}
    kp, vp = pc.new_pages()
    rope = ice.Rope(c[0]["freq"], c[0]["axis"])
    x = {k: c[0][k].cuda() for k in ("q", "k", "v", "pos", "slots")}
    y = {m: [None if t is None else t.cuda() for t in v[m][0]] for m in v}
    q_out = torch.zeros_like(x["q"])
    outs = {m: pc.verify(*y[m]) for m in v}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pc.rope_append(x["q"], x["k"], x["v"], x["pos"], rope, x["slots"], kp, vp, 5, q_out)
        for m in v:
            pc.verify(*y[m], *outs[m])
    for k in (1, 0, 1):
        for t in (kp, vp, q_out):
            t.fill_(7.0)
        for name in x:
            x[name].copy_(c[k][name])
        for m in v:
            for a, b in zip(y[m], v[m][k]):
                if a is not None:
                    a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        code = pc.get_error()
        _rope_check(c[k], False, 5, q_out.cpu(), kp.cpu(), vp.cpu())
        for m in v:
            answers = plain_verify(*v[m][k])
            assert code == 0 and not any(a[0] for a in answers)
            tokens, accepted, n_new = (t.cpu() for t in outs[m])
            for r, (_, kept, check) in enumerate(answers):
                assert int(accepted[r]) == kept and check(int(tokens[r, kept])), (m, r)


def test_two_handles_at_once(ice):
    """Steps of two pools on two streams, none waiting for the other; one by one cluster, one by three launches."""
    from tests.step_helpers import plain_tables_shared
    sizes = ((60, 4, 9, 400), (1100, 4, 9, 7000))
    pools = [Pool(7 + i, *x) for i, x in enumerate(sizes)]
    pcs = [_cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=n_pages, max_requests=n, max_blocks=cols, max_tokens=1)
           for n, P, cols, n_pages in sizes]
    gpus = [Shared(pool, pc=pc) for pool, pc in zip(pools, pcs)]
    streams = [torch.cuda.Stream() for _ in pools]
    refs = [[], []]
    changes = [[], []]
    for i, pool in enumerate(pools):
        for _ in range(8):
            new = pool.change()
            ref = plain_tables_shared(pool.lens, new, pool.table, pool.ring, pool.state, pool.refs, 9000, pool.P)
            assert ref[0] == 0
            _, pool.lens, pool.state, *rest, pool.table, pool.ring, pool.refs = ref
            refs[i].append(rest)
            changes[i].append(_i32(new))
    torch.cuda.synchronize()
    outs = [[], []]
    for t in range(8):
        for i, (pc, gpu, st) in enumerate(zip(pcs, gpus, streams)):
            outs[i].append(pc.tables_shared(gpu.lens, changes[i][t], gpu.table, gpu.ring, gpu.state, gpu.refs, 9000, gpu.lens, gpu.state,
                                            stream=st)[2:])
    torch.cuda.synchronize()
    for i in range(2):
        assert pcs[i].get_error() == 0
        for t in range(8):
            assert [x.tolist() for x in outs[i][t]] == list(refs[i][t]), (i, t)
        assert gpus[i].lists() == _pool_lists(pools[i])


def test_shared_pages_in_a_graph(ice):
    """Forks, steps and a compaction, captured once and replayed as lengths change, in place."""
    n, P, cols, n_pages = 40, 4, 9, 260
    pool = Pool(3, n, P, cols, n_pages)
    pc = _cache(ice, n_kv_heads=1, n_q_heads=1, page_size=P, n_pages=n_pages, max_requests=n, max_blocks=cols, max_tokens=1)
    gpu = Shared(pool, pc=pc)
    from tests.step_helpers import plain_compact, plain_fork, plain_tables_shared
    new, src, dst = _i32([0] * n), _i32([0] * 4), _i32([0] * 4)
    ms, md = _i32([0] * (n_pages // 2)), _i32([0] * (n_pages // 2))

    def step():
        pc.tables_shared(gpu.lens, new, gpu.table, gpu.ring, gpu.state, gpu.refs, 600, gpu.lens, gpu.state, *outs[2:])
        pc.fork(src, dst, gpu.lens, gpu.table, gpu.refs, None, gpu.lens)
        pc.compact(gpu.lens, gpu.table, gpu.refs, gpu.ring, gpu.state, move_src=ms, move_dst=md)

    outs = pc.tables_shared(gpu.lens, new, gpu.table, gpu.ring, gpu.state, gpu.refs, 600)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in range(12):
        change = pool.change()
        ref = plain_tables_shared(pool.lens, change, pool.table, pool.ring, pool.state, pool.refs, 600, P)
        assert ref[0] == 0
        _, pool.lens, pool.state, *rest, pool.table, pool.ring, pool.refs = ref
        empty, full = [r for r in range(n) if not pool.lens[r]], [r for r in range(n) if pool.lens[r]]
        d = empty[:4]
        while len(d) < 4:  # no room: not a destination twice, but a call that is refused whole
            d.append(d[-1] if d else 0)
        s = [full[(t + i) % len(full)] for i in range(4)] if full else d
        f = plain_fork(s, d, None, pool.lens, pool.table, pool.refs, P)
        _, pool.lens, pool.table, pool.refs = f
        c = plain_compact(pool.lens, pool.table, [], pool.refs, pool.ring, pool.state, n_pages // 2, P)
        assert c[0] == 0
        _, msrc, mdst, pool.table, _, pool.refs, pool.ring, pool.state = c
        new.copy_(_i32(change))
        src.copy_(_i32(s))
        dst.copy_(_i32(d))
        g.replay()
        torch.cuda.synchronize()
        assert pc.get_error() == f[0], t
        assert [x.tolist() for x in outs[2:]] == list(rest), t
        assert [ms.tolist(), md.tolist()] == [msrc, mdst]
        assert gpu.lists() == _pool_lists(pool), t
        pool.check()


@pytest.mark.parametrize("axes", [1, 3])
def test_readme_examples(ice, axes):
    """The examples of the paged cache, as they are written, one after the other."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "pc." in b]
    assert len(blocks) == 2 and "PagedCache" in blocks[0] and "compact" in blocks[1]
    g = torch.Generator().manual_seed(1)
    n_req, drafts, V, L = 8, 3, 500, 37
    new = [1 + min(r, drafts) for r in range(n_req)]
    n_slots = sum(new) + 5
    rows = [torch.randn((n_slots, h, D), generator=g).to(BF16).cuda() for h in (32, 8, 8)]
    probs = torch.softmax(torch.randn((n_req, drafts + 1, V), generator=g), -1).cuda()
    here = dict(ice=ice, torch=torch, n_req=n_req, n_slots=n_slots, n_new=_i32(new), prefix_len=L, n_prefix_pages=pages_of(L, 16),
                prefix_table=_i32([4095, 4094, 4093]), freq=[10000.0 ** (-i / 64) for i in range(64)], axis=[i % 3 for i in range(64)],
                draft_tokens=torch.zeros((n_req, drafts), dtype=torch.int32, device="cuda"), n_draft=_i32(new) - 1, target_probs=probs,
                draft_probs=probs[:, :drafts].flip(2).contiguous(), uniform=torch.rand((n_req, drafts + 1), generator=g).cuda())
    for i, b in enumerate(blocks):
        if axes > 1:  # as the comments beside the two lines say
            b = b.replace("ice.Rope(freq)", "ice.Rope(freq, axis)").replace(", pos, rope", f", torch.stack([pos] * {axes}), rope")
        here.update(q=rows[0], k=rows[1], v=rows[2], src=_i32([0, 0]), dst=_i32([6, 7]))
        if i:
            here["k_pages"].zero_(), here["v_pages"].zero_()
        exec(b, here)
        assert here["pc"].get_error() == 0
    assert bool(torch.isfinite(here["out"][:sum(new)]).all())
    lens, kept = here["seq_len"].tolist(), here["n_accepted"].tolist()
    assert lens == [1 + a for a in kept]
    pages = here["n_prefix_pages"] + n_req  # a page a request
    assert here["state"].tolist() == [0, 4096 - pages] and int(here["refs"][:pages].sum()) == pages


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("graph", [False, True])
def test_speculative_serving_loop(ice, dtype, graph):
    """A batch over a shared prefix, two layers: forks, drafts, tables, copies on write, rotating append, attention, verification,
    rejected drafts given up, ends and compaction; eagerly on a stream of its own or as a captured step. Against requests that keep
    every row of theirs."""
    B, H, G, P, L, layers, K, V, cap, n_pages, cols = 6, 2, 4, 8, 21, 2, 3, 700, 128, 120, 10
    n = B + 1  # the last request is the prefix
    pc = _cache(ice, n_kv_heads=H, n_q_heads=H * G, page_size=P, n_pages=n_pages, max_requests=n, max_blocks=cols, max_tokens=cap, dtype=dtype)
    g, rng = torch.Generator().manual_seed(4), random.Random(4)
    freq = [500.0 ** (-i / 64) for i in range(64)]
    rope = ice.Rope(freq)
    pools = [torch.full((layers, n_pages, H, P, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    lens, table, ring, state = pc.new_tables(n)
    refs = pc.new_refs()
    new, n_draft = _i32([0] * n), _i32([-1] * n)
    q = torch.zeros((layers, cap, H * G, D), dtype=dtype, device="cuda")
    kn, vn = (torch.zeros((layers, cap, H, D), dtype=dtype, device="cuda") for _ in range(2))
    qr, out = torch.zeros_like(q), torch.zeros_like(q)
    target, draft = torch.zeros((n, K + 1, V), device="cuda"), torch.zeros((n, K, V), device="cuda")
    tokens, uniform = torch.zeros((n, K), dtype=torch.int32, device="cuda"), torch.zeros((n, K + 1), device="cuda")
    step_out = pc.tables_shared(lens, new, table, ring, state, refs, cap)
    ver_out = pc.verify(tokens, n_draft, target, draft, uniform)
    # the prefix's rows, through the same calls
    one = pc.tables_shared(lens, _i32([0] * B + [L]), table, ring, state, refs, cap, lens, state)
    pre = [torch.randn((layers, L, H, D), generator=g).to(dtype) for _ in range(2)]
    for y in range(layers):
        kn[y, :L], vn[y, :L] = pre[0][y].cuda(), pre[1][y].cuda()
        pc.rope_append(None, kn[y], vn[y], one[4], rope, one[3], pools[0][y], pools[1][y])
    prefix = table[B, :pages_of(L, P)].clone()
    plain = [[(pre[0][y].new_zeros((0, H, D)), pre[1][y].new_zeros((0, H, D))) for y in range(layers)] for _ in range(B)]  # k as given

    def step():
        pc.tables_shared(lens, new, table, ring, state, refs, cap, lens, state, *step_out[2:])
        _, _, q_start, slots, pos, csrc, cdst = step_out
        pc.copy(csrc, cdst, *pools)
        for y in range(layers):
            pc.rope_append(q[y], kn[y], vn[y], pos, rope, slots, pools[0][y], pools[1][y], L, qr[y])
            pc.attn(qr[y], q_start, lens, table, pools[0][y], pools[1][y], prefix, L, out=out[y])
        pc.verify(tokens, n_draft, target, draft, uniform, *ver_out)

    after = [t.clone() for t in step_out]

    def settle():
        pc.tables_shared(lens, ver_out[2], table, ring, state, refs, 0, lens, state, after[2], after[3][:0], after[4][:0], *after[5:])

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    replay = None
    if graph:
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay):
            step()
    forks = copies = rejected = moved = 0
    for t in range(22):
        have = [x[0][0].shape[0] for x in plain]
        # forks: empty rows continue others, some from an earlier token on
        full, empty = [r for r in range(B) if have[r]], [r for r in range(B) if not have[r]]
        if t % 3 == 1 and full and empty:
            dst = empty[:rng.randint(1, len(empty))]
            src = [rng.choice(full) for _ in dst]
            cut = [rng.randint(1, have[s]) if rng.random() < 0.5 else have[s] for s in src]
            pc.fork(_i32(src), _i32(dst), lens, table, refs, _i32(cut), lens)
            for s, d, c in zip(src, dst, cut):
                plain[d] = [(k[:c], v[:c]) for k, v in plain[s]]
            forks += len(dst)
        have = [x[0][0].shape[0] for x in plain]
        # a prompt, a token with drafts, nothing, or the end
        change, drafts = [], []
        for r in range(B):
            if have[r] == 0:
                x = rng.choice([0, rng.randint(1, 20)])
                d = -1
            elif have[r] > cols * P - 12 or (t % 6 == 5 and r % 2):
                x, d = -have[r], -1
            else:
                d = rng.randint(0, K)
                x = 1 + d
            change.append(x)
            drafts.append(d)
        total = sum(max(0, x) for x in change)
        base = torch.randn((n, K + 1, V), generator=g) * 2
        tp = torch.softmax(base, -1)
        dp = torch.softmax(base[:, :K] + 0.6 * torch.randn((n, K, V), generator=g), -1)
        tk = torch.multinomial(dp.reshape(-1, V), 1, generator=g).view(n, K).to(torch.int32)
        u = torch.rand((n, K + 1), generator=g)
        rows = {a: torch.randn(b.shape, generator=g).to(dtype) for a, b in (("q", q), ("k", kn), ("v", vn))}
        for a, b in ((q, rows["q"]), (kn, rows["k"]), (vn, rows["v"]), (target, tp), (draft, dp), (tokens, tk), (uniform, u)):
            a.copy_(b)
        new.copy_(_i32(change + [0]))
        n_draft.copy_(_i32(drafts + [-1]))
        out.fill_(5.0)
        qr.fill_(5.0)
        torch.cuda.synchronize()
        if graph:
            replay.replay()
        else:
            with torch.cuda.stream(side):
                step()
        torch.cuda.synchronize()
        assert pc.get_error() == 0, t
        copies += int((step_out[5] >= 0).sum())
        at = 0
        for r, x in enumerate(change):
            plain[r] = [((torch.cat([k, rows["k"][y, at:at + x]]), torch.cat([v, rows["v"][y, at:at + x]])) if x > 0 else
                         (k[:k.shape[0] + x], v[:v.shape[0] + x])) for y, (k, v) in enumerate(plain[r])]
            at += max(0, x)
        have = [x[0][0].shape[0] for x in plain]
        assert lens.tolist() == have + [L]
        tb, q0 = table.cpu(), step_out[2].cpu()
        for y in range(layers):
            # what the pages hold: each request's keys, rotated, and values
            kc, vc = pools[0][y].cpu(), pools[1][y].cpu()
            S = max(max(have), L, 1)
            kf, vf = (torch.zeros((B + 1, H, S, D), dtype=dtype) for _ in range(2))
            for i, (first, (k, v)) in enumerate([(0, (pre[0][y], pre[1][y]))] + [(L, plain[r][y]) for r in range(B)]):
                m = k.shape[0]
                ids = tb[B if i == 0 else i - 1, :pages_of(m, P)].long()
                got = [x[ids].transpose(1, 2).reshape(-1, H, D)[:m] for x in (kc, vc)]
                want, tol = plain_rope(k, torch.arange(m)[None], first, freq, [0] * 64, False)
                assert bool(((got[0].double() - want).abs() <= tol).all()), (t, y, i)
                assert torch.equal(got[1], v), (t, y, i)
                kf[i, :, :m], vf[i, :, :m] = got[0].transpose(0, 1), got[1].transpose(0, 1)
            where = torch.cat([torch.arange(x) + h - x for x, h in zip(change, have) if x > 0] or [torch.zeros(0)]).long()
            want, tol = plain_rope(rows["q"][y, :total], where[None], L, freq, [0] * 64, False)
            assert bool(((qr[y, :total].cpu().double() - want).abs() <= tol).all())
            assert bool((qr[y, total:] == 5.0).all())
            ref, tol = plain_attn(qr[y, :total].cpu(), q0[:B + 1], torch.tensor(have), torch.arange(1, B + 1, dtype=torch.int32)[:, None], kf, vf,
                                  torch.tensor([0], dtype=torch.int32), L)
            assert bool(((out[y, :total].cpu().double() - ref).abs() <= tol).all()), (t, y)
            assert bool((out[y, total:] == 5.0).all())
        kept = ver_out[1].tolist()
        for r, (code, a, check) in enumerate(plain_verify(tk, torch.tensor(drafts + [-1], dtype=torch.int32), tp, dp, u)):
            assert code == 0 and kept[r] == a and check(int(ver_out[0][r, a])), (t, r)
        give = [k - d if d >= 0 else 0 for k, d in zip(kept, drafts)]
        assert ver_out[2].tolist() == give + [0]
        settle()
        assert pc.get_error() == 0
        plain = [[(k[:k.shape[0] + x], v[:v.shape[0] + x]) for k, v in p] for p, x in zip(plain, give)]
        rejected -= sum(give)
        if t % 4 == 3:
            src, dst, *_ = pc.compact(lens, table, refs, ring, state, prefix)
            pc.copy(src, dst, *pools)
            assert pc.get_error() == 0
            moved += int((dst >= 0).sum())
            used = int((refs > 0).sum())
            assert bool((refs[:used] > 0).all()) and state.tolist() == [0, n_pages - used]
    assert forks and copies and rejected and moved
    pc.tables_shared(lens, -lens, table, ring, state, refs, 0, lens, state)
    assert pc.get_error() == 0
    assert not bool(refs.any()) and int(state[1] - state[0]) == n_pages  # no page was lost
    assert sorted(ring.tolist()) == list(range(n_pages))
