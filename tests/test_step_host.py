"""What surrounds the paged cache's attention, without a GPU: refusals of the C entries and of the binding, the ctypes mirror, where
the kernels wait, and the plain statements that the GPU tests compare with."""
import ctypes
import math
import os
import random
import re
import shutil
import subprocess
from fractions import Fraction

import pytest
import torch

from tests import paged_helpers, step_helpers as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "semantic_paged_kv_head_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    from semantic_paged_kv_head_gb300 import build
    build.build_lib()
    from semantic_paged_kv_head_gb300 import ice
    return ice


def test_null_handles(lib):
    raw, E = lib.raw_library(), lib.ICE_ERR_INVALID_ARG
    rope = lib.Rope([1.0] * 8)
    assert raw.ice_paged_rope_append(None, 1, rope._ref, 16, 1, 0, 16, 1024, 32, 1024, 16, 1024, 16, 1024, 16, 16, 16, None) == E
    assert raw.ice_paged_fork(None, 1, 16, 16, None, 1, 16, 16, 16, 16, None) == E
    assert raw.ice_paged_tables_shared(None, 1, *[16] * 11, 1, 16, 16, None) == E
    assert raw.ice_paged_copy(None, 1, 16, 16, 1, 0, 16, 16, None) == E
    assert raw.ice_paged_compact(None, 1, 16, 16, 0, None, 16, 16, 16, 1, 16, 16, 16, None, 16, None) == E
    assert raw.ice_paged_verify(None, 1, 1, 10, 0, 16, 16, 16, 10, 10, None, 0, 0, None, 16, 16, 16, None) == E


def test_struct_layout_matches_the_header(lib, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    cls = lib.ice_rope
    lines = ['#include <stdio.h>', '#include "ice.h"', "int main(void) {", 'printf("size %zu\\n", sizeof(ice_rope));']
    lines += [f'printf("{f} %zu\\n", offsetof(ice_rope, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]) + "\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f, _ in cls._fields_:
        assert int(got[f]) == getattr(cls, f).offset, f


def test_kernels_wait_before_they_read():
    """The kernels are launched before the kernels ahead of them have ended: what comes before the wait touches no buffer of the
    call."""
    seen = []
    for name in ("ice_paged_rope.cu", "ice_paged_share.cu", "ice_paged_verify.cu"):
        text = open(os.path.join(CSRC, name)).read()
        for m in re.finditer(r"__global__ void __launch_bounds__\(.*?\) (\w+_kernel)\((.*?)\) \{", text, re.S):
            before = text[m.end():text.index("pdl_wait_then_release();", m.end())]
            assert "__global__" not in before, m.group(1)
            before = re.sub(r"//[^\n]*", "", before)
            if re.search(r"\b\w+ a$", m.group(2).strip()):  # one struct; the arrays in it are passed by value
                assert not re.search(r"\ba\.(?!turn\b|axis\b)\w+\s*(\[|->)|[=(,!]\s*\*\s*\(?a\.", before), m.group(1)
            else:
                for p in re.findall(r"\*\s*(\w+)", m.group(2)):
                    assert not re.search(r"\b" + p + r"\s*\[|\*\s*" + p + r"\b(?!\s*[\w(])", before), (m.group(1), p)
            assert not re.search(r"__ld\w+\(|atomic|share_|compact_|tokens|uniform", before), m.group(1)
            seen.append(m.group(1))
    assert sorted(seen) == ["compact_apply_kernel", "compact_count_kernel", "compact_move_kernel", "compact_step_kernel", "fork_kernel",
                            "page_copy_kernel", "rope_append_kernel", "share_claim_kernel", "share_count_kernel", "share_fill_kernel",
                            "share_step_kernel", "verify_greedy_kernel", "verify_sample_kernel"]


def test_words_that_others_change_decide_by_a_vote():
    """A word that other blocks change meanwhile may read differently in each lane. What it decides is a vote of the warp, so that
    all lanes go the same way and meet in the shuffles and reductions behind it."""
    seen = 0
    for name in ("ice_paged_rope.cu", "ice_paged_share.cu", "ice_paged_verify.cu"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"(?<!asm )volatile", text):
            start = max(text.rfind(c, 0, m.start()) for c in ";{}")
            statement = text[start + 1:text.index(";", m.end())]
            # one declaration, nothing but the vote on the load
            assert re.fullmatch(r"\s*const bool \w+ = __any_sync\(0xffffffffu, [\w +]+ <= [\w +]+ - \*\(volatile int\*\)&[\w>-]+\)", statement), statement
            seen += 1
    assert seen == 1


TURNS = r"""
#include <cstdio>
#include <cstdlib>
#include "ice_paged_turns.h"

int main() {
    char line[64];
    while (std::fgets(line, sizeof line, stdin)) std::printf("%llu\n", ice::turns(std::strtod(line, nullptr)));
}
"""


def test_frequencies_to_the_nearest_part_of_a_turn(tmp_path):
    """The 64-bit fraction of a turn that a frequency is held as, against exact fractions: to the nearest, 2^-65 turns. 2 pi is taken in
    106 bits: a quotient t moves by t 2^-106 at most, 2^-42 t units of 2^-64."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "turns.cpp", tmp_path / "turns"
    src.write_text(TURNS)
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    turn = Fraction("6.2831853071795864769252867665590057683943387987502116419498891846156")
    rng = random.Random(1)
    freq = [base ** (-i / 64) for base in (10000.0, 500000.0, 5e6) for i in range(64)]
    freq += [math.ldexp(1 + rng.random(), rng.randint(-70, 31)) for _ in range(3000)] + [0.0, 5e-324, 2.0 ** -1022, 2.0 ** -65, 2.0 ** -60, 1.0, 6.5, 2.0 ** 32]
    freq += [k * float(turn) for k in (0.25, 0.5, 1, 2, 1000)] + [float(turn) * 2.0 ** -k for k in (11, 12, 13, 40, 64, 65)]
    freq += [-f for f in freq]
    r = subprocess.run([str(exe)], input="\n".join(f.hex() for f in freq) + "\n", capture_output=True, text=True, check=True)
    for f, got in zip(freq, r.stdout.split(), strict=True):
        units = Fraction(f) / turn * 2 ** 64
        off = (int(got) - units + 2 ** 63) % 2 ** 64 - 2 ** 63
        assert abs(off) <= Fraction(1, 2) + Fraction(1, 2 ** 16) + abs(Fraction(f) / turn) / 2 ** 42, (f, float(off))


@pytest.mark.parametrize("freq,axis", [
    ([], None), ([1.0] * 7, None), ([1.0] * 72, None), ([1.0] * 12, None), ([math.nan] + [1.0] * 7, None), ([math.inf] + [1.0] * 7, None),
    ([1.0] * 8, [0] * 7), ([1.0] * 8, [0] * 7 + [4]), ([1.0] * 8, [0] * 7 + [-1]), ([1.0] * 8, [0] * 7 + [1 << 32])])
def test_rope_refuses(lib, freq, axis):
    with pytest.raises(ValueError):
        lib.Rope(freq, axis)


def test_rope_parameters(lib):
    r = lib.Rope([1.0, 0.5] * 8, [0, 2] * 8, interleaved=True)
    assert (r.n_axes, r.params.n_axes, r.params.n_pairs, r.params.interleaved, r.params.reserved) == (3, 3, 16, 1, 0)
    assert list(r.params.freq)[:18] == [1.0, 0.5] * 8 + [0, 0] and list(r.params.axis)[:16] == [0, 2] * 8


def test_binding_refuses_without_a_gpu(lib):
    """Arguments that are no CUDA tensors, or numbers that do not fit, before anything is launched."""
    pc = lib.PagedCache.__new__(lib.PagedCache)
    pc.params = lib.ice_paged_params(d=128, n_kv_heads=2, n_q_heads=8, page_size=16, dtype=lib.ICE_BF16, max_requests=4, max_blocks=8,
                                     max_tokens=16, n_pages=64)
    pc.dtype, pc._page_shape, pc.device = torch.bfloat16, (64, 2, 16, 128), torch.device("cpu")
    pc._d, pc._n_pages, pc._columns, pc._index = 128, 64, 8, 0
    i, l = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    kv, q = torch.zeros((4, 2, 128), dtype=torch.bfloat16), torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    pages = torch.zeros((64, 2, 16, 128), dtype=torch.bfloat16)
    rope = lib.Rope([1.0] * 64)
    for call in (lambda: pc.rope_append(q, kv, kv, i, rope, l, pages, pages), lambda: pc.rope_append(q, kv, kv, i, None, l, pages, pages),
                 lambda: pc.fork(i, i, i, i, i), lambda: pc.fork(None, i, i, i, i), lambda: pc.tables_shared(i, i, i, i, i, i, 4),
                 lambda: pc.copy(i, i, pages, pages), lambda: pc.compact(i, i, i, i, i), lambda: pc.verify(i, i, pages),
                 lambda: pc.verify(i, i, None)):
        with pytest.raises(ValueError):
            call()
    for n in (-1, (1 << 30) + 1, 1 << 32):
        with pytest.raises(ValueError, match="n_slots"):
            pc.tables_shared(i, i, i, i, i, i, n)
    for n in (-1, 1 << 31, 1 << 32):
        with pytest.raises(ValueError, match="n_moves"):
            pc.compact(i, i, i, i, i, n_moves=n)


# ---- the plain statements ---------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(6))
def test_plain_shared_tables_without_sharing(seed):
    """Where no page is shared: plain_tables, and counts of 1 for the pages held."""
    rng = random.Random(seed)
    P, cols, n = rng.choice([1, 4, 5]), 6, 9
    lens = [rng.randint(0, cols * P // 2) for _ in range(n)]
    new = [rng.choice([-a, 1, 0, 2 * P, -min(a, 2)]) for a in lens]
    table, ids = [], list(range(80))
    rng.shuffle(ids)
    at = 0
    for a in lens:
        k = H.pages_of(a, P)
        table.append(ids[at:at + k] + [-1] * (cols - k))
        at += k
    ring, state = ids[at:] + [-1] * at, [0, 80 - at]
    refs = [0] * 80
    for p in ids[:at]:
        refs[p] = 1
    slots = sum(max(0, x) for x in new) + 2
    one = paged_helpers.plain_tables(lens, new, table, ring, state, slots, P)
    two = H.plain_tables_shared(lens, new, table, ring, state, refs, slots, P)
    assert one[0] == 0 and two[:6] == one[:6] and two[8:10] == one[6:8]
    assert two[6] == two[7] == [-1] * n
    held = [0] * 80
    for a, row in zip(two[1], two[8]):
        for p in row[:H.pages_of(a, P)]:
            held[p] += 1
    assert held == two[10]


def test_plain_shared_tables_by_hand():
    # P = 4: requests 0 and 1 share page 2 (full) and page 5 (two tokens); both write a token; request 2 ends, alone on page 0
    table = [[2, 5, -1], [2, 5, -1], [0, -1, -1]]
    got = H.plain_tables_shared([6, 6, 3], [1, 3, -3], table, [1, 3, 4, -1, -1, -1], [0, 3], [1, 0, 2, 0, 0, 2], 6, 4)
    code, lens, state, q0, slots, pos, src, dst, table, ring, refs = got
    # the first of the two copies page 5 to page 1, the second keeps it and takes page 3 besides; page 0 goes back
    assert code == 0 and lens == [7, 9, 0] and state == [2, 4] and q0 == [0, 1, 4, 4]
    assert src == [5, -1, -1] and dst == [1, -1, -1]
    assert slots == [1 * 4 + 2, 5 * 4 + 2, 5 * 4 + 3, 3 * 4, -1, -1] and pos == [6, 6, 7, 8, 0, 0]
    assert table == [[2, 1, -1], [2, 5, 3], [0, -1, -1]] and ring == [1, 3, 4, 0, -1, -1] and refs == [0, 1, 2, 1, 0, 1]


def test_plain_fork_and_compact_by_hand():
    code, lens, table, refs = H.plain_fork([0, 0], [2, 1], [5, 3], [5, 0, 0], [[4, 1], [-1, -1], [-1, -1]], [0, 1, 0, 0, 1], 4)
    assert code == 0 and lens == [5, 3, 5] and table == [[4, 1], [4, -1], [4, 1]] and refs == [0, 2, 0, 0, 3]
    code, src, dst, table, extra, refs, ring, state = H.plain_compact(lens, table, [1], refs, [9] * 5, [7, 8], 2, 4)
    assert code == 0 and src == [4, -1] and dst == [0, -1] and extra == [1]
    assert table == [[0, 1], [0, -1], [0, 1]] and refs == [3, 2, 0, 0, 0] and ring == [2, 3, 4, 9, 9] and state == [0, 3]


def test_plain_rope_by_hand():
    x = torch.zeros((2, 1, 128), dtype=torch.float32)
    x[:, 0, 0], x[:, 0, 1], x[:, 0, 8], x[:, 0, 100] = 1.0, 2.0, 3.0, 7.0
    pos = torch.tensor([[1, 0], [5, 2]])
    freq = [math.pi / 2] * 8
    y, tol = H.plain_rope(x, pos, 0, freq, [0, 1] + [0] * 6, False)
    # token 0: pair 0 (elements 0, 8) a quarter turn, pair 1 (1, 9) five; token 1: none, and a half
    assert torch.allclose(y[0, 0, [0, 8, 1, 9, 100]], torch.tensor([-3.0, 1.0, 0.0, 2.0, 7.0], dtype=torch.float64), atol=1e-12)
    assert torch.allclose(y[1, 0, [0, 8, 1, 9]], torch.tensor([1.0, 3.0, -2.0, 0.0], dtype=torch.float64), atol=1e-12)
    assert float(tol[0, 0, 0]) > 0 and float(tol[0, 0, 100]) == 0
    y, _ = H.plain_rope(x, pos, 0, freq, [0] * 8, True)
    assert torch.allclose(y[0, 0, [0, 1, 8, 9]], torch.tensor([-2.0, 1.0, 0.0, 3.0], dtype=torch.float64), atol=1e-12)


def test_plain_verify_by_hand():
    p = torch.tensor([[[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]]])
    q = torch.tensor([[[0.25, 0.5, 0.25], [0.5, 0.5, 0.0]]])
    n = torch.tensor([2], dtype=torch.int32)

    def one(tokens, u, draft=q):
        (code, kept, check), = H.plain_verify(torch.tensor([tokens], dtype=torch.int32), n, p, draft, torch.tensor([u]))
        return code, kept, [x for x in range(3) if check(x)]
    assert one([0, 1], [0.9, 0.9, 0.6]) == (0, 2, [2])       # both stay; 0.6 lies in the third entry
    assert one([1, 1], [0.6, 0.9, 0.9]) == (0, 0, [0])       # 0.6 * 0.5 >= 0.25; only token 0 is above the draft
    assert one([0, 0], [0.9, 0.1, 0.2]) == (0, 1, [1])       # p is 0 there
    assert one([0, 0], [0.9, 0.1, 0.2], None) == (0, 0, [1])  # 0.9 >= 0.5: what is left is 0.25, 0.25 of tokens 1 and 2
    assert one([0, 3], [0.2, 0.1, 0.2], None)[:2] == (-5, 1)
    (code, kept, check), = H.plain_verify(torch.tensor([[0, 0]], dtype=torch.int32), n, p, None, None)
    assert (code, kept, check(1)) == (0, 1, True)
