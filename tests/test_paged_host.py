"""Argument checks of the paged cache's C entries that need no GPU, its ctypes mirror, and
the plain statement of the tables that the GPU tests compare with."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from tests import paged_helpers as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from semantic_paged_kv_head_gb300 import build
    build.build_lib()
    from semantic_paged_kv_head_gb300 import ice
    return ice


def _params(lib, **over):
    p = dict(d=128, n_kv_heads=8, n_q_heads=32, page_size=16, dtype=lib.ICE_BF16, max_requests=4, max_blocks=8,
             max_tokens=16, n_pages=64)
    p.update(over)
    return lib.ice_paged_params(**p)


@pytest.mark.parametrize("field,value,code", [
    ("d", 64, "UNSUPPORTED"), ("n_kv_heads", 0, "INVALID_ARG"), ("n_q_heads", 30, "INVALID_ARG"),
    ("n_q_heads", 4, "INVALID_ARG"), ("n_q_heads", 24, "UNSUPPORTED"), ("n_q_heads", 128, "UNSUPPORTED"),
    ("page_size", 0, "INVALID_ARG"), ("page_size", 65, "INVALID_ARG"), ("dtype", 7, "INVALID_ARG"),
    ("max_requests", 0, "INVALID_ARG"), ("max_requests", 8193, "INVALID_ARG"), ("max_blocks", 0, "INVALID_ARG"),
    ("max_blocks", (1 << 26) + 1, "INVALID_ARG"), ("max_tokens", 0, "INVALID_ARG"),
    ("max_tokens", (1 << 20) + 1, "INVALID_ARG"), ("n_pages", 0, "INVALID_ARG"), ("n_pages", 1 << 24, "UNSUPPORTED")])
def test_refused_parameters(lib, field, value, code):
    out = ctypes.c_void_p(1)
    p = _params(lib, **{field: value})
    assert lib.raw_library().ice_paged_create(ctypes.byref(p), ctypes.byref(out)) == getattr(lib, "ICE_ERR_" + code)
    assert out.value is None


def test_null_arguments(lib):
    raw, E = lib.raw_library(), lib.ICE_ERR_INVALID_ARG
    out = ctypes.c_void_p()
    assert raw.ice_paged_create(None, ctypes.byref(out)) == E
    assert raw.ice_paged_create(ctypes.byref(_params(lib)), None) == E
    assert raw.ice_paged_get_error(None, None) == E
    assert raw.ice_paged_tables(None, 1, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16, 1, None) == E
    assert raw.ice_paged_append(None, 1, 16, 1024, 16, 1024, 16, 16, 16, None) == E
    assert raw.ice_paged_attn(None, 1, 1, 16, 4096, 16, 16, 16, None, 0, 16, 16, 16, None) == E
    raw.ice_paged_destroy(None)  # a no-op


def test_struct_layout_matches_the_header(lib, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    cls = lib.ice_paged_params
    lines = ['#include <stdio.h>', '#include "ice.h"', "int main(void) {",
             'printf("size %zu\\n", sizeof(ice_paged_params));']
    lines += [f'printf("{f} %zu\\n", offsetof(ice_paged_params, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]) + "\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f, _ in cls._fields_:
        assert int(got[f]) == getattr(cls, f).offset, f


def test_plain_tables_by_hand():
    # P = 4, 6 pages, ring holding 5, 3, 1 from head 4; request 0 has page 2, request 1 pages 0 and 4
    table = [[2, -1, -1], [0, 4, -1]]
    code, lens, state, q0, slots, pos, table, ring = H.plain_tables(
        [3, 6], [3, -4], table, [1, -1, -1, -1, 5, 3], [4, 7], 5, 4)
    assert code == 0 and lens == [6, 2] and state == [5, 8] and q0 == [0, 3, 3]
    assert slots == [11, 20, 21, -1, -1] and pos == [3, 4, 5, 0, 0]
    assert table == [[2, 5, -1], [0, 4, -1]] and ring == [1, 4, -1, -1, 5, 3]


@pytest.mark.parametrize("field", ["d", "n_kv_heads", "n_q_heads", "page_size", "max_requests", "max_blocks", "max_tokens", "n_pages"])
def test_binding_refuses_sizes_that_do_not_fit(lib, field):
    """A size whose low bits would be a valid one."""
    sizes = dict(d=128, n_kv_heads=8, n_q_heads=32, page_size=16, max_requests=4, max_blocks=8, max_tokens=16, n_pages=64)
    sizes[field] += 1 << (64 if field == "n_pages" else 32)
    with pytest.raises(ValueError, match=field):
        lib.PagedCache(**sizes)


def test_binding_refuses_counts_that_do_not_fit(lib):
    pc = lib.PagedCache.__new__(lib.PagedCache)
    pc.params = _params(lib)
    lens = torch.zeros(1, dtype=torch.int32)
    for n in (1 << 32, -(1 << 31) - 1, -1):
        with pytest.raises(ValueError, match="n_slots"):
            pc.tables(lens, lens, lens, lens, lens, n)
    for n in (1 << 32, (1 << 32) + 5, 1 << 31):
        with pytest.raises(ValueError, match="prefix_len"):
            pc.attn(lens, lens, lens, lens, lens, lens, lens, n)


def test_debug_flags_need_a_handle(lib):
    assert lib.raw_library().ice_paged_debug_set_flags(None, 0) == lib.ICE_ERR_INVALID_ARG


SEARCH = r"""
#include <algorithm>
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "ice_paged_search.h"

static int bad = 0;
// Entry i of the list, with the index checked first.
static int at(const std::vector<int>& q, int i) {
    if (i < 0 || i >= (int)q.size()) { ++bad; return INT_MIN; }
    return q[i];
}
// The search of one row as the kernel makes it, 32 lanes in turn; the request found.
static int find(const std::vector<int>& q, int tok) {
    const int n = (int)q.size() - 1;
    ice::RowSearch f(n);
    for (int step = 0; f.open(); ++step) {
        unsigned le = 0;
        for (int lane = 0; lane < 32; ++lane)
            if (f.has_probe(lane) && at(q, f.probe(lane)) <= tok) le |= 1u << lane;
        f.narrow(le);
        if (f.lo < 0 || f.hi > n || f.lo >= f.hi || step > 4) { ++bad; return -1; }
    }
    at(q, f.lo), at(q, f.lo + 1);
    return f.lo;
}

int main() {
    unsigned long long x = 88172645463325252ull;
    auto rnd = [&](int m) { x ^= x << 13, x ^= x >> 7, x ^= x << 17; return (int)(x % (unsigned long long)m); };
    for (int n : {1, 2, 3, 31, 32, 33, 64, 65, 1000, 1024, 1025, 2047, 2500, 8191, 8192}) {
        // in order: a request of its own for every row, however many are empty
        std::vector<int> q(n + 1, 0);
        for (int r = 0; r < n; ++r) q[r + 1] = q[r] + (rnd(3) ? rnd(5) : 0);
        for (int r = 0; r < n; ++r)
            for (int t = q[r]; t < q[r + 1]; ++t)
                if (find(q, t) != r) ++bad;
        // out of order or out of range: some request, and no entry outside the list
        for (int kind = 0; kind < 7; ++kind)
            for (int rep = 0; rep < 40; ++rep) {
                std::vector<int> b = q;
                if (kind == 0) b[0] = 1 + rnd(1000);
                if (kind == 1) std::fill(b.begin(), b.end(), INT_MAX);
                if (kind == 2) std::fill(b.begin(), b.end(), INT_MIN);
                if (kind == 3) for (int& e : b) e = rnd(2 * n + 2) - n;
                if (kind == 4) std::reverse(b.begin(), b.end());
                if (kind == 5) b[rnd(n + 1)] = rnd(2) ? INT_MAX : INT_MIN;
                if (kind == 6) for (int& e : b) e = 1 + rnd(3);
                find(b, 0), find(b, rnd(4 * n + 1)), find(b, (1 << 20) - 1);
            }
    }
    std::printf("%d\n", bad);
    return bad != 0;
}
"""


def test_row_search_stays_in_the_list(tmp_path):
    """The joining kernel's search reads q_start before it is known to be in order: every index that it makes lies in the
    list for any contents, and it finds the right request of a list that is in order."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "search.cpp", tmp_path / "search"
    src.write_text(SEARCH)
    csrc = os.path.join(ROOT, "semantic_paged_kv_head_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", csrc, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_kernels_wait_before_they_read():
    """The paged kernels are launched before the kernels ahead of them have ended: what comes before the wait touches no
    buffer of the call."""
    csrc = os.path.join(ROOT, "semantic_paged_kv_head_gb300", "csrc")
    seen = []
    for name in ("ice_paged_attn.cu", "ice_paged_attn_tc.cu", "ice_paged_tables.cu"):
        text = open(os.path.join(csrc, name)).read()
        for m in re.finditer(r"__global__ void __\w+__\([^)]*\)\s*(\w+)\((.*?)\) \{", text, re.S):
            kernel, params = m.group(1), m.group(2)
            before = text[m.end():text.index("pdl_wait_then_release();", m.end())]
            assert "__global__" not in before, kernel
            before = re.sub(r"//[^\n]*", "", before)
            # PagedAttn's pointers, and pointer parameters
            pointers = [r"a\.\w+"] if "PagedAttn a" in params else re.findall(r"\*\s*(\w+)", params)
            for p in pointers:
                assert not re.search(r"\b" + p + r"\s*\[|\*\s*" + p + r"\b(?!\s*[\w(])", before), (kernel, p)
            seen.append(kernel)
    assert sorted(seen) == ["append_kernel", "paged_join_kernel", "paged_simt_kernel", "paged_tc_kernel", "tables_kernel"]
