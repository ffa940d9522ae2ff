"""ctypes binding of libice.so (the C ABI declared in include/ice.h).

Argument marshalling only: torch supplies device memory (or, for the decode-step
calls, page-locked CPU tensors that the kernels read and write in place) and the
current CUDA stream; every step of the decode path runs in the library's CUDA
kernels.
There is no CPU fallback. If libice.so is missing or cannot be loaded the
import of this module raises.

    from semantic_paged_kv_head_gb300 import ice
    ix = ice.IceIndex.build(keys, values, page_size=16, n_q_heads=32, n_composite=2)
    page_ids, n_pages = ix.select(q, token_budget=256)
    out = ix.sparse_attn(q, page_ids, n_pages)
    ix.insert(k_new, v_new)
"""
from __future__ import annotations

import ctypes
import operator
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libice.so")

ICE_OK = 0
ICE_ERR_INVALID_ARG = -1
ICE_ERR_CAPACITY = -2
ICE_ERR_CUDA = -3
ICE_ERR_TIMEOUT = -4
ICE_ERR_BOUNDS = -5
ICE_ERR_UNSUPPORTED = -6
ICE_F32 = 0
ICE_BF16 = 1

# every symbol include/ice.h declares
EXPORTS = ["ice_build", "ice_insert", "ice_select", "ice_select_attn", "ice_sparse_attn", "ice_get_error",
           "ice_destroy", "ice_status_string", "ice_get_info", "ice_debug_dump", "ice_debug_page",
           "ice_key_codes_noalloc", "ice_select_attn_reuse", "ice_reuse_reset",
           "ice_debug_set_flags", "ice_select_heads", "ice_decode_step", "ice_set_cluster_size",
           "ice_paged_create", "ice_paged_destroy", "ice_paged_get_error", "ice_paged_tables",
           "ice_paged_append", "ice_paged_attn", "ice_paged_debug_set_flags"]


class ice_params(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_proj", ctypes.c_int32), ("n_composite", ctypes.c_int32),
                ("n_cand", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("max_tokens", ctypes.c_int64), ("seed", ctypes.c_uint64),
                ("kv_location", ctypes.c_int32), ("dir_kind", ctypes.c_int32)]


DIR_RADEMACHER, DIR_GAUSSIAN = 0, 1  # ice_params.dir_kind
KV_DEVICE, KV_HOST = 0, 1  # ice_params.kv_location
DEBUG_STALL_ATTN = 1       # ice_debug_set_flags


class ice_info(ctypes.Structure):
    _fields_ = [("n_units", ctypes.c_int64), ("n_tokens", ctypes.c_int64),
                ("max_tokens", ctypes.c_int64), ("list_capacity", ctypes.c_int64),
                ("pool_bytes", ctypes.c_int64), ("group", ctypes.c_int32),
                ("n_composite", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("host_bytes", ctypes.c_int64),
                ("kv_location", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ice_paged_params(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("max_requests", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("n_pages", ctypes.c_int64)]


class IceError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})" if what else status_string(code))


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libice.so and declare the signatures of include/ice.h."""
    if not os.path.exists(path):
        raise ImportError(f"libice.so not built ({path}); run semantic_paged_kv_head_gb300/build.py")
    lib = ctypes.CDLL(path)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    P = ctypes.POINTER
    lib.ice_build.argtypes = [P(ice_params), vp, vp, i64, vp, P(vp)]
    lib.ice_build.restype = ctypes.c_int
    lib.ice_insert.argtypes = [vp, vp, vp, vp]
    lib.ice_insert.restype = ctypes.c_int
    lib.ice_select.argtypes = [vp, vp, i32, vp, vp, vp, vp]
    lib.ice_select.restype = ctypes.c_int
    lib.ice_select_attn.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp]
    lib.ice_select_attn.restype = ctypes.c_int
    lib.ice_sparse_attn.argtypes = [vp, vp, vp, vp, i32, vp, vp]
    lib.ice_sparse_attn.restype = ctypes.c_int
    lib.ice_get_error.argtypes = [vp, vp]
    lib.ice_get_error.restype = ctypes.c_int
    lib.ice_destroy.argtypes = [vp]
    lib.ice_destroy.restype = None
    lib.ice_status_string.argtypes = [ctypes.c_int]
    lib.ice_status_string.restype = ctypes.c_char_p
    lib.ice_get_info.argtypes = [vp, P(ice_info)]
    lib.ice_get_info.restype = ctypes.c_int
    lib.ice_debug_dump.argtypes = [vp, i32, vp, i64, vp]
    lib.ice_debug_dump.restype = i64
    lib.ice_debug_page.argtypes = [vp, i32, i32, vp, vp, vp]
    lib.ice_debug_page.restype = ctypes.c_int
    lib.ice_key_codes_noalloc.argtypes = [P(ice_params), vp, i64, vp, vp, vp]
    lib.ice_key_codes_noalloc.restype = ctypes.c_int
    lib.ice_select_attn_reuse.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp]
    lib.ice_select_attn_reuse.restype = ctypes.c_int
    lib.ice_reuse_reset.argtypes = [vp, vp]
    lib.ice_reuse_reset.restype = ctypes.c_int
    lib.ice_decode_step.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp]
    lib.ice_decode_step.restype = ctypes.c_int
    lib.ice_select_heads.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp]
    lib.ice_select_heads.restype = ctypes.c_int
    lib.ice_debug_set_flags.argtypes = [vp, i32]
    lib.ice_debug_set_flags.restype = ctypes.c_int
    lib.ice_set_cluster_size.argtypes = [vp, i32]
    lib.ice_set_cluster_size.restype = ctypes.c_int
    lib.ice_paged_create.argtypes = [P(ice_paged_params), P(vp)]
    lib.ice_paged_create.restype = ctypes.c_int
    lib.ice_paged_destroy.argtypes = [vp]
    lib.ice_paged_destroy.restype = None
    lib.ice_paged_get_error.argtypes = [vp, vp]
    lib.ice_paged_get_error.restype = ctypes.c_int
    lib.ice_paged_tables.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp]
    lib.ice_paged_tables.restype = ctypes.c_int
    lib.ice_paged_append.argtypes = [vp, i32, vp, i64, vp, i64, vp, vp, vp, vp]
    lib.ice_paged_append.restype = ctypes.c_int
    lib.ice_paged_attn.argtypes = [vp, i32, i32, vp, i64, vp, vp, vp, vp, i32, vp, vp, vp, vp]
    lib.ice_paged_attn.restype = ctypes.c_int
    lib.ice_paged_debug_set_flags.argtypes = [vp, i32]
    lib.ice_paged_debug_set_flags.restype = ctypes.c_int
    return lib


_lib = load_library()


def status_string(code: int) -> str:
    return _lib.ice_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != ICE_OK:
        raise IceError(code, what)


# the current stream's handle without a Stream object around it (0.1 against 2.9 us a call)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _dev_ptr(t: torch.Tensor, dtype=None, name="tensor", host_ok=True) -> int:
    """Address of a buffer argument: a CUDA tensor or, where the call allows it,
    a page-locked CPU tensor that the kernels read or write in place."""
    ok = isinstance(t, torch.Tensor) and (
        t.is_cuda or (host_ok and t.device.type == "cpu" and t.is_pinned()))
    if not ok:
        raise ValueError(f"{name} must be a CUDA tensor" + (" or page-locked CPU tensor" if host_ok else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _like(t: torch.Tensor) -> torch.Tensor:
    """An uninitialised buffer like t, page-locked when t is a CPU tensor."""
    if t.is_cuda:
        return torch.empty_like(t)
    return torch.empty(t.shape, dtype=t.dtype, pin_memory=True)


def _code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return ICE_BF16
    if dtype == torch.float32:
        return ICE_F32
    raise ValueError(f"unsupported dtype {dtype}")


class IceIndex:
    """Owner of one ice_index handle (all units of a batch x layers x KV heads grid)."""

    def __init__(self, handle: int, params: ice_params, dtype: torch.dtype):
        self._h = ctypes.c_void_p(handle)
        self.params = params
        self.dtype = dtype

    # -- the four calls ------------------------------------------------------------
    @classmethod
    def build(cls, keys: torch.Tensor, values: torch.Tensor, *, page_size: int, n_q_heads: int,
              n_composite: int = 2, n_proj: int = 8, n_cand: int = 0, max_tokens: int | None = None,
              seed: int = 0, kv_host: bool = False, dir_kind: int = 0, stream=None) -> "IceIndex":
        """ice_build over keys/values shaped [batch, layers, kv_heads, n, d].

        kv_host places the page pool in pinned host memory (ICE_KV_HOST)."""
        if keys.dim() != 5 or keys.shape != values.shape:
            raise ValueError("keys/values must be [batch, layers, kv_heads, n, d] and equal in shape")
        B, Ly, H, n, d = keys.shape
        p = ice_params(d=d, n_kv_heads=H, n_q_heads=n_q_heads, n_layers=Ly, batch=B,
                       page_size=page_size, n_proj=n_proj, n_composite=n_composite, n_cand=n_cand,
                       dtype=_code(keys.dtype), max_tokens=n if max_tokens is None else max_tokens,
                       seed=seed, kv_location=KV_HOST if kv_host else KV_DEVICE, dir_kind=dir_kind)
        h = ctypes.c_void_p()
        kp = _dev_ptr(keys, values.dtype, "keys", host_ok=False) if n else 0
        vp = _dev_ptr(values, keys.dtype, "values", host_ok=False) if n else 0
        _check(_lib.ice_build(ctypes.byref(p), kp, vp, n, _stream(stream), ctypes.byref(h)),
               "ice_build")
        return cls(h.value, p, keys.dtype)

    def insert(self, k: torch.Tensor, v: torch.Tensor, stream=None):
        """ice_insert of one token per unit, k/v shaped [batch, layers, kv_heads, d]."""
        _check(_lib.ice_insert(self._h, _dev_ptr(k, self.dtype, "k"), _dev_ptr(v, self.dtype, "v"),
                               _stream(stream)), "ice_insert")

    def select(self, q: torch.Tensor, token_budget: int, page_ids: torch.Tensor | None = None,
               n_pages: torch.Tensor | None = None, stats: torch.Tensor | None = None, stream=None):
        """ice_select; returns (page_ids [units, n_sel] int32, n_pages [units] int32)."""
        U = self.n_units
        n_sel = token_budget // self.params.page_size
        dev = q.device if q.is_cuda else torch.device("cuda")  # q may be page-locked host memory
        if page_ids is None:
            page_ids = torch.empty((U, n_sel), dtype=torch.int32, device=dev)
        if n_pages is None:
            n_pages = torch.empty((U,), dtype=torch.int32, device=dev)
        sp = _dev_ptr(stats, torch.int32, "stats") if stats is not None else None
        _check(_lib.ice_select(self._h, _dev_ptr(q, self.dtype, "q"), int(token_budget),
                               _dev_ptr(page_ids, torch.int32, "page_ids"),
                               _dev_ptr(n_pages, torch.int32, "n_pages"), sp, _stream(stream)),
               "ice_select")
        return page_ids, n_pages

    def select_attn(self, q: torch.Tensor, token_budget: int, out: torch.Tensor | None = None,
                    page_ids: torch.Tensor | None = None, n_pages: torch.Tensor | None = None,
                    stats: torch.Tensor | None = None, stream=None):
        """ice_select_attn; returns (out, page_ids, n_pages)."""
        U = self.n_units
        n_sel = token_budget // self.params.page_size
        dev = q.device if q.is_cuda else torch.device("cuda")  # q may be page-locked host memory
        if page_ids is None:
            page_ids = torch.empty((U, n_sel), dtype=torch.int32, device=dev)
        if n_pages is None:
            n_pages = torch.empty((U,), dtype=torch.int32, device=dev)
        if out is None:
            out = _like(q)
        sp = _dev_ptr(stats, torch.int32, "stats") if stats is not None else None
        _check(_lib.ice_select_attn(self._h, _dev_ptr(q, self.dtype, "q"), int(token_budget),
                                    _dev_ptr(page_ids, torch.int32, "page_ids"),
                                    _dev_ptr(n_pages, torch.int32, "n_pages"), sp,
                                    _dev_ptr(out, self.dtype, "out"), _stream(stream)),
               "ice_select_attn")
        return out, page_ids, n_pages

    def select_attn_reuse(self, q: torch.Tensor, token_budget: int, r: int, page_ids: torch.Tensor,
                          n_pages: torch.Tensor, out: torch.Tensor | None = None,
                          reselected: torch.Tensor | None = None, stream=None):
        """ice_select_attn_reuse; page_ids/n_pages carry the selection between calls
        (pass the same tensors every step). Returns (out, page_ids, n_pages)."""
        if out is None:
            out = _like(q)
        _check(_lib.ice_select_attn_reuse(self._h, _dev_ptr(q, self.dtype, "q"), int(token_budget),
                                          int(r), _dev_ptr(page_ids, torch.int32, "page_ids"),
                                          _dev_ptr(n_pages, torch.int32, "n_pages"),
                                          (_dev_ptr(reselected, torch.int32, "reselected")
                                           if reselected is not None else None),
                                          _dev_ptr(out, self.dtype, "out"), _stream(stream)),
               "ice_select_attn_reuse")
        return out, page_ids, n_pages

    def debug_set_flags(self, flags: int):
        """ice_debug_set_flags (tests only): DEBUG_STALL_ATTN forces the fused call's
        bounded wait to run out."""
        _check(_lib.ice_debug_set_flags(self._h, int(flags)), "ice_debug_set_flags")

    def set_cluster_size(self, k: int):
        """ice_set_cluster_size: blocks per unit of the selection (0 automatic, 1, 2,
        4, 8 or 16)."""
        _check(_lib.ice_set_cluster_size(self._h, int(k)), "ice_set_cluster_size")

    def decode_step(self, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, token_budget: int,
                    page_ids: torch.Tensor, n_pages: torch.Tensor, out: torch.Tensor, stream=None):
        """ice_decode_step: insert (k, v) into every unit, then select + attend for q.
        Capturable in a CUDA graph (all buffers preallocated by the caller)."""
        _check(_lib.ice_decode_step(self._h, _dev_ptr(k, self.dtype, "k"), _dev_ptr(v, self.dtype, "v"),
                                    _dev_ptr(q, self.dtype, "q"), int(token_budget),
                                    _dev_ptr(page_ids, torch.int32, "page_ids"),
                                    _dev_ptr(n_pages, torch.int32, "n_pages"),
                                    _dev_ptr(out, self.dtype, "out"), _stream(stream)),
               "ice_decode_step")
        return out

    def select_heads(self, q: torch.Tensor, token_budget: int, stream=None):
        """ice_select_heads; returns (page_ids [units, G*n_sel] union, n_pages [units],
        head_page_ids [units, G, n_sel], head_n_pages [units, G])."""
        U, G = self.n_units, self.params.n_q_heads // self.params.n_kv_heads
        n_sel = token_budget // self.params.page_size
        dev = q.device if q.is_cuda else torch.device("cuda")
        hid = torch.empty((U, G, n_sel), dtype=torch.int32, device=dev)
        hn = torch.empty((U, G), dtype=torch.int32, device=dev)
        ids = torch.empty((U, G * n_sel), dtype=torch.int32, device=dev)
        n = torch.empty((U,), dtype=torch.int32, device=dev)
        _check(_lib.ice_select_heads(self._h, _dev_ptr(q, self.dtype, "q"), int(token_budget),
                                     hid.data_ptr(), hn.data_ptr(), ids.data_ptr(), n.data_ptr(),
                                     _stream(stream)), "ice_select_heads")
        return ids, n, hid, hn

    def reuse_reset(self, stream=None):
        _check(_lib.ice_reuse_reset(self._h, _stream(stream)), "ice_reuse_reset")

    def sparse_attn(self, q: torch.Tensor, page_ids: torch.Tensor, n_pages: torch.Tensor,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """ice_sparse_attn; returns out shaped like q."""
        if out is None:
            out = _like(q)
        _check(_lib.ice_sparse_attn(self._h, _dev_ptr(q, self.dtype, "q"),
                                    _dev_ptr(page_ids, torch.int32, "page_ids"),
                                    _dev_ptr(n_pages, torch.int32, "n_pages"),
                                    int(page_ids.shape[-1]), _dev_ptr(out, self.dtype, "out"),
                                    _stream(stream)), "ice_sparse_attn")
        return out

    # -- status, info, teardown ---------------------------------------------------------
    def get_error(self, stream=None) -> int:
        return int(_lib.ice_get_error(self._h, _stream(stream)))

    def check(self, stream=None):
        _check(self.get_error(stream), "device status")

    def info(self) -> ice_info:
        inf = ice_info()
        _check(_lib.ice_get_info(self._h, ctypes.byref(inf)), "ice_get_info")
        return inf

    @property
    def n_units(self) -> int:
        p = self.params
        return p.batch * p.n_layers * p.n_kv_heads

    def destroy(self):
        if self._h and self._h.value:
            _lib.ice_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    # -- debug views --------------------------------------------------------------------
    def dump(self, unit: int, stream=None) -> dict:
        """Decoded ice_debug_dump of one unit (see include/ice.h for the layout)."""
        need = int(_lib.ice_debug_dump(self._h, unit, None, 0, _stream(stream)))
        if need < 0:
            raise IceError(need, "ice_debug_dump")
        buf = np.zeros(need, dtype=np.uint8)
        _check(int(_lib.ice_debug_dump(self._h, unit, buf.ctypes.data, need, _stream(stream))),
               "ice_debug_dump")
        hdr = buf[:128].view(np.int64)
        L, P, C, n, e = (int(x) for x in hdr[:5])
        out = {"L": L, "P": P, "C": C, "n": n, "e": e, "n_leaf": hdr[5:5 + L].tolist(),
               "next_id": hdr[9:9 + L].tolist(), "comp": []}
        o = 128
        for _ in range(L):
            lk = buf[o:o + C * 16].view(np.uint32).reshape(C, 4)
            o += C * 16
            rec = buf[o:o + C * 16].reshape(C, 16)
            o += C * 16
            meta = rec[:, 8:12].copy().view(np.uint32).reshape(C)
            lo = rec[:, :8].astype(np.int32)
            t = lk[:, 3].astype(np.int32)
            # known bits of code j at prefix length t (Morton order, code j at bit j of each byte)
            jj = np.arange(8)[None, :]
            bj = np.where(t[:, None] >= 64, 8, np.clip((t[:, None] + 7 - jj) >> 3, 0, 8))
            hi = lo | ((1 << (8 - bj)) - 1)
            rec_t = rec[:, 12:16].copy().view(np.uint32).reshape(C).astype(np.int32)
            cnt = buf[o:o + C * 4].view(np.int32)
            o += C * 4
            stok = buf[o:o + C * P * 4].view(np.int32).reshape(C, P)
            o += C * P * 4
            skey = buf[o:o + C * P * 8].view(np.uint64).reshape(C, P)
            o += C * P * 8
            pm = lk[:, 0].astype(np.uint64) | (lk[:, 1].astype(np.uint64) << np.uint64(32))
            out["comp"].append({"pm": pm, "pt": lk[:, 2].copy(), "t": t, "rec_t": rec_t,
                                "lo": lo, "hi": hi,
                                "id": (meta >> 8).astype(np.int32), "cnt": (meta & 0xFF).astype(np.int32),
                                "list_cnt": cnt.copy(), "slot_tok": stok.copy(), "slot_key": skey.copy()})
        mt = self.info().max_tokens
        out["tok_loc"] = buf[o:o + 4 * mt].view(np.int32).copy()
        o += 4 * mt
        if L > 1:
            out["slot_loc1"] = buf[o:o + C * P * 4].view(np.int32).reshape(C, P).copy()
            o += C * P * 4
            out["tok_slot1"] = buf[o:o + 4 * mt].view(np.int32).copy()
        return out

    def page(self, unit: int, page_id: int, stream=None):
        """K and V rows of one page as torch CPU tensors [P, d]."""
        P, d = self.params.page_size, self.params.d
        hk = torch.empty((P, d), dtype=self.dtype)
        hv = torch.empty((P, d), dtype=self.dtype)
        _check(_lib.ice_debug_page(self._h, unit, page_id, hk.data_ptr(), hv.data_ptr(),
                                   _stream(stream)), "ice_debug_page")
        return hk, hv


def _int(x, name: str, bits: int = 32) -> int:
    """x as a C integer argument; ctypes would cut a larger number to its low bits."""
    x = operator.index(x)
    if not -(1 << (bits - 1)) <= x < 1 << (bits - 1):
        raise ValueError(f"{name} = {x} does not fit {bits} bits")
    return x


class PagedCache:
    """The plain paged cache of a batch whose requests share a prefix (an ice_paged
    handle: geometry, scratch and status word; the pages and tables are the caller's
    tensors). One step, for each layer the last two calls:

        seq_len, state, q_start, slots, pos = pc.tables(seq_len, n_new, table, ring, state, n)
        pc.append(k, v, slots, k_pages, v_pages)
        out = pc.attn(q, q_start, seq_len, table, k_pages, v_pages, prefix_table, prefix_len)
    """

    def __init__(self, *, n_kv_heads: int, n_q_heads: int, page_size: int, n_pages: int,
                 max_requests: int, max_blocks: int, max_tokens: int,
                 dtype: torch.dtype = torch.bfloat16, d: int = 128):
        sizes = dict(d=d, n_kv_heads=n_kv_heads, n_q_heads=n_q_heads, page_size=page_size,
                     max_requests=max_requests, max_blocks=max_blocks, max_tokens=max_tokens)
        self.params = ice_paged_params(dtype=_code(dtype), n_pages=_int(n_pages, "n_pages", 64),
                                       **{k: _int(x, k) for k, x in sizes.items()})
        self.dtype = dtype
        self._h = ctypes.c_void_p()
        self.device = torch.device("cuda", torch.cuda.current_device())
        _check(_lib.ice_paged_create(ctypes.byref(self.params), ctypes.byref(self._h)),
               "ice_paged_create")
        self._page_shape = (n_pages, n_kv_heads, page_size, d)

    # -- tensors of the shapes that the calls take -----------------------------------
    def new_pages(self):
        """(k_pages, v_pages) of one layer, uninitialised."""
        return (torch.empty(self._page_shape, dtype=self.dtype, device=self.device),
                torch.empty(self._page_shape, dtype=self.dtype, device=self.device))

    def new_tables(self, n_req: int):
        """(seq_len, block_table, free_pages, free_state) of n_req empty requests and a pool
        whose pages are all free."""
        n_pages = self.params.n_pages
        return (torch.zeros((n_req,), dtype=torch.int32, device=self.device),
                torch.full((n_req, self.params.max_blocks), -1, dtype=torch.int32, device=self.device),
                torch.arange(n_pages, dtype=torch.int32, device=self.device),
                torch.tensor([0, n_pages], dtype=torch.int64, device=self.device))

    # -- checks ------------------------------------------------------------------------
    @staticmethod
    def _count(t, name):
        """Entries of a list."""
        try:
            n, = t.shape
        except (AttributeError, ValueError):
            raise ValueError(f"{name} must be a CUDA tensor of one dimension") from None
        return n

    def _ints(self, t, dtype, shape, name):
        try:
            if t.shape == shape and t.dtype is dtype and t.is_cuda and t.is_contiguous():
                return t.data_ptr()
        except AttributeError:
            raise ValueError(f"{name} must be a CUDA tensor") from None
        if t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        return _dev_ptr(t, dtype, name, host_ok=False)

    def _rows(self, t, heads, name):
        """Pointer and token stride of [tokens, heads, d] whose rows of heads are contiguous."""
        d = self.params.d
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != self.dtype:
            raise ValueError(f"{name} must be {self.dtype}, got {t.dtype}")
        if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
            raise ValueError(f"{name} must be [tokens, {heads}, {d}], got {tuple(t.shape)}")
        stride, head, one = t.stride()
        if one != 1 or (head != d and heads > 1):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        return t.data_ptr(), stride if t.shape[0] > 1 else heads * d

    def _pages(self, k_pages, v_pages):
        return (self._ints(k_pages, self.dtype, self._page_shape, "k_pages"),
                self._ints(v_pages, self.dtype, self._page_shape, "v_pages"))

    # -- the three calls -----------------------------------------------------------------
    def tables(self, seq_len: torch.Tensor, n_new: torch.Tensor, block_table: torch.Tensor,
               free_pages: torch.Tensor, free_state: torch.Tensor, n_slots: int,
               seq_len_out: torch.Tensor | None = None, free_state_out: torch.Tensor | None = None,
               q_start: torch.Tensor | None = None, slot_map: torch.Tensor | None = None,
               positions: torch.Tensor | None = None, stream=None):
        """ice_paged_tables; returns (seq_len_out, free_state_out, q_start, slot_map, positions).

        block_table and free_pages are updated in place; seq_len_out and free_state_out may
        be seq_len and free_state. n_slots: room for new tokens (entries behind the last
        are -1 in slot_map)."""
        if stream is not None:  # what is allocated here belongs to the stream that writes it
            with torch.cuda.stream(stream):
                return self.tables(seq_len, n_new, block_table, free_pages, free_state, n_slots, seq_len_out,
                                   free_state_out, q_start, slot_map, positions)
        if not 0 <= n_slots <= 1 << 30:
            raise ValueError(f"n_slots = {n_slots} must be from 0 to 2^30")
        n, i32, i64, check = self._count(seq_len, "seq_len"), torch.int32, torch.int64, self._ints
        ins = (check(seq_len, i32, (n,), "seq_len"), check(n_new, i32, (n,), "n_new"),
               check(block_table, i32, (n, self.params.max_blocks), "block_table"),
               check(free_pages, i32, (self.params.n_pages,), "free_pages"),
               check(free_state, i64, (2,), "free_state"))
        dev, outs = self.device, []
        for t, dtype, shape, name in ((seq_len_out, i32, (n,), "seq_len_out"), (free_state_out, i64, (2,), "free_state_out"),
                                      (q_start, i32, (n + 1,), "q_start"), (slot_map, i64, (n_slots,), "slot_map"),
                                      (positions, i32, (n_slots,), "positions")):
            if t is None:
                t = torch.empty(shape, dtype=dtype, device=dev)
            else:
                check(t, dtype, shape, name)
            outs.append(t)
        _check(_lib.ice_paged_tables(self._h, n, *ins, *[t.data_ptr() for t in outs], n_slots, _stream()),
               "ice_paged_tables")
        return tuple(outs)

    def append(self, k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
               k_pages: torch.Tensor, v_pages: torch.Tensor, stream=None):
        """ice_paged_append of k, v [tokens, kv_heads, d] (a token stride is allowed)."""
        n = self._count(slot_map, "slot_map")
        kp, ks = self._rows(k, self.params.n_kv_heads, "k")
        vp, vs = self._rows(v, self.params.n_kv_heads, "v")
        if k.shape[0] != n or v.shape[0] != n:
            raise ValueError("k, v and slot_map must have as many tokens")
        kg, vg = self._pages(k_pages, v_pages)
        _check(_lib.ice_paged_append(self._h, n, kp, ks, vp, vs,
                                     self._ints(slot_map, torch.int64, (n,), "slot_map"), kg, vg,
                                     _stream(stream)), "ice_paged_append")

    def attn(self, q: torch.Tensor, q_start: torch.Tensor, seq_len: torch.Tensor,
             block_table: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
             prefix_table: torch.Tensor | None = None, prefix_len: int = 0,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """ice_paged_attn of q [tokens, q_heads, d] (a token stride is allowed); returns out,
        contiguous."""
        if stream is not None:  # what is allocated here belongs to the stream that writes it
            with torch.cuda.stream(stream):
                return self.attn(q, q_start, seq_len, block_table, k_pages, v_pages, prefix_table, prefix_len, out)
        p, n, prefix_len = self.params, self._count(seq_len, "seq_len"), _int(int(prefix_len), "prefix_len")
        qp, qs = self._rows(q, p.n_q_heads, "q")
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif not isinstance(out, torch.Tensor) or out.shape != q.shape:
            raise ValueError("out must be shaped like q")
        kg, vg = self._pages(k_pages, v_pages)
        pt = None
        if prefix_len:
            if not isinstance(prefix_table, torch.Tensor) or prefix_table.numel() * p.page_size < prefix_len:
                raise ValueError("prefix_table must hold the pages of prefix_len tokens")
            pt = _dev_ptr(prefix_table, torch.int32, "prefix_table", host_ok=False)
        _check(_lib.ice_paged_attn(
            self._h, n, q.shape[0], qp, qs, self._ints(q_start, torch.int32, (n + 1,), "q_start"),
            self._ints(seq_len, torch.int32, (n,), "seq_len"),
            self._ints(block_table, torch.int32, (n, p.max_blocks), "block_table"), pt, prefix_len,
            kg, vg, _dev_ptr(out, self.dtype, "out", host_ok=False), _stream()), "ice_paged_attn")
        return out

    # -- status, teardown ------------------------------------------------------------------
    def debug_set_flags(self, flags: int):
        """ice_paged_debug_set_flags (tests only): DEBUG_STALL_ATTN forces the bounded waits of a
        bf16 attn call to run out."""
        _check(_lib.ice_paged_debug_set_flags(self._h, int(flags)), "ice_paged_debug_set_flags")

    def get_error(self, stream=None) -> int:
        return int(_lib.ice_paged_get_error(self._h, _stream(stream)))

    def check(self, stream=None):
        _check(self.get_error(stream), "device status")

    def destroy(self):
        if self._h and self._h.value:
            _lib.ice_paged_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def key_codes_noalloc(keys: torch.Tensor, *, n_composite: int = 2, n_proj: int = 8, seed: int = 0,
                      morton_out: torch.Tensor | None = None, e_out: torch.Tensor | None = None,
                      stream=None):
    """ice_key_codes_noalloc on keys [batch, layers, kv_heads, n, d].

    Returns (morton [n_composite, units, n] as int64 bit patterns, e [units]).
    Pass preallocated outputs to keep the call free of allocations."""
    B, Ly, H, n, d = keys.shape
    U = B * Ly * H
    p = ice_params(d=d, n_kv_heads=H, n_q_heads=H, n_layers=Ly, batch=B, page_size=1,
                   n_proj=n_proj, n_composite=n_composite, n_cand=0, dtype=_code(keys.dtype),
                   max_tokens=n, seed=seed)
    if morton_out is None:
        morton_out = torch.empty((n_composite, U, n), dtype=torch.int64, device=keys.device)
    if e_out is None:
        e_out = torch.empty((U,), dtype=torch.int32, device=keys.device)
    _check(_lib.ice_key_codes_noalloc(ctypes.byref(p), _dev_ptr(keys, None, "keys", host_ok=False), n,
                                      _dev_ptr(morton_out, torch.int64, "morton_out", host_ok=False),
                                      _dev_ptr(e_out, torch.int32, "e_out", host_ok=False),
                                      _stream(stream)),
           "ice_key_codes_noalloc")
    return morton_out, e_out


def raw_library() -> ctypes.CDLL:
    """The loaded libice.so (for tests that call the C ABI directly)."""
    return _lib
