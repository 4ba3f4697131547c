"""Python binding of libzha (the C ABI in include/zha.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels. Tensors are torch CUDA tensors (PyTorch supplies device memory
and streams); their data pointers and the current stream are handed to the C
calls. Importing this module raises if libzha.so has not been built -- there is
no fallback implementation.
"""

from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, byref, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_uint64, c_void_p

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libzha.so")

ZHA_OK = 0
ZHA_ERR_INVALID = -1
ZHA_ERR_CAPACITY = -2
ZHA_ERR_STATE = -3
ZHA_ERR_CUDA = -4
ZHA_ERR_UNSUPPORTED = -6
ZHA_F32 = 0
ZHA_BF16 = 1
ZHA_DEV_SELECTION_TRUNCATED = 1
ZHA_DEV_BAD_SELECTION = 2
ZHA_DEV_TIMEOUT = 4
ZHA_DEV_BAD_PAGE = 8
ZHA_DEV_BAD_LENGTH = 16
ZHA_DEV_NO_PAGES = 32
ZHA_DEV_BAD_SEQUENCE = 64


class ZhaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


ZHA_SELECT_TOP_P = 0
ZHA_SELECT_TOP_K = 1


class RoutePolicy(ctypes.Structure):
    """zha_route_policy: per-level top-p masses or top-k budgets (level l at index l-1)."""
    _fields_ = [("mode", c_int32), ("reserved", c_int32), ("p", c_float * 8), ("k", c_int32 * 8)]


def top_p_policy(p_by_level) -> RoutePolicy:
    """Top-p with p_by_level[l-1] at level l (a sequence of up to 8 masses)."""
    pol = RoutePolicy()
    pol.mode = ZHA_SELECT_TOP_P
    for i, v in enumerate(p_by_level):
        pol.p[i] = float(v)
    return pol


def top_k_policy(k_by_level) -> RoutePolicy:
    """Fixed-budget top-K with k_by_level[l-1] nodes kept at level l."""
    pol = RoutePolicy()
    pol.mode = ZHA_SELECT_TOP_K
    for i, v in enumerate(k_by_level):
        pol.k[i] = int(v)
    return pol


_DTYPE = {torch.float32: ZHA_F32, torch.bfloat16: ZHA_BF16}


class KvCache(ctypes.Structure):
    """zha_kv_cache: a contiguous [Hkv, ld, d] cache, or page pools [n_pages, C, d]
    with a block table [Hkv, max_blocks] (int32 page ids)."""
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("ld", c_int64), ("block_table", c_void_p),
                ("max_blocks", c_int64)]


def _some(block_table: torch.Tensor) -> None:
    """A table without entries has no address, and a cache without a table is a contiguous one."""
    if block_table.numel() == 0:
        raise ValueError("block_table must have at least one entry per sequence and KV head")


def kv_cache(K: torch.Tensor, V: torch.Tensor | None = None,
             block_table: torch.Tensor | None = None) -> KvCache:
    """A zha_kv_cache over torch tensors: contiguous when block_table is None
    (K [Hkv, ld, d]), else page pools K, V [n_pages, C, d] and block_table
    [Hkv, max_blocks] int32."""
    c = KvCache()
    c.k = K.data_ptr()
    c.v = V.data_ptr() if V is not None else None
    c.ld = K.shape[0] if block_table is not None else K.shape[1]
    if block_table is not None:
        if not (block_table.is_cuda and block_table.dtype == torch.int32 and block_table.is_contiguous()):
            raise ValueError("block_table must be a contiguous int32 CUDA tensor [Hkv, max_blocks]")
        _some(block_table)
        c.block_table = block_table.data_ptr()
        c.max_blocks = block_table.shape[1]
    return c


def kv_batch(K: torch.Tensor, V: torch.Tensor, block_table: torch.Tensor | None = None) -> KvCache:
    """A zha_kv_cache over the caches of a batch: contiguous K, V [n_seqs, Hkv, ld, d]
    when block_table is None, else page pools [n_pages, C, d] and block_table
    [n_seqs, Hkv, max_blocks] int32. It keeps the tensors alive."""
    for x in (K, V):
        if not (x.is_cuda and x.is_contiguous() and x.dim() == (4 if block_table is None else 3)):
            raise ValueError("caches must be contiguous CUDA tensors [n_seqs, Hkv, ld, d], or pools [n_pages, C, d]")
    if K.shape != V.shape or K.dtype != V.dtype or K.device != V.device:
        raise ValueError("K and V must have one shape, type and device")
    if K.dtype not in _DTYPE:
        raise ValueError("K and V must be float32 or bfloat16")
    c = KvCache()
    c.k, c.v = K.data_ptr(), V.data_ptr()
    c.ld = K.shape[2] if block_table is None else K.shape[0]
    if block_table is not None:
        if not (block_table.device == K.device and block_table.dtype == torch.int32
                and block_table.is_contiguous() and block_table.dim() == 3):
            raise ValueError("block_table must be a contiguous int32 CUDA tensor [n_seqs, Hkv, max_blocks]")
        _some(block_table)
        c.block_table = block_table.data_ptr()
        c.max_blocks = block_table.shape[2]
    # what the calls check a configuration against (not part of the C struct)
    c.tensors = (K, V, block_table)
    c.shape = tuple(K.shape)
    c.dtype = _DTYPE[K.dtype]
    c.seqs = K.shape[0] if block_table is None else block_table.shape[0]
    c.heads = K.shape[1] if block_table is None else block_table.shape[1]
    c.device, c.index = K.device, K.get_device()
    return c


class Rows(ctypes.Structure):
    """zha_rows: rows of one head each, with token and head strides in elements."""
    _fields_ = [("data", c_void_p), ("token_stride", c_int64), ("head_stride", c_int64)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("head_dim", c_int32), ("pairs", c_int32), ("layout", c_int32), ("scaling", c_int32),
                ("freq_dim", c_int32), ("reserved", c_int32), ("base", c_double), ("factor", c_double),
                ("original_tokens", c_double), ("low", c_double), ("high", c_double), ("amplitude", c_double)]


class RopeTable(ctypes.Structure):
    _fields_ = [("head_dim", c_int32), ("pairs", c_int32), ("layout", c_int32), ("amplitude", c_float),
                ("turn", c_uint64 * 64)]


class PagePool(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("n_pages", c_int64), ("block_table", c_void_p),
                ("max_blocks", c_int64), ("refs", c_void_p), ("n_seqs", c_int32), ("reserved", c_int32)]


class Config(ctypes.Structure):
    _fields_ = [
        ("n_kv_heads", c_int32), ("n_q_heads", c_int32), ("head_dim", c_int32),
        ("chunk", c_int32), ("levels", c_int32), ("n_ref", c_int32),
        ("kv_dtype", c_int32), ("rope_pairs", c_int32), ("max_tokens", c_int64),
        ("rope_base", c_float), ("reserved", c_int32),
    ]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m "
            "hierarchical_sparse_attention_zha_b200.build` (there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P = c_void_p
    sig = {
        "zha_abi_version": (c_int32, []),
        "zha_status_str": (c_char_p, [c_int32]),
        "zha_last_error": (c_char_p, []),
        "zha_launch_count": (c_uint64, []),
        "zha_tree_bytes": (c_size_t, [POINTER(Config)]),
        "zha_tree_create": (c_int32, [POINTER(Config), P, c_size_t, P, POINTER(P)]),
        "zha_tree_destroy": (None, [P]),
        "zha_tree_built_tokens": (c_int64, [P]),
        "zha_tree_level_layout": (c_int32, [P, c_int32, POINTER(c_int64), POINTER(c_int64),
                                            POINTER(c_int32)]),
        "zha_build": (c_int32, [P, P, c_int64, c_int64, P]),
        "zha_append_chunk": (c_int32, [P, P, c_int64, c_int64, P]),
        "zha_route_workspace_bytes": (c_size_t, [POINTER(Config), c_int32, c_int64]),
        "zha_route_kept_words": (c_size_t, [POINTER(Config), c_int32, c_int64]),
        "zha_route": (c_int32, [P, P, c_int32, c_int64, c_float, P, P, c_int32, P, P, c_size_t,
                                P, P]),
        "zha_route_noalloc": (c_int32, [P, P, c_int32, c_int64, c_float, P, P, c_int32, P, P, P]),
        "zha_route_ex": (c_int32, [P, P, c_int32, c_int64, POINTER(RoutePolicy), P, P, c_int32, P, P,
                                   c_size_t, P, P]),
        "zha_attend_workspace_bytes": (c_size_t, [POINTER(Config), c_int32, c_int64]),
        "zha_sparse_attend": (c_int32, [P, P, P, P, c_int64, c_int64, c_int32, P, P, c_int32, P,
                                        P, P, c_size_t, P, P]),
        "zha_build_kv": (c_int32, [P, POINTER(KvCache), c_int64, P]),
        "zha_append_chunk_kv": (c_int32, [P, POINTER(KvCache), c_int64, P]),
        "zha_sparse_attend_kv": (c_int32, [P, P, POINTER(KvCache), c_int64, c_int32, P, P, c_int32, P, P,
                                           P, c_size_t, P, P]),
        "zha_rope_init": (c_int32, [POINTER(RopeSpec), POINTER(RopeTable)]),
        "zha_rope_apply": (c_int32, [P, P, c_int32, P, c_int64, c_int32, c_int32, P, c_int32, P]),
        "zha_rope_append_kv": (c_int32, [P, P, P, P, P, c_int32, c_int64, P, c_int32, P, P, P, P, c_int32, P, P]),
        "zha_attend_batch_workspace_bytes": (c_size_t, [P, c_int32, c_int64]),
        "zha_attend_batch_kv": (c_int32, [P, P, c_int32, P, c_int32, P, c_int64, P, P, P, c_size_t, P, P]),
        "zha_pages_workspace_bytes": (c_size_t, [P, P, c_int32]),
        "zha_pages_extend": (c_int32, [P, P, P, P, c_int32, P, c_size_t, P, P]),
        "zha_pages_fork": (c_int32, [P, P, P, P, P, c_int32, P, c_size_t, P, P]),
        "zha_pages_free": (c_int32, [P, P, P, P, c_int32, P, P]),
        "zha_pages_compact": (c_int32, [P, P, P, P, P, c_size_t, P, P]),
        "zha_diagnostics_workspace_bytes": (c_size_t, [POINTER(Config), c_int32, c_int64]),
        "zha_route_diagnostics": (c_int32, [P, P, P, c_int64, c_int32, c_int64, P, P, P, c_size_t, P]),
        "zha_tree_debug": (c_int32, [P, ctypes.c_uint32, c_int32]),
        "zha_trace_enable": (c_int32, [c_int32, c_char_p, c_int32]),
        "zha_trace_count": (c_int32, []),
        "zha_trace_dropped": (c_int32, []),
        "zha_trace_read": (c_int32, [c_int32, POINTER(c_char_p), POINTER(c_int32), POINTER(c_float)]),
        "zha_trace_clear": (None, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def status_str(status: int) -> str:
    return lib.zha_status_str(status).decode()


def last_error() -> str:
    return lib.zha_last_error().decode()


def launch_count() -> int:
    return int(lib.zha_launch_count())


def check(status: int, what: str) -> None:
    if status != ZHA_OK:
        raise ZhaError(status, f"{what}: {status_str(status)}: {last_error()}")


def ptr(t: torch.Tensor | None):
    return None if t is None else c_void_p(t.data_ptr())


def stream_ptr(stream: torch.cuda.Stream | None = None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return c_void_p(s.cuda_stream)


def trace_enable(max_records: int, name_filter: str | None = None, tag_filter: int = -1) -> None:
    """Record CUDA events around the library's kernel launches (see zha.h)."""
    check(lib.zha_trace_enable(max_records, name_filter.encode() if name_filter else None, tag_filter),
          "zha_trace_enable")


def trace_records() -> list[tuple[str, int, float]]:
    """(kernel name, tag, device ms) of every recorded launch; synchronise first."""
    out = []
    for i in range(int(lib.zha_trace_count())):
        name, tag, ms = c_char_p(), c_int32(), c_float()
        check(lib.zha_trace_read(i, byref(name), byref(tag), byref(ms)), "zha_trace_read")
        out.append((name.value.decode(), int(tag.value), float(ms.value)))
    return out


def trace_dropped() -> int:
    return int(lib.zha_trace_dropped())


def trace_clear() -> None:
    lib.zha_trace_clear()


def make_config(n_kv_heads: int, n_q_heads: int, head_dim: int, chunk: int, levels: int,
                n_ref: int, kv_dtype: torch.dtype, max_tokens: int, rope_pairs: int = 0,
                rope_base: float = 10000.0) -> Config:
    """zha_config; rope_pairs > 0 declares rotary positions (see zha.h)."""
    dt = {torch.float32: ZHA_F32, torch.bfloat16: ZHA_BF16}[kv_dtype]
    return Config(n_kv_heads, n_q_heads, head_dim, chunk, levels, n_ref, dt, rope_pairs, max_tokens,
                  rope_base if rope_pairs > 0 else 0.0, 0)


def tree_bytes(cfg: Config) -> int:
    return int(lib.zha_tree_bytes(byref(cfg)))


def route_workspace_bytes(cfg: Config, batch: int, n_tokens: int) -> int:
    return int(lib.zha_route_workspace_bytes(byref(cfg), batch, n_tokens))


def route_kept_words(cfg: Config, batch: int, n_tokens: int) -> int:
    return int(lib.zha_route_kept_words(byref(cfg), batch, n_tokens))


def attend_workspace_bytes(cfg: Config, batch: int, n_tokens: int) -> int:
    return int(lib.zha_attend_workspace_bytes(byref(cfg), batch, n_tokens))


def _bytes_tensor(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(1, (nbytes + 255) // 256) * 64, dtype=torch.float32, device=device)


class Tree:
    """One summary store (all KV heads) plus its C handle.

    ``ref_q``: float32 CUDA tensor [n_kv_heads, n_ref, head_dim], kept alive here.
    """

    def __init__(self, cfg: Config, ref_q: torch.Tensor):
        if not (ref_q.is_cuda and ref_q.dtype == torch.float32 and ref_q.is_contiguous()):
            raise ValueError("ref_q must be a contiguous float32 CUDA tensor")
        if tuple(ref_q.shape) != (cfg.n_kv_heads, cfg.n_ref, cfg.head_dim):
            raise ValueError("ref_q shape does not match the config")
        self.cfg = cfg
        self.ref_q = ref_q
        self.device = ref_q.device
        nbytes = tree_bytes(cfg)
        if nbytes == 0:
            check(ZHA_ERR_INVALID, "zha_tree_bytes")
        self.store = _bytes_tensor(nbytes, self.device)
        handle = c_void_p()
        check(lib.zha_tree_create(byref(cfg), ptr(self.store), self.store.numel() * 4, ptr(ref_q),
                                  byref(handle)), "zha_tree_create")
        self.handle = handle

    def __del__(self):
        h = getattr(self, "handle", None)
        # (at interpreter exit the module's globals may already be gone)
        if h is not None and h.value and lib is not None:
            lib.zha_tree_destroy(h)
            self.handle = None

    @property
    def built_tokens(self) -> int:
        return int(lib.zha_tree_built_tokens(self.handle))

    def _kv(self, K: torch.Tensor) -> None:
        want = torch.float32 if self.cfg.kv_dtype == ZHA_F32 else torch.bfloat16
        if not (K.is_cuda and K.dtype == want and K.is_contiguous() and K.dim() == 3
                and K.shape[0] == self.cfg.n_kv_heads and K.shape[2] == self.cfg.head_dim):
            raise ValueError(f"cache must be a contiguous {want} CUDA tensor [Hkv, ld, d]")

    def build(self, K: torch.Tensor, n_tokens: int, stream=None) -> None:
        self._kv(K)
        check(lib.zha_build(self.handle, ptr(K), K.shape[1], n_tokens, stream_ptr(stream)),
              "zha_build")

    def append_chunk(self, K: torch.Tensor, n_tokens: int, stream=None) -> None:
        self._kv(K)
        check(lib.zha_append_chunk(self.handle, ptr(K), K.shape[1], n_tokens, stream_ptr(stream)),
              "zha_append_chunk")

    def build_kv(self, kv: KvCache, n_tokens: int, stream=None) -> None:
        """zha_build_kv over a zha_kv_cache (see kv_cache())."""
        check(lib.zha_build_kv(self.handle, byref(kv), n_tokens, stream_ptr(stream)), "zha_build_kv")

    def append_chunk_kv(self, kv: KvCache, n_tokens: int, stream=None) -> None:
        check(lib.zha_append_chunk_kv(self.handle, byref(kv), n_tokens, stream_ptr(stream)),
              "zha_append_chunk_kv")

    def sparse_attend_kv(self, Q: torch.Tensor, kv: KvCache, n_tokens: int, chunk_ids: torch.Tensor,
                         n_chunks: torch.Tensor, out: torch.Tensor | None = None,
                         lse: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                         status: torch.Tensor | None = None, stream=None):
        B = Q.shape[0]
        if out is None:
            out = torch.empty(B, self.cfg.n_q_heads, self.cfg.head_dim, dtype=torch.float32,
                              device=self.device)
        if lse is None:
            lse = torch.empty(B, self.cfg.n_q_heads, dtype=torch.float32, device=self.device)
        if ws is None:
            ws = _bytes_tensor(attend_workspace_bytes(self.cfg, B, n_tokens), self.device)
        check(lib.zha_sparse_attend_kv(self.handle, ptr(Q), byref(kv), n_tokens, B, ptr(chunk_ids),
                                       ptr(n_chunks), chunk_ids.shape[-1], ptr(out), ptr(lse), ptr(ws),
                                       ws.numel() * ws.element_size(), ptr(status), stream_ptr(stream)),
              "zha_sparse_attend_kv")
        return out, lse

    def level(self, level: int) -> tuple[torch.Tensor, torch.Tensor]:
        """Views of level `level`'s summaries: khat [Hkv, cap, R, d], bhat [Hkv, cap, R]."""
        off, cap, nf = c_int64(), c_int64(), c_int32()
        check(lib.zha_tree_level_layout(self.handle, level, byref(off), byref(cap), byref(nf)),
              "zha_tree_level_layout")
        H, R, d = self.cfg.n_kv_heads, self.cfg.n_ref, self.cfg.head_dim
        blk = self.store[off.value: off.value + H * cap.value * nf.value].view(H, cap.value, nf.value)
        return blk[:, :, : R * d].reshape(H, cap.value, R, d), blk[:, :, R * d: R * d + R]

    def route(self, Q: torch.Tensor, n_tokens: int, p: "float | RoutePolicy", max_sel: int,
              chunk_ids: torch.Tensor | None = None, n_chunks: torch.Tensor | None = None,
              kept_bits: torch.Tensor | None = None, ws: torch.Tensor | None = None,
              status: torch.Tensor | None = None, stream=None):
        B = Q.shape[0]
        if chunk_ids is None:
            chunk_ids = torch.empty(B, self.cfg.n_q_heads, max_sel, dtype=torch.int32, device=self.device)
        if n_chunks is None:
            n_chunks = torch.empty(B, self.cfg.n_q_heads, dtype=torch.int32, device=self.device)
        if ws is None:
            ws = _bytes_tensor(route_workspace_bytes(self.cfg, B, n_tokens), self.device)
        if isinstance(p, RoutePolicy):
            check(lib.zha_route_ex(self.handle, ptr(Q), B, n_tokens, byref(p), ptr(chunk_ids),
                                   ptr(n_chunks), max_sel, ptr(kept_bits), ptr(ws),
                                   ws.numel() * ws.element_size(), ptr(status), stream_ptr(stream)),
                  "zha_route_ex")
        else:
            check(lib.zha_route(self.handle, ptr(Q), B, n_tokens, p, ptr(chunk_ids), ptr(n_chunks),
                                max_sel, ptr(kept_bits), ptr(ws), ws.numel() * ws.element_size(),
                                ptr(status), stream_ptr(stream)), "zha_route")
        return chunk_ids, n_chunks

    def diagnostics(self, Q: torch.Tensor, K: torch.Tensor, n_tokens: int, usage: bool = True,
                    stream=None):
        """zha_route_diagnostics: (kl [L, B, Hq] float32, usage [L, R] int64 or None)."""
        self._kv(K)
        B = Q.shape[0]
        L = self.cfg.levels
        kl = torch.empty(L, B, self.cfg.n_q_heads, dtype=torch.float32, device=self.device)
        use = torch.zeros(L, self.cfg.n_ref, dtype=torch.int32, device=self.device) if usage else None
        ws = _bytes_tensor(int(lib.zha_diagnostics_workspace_bytes(byref(self.cfg), B, n_tokens)),
                           self.device)
        check(lib.zha_route_diagnostics(self.handle, ptr(Q), ptr(K), K.shape[1], B, n_tokens, ptr(kl),
                                        ptr(use), ptr(ws), ws.numel() * 4, stream_ptr(stream)),
              "zha_route_diagnostics")
        return kl, (use.to(torch.int64) if use is not None else None)

    def sparse_attend(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, n_tokens: int,
                      chunk_ids: torch.Tensor, n_chunks: torch.Tensor,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      ws: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      stream=None):
        self._kv(K)
        self._kv(V)
        B = Q.shape[0]
        if out is None:
            out = torch.empty(B, self.cfg.n_q_heads, self.cfg.head_dim, dtype=torch.float32,
                              device=self.device)
        if lse is None:
            lse = torch.empty(B, self.cfg.n_q_heads, dtype=torch.float32, device=self.device)
        if ws is None:
            ws = _bytes_tensor(attend_workspace_bytes(self.cfg, B, n_tokens), self.device)
        check(lib.zha_sparse_attend(self.handle, ptr(Q), ptr(K), ptr(V), K.shape[1], n_tokens, B,
                                    ptr(chunk_ids), ptr(n_chunks), chunk_ids.shape[-1], ptr(out),
                                    ptr(lse), ptr(ws), ws.numel() * ws.element_size(), ptr(status),
                                    stream_ptr(stream)), "zha_sparse_attend")
        return out, lse


# ---- Batches of caches -------------------------------------------------------
# The wrappers below check what the C calls cannot see (shapes, types, devices)
# and pass pointers; checks of values are the library's. Like all calls here they
# run on the current device's current stream unless given one.

def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


# A small call costs its time on the host, so the checks below are plain comparisons,
# devices are compared by number, and pointers go to C as integers.
_get_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _run_on(index: int, stream) -> int:
    """The stream of a call on tensors of device `index` (-1: not a GPU), which must be the
    current one. (torch.cuda.current_stream() makes an object of it, which takes 3 us.)"""
    if index < 0 or index != _get_device():
        raise ValueError("tensors must lie on the current CUDA device")
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """Memory for a call on `stream`, which is given back to that stream's later calls."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _status_ptr(status: torch.Tensor | None, index: int):
    if status is None:
        return None
    if status.dtype is not torch.int32 or status.get_device() != index or status.numel() < 1:
        raise ValueError("status must be an int32 tensor on the same device")
    return status.data_ptr()


def _scratch(ws: torch.Tensor, index: int) -> tuple[int, int]:
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the same device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _list_ptr(x: torch.Tensor, dtype, n: int, index: int, name: str) -> int:
    if x.dtype is not dtype or x.get_device() != index or x.dim() != 1 or x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor [{n}] on the same device")
    return x.data_ptr()


_three_rows = c_int64 * 9                        # zha_rows one behind the other


def _row_args(x: torch.Tensor, shape: tuple, index: int, name: str) -> tuple[int, int, int]:
    stride = x.stride()
    if x.shape != shape or x.get_device() != index or stride[2] != 1:
        raise ValueError(f"{name} must be {list(shape)} with rows of adjacent elements, on the same device")
    return x.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0


def _same_cache(cfg: Config, c, kind: type) -> None:
    """A configuration and a kv_batch() (kind KvCache) or page_pool() (kind PagePool) that
    describe one cache. The two have C structs of different sizes: one for the other is refused."""
    s = getattr(c, "shape", None)
    if s is None or not isinstance(c, kind):
        raise ValueError("the cache must come from " + ("kv_batch()" if kind is KvCache else "page_pool()"))
    if (c.heads != cfg.n_kv_heads or s[-1] != cfg.head_dim or c.dtype != cfg.kv_dtype
            or (len(s) == 3 and s[1] != cfg.chunk)):
        raise ValueError("the cache does not match the configuration")


class Rope:
    """A rotation (zha_rope_init): `layout` "interleaved" or "half", `scaling` "none",
    "linear", "ntk", "yarn" or "bands". pairs None: the whole head."""

    LAYOUTS = {"interleaved": 0, "half": 1}
    SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}

    def __init__(self, head_dim: int, pairs: int | None = None, layout: str = "interleaved",
                 base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_tokens: float = 0.0, low: float = 0.0, high: float = 0.0,
                 freq_dim: int = 0, amplitude: float = 0.0):
        _need(layout in self.LAYOUTS and scaling in self.SCALINGS, "unknown layout or scaling")
        spec = RopeSpec(head_dim, head_dim // 2 if pairs is None else pairs, self.LAYOUTS[layout],
                        self.SCALINGS[scaling], freq_dim, 0, base, factor, original_tokens, low, high, amplitude)
        self.table = RopeTable()
        check(lib.zha_rope_init(byref(spec), byref(self.table)), "zha_rope_init")
        self.at = ctypes.addressof(self.table)


def rope_apply(rope: Rope, x: torch.Tensor, pos: torch.Tensor, out: torch.Tensor | None = None,
               inverse: bool = False, stream=None) -> torch.Tensor:
    """zha_rope_apply: x [T, heads, d] (float32 or bf16, any token and head strides) turned
    at pos [T] int64, or turned back (the gradient's direction). `out` may be x."""
    shape, index, dtype = x.shape, x.get_device(), _DTYPE.get(x.dtype)
    if len(shape) != 3 or dtype is None or shape[2] != rope.table.head_dim:
        raise ValueError("x must be [T, heads, head_dim] of the rotation, float32 or bfloat16")
    on = _run_on(index, stream)
    if out is None:
        out = _new(shape, x.dtype, x.device, stream)
    to = _DTYPE.get(out.dtype)
    if to is None:
        raise ValueError("out must be float32 or bfloat16")
    T, H, _ = shape
    where = _list_ptr(pos, torch.int64, T, index, "pos")
    if T == 0 or H == 0:
        return out
    rows = _three_rows(*_row_args(x, shape, index, "x"), *_row_args(out, shape, index, "out"))
    at = ctypes.addressof(rows)
    st = lib.zha_rope_apply(rope.at, at, dtype, where, T, H, inverse, at + 24, to, on)
    if st:
        check(st, "zha_rope_apply")
    return out


def rope_append_kv(cfg: Config, rope: Rope | None, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                   kv: KvCache, n_seqs: int, seq: torch.Tensor, index: torch.Tensor,
                   pos: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                   q_dtype: torch.dtype = torch.float32, status: torch.Tensor | None = None, stream=None):
    """zha_rope_append_kv: k, v [T, Hkv, d] into the caches of kv_batch() at row index[t] of
    sequence seq[t], keys turned at pos (None: index); q [T, Hq, d] turned into q_out, which
    is returned (None without q). rope None: nothing is turned."""
    _same_cache(cfg, kv, KvCache)
    if not 1 <= n_seqs <= kv.seqs:
        raise ValueError("n_seqs is more than the caches hold")
    H, Hq, d, dev = cfg.n_kv_heads, cfg.n_q_heads, cfg.head_dim, kv.index
    T, dtype = k.shape[0], _DTYPE.get(k.dtype)
    on = _run_on(dev, stream)
    if dtype is None or v.dtype is not k.dtype or (q is not None and q.dtype is not k.dtype):
        raise ValueError("q, k and v must have one type, float32 or bfloat16")
    to, q_type, q_rows = None, ZHA_F32, (0, 0, 0)
    if q is not None:
        shape = (T, Hq, d)
        if q_out is None:
            q_out = _new(shape, q_dtype, kv.device, stream)
        q_type = _DTYPE.get(q_out.dtype)
        if q_type is None or q_out.shape != shape or q_out.get_device() != dev or not q_out.is_contiguous():
            raise ValueError(f"q_out must be a contiguous float32 or bfloat16 tensor {list(shape)}")
        to = q_out.data_ptr()
        q_rows = _row_args(q, shape, dev, "q")
    shape = (T, H, d)
    rows = _three_rows(*_row_args(k, shape, dev, "k"), *_row_args(v, shape, dev, "v"), *q_rows)
    at = ctypes.addressof(rows)
    st = lib.zha_rope_append_kv(
        byref(cfg), None if rope is None else rope.at, None if q is None else at + 48, at, at + 24, dtype, T, byref(kv),
        n_seqs, _list_ptr(seq, torch.int32, T, dev, "seq"), _list_ptr(index, torch.int64, T, dev, "index"),
        None if pos is None else _list_ptr(pos, torch.int64, T, dev, "pos"), to, q_type, _status_ptr(status, dev), on)
    if st:
        check(st, "zha_rope_append_kv")
    return None if q is None else q_out


def attend_batch_workspace_bytes(cfg: Config, n_seqs: int, max_tokens: int) -> int:
    return int(lib.zha_attend_batch_workspace_bytes(byref(cfg), n_seqs, max_tokens))


def attend_batch_kv(cfg: Config, Q: torch.Tensor, kv: KvCache, n_seqs: int, n_tokens: torch.Tensor, max_tokens: int,
                    out: torch.Tensor | None = None, lse: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, stream=None):
    """zha_attend_batch_kv: Q [n_seqs, Hq, d] (float32 or bf16) over the first n_tokens [n_seqs]
    (int64) tokens of each cache of kv_batch(); (out, lse), out of Q's type."""
    _same_cache(cfg, kv, KvCache)
    if not 1 <= n_seqs <= kv.seqs:
        raise ValueError("n_seqs is more than the caches hold")
    dev, dtype = kv.index, _DTYPE.get(Q.dtype)
    on = _run_on(dev, stream)
    want = (n_seqs, cfg.n_q_heads, cfg.head_dim)
    if dtype is None or Q.shape != want or Q.get_device() != dev or not Q.is_contiguous():
        raise ValueError(f"Q must be a contiguous float32 or bfloat16 tensor {list(want)} on the cache's device")
    if out is None:
        out = _new(want, Q.dtype, kv.device, stream)
    elif out.shape != want or out.dtype is not Q.dtype or out.get_device() != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of Q's shape and type")
    if lse is None:
        lse = _new(want[:2], torch.float32, kv.device, stream)
    elif lse.shape != want[:2] or lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [n_seqs, Hq]")
    if ws is None:
        ws = _new(max(1, attend_batch_workspace_bytes(cfg, n_seqs, max_tokens)), torch.uint8, kv.device, stream)
    st = lib.zha_attend_batch_kv(byref(cfg), Q.data_ptr(), dtype, byref(kv), n_seqs,
                                 _list_ptr(n_tokens, torch.int64, n_seqs, dev, "n_tokens"), max_tokens, out.data_ptr(),
                                 lse.data_ptr(), *_scratch(ws, dev), _status_ptr(status, dev), on)
    if st:
        check(st, "zha_attend_batch_kv")
    return out, lse


def page_pool(K: torch.Tensor, V: torch.Tensor, block_table: torch.Tensor, refs: torch.Tensor) -> PagePool:
    """A zha_page_pool over K, V [n_pages, C, d], block_table [n_seqs, Hkv, max_blocks] and refs
    [n_pages] (both int32). It keeps the tensors alive."""
    _need(block_table is not None, "a page pool needs a block table")
    kv = kv_batch(K, V, block_table)
    p = PagePool(kv.k, kv.v, kv.ld, kv.block_table, kv.max_blocks,
                 _list_ptr(refs, torch.int32, K.shape[0], K.get_device(), "refs"), block_table.shape[0], 0)
    p.tensors = (*kv.tensors, refs)
    p.shape, p.dtype, p.heads, p.seqs, p.device, p.index = (kv.shape, kv.dtype, kv.heads, kv.seqs,
                                                                   kv.device, kv.index)
    return p


def pages_workspace_bytes(cfg: Config, pool: PagePool, n_items: int) -> int:
    if not isinstance(pool, PagePool):
        raise ValueError("the pool must come from page_pool()")
    return int(lib.zha_pages_workspace_bytes(byref(cfg), byref(pool), n_items))


def pages_extend(cfg: Config, pool: PagePool, seqs: torch.Tensor, n_tokens: torch.Tensor,
                 ws: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> None:
    """zha_pages_extend: pages for the first n_tokens[i] (int64) tokens of sequence seqs[i] (int32)."""
    _same_cache(cfg, pool, PagePool)
    n, dev = seqs.numel(), pool.index
    on = _run_on(dev, stream)
    if ws is None:
        ws = _new(max(1, pages_workspace_bytes(cfg, pool, n)), torch.uint8, pool.device, stream)
    st = lib.zha_pages_extend(byref(cfg), byref(pool), _list_ptr(seqs, torch.int32, n, dev, "seqs"),
                              _list_ptr(n_tokens, torch.int64, n, dev, "n_tokens"), n, *_scratch(ws, dev),
                              _status_ptr(status, dev), on)
    if st:
        check(st, "zha_pages_extend")


def pages_fork(cfg: Config, pool: PagePool, src: torch.Tensor, dst: torch.Tensor, n_tokens: torch.Tensor,
               ws: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> None:
    """zha_pages_fork: the empty sequence dst[i] becomes the first n_tokens[i] tokens of src[i]."""
    _same_cache(cfg, pool, PagePool)
    n, dev = dst.numel(), pool.index
    on = _run_on(dev, stream)
    if ws is None:
        ws = _new(max(1, pages_workspace_bytes(cfg, pool, n)), torch.uint8, pool.device, stream)
    st = lib.zha_pages_fork(byref(cfg), byref(pool), _list_ptr(src, torch.int32, n, dev, "src"),
                            _list_ptr(dst, torch.int32, n, dev, "dst"),
                            _list_ptr(n_tokens, torch.int64, n, dev, "n_tokens"), n, *_scratch(ws, dev),
                            _status_ptr(status, dev), on)
    if st:
        check(st, "zha_pages_fork")


def pages_free(cfg: Config, pool: PagePool, seqs: torch.Tensor, keep: torch.Tensor | None = None,
               ws: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> None:
    """zha_pages_free: sequences seqs [n] give up their pages behind the first keep [n] (int64)
    tokens (None: all). Needs no workspace; ws is taken for symmetry and not used."""
    _same_cache(cfg, pool, PagePool)
    n, dev = seqs.numel(), pool.index
    on = _run_on(dev, stream)
    st = lib.zha_pages_free(byref(cfg), byref(pool), _list_ptr(seqs, torch.int32, n, dev, "seqs"),
                            None if keep is None else _list_ptr(keep, torch.int64, n, dev, "keep"), n,
                            _status_ptr(status, dev), on)
    if st:
        check(st, "zha_pages_free")


def pages_compact(cfg: Config, pool: PagePool, page_map: torch.Tensor | None = None, n_live: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> None:
    """zha_pages_compact: the pages in use become [0, n); page_map [n_pages] and n_live [1]
    (int32, both may be None) say where each went and how many they are."""
    _same_cache(cfg, pool, PagePool)
    dev = pool.index
    on = _run_on(dev, stream)
    if ws is None:
        ws = _new(max(1, pages_workspace_bytes(cfg, pool, 0)), torch.uint8, pool.device, stream)
    st = lib.zha_pages_compact(
        byref(cfg), byref(pool),
        None if page_map is None else _list_ptr(page_map, torch.int32, pool.shape[0], dev, "page_map"),
        None if n_live is None else _list_ptr(n_live, torch.int32, 1, dev, "n_live"), *_scratch(ws, dev),
        _status_ptr(status, dev), on)
    if st:
        check(st, "zha_pages_compact")
