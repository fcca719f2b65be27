"""ctypes binding of libdsa.so: same names and argument order as include/dsa.h.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (their data pointers are passed);
``stream`` defaults to torch's current stream; with another one, the caller orders
it after the work that made the tensors and keeps them alive until it is done. A
non-zero return code raises DsaError. If libdsa.so cannot be built or loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import buildlib as _build

RATIO, INDEX_HEADS, INDEX_DIM, HEADS, DIM = 4, 64, 128, 64, 512

DSA_OK = 0
DSA_ERR_ARG, DSA_ERR_SHAPE, DSA_ERR_OFFSET, DSA_ERR_CAPACITY = -1, -2, -3, -4
DSA_ERR_DIVERGED, DSA_ERR_SCRATCH, DSA_ERR_CUDA, DSA_ERR_TIMEOUT = -5, -6, -7, -8
DSA_ERR_BOUNDS, DSA_ERR_RAW_RANGE = -9, -10

EXPORTS = ("dsa_pool_append", "dsa_score_scratch_bytes", "dsa_index_score_topk",
           "dsa_window_sparse_attn", "dsa_prefill_chunk", "dsa_strerror",
           "dsa_index_score_topk_noalloc", "dsa_bounded_wait_selftest", "dsa_prefill_chunk_host",
           "dsa_paged_append", "dsa_paged_attn", "dsa_qk_norm_rope", "dsa_paged_q4_append",
           "dsa_paged_q4_read", "dsa_paged_q4_attn")
DSA_STATIC_SCRATCH_BYTES = 16 << 20
DSA_PAGED_WORKSPACE_BYTES = 40 << 20
ROPE_DIM, MAX_PAGE_SIZE, MAX_PAGED_HEADS, MAX_PAGED_TOKENS = 64, 1024, 128, 1 << 24
Q4_ROW_BYTES, MAX_SINKS = 384, 128


class DsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {dsa_strerror(code)} (code {code})")


class dsa_pool_state(ctypes.Structure):
    _fields_ = [("pooled_kv", ctypes.c_void_p), ("pooled_ik", ctypes.c_void_p),
                ("rem_kv", ctypes.c_void_p), ("rem_ik", ctypes.c_void_p),
                ("cap", ctypes.c_int64), ("n_pooled_kv", ctypes.c_int64),
                ("n_pooled_ik", ctypes.c_int64), ("n_tokens", ctypes.c_int64),
                ("n_rem", ctypes.c_int32), ("ratio", ctypes.c_int32)]


class dsa_prefill_workspace(ctypes.Structure):
    _fields_ = [("raw_kv", ctypes.c_void_p), ("raw_kv_rows", ctypes.c_int64),
                ("raw_ik", ctypes.c_void_p), ("q_idx", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("sel", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("scratch", ctypes.c_void_p), ("scratch_bytes", ctypes.c_size_t),
                ("max_chunk", ctypes.c_int64), ("max_topk", ctypes.c_int32)]


_lib = None


def load(path: str | None = None):
    """Load libdsa.so (building it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.build()
    lib = ctypes.CDLL(path)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    S = ctypes.POINTER(dsa_pool_state)
    lib.dsa_pool_append.argtypes = [S, P, P, i64, i64, i32, P]
    lib.dsa_score_scratch_bytes.argtypes = [i64, i64]
    lib.dsa_score_scratch_bytes.restype = sz
    lib.dsa_index_score_topk.argtypes = [P, P, P, i64, i64, i64, i32, i32, i64, P, sz, P, P, P]
    lib.dsa_window_sparse_attn.argtypes = [P, P, i64, i64, P, i64, P, i32, i64, i64, i32, i32,
                                           ctypes.c_float, P, P, P]
    lib.dsa_prefill_chunk.argtypes = [S, P, i64, i64, P, P, P, P, i64, i64, i32, i32,
                                      ctypes.c_float, i64, P, sz, P, P, P, P]
    lib.dsa_index_score_topk_noalloc.argtypes = [P, P, P, i64, i64, i64, i32, i32, i64, P, P, P]
    lib.dsa_bounded_wait_selftest.argtypes = [i32, P, P]
    lib.dsa_prefill_chunk_host.argtypes = [S, ctypes.POINTER(dsa_prefill_workspace), P, i64, i64,
                                           P, P, P, P, i64, i64, i32, i32, ctypes.c_float, i64,
                                           P, P, P, P, P]
    lib.dsa_paged_append.argtypes = [P, i64, P, P, i32, P, i32, P, i64, i64, i32, P, i64, P, P]
    lib.dsa_paged_attn.argtypes = [P, i32, i64, P, P, i32, P, i32, P, i64, i64, i32, P, i64, i32,
                                   ctypes.c_float, P, sz, P, P, P]
    lib.dsa_qk_norm_rope.argtypes = [P, i32, P, i64, P, P, i32, P, P, ctypes.c_float, P, i64, P, P,
                                     P, P]
    lib.dsa_paged_q4_append.argtypes = lib.dsa_paged_append.argtypes
    lib.dsa_paged_q4_read.argtypes = [P, P, i32, P, i32, P, i64, i64, i32, P, i64, P, i64, P, P]
    lib.dsa_paged_q4_attn.argtypes = [P, i32, i64, P, P, i32, P, i32, P, i64, i64, i32, P, i64, i32,
                                      i32, i32, ctypes.c_float, P, sz, P, P, P]
    lib.dsa_strerror.argtypes = [ctypes.c_int]
    lib.dsa_strerror.restype = ctypes.c_char_p
    for f in ("dsa_pool_append", "dsa_index_score_topk", "dsa_window_sparse_attn",
              "dsa_prefill_chunk", "dsa_index_score_topk_noalloc", "dsa_bounded_wait_selftest",
              "dsa_prefill_chunk_host", "dsa_paged_append", "dsa_paged_attn", "dsa_qk_norm_rope",
              "dsa_paged_q4_append", "dsa_paged_q4_read", "dsa_paged_q4_attn"):
        getattr(lib, f).restype = ctypes.c_int
    _lib = lib
    return lib


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _s(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != DSA_OK:
        raise DsaError(rc, where)


def dsa_strerror(code: int) -> str:
    return load().dsa_strerror(int(code)).decode()


class PoolState:
    """Caller-side PoolingCache: device buffers (torch) plus the C struct."""

    def __init__(self, cap: int, device="cuda", ratio: int = RATIO):
        self.ratio = ratio
        self.pooled_kv = torch.zeros(max(cap, 1), DIM, dtype=torch.bfloat16, device=device)
        self.pooled_ik = torch.zeros(max(cap, 1), INDEX_DIM, dtype=torch.bfloat16, device=device)
        self.rem_kv = torch.zeros(max(ratio - 1, 1), DIM, dtype=torch.bfloat16, device=device)
        self.rem_ik = torch.zeros(max(ratio - 1, 1), INDEX_DIM, dtype=torch.bfloat16, device=device)
        self.c = dsa_pool_state(self.pooled_kv.data_ptr(), self.pooled_ik.data_ptr(),
                                self.rem_kv.data_ptr(), self.rem_ik.data_ptr(), cap, 0, 0, 0, 0,
                                ratio)

    @classmethod
    def from_prefix(cls, pooled_ik, pooled_kv, n_tokens: int, cap: int, device="cuda",
                    ratio: int = RATIO):
        """A cache that already holds `pooled_*` rows after n_tokens tokens (no remainder)."""
        s = cls(cap, device, ratio)
        P = pooled_ik.shape[0]
        assert n_tokens == P * ratio and pooled_kv.shape[0] == P and P <= cap
        s.pooled_ik[:P].copy_(pooled_ik)
        s.pooled_kv[:P].copy_(pooled_kv)
        s.c.n_pooled_kv = s.c.n_pooled_ik = P
        s.c.n_tokens = n_tokens
        return s

    @property
    def n_pooled(self) -> int:
        return self.c.n_pooled_kv

    @property
    def n_tokens(self) -> int:
        return self.c.n_tokens

    @property
    def n_rem(self) -> int:
        return self.c.n_rem

    def snapshot(self):
        """O(1) rollback point: the counters and the (at most 3) remainder rows."""
        return (self.c.n_pooled_kv, self.c.n_pooled_ik, self.c.n_tokens, self.c.n_rem,
                self.rem_kv.clone(), self.rem_ik.clone())

    def restore(self, snap) -> None:
        (self.c.n_pooled_kv, self.c.n_pooled_ik, self.c.n_tokens, self.c.n_rem, rk, ri) = snap
        self.rem_kv.copy_(rk)
        self.rem_ik.copy_(ri)


def dsa_pool_append(state: PoolState, raw_kv, raw_ik, chunk: int, offset: int,
                    ratio: int | None = None, stream=None) -> None:
    ratio = state.ratio if ratio is None else ratio
    rc = load().dsa_pool_append(ctypes.byref(state.c), _p(raw_kv), _p(raw_ik), chunk, offset,
                                ratio, _s(stream))
    _check(rc, "dsa_pool_append")


def dsa_score_scratch_bytes(tile_rows: int, n_pooled: int) -> int:
    return int(load().dsa_score_scratch_bytes(tile_rows, n_pooled))


def _nbytes(t):
    if t is None:
        return 0
    return t.numel() * t.element_size()


def dsa_index_score_topk(q_idx, w, pooled_ik, n_pooled: int, chunk: int, offset: int,
                         ratio: int, index_topk: int, tile_rows: int, scratch, sel,
                         dev_status=None, stream=None) -> None:
    rc = load().dsa_index_score_topk(_p(q_idx), _p(w), _p(pooled_ik), n_pooled, chunk, offset,
                                     ratio, index_topk, tile_rows, _p(scratch), _nbytes(scratch),
                                     _p(sel), _p(dev_status), _s(stream))
    _check(rc, "dsa_index_score_topk")


def dsa_index_score_topk_noalloc(q_idx, w, pooled_ik, n_pooled: int, chunk: int, offset: int,
                                 ratio: int, index_topk: int, tile_rows: int, sel,
                                 dev_status=None, stream=None) -> None:
    """dsa_index_score_topk with the library's own score scratch (no allocation)."""
    rc = load().dsa_index_score_topk_noalloc(_p(q_idx), _p(w), _p(pooled_ik), n_pooled, chunk,
                                             offset, ratio, index_topk, tile_rows, _p(sel),
                                             _p(dev_status), _s(stream))
    _check(rc, "dsa_index_score_topk_noalloc")


def dsa_bounded_wait_selftest(arrive: int, dev_status, stream=None) -> None:
    """Run the library's bounded mbarrier waits on a barrier that gets its arrival (1) or none (0),
    or gets it late while blocks of work move on (2) or stand still (3)."""
    rc = load().dsa_bounded_wait_selftest(int(arrive), _p(dev_status), _s(stream))
    _check(rc, "dsa_bounded_wait_selftest")


def dsa_window_sparse_attn(q, raw_kv, raw_start: int, pooled_kv, n_pooled: int, sel,
                           index_topk: int, chunk: int, offset: int, ratio: int, window: int,
                           scale: float, out, dev_status=None, stream=None,
                           raw_rows: int | None = None) -> None:
    rows = raw_kv.shape[0] if raw_rows is None else raw_rows
    rc = load().dsa_window_sparse_attn(_p(q), _p(raw_kv), raw_start, rows, _p(pooled_kv),
                                       n_pooled, _p(sel), index_topk, chunk, offset, ratio,
                                       window, scale, _p(out), _p(dev_status), _s(stream))
    _check(rc, "dsa_window_sparse_attn")


def dsa_prefill_chunk(state: PoolState, raw_kv, raw_start: int, raw_ik, q_idx, w, q,
                      chunk: int, offset: int, index_topk: int, window: int, scale: float,
                      tile_rows: int, scratch, sel, out, dev_status=None, stream=None,
                      raw_rows: int | None = None) -> None:
    rows = raw_kv.shape[0] if raw_rows is None else raw_rows
    rc = load().dsa_prefill_chunk(ctypes.byref(state.c), _p(raw_kv), raw_start, rows,
                                  _p(raw_ik), _p(q_idx), _p(w), _p(q), chunk, offset, index_topk,
                                  window, scale, tile_rows, _p(scratch), _nbytes(scratch),
                                  _p(sel), _p(out), _p(dev_status), _s(stream))
    _check(rc, "dsa_prefill_chunk")


class PrefillWorkspace:
    """Device buffers for dsa_prefill_chunk_host (torch allocations, caller-owned)."""

    def __init__(self, max_chunk: int, max_topk: int, raw_kv_rows: int, n_pooled_max: int,
                 tile_rows: int, device="cuda"):
        dev = torch.device(device)
        self.raw_kv = torch.empty(raw_kv_rows, DIM, dtype=torch.bfloat16, device=dev)
        self.raw_ik = torch.empty(max_chunk, INDEX_DIM, dtype=torch.bfloat16, device=dev)
        self.q_idx = torch.empty(max_chunk, INDEX_HEADS, INDEX_DIM, dtype=torch.bfloat16,
                                 device=dev)
        self.w = torch.empty(max_chunk, INDEX_HEADS, dtype=torch.float32, device=dev)
        self.q = torch.empty(max_chunk, HEADS, DIM, dtype=torch.bfloat16, device=dev)
        self.sel = torch.empty(max_chunk, max_topk, dtype=torch.int32, device=dev)
        self.out = torch.empty(max_chunk, HEADS, DIM, dtype=torch.bfloat16, device=dev)
        nbytes = dsa_score_scratch_bytes(min(tile_rows, max_chunk), n_pooled_max)
        self.scratch = torch.empty(max(nbytes // 4, 1), dtype=torch.float32, device=dev)
        self.c = dsa_prefill_workspace(
            self.raw_kv.data_ptr(), raw_kv_rows, self.raw_ik.data_ptr(), self.q_idx.data_ptr(),
            self.w.data_ptr(), self.q.data_ptr(), self.sel.data_ptr(), self.out.data_ptr(),
            self.scratch.data_ptr(), self.scratch.numel() * 4, max_chunk, max_topk)


def dsa_prefill_chunk_host(state: "PoolState", ws: PrefillWorkspace, raw_kv_h, raw_start: int,
                           raw_ik_h, q_idx_h, w_h, q_h, chunk: int, offset: int,
                           index_topk: int, window: int, scale: float, tile_rows: int,
                           sel_h, out_h, dev_status=None, stream=None,
                           copy_stream=None) -> None:
    """The whole path from host tensors (pinned for overlap) to host tensors."""
    rc = load().dsa_prefill_chunk_host(
        ctypes.byref(state.c), ctypes.byref(ws.c), _p(raw_kv_h), raw_start, raw_kv_h.shape[0],
        _p(raw_ik_h), _p(q_idx_h), _p(w_h), _p(q_h), chunk, offset, index_topk, window, scale,
        tile_rows, _p(sel_h), _p(out_h), _p(dev_status), _s(stream),
        _s(copy_stream) if copy_stream is not None else _s(stream))
    _check(rc, "dsa_prefill_chunk_host")


_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # absent from CPU builds


def _stream_of(stream, device):
    """As _s, by the shorter way to the current stream of `device`."""
    return _raw_stream(device) if stream is None and _raw_stream is not None else _s(stream)


def _refuse(where: str, name: str, dtype, want: str, device):
    raise DsaError(DSA_ERR_ARG, f"{where}: {name} has to be a packed {dtype} tensor [{want}] on "
                                f"cuda:{device}")


def _paged(where: str, new_start, seq_len, page_table, pages, cos_sin, device, width=DIM,
           dtype=_BF16):
    """The arguments the paged calls share, checked, in the ABI's order. A row of the pages is
    `width` elements of `dtype`."""
    table, shape, strides = page_table.shape, pages.shape, pages.stride()
    if not (len(table) == 2 and page_table.dtype is _I32 and page_table.get_device() == device
            and page_table.is_contiguous()):
        _refuse(where, "page_table", _I32, "*, *", device)
    n_seqs, max_pages = table
    if not (new_start.shape == (n_seqs + 1,) and new_start.dtype is _I32
            and new_start.get_device() == device and new_start.is_contiguous()):
        _refuse(where, "new_start", _I32, n_seqs + 1, device)
    if not (seq_len.shape == (n_seqs,) and seq_len.dtype is _I32
            and seq_len.get_device() == device and seq_len.is_contiguous()):
        _refuse(where, "seq_len", _I32, n_seqs, device)
    if not (len(shape) == 3 and shape[2] == width and strides[2] == 1 and strides[1] == width
            and pages.dtype is dtype and pages.get_device() == device):
        raise DsaError(DSA_ERR_ARG, f"{where}: pages has to be a {dtype} tensor "
                                    f"[*, *, {width}] on cuda:{device} with packed pages")
    n_pages, page_size, _ = shape
    if (n_seqs | max_pages | page_size) >> 31:   # ctypes would drop the upper bits
        raise DsaError(DSA_ERR_SHAPE, f"{where}: {n_seqs} sequences of {max_pages} pages of "
                                      f"{page_size} rows are no 32-bit counts")
    angles, n_pos = None, 0
    if cos_sin is not None:
        n_pos = cos_sin.shape[0] if cos_sin.dim() else 0
        if not (cos_sin.shape == (n_pos, ROPE_DIM // 2, 2) and cos_sin.dtype is _F32
                and cos_sin.get_device() == device and cos_sin.is_contiguous()):
            _refuse(where, "cos_sin", _F32, f"*, {ROPE_DIM // 2}, 2", device)
        angles = cos_sin.data_ptr()
    return (new_start.data_ptr(), seq_len.data_ptr(), n_seqs, page_table.data_ptr(), max_pages,
            pages.data_ptr(), n_pages, strides[0] if n_pages > 1 else page_size * width, page_size,
            angles, n_pos)


def _status(where: str, dev_status, device):
    if dev_status is None:
        return None
    if not (dev_status.shape == (1,) and dev_status.dtype is _I32
            and dev_status.get_device() == device):
        _refuse(where, "dev_status", _I32, 1, device)
    return dev_status.data_ptr()


def dsa_paged_append(kv, new_start, seq_len, page_table, pages, cos_sin=None, dev_status=None,
                     stream=None) -> None:
    """Rotate the new tokens' rows kv [n_new, 512] by their positions into their pages
    [n_pages, page_size, 512]. Tensors are on the current device; see include/dsa.h."""
    dev = torch.cuda.current_device()
    shape = kv.shape
    if not (len(shape) == 2 and shape[1] == DIM and kv.dtype is _BF16 and kv.get_device() == dev
            and kv.is_contiguous()):
        _refuse("dsa_paged_append", "kv", _BF16, f"*, {DIM}", dev)
    rc = (_lib or load()).dsa_paged_append(
        kv.data_ptr(), shape[0],
        *_paged("dsa_paged_append", new_start, seq_len, page_table, pages, cos_sin, dev),
        _status("dsa_paged_append", dev_status, dev), _stream_of(stream, dev))
    _check(rc, "dsa_paged_append")


def dsa_paged_attn(q, new_start, seq_len, page_table, pages, window: int, scale: float, workspace,
                   out, cos_sin=None, dev_status=None, stream=None) -> None:
    """Attention of the new tokens q [n_new, heads, 512] over their sequences' paged rows
    (window 0: all of them) into out. `workspace` is any packed tensor of at least
    DSA_PAGED_WORKSPACE_BYTES. Tensors are on the current device; see include/dsa.h."""
    where = "dsa_paged_attn"
    dev = torch.cuda.current_device()
    shape = q.shape
    if not (len(shape) == 3 and shape[2] == DIM and q.dtype is _BF16 and q.get_device() == dev
            and q.is_contiguous()):
        _refuse(where, "q", _BF16, f"*, *, {DIM}", dev)
    if not (out.shape == shape and out.dtype is _BF16 and out.get_device() == dev
            and out.is_contiguous()):
        _refuse(where, "out", _BF16, ", ".join(map(str, shape)), dev)
    if not (workspace.get_device() == dev and workspace.is_contiguous()):
        _refuse(where, "workspace", workspace.dtype, "*", dev)
    if (window | shape[1]) >> 31:   # ctypes would drop the upper bits
        raise DsaError(DSA_ERR_SHAPE, f"{where}: window {window} or heads {shape[1]} is no 32-bit "
                                      "count")
    rc = (_lib or load()).dsa_paged_attn(
        q.data_ptr(), shape[1], shape[0],
        *_paged(where, new_start, seq_len, page_table, pages, cos_sin, dev), window, scale,
        workspace.data_ptr(), _nbytes(workspace), out.data_ptr(),
        _status(where, dev_status, dev), _stream_of(stream, dev))
    _check(rc, where)


def _rows(where: str, name: str, t, device, shape=None):
    """A packed bf16 tensor [*, 512] or [*, *, 512], of `shape` where one is given."""
    have = t.shape
    if not ((have == shape if shape is not None else len(have) == 2 and have[1] == DIM)
            and t.dtype is _BF16 and t.get_device() == device and t.is_contiguous()):
        _refuse(where, name, _BF16, ", ".join(map(str, shape or ("*", DIM))), device)


def dsa_qk_norm_rope(q, kv, new_start, seq_len, q_out, kv_out, cos_sin=None, q_weight=None,
                     kv_weight=None, eps: float = 1e-6, dev_status=None, stream=None) -> None:
    """Normalise the new tokens' query heads q [n_new, heads, 512] and rows kv [n_new, 512] and
    rotate them by position into q_out and kv_out (which may be q and kv). Weights are fp32 [512]
    or None. Tensors are on the current device; see include/dsa.h."""
    where = "dsa_qk_norm_rope"
    dev = torch.cuda.current_device()
    shape = q.shape
    if not (len(shape) == 3 and shape[2] == DIM and q.dtype is _BF16 and q.get_device() == dev
            and q.is_contiguous()):
        _refuse(where, "q", _BF16, f"*, *, {DIM}", dev)
    _rows(where, "kv", kv, dev, (shape[0], DIM))
    _rows(where, "q_out", q_out, dev, tuple(shape))
    _rows(where, "kv_out", kv_out, dev, (shape[0], DIM))
    for name, w in (("q_weight", q_weight), ("kv_weight", kv_weight)):
        if w is not None and not (w.shape == (DIM,) and w.dtype is _F32 and w.get_device() == dev
                                  and w.is_contiguous()):
            _refuse(where, name, _F32, DIM, dev)
    n_seqs = seq_len.shape[0] if seq_len.dim() else 0
    if not (seq_len.shape == (n_seqs,) and seq_len.dtype is _I32 and seq_len.get_device() == dev
            and seq_len.is_contiguous()):
        _refuse(where, "seq_len", _I32, "*", dev)
    if not (new_start.shape == (n_seqs + 1,) and new_start.dtype is _I32
            and new_start.get_device() == dev and new_start.is_contiguous()):
        _refuse(where, "new_start", _I32, n_seqs + 1, dev)
    n_pos = 0
    if cos_sin is not None:
        n_pos = cos_sin.shape[0] if cos_sin.dim() else 0
        if not (cos_sin.shape == (n_pos, ROPE_DIM // 2, 2) and cos_sin.dtype is _F32
                and cos_sin.get_device() == dev and cos_sin.is_contiguous()):
            _refuse(where, "cos_sin", _F32, f"*, {ROPE_DIM // 2}, 2", dev)
    if (n_seqs | shape[1]) >> 31:   # ctypes would drop the upper bits
        raise DsaError(DSA_ERR_SHAPE, f"{where}: {n_seqs} sequences or {shape[1]} heads are no "
                                      "32-bit counts")
    rc = (_lib or load()).dsa_qk_norm_rope(
        q.data_ptr(), shape[1], kv.data_ptr(), shape[0], new_start.data_ptr(), seq_len.data_ptr(),
        n_seqs, _p(q_weight), _p(kv_weight), eps, _p(cos_sin), n_pos, q_out.data_ptr(),
        kv_out.data_ptr(), _status(where, dev_status, dev), _stream_of(stream, dev))
    _check(rc, where)


def dsa_paged_q4_append(kv, new_start, seq_len, page_table, pages, cos_sin=None, dev_status=None,
                        stream=None) -> None:
    """dsa_paged_append into pages [n_pages, page_size, 384] uint8 of 4-bit rows. Tensors are on
    the current device; see include/dsa.h."""
    where = "dsa_paged_q4_append"
    dev = torch.cuda.current_device()
    _rows(where, "kv", kv, dev)
    rc = (_lib or load()).dsa_paged_q4_append(
        kv.data_ptr(), kv.shape[0],
        *_paged(where, new_start, seq_len, page_table, pages, cos_sin, dev, Q4_ROW_BYTES, _U8),
        _status(where, dev_status, dev), _stream_of(stream, dev))
    _check(rc, where)


def dsa_paged_q4_read(new_start, seq_len, page_table, pages, out, cos_sin=None, dev_status=None,
                      stream=None) -> None:
    """What the sequences' 4-bit rows stand for into out [n_new, 512] bf16, turned back with
    cos_sin. Tensors are on the current device; see include/dsa.h."""
    where = "dsa_paged_q4_read"
    dev = torch.cuda.current_device()
    _rows(where, "out", out, dev)
    rc = (_lib or load()).dsa_paged_q4_read(
        *_paged(where, new_start, seq_len, page_table, pages, cos_sin, dev, Q4_ROW_BYTES, _U8),
        out.data_ptr(), out.shape[0], _status(where, dev_status, dev), _stream_of(stream, dev))
    _check(rc, where)


def dsa_paged_q4_attn(q, new_start, seq_len, page_table, pages, window: int, sinks: int,
                      scale: float, workspace, out, cos_sin=None, q_turned: bool = False,
                      dev_status=None, stream=None) -> None:
    """Attention of the new tokens q [n_new, heads, 512] over their sequences' 4-bit rows into
    out: all of them (window 0), or the last `window` and the first `sinks`. q_turned: q comes
    turned by its positions. `workspace` as for dsa_paged_attn. Tensors are on the current device;
    see include/dsa.h."""
    where = "dsa_paged_q4_attn"
    dev = torch.cuda.current_device()
    shape = q.shape
    if not (len(shape) == 3 and shape[2] == DIM and q.dtype is _BF16 and q.get_device() == dev
            and q.is_contiguous()):
        _refuse(where, "q", _BF16, f"*, *, {DIM}", dev)
    _rows(where, "out", out, dev, tuple(shape))
    if not (workspace.get_device() == dev and workspace.is_contiguous()):
        _refuse(where, "workspace", workspace.dtype, "*", dev)
    if (window | sinks | shape[1]) >> 31:   # ctypes would drop the upper bits
        raise DsaError(DSA_ERR_SHAPE, f"{where}: window {window}, sinks {sinks} or heads "
                                      f"{shape[1]} is no 32-bit count")
    rc = (_lib or load()).dsa_paged_q4_attn(
        q.data_ptr(), shape[1], shape[0],
        *_paged(where, new_start, seq_len, page_table, pages, cos_sin, dev, Q4_ROW_BYTES, _U8),
        window, sinks, bool(q_turned), scale, workspace.data_ptr(), _nbytes(workspace),
        out.data_ptr(), _status(where, dev_status, dev), _stream_of(stream, dev))
    _check(rc, where)
