"""SegmentAttention for B200: Python binding of the C-ABI library ``libsegattn.so``.

Every function here only marshals arguments for the C entry points declared
in ``include/seg_attn.h``, ``include/seg_la.h`` and ``include/seg_draft.h`` (same
names).  All compute runs in the library's sm_100a kernels; there is no fallback
path.  PyTorch supplies device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from ._build import LIB as LIB_PATH

__all__ = [
    "SegAttnError", "seg_attn_table_desc", "seg_attn_build_table", "seg_attn_workspace_size",
    "seg_attn_prefill", "seg_attn_decode", "seg_attn_status_string", "seg_attn_version",
    "seg_attn_take_device_error", "seg_attn_wait_selftest", "seg_attn_stall_test", "seg_attn_order_test", "SegTable", "load_library", "LIB_PATH",
    "MODE_PREFILL", "MODE_DECODE", "STATUS", "SegPool", "seg_attn_kv_append",
    "seg_attn_decode_fp8", "seg_attn_prefill_fp8", "seg_attn_kv_append_fp8", "SHARE_PREFIX",
    "seg_la_table_desc", "seg_la_build_table", "seg_la_workspace_size", "seg_la_prefill",
    "seg_la_decode", "LATable",
    "RopeScaling", "seg_attn_rope_desc", "seg_attn_rope_plan", "seg_attn_rope",
    "seg_attn_rope_append", "seg_attn_rope_append_fp8", "seg_attn_tree_desc",
    "seg_attn_build_tree_table", "seg_attn_tree_workspace_size", "seg_attn_tree",
    "seg_attn_tree_fp8", "TreeTable", "seg_attn_kv_move",
]

MODE_PREFILL = 0
MODE_DECODE = 1
SHARE_PREFIX = 0x100  # OR into the mode: plan shared prefixes
STATUS = {
    "OK": 0, "INVALID_ARG": -1, "SEGMENT_OOB": -2, "SEGMENT_OVERLAP": -3, "QLEN_GT_KLEN": -4,
    "WORKSPACE": -5, "UNSUPPORTED": -6, "CUDA": -7, "BUFFER_TOO_SMALL": -8, "NO_SPACE": -9,
}


class seg_attn_table_desc(ctypes.Structure):
    """Mirror of ``seg_attn_table_desc`` in include/seg_attn.h."""
    _fields_ = [
        ("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
        ("mode", ctypes.c_int32), ("causal", ctypes.c_int32),
        ("batch", ctypes.c_int32), ("q_heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("num_slots", ctypes.c_int64), ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64),
        ("num_segments", ctypes.c_int32), ("num_work", ctypes.c_int32),
        ("queries_per_tile", ctypes.c_int32), ("chunk_len", ctypes.c_int32),
        ("max_k_tiles", ctypes.c_int32), ("num_merge", ctypes.c_int32),
        ("num_parts", ctypes.c_int32), ("shared", ctypes.c_int32),
        ("off_q_offsets", ctypes.c_int64), ("off_k_lens", ctypes.c_int64),
        ("off_seg_offsets", ctypes.c_int64), ("off_seg_start", ctypes.c_int64),
        ("off_seg_kstart", ctypes.c_int64), ("off_seg_len", ctypes.c_int64),
        ("off_work", ctypes.c_int64), ("off_req_chunks", ctypes.c_int64),
        ("off_merge", ctypes.c_int64),
        ("table_bytes", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64),
        ("num_groups", ctypes.c_int32), ("num_group_segments", ctypes.c_int32),
        ("num_group_work", ctypes.c_int32), ("num_group_parts", ctypes.c_int32),
        ("num_citems", ctypes.c_int32), ("num_cascade", ctypes.c_int32),
        ("num_single", ctypes.c_int32), ("num_group_single", ctypes.c_int32),
        ("group_total_k", ctypes.c_int64),
        ("off_group_req", ctypes.c_int64), ("off_group_q_offsets", ctypes.c_int64),
        ("off_group_k_lens", ctypes.c_int64), ("off_group_seg_offsets", ctypes.c_int64),
        ("off_group_seg_start", ctypes.c_int64), ("off_group_seg_kstart", ctypes.c_int64),
        ("off_group_seg_len", ctypes.c_int64), ("off_group_work", ctypes.c_int64),
        ("off_citem", ctypes.c_int64), ("off_cascade", ctypes.c_int64),
    ]


class seg_la_table_desc(ctypes.Structure):
    """Mirror of ``seg_la_table_desc`` in include/seg_la.h."""
    _fields_ = [
        ("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
        ("mode", ctypes.c_int32), ("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("chunk_len", ctypes.c_int32),
        ("num_chunks", ctypes.c_int32),
        ("total_q", ctypes.c_int64), ("num_state_slots", ctypes.c_int64),
        ("off_q_offsets", ctypes.c_int64), ("off_in_slot", ctypes.c_int64),
        ("off_out_slot", ctypes.c_int64), ("off_req_chunks", ctypes.c_int64),
        ("off_chunks", ctypes.c_int64),
        ("table_bytes", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64),
    ]


class seg_attn_rope_scaling(ctypes.Structure):
    """Mirror of ``seg_attn_rope_scaling`` in include/seg_draft.h."""
    _fields_ = [
        ("kind", ctypes.c_int32), ("num_factors", ctypes.c_int32), ("factor", ctypes.c_double),
        ("original_len", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
        ("amp", ctypes.c_double), ("factors", ctypes.c_void_p),
    ]


class seg_attn_rope_desc(ctypes.Structure):
    """Mirror of ``seg_attn_rope_desc`` in include/seg_draft.h."""
    _fields_ = [("magic", ctypes.c_uint32), ("rotary_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("amp", ctypes.c_float),
                ("turns", ctypes.c_uint64 * 128)]


class seg_attn_tree_desc(ctypes.Structure):
    """Mirror of ``seg_attn_tree_desc`` in include/seg_draft.h."""
    _fields_ = [
        ("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
        ("batch", ctypes.c_int32), ("max_draft", ctypes.c_int32),
        ("off_mask", ctypes.c_int64), ("off_draft_slot", ctypes.c_int64),
        ("pass_", seg_attn_table_desc),
        ("table_bytes", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64),
    ]


class seg_attn_pool_stats(ctypes.Structure):
    """Mirror of ``seg_attn_pool_stats`` in include/seg_attn.h."""
    _fields_ = [("num_slots", ctypes.c_int64), ("free_slots", ctypes.c_int64),
                ("free_runs", ctypes.c_int64), ("largest_free_run", ctypes.c_int64),
                ("sequences", ctypes.c_int64), ("segments", ctypes.c_int64)]


class SegAttnError(RuntimeError):
    def __init__(self, fn: str, code: int, detail: str = ""):
        self.code = code
        super().__init__(f"{fn}: {seg_attn_status_string(code)} (status {code})"
                         + (f": {detail}" if detail else ""))


_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libsegattn.so (built in-tree by ``__graft_entry__.build()``); fail loudly if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise ImportError(f"CUDA library not built: {path} is missing "
                              "(run python -c 'import __graft_entry__; __graft_entry__.build()')")
        lib = ctypes.CDLL(path)
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        D = ctypes.POINTER(seg_attn_table_desc)
        lib.seg_attn_build_table.argtypes = [I, P, P, P, P, I64, I, I, I, I, I, P, SZ, D]
        lib.seg_attn_build_table.restype = I
        lib.seg_attn_workspace_size.argtypes = [D]
        lib.seg_attn_workspace_size.restype = SZ
        for fn in (lib.seg_attn_prefill, lib.seg_attn_decode):
            fn.argtypes = [P, P, P, P, P, P, D, ctypes.c_float, P, SZ, P]
            fn.restype = I
        lib.seg_attn_status_string.argtypes = [I]
        lib.seg_attn_status_string.restype = ctypes.c_char_p
        lib.seg_attn_version.argtypes = []
        lib.seg_attn_version.restype = I
        lib.seg_attn_take_device_error.argtypes = [ctypes.POINTER(ctypes.c_int)]
        lib.seg_attn_take_device_error.restype = I
        lib.seg_attn_wait_selftest.argtypes = [I, P]
        lib.seg_attn_wait_selftest.restype = I
        lib.seg_attn_stall_test.argtypes = [I, I]
        lib.seg_attn_stall_test.restype = I
        lib.seg_attn_order_test.argtypes = [I]
        lib.seg_attn_order_test.restype = I
        PP = ctypes.POINTER(ctypes.c_void_p)
        lib.seg_attn_pool_create.argtypes = [I64, PP]
        lib.seg_attn_pool_destroy.argtypes = [P]
        lib.seg_attn_pool_append.argtypes = [P, I64, I64, P]
        lib.seg_attn_pool_release.argtypes = [P, I64]
        lib.seg_attn_pool_segments.argtypes = [P, I64, P, P, I, ctypes.POINTER(I)]
        lib.seg_attn_pool_get_stats.argtypes = [P, ctypes.POINTER(seg_attn_pool_stats)]
        for fn in (lib.seg_attn_pool_create, lib.seg_attn_pool_destroy, lib.seg_attn_pool_append,
                   lib.seg_attn_pool_release, lib.seg_attn_pool_segments,
                   lib.seg_attn_pool_get_stats):
            fn.restype = I
        lib.seg_attn_kv_append.argtypes = [P, P, P, I64, I, I, P, P, I64, P]
        lib.seg_attn_kv_append.restype = I
        lib.seg_attn_kv_append_fp8.argtypes = [P, P, P, I64, I, I, P, P, P, P, I64, P]
        lib.seg_attn_kv_append_fp8.restype = I
        for fn in (lib.seg_attn_decode_fp8, lib.seg_attn_prefill_fp8):
            fn.argtypes = [P, P, P, P, P, P, P, P, D, ctypes.c_float, P, SZ, P]
            fn.restype = I
        LD = ctypes.POINTER(seg_la_table_desc)
        lib.seg_la_build_table.argtypes = [I, P, P, P, I64, I, I, I, P, SZ, LD]
        lib.seg_la_build_table.restype = I
        lib.seg_la_workspace_size.argtypes = [LD]
        lib.seg_la_workspace_size.restype = SZ
        lib.seg_la_prefill.argtypes = [P, P, P, P, P, P, P, LD, ctypes.c_float, P, SZ, P]
        lib.seg_la_prefill.restype = I
        lib.seg_la_decode.argtypes = [P, P, P, P, P, P, P, LD, ctypes.c_float, P]
        lib.seg_la_decode.restype = I
        RD, F = ctypes.POINTER(seg_attn_rope_desc), ctypes.c_float
        TD = ctypes.POINTER(seg_attn_tree_desc)
        lib.seg_attn_rope_plan.argtypes = [I, I, ctypes.c_double,
                                           ctypes.POINTER(seg_attn_rope_scaling), RD]
        lib.seg_attn_rope.argtypes = [P, I64, P, I64, P, I64, I, I, RD, I, P]
        rows = [P, I64] * 4 + [P, P, I64, I, I, I, RD]
        lib.seg_attn_rope_append.argtypes = rows + [P, P, I64, P]
        lib.seg_attn_rope_append_fp8.argtypes = rows + [P, P, P, P, I64, P]
        lib.seg_attn_build_tree_table.argtypes = [I, P, P, P, P, P, P, I64, I, I, I, P, SZ, TD]
        lib.seg_attn_tree_workspace_size.argtypes = [TD]
        lib.seg_attn_tree_workspace_size.restype = SZ
        lib.seg_attn_tree.argtypes = [P, P, P, P, P, P, TD, F, P, SZ, P]
        lib.seg_attn_tree_fp8.argtypes = [P, P, P, P, P, P, P, P, TD, F, P, SZ, P]
        lib.seg_attn_kv_move.argtypes = [P, P, P, P, I64, P, I64, I, I, I, I64, P]
        for fn in (lib.seg_attn_rope_plan, lib.seg_attn_rope, lib.seg_attn_rope_append,
                   lib.seg_attn_rope_append_fp8, lib.seg_attn_build_tree_table,
                   lib.seg_attn_tree, lib.seg_attn_tree_fp8, lib.seg_attn_kv_move):
            fn.restype = I
        _lib = lib
        return lib


def seg_attn_status_string(code: int) -> str:
    return load_library().seg_attn_status_string(int(code)).decode()


def seg_attn_version() -> int:
    return load_library().seg_attn_version()


def _i32(x) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(x, dtype=np.int32).reshape(-1))


def _np_ptr(a: Optional[np.ndarray]):
    return ctypes.c_void_p(a.ctypes.data) if a is not None and a.size else ctypes.c_void_p(0)


def seg_attn_build_table(batch: int, q_lens: Optional[Sequence[int]], seg_counts: Sequence[int],
                         seg_starts: Sequence[int], seg_lens: Sequence[int], num_slots: int,
                         causal: bool, mode: int, q_heads: int, kv_heads: int, head_dim: int,
                         pin: bool = False):
    """Returns (host table as an int32 torch tensor, seg_attn_table_desc).  Raises SegAttnError."""
    lib = load_library()
    ql = _i32(q_lens) if q_lens is not None else None
    sc, ss, sl = _i32(seg_counts), _i32(seg_starts), _i32(seg_lens)
    desc = seg_attn_table_desc()
    args = [int(batch), _np_ptr(ql), _np_ptr(sc), _np_ptr(ss), _np_ptr(sl), int(num_slots),
            int(bool(causal)), int(mode), int(q_heads), int(kv_heads), int(head_dim)]
    rc = lib.seg_attn_build_table(*args, ctypes.c_void_p(0), 0, ctypes.byref(desc))
    if rc != 0:
        raise SegAttnError("seg_attn_build_table", rc)
    n = max(1, (desc.table_bytes + 3) // 4)
    host = torch.zeros(n, dtype=torch.int32, pin_memory=pin)
    rc = lib.seg_attn_build_table(*args, ctypes.c_void_p(host.data_ptr()), int(desc.table_bytes),
                                  ctypes.byref(desc))
    if rc != 0:
        raise SegAttnError("seg_attn_build_table", rc)
    return host, desc


def seg_attn_workspace_size(desc: seg_attn_table_desc) -> int:
    return int(load_library().seg_attn_workspace_size(ctypes.byref(desc)))


def _dptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _compute(fn_name, q, k_pool, v_pool, out, lse, dev_table, desc, softmax_scale, workspace,
             stream):
    lib = load_library()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = getattr(lib, fn_name)(_dptr(q), _dptr(k_pool), _dptr(v_pool), _dptr(out), _dptr(lse),
                               _dptr(dev_table), ctypes.byref(desc), float(softmax_scale),
                               _dptr(workspace), int(ws_bytes), _stream_ptr(stream))
    if rc != 0:
        raise SegAttnError(fn_name, rc)


def seg_attn_prefill(q, k_pool, v_pool, out, lse, dev_table, desc, softmax_scale,
                     workspace=None, stream=None) -> None:
    """Launch chunked-prefill attention on ``stream`` (default: torch's current stream)."""
    _compute("seg_attn_prefill", q, k_pool, v_pool, out, lse, dev_table, desc, softmax_scale,
             workspace, stream)


def seg_attn_decode(q, k_pool, v_pool, out, lse, dev_table, desc, softmax_scale,
                    workspace=None, stream=None) -> None:
    """Launch split-K decode attention on ``stream`` (default: torch's current stream)."""
    _compute("seg_attn_decode", q, k_pool, v_pool, out, lse, dev_table, desc, softmax_scale,
             workspace, stream)


def seg_attn_wait_selftest(wait_us: int, stream=None) -> None:
    """Launch the bounded-wait diagnostic: a wait that nothing completes gives up after
    ``wait_us`` and sets bit 0 of the device error word."""
    rc = load_library().seg_attn_wait_selftest(int(wait_us), _stream_ptr(stream))
    if rc != 0:
        raise SegAttnError("seg_attn_wait_selftest", rc)


def seg_attn_stall_test(withhold_k_tile: int, wait_us: int = 1000000) -> None:
    """Stall test switch of later prefill launches: the producer stops before K tile
    ``withhold_k_tile`` (< 0: off) and every bounded wait gives up after ``wait_us``."""
    rc = load_library().seg_attn_stall_test(int(withhold_k_tile), int(wait_us))
    if rc != 0:
        raise SegAttnError("seg_attn_stall_test", rc)


def seg_attn_order_test(delay_ns: int) -> None:
    """Order test switch of later prefill launches: every softmax warp of a one-tile item
    sleeps ``delay_ns`` after signalling P of the item's last K tile (0: off)."""
    rc = load_library().seg_attn_order_test(int(delay_ns))
    if rc != 0:
        raise SegAttnError("seg_attn_order_test", rc)


def seg_attn_take_device_error() -> int:
    v = ctypes.c_int(0)
    rc = load_library().seg_attn_take_device_error(ctypes.byref(v))
    if rc != 0:
        raise SegAttnError("seg_attn_take_device_error", rc)
    return v.value


@dataclass
class SegTable:
    """A built table: host copy, description, device copy and workspace size."""
    host: torch.Tensor
    desc: seg_attn_table_desc
    device: Optional[torch.Tensor] = None

    @classmethod
    def build(cls, q_lens, seg_starts, seg_lens, num_slots, causal, mode, q_heads, kv_heads,
              head_dim, pin=False):
        """Per-request lists in, flattened for seg_attn_build_table."""
        counts = [len(s) for s in seg_starts]
        starts = [x for s in seg_starts for x in s]
        lens = [x for s in seg_lens for x in s]
        host, desc = seg_attn_build_table(len(counts), q_lens, counts, starts, lens, num_slots,
                                          causal, mode, q_heads, kv_heads, head_dim, pin=pin)
        return cls(host=host, desc=desc)

    def to(self, device, non_blocking=False) -> "SegTable":
        self.device = self.host.to(device, non_blocking=non_blocking)
        return self

    @property
    def workspace_bytes(self) -> int:
        return seg_attn_workspace_size(self.desc)


class SegPool:
    """Host segment allocator of a slot pool (wraps the seg_attn_pool_* calls)."""

    def __init__(self, num_slots: int):
        self._lib = load_library()
        self._h = ctypes.c_void_p()
        rc = self._lib.seg_attn_pool_create(int(num_slots), ctypes.byref(self._h))
        if rc != 0:
            raise SegAttnError("seg_attn_pool_create", rc)

    def close(self):
        if self._h:
            self._lib.seg_attn_pool_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, seq: int, n_tokens: int) -> np.ndarray:
        """Slots (int32, logical order) of n_tokens new tokens of sequence ``seq``."""
        out = np.zeros(max(1, int(n_tokens)), dtype=np.int32)
        rc = self._lib.seg_attn_pool_append(self._h, int(seq), int(n_tokens),
                                            ctypes.c_void_p(out.ctypes.data))
        if rc != 0:
            raise SegAttnError("seg_attn_pool_append", rc)
        return out[:n_tokens]

    def release(self, seq: int) -> None:
        rc = self._lib.seg_attn_pool_release(self._h, int(seq))
        if rc != 0:
            raise SegAttnError("seg_attn_pool_release", rc)

    def segments(self, seq: int):
        """(starts, lens) lists of ``seq`` in logical order."""
        count = ctypes.c_int(0)
        self._lib.seg_attn_pool_segments(self._h, int(seq), None, None, 0, ctypes.byref(count))
        n = count.value
        st = np.zeros(max(1, n), dtype=np.int32)
        ln = np.zeros(max(1, n), dtype=np.int32)
        rc = self._lib.seg_attn_pool_segments(self._h, int(seq), ctypes.c_void_p(st.ctypes.data),
                                              ctypes.c_void_p(ln.ctypes.data), n,
                                              ctypes.byref(count))
        if rc != 0:
            raise SegAttnError("seg_attn_pool_segments", rc)
        return st[:n].tolist(), ln[:n].tolist()

    def stats(self) -> dict:
        st = seg_attn_pool_stats()
        rc = self._lib.seg_attn_pool_get_stats(self._h, ctypes.byref(st))
        if rc != 0:
            raise SegAttnError("seg_attn_pool_get_stats", rc)
        return {name: getattr(st, name) for name, _ in st._fields_}


def seg_attn_kv_append(k_new, v_new, slots, k_pool, v_pool, stream=None) -> None:
    """Write k_new / v_new [n, Hkv, d] (device bf16) into the pools at ``slots`` (device int32)."""
    lib = load_library()
    rc = lib.seg_attn_kv_append(_dptr(k_new), _dptr(v_new), _dptr(slots), int(slots.numel()),
                                int(k_pool.shape[1]), int(k_pool.shape[2]), _dptr(k_pool),
                                _dptr(v_pool), int(k_pool.shape[0]), _stream_ptr(stream))
    if rc != 0:
        raise SegAttnError("seg_attn_kv_append", rc)


def seg_attn_kv_append_fp8(k_new, v_new, slots, k_scale, v_scale, k_pool, v_pool,
                           stream=None) -> None:
    """Quantise k_new / v_new (bf16 [n, Hkv, d]) with per-kv-head scales and write the E4M3
    codes into uint8 pools [S, Hkv, d] at ``slots``."""
    lib = load_library()
    rc = lib.seg_attn_kv_append_fp8(_dptr(k_new), _dptr(v_new), _dptr(slots), int(slots.numel()),
                                    int(k_pool.shape[1]), int(k_pool.shape[2]), _dptr(k_scale),
                                    _dptr(v_scale), _dptr(k_pool), _dptr(v_pool),
                                    int(k_pool.shape[0]), _stream_ptr(stream))
    if rc != 0:
        raise SegAttnError("seg_attn_kv_append_fp8", rc)


def _compute_fp8(fn_name, q, k_pool, v_pool, k_scale, v_scale, out, lse, dev_table, desc,
                 softmax_scale, workspace, stream):
    lib = load_library()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = getattr(lib, fn_name)(_dptr(q), _dptr(k_pool), _dptr(v_pool), _dptr(k_scale),
                               _dptr(v_scale), _dptr(out), _dptr(lse), _dptr(dev_table),
                               ctypes.byref(desc), float(softmax_scale), _dptr(workspace),
                               int(ws_bytes), _stream_ptr(stream))
    if rc != 0:
        raise SegAttnError(fn_name, rc)


def seg_attn_decode_fp8(q, k_pool, v_pool, k_scale, v_scale, out, lse, dev_table, desc,
                        softmax_scale, workspace=None, stream=None) -> None:
    """Decode over E4M3 pools (uint8 [S, Hkv, d]) with per-kv-head fp32 scales."""
    _compute_fp8("seg_attn_decode_fp8", q, k_pool, v_pool, k_scale, v_scale, out, lse, dev_table,
                 desc, softmax_scale, workspace, stream)


def seg_attn_prefill_fp8(q, k_pool, v_pool, k_scale, v_scale, out, lse, dev_table, desc,
                         softmax_scale, workspace=None, stream=None) -> None:
    """Chunked prefill over E4M3 pools (uint8 [S, Hkv, d]) with per-kv-head fp32 scales."""
    _compute_fp8("seg_attn_prefill_fp8", q, k_pool, v_pool, k_scale, v_scale, out, lse,
                 dev_table, desc, softmax_scale, workspace, stream)


# ----------------------------------------------------------------- segment linear attention
def seg_la_build_table(q_lens, in_slot, out_slot, num_state_slots: int, mode: int, heads: int,
                       head_dim: int, pin: bool = False):
    """Returns (host table int32 tensor, seg_la_table_desc).  ``q_lens`` may be None in decode
    mode.  Raises SegAttnError."""
    lib = load_library()
    ins, outs = _i32(in_slot), _i32(out_slot)
    ql = _i32(q_lens) if q_lens is not None else None
    desc = seg_la_table_desc()
    args = [int(ins.size), _np_ptr(ql), _np_ptr(ins), _np_ptr(outs), int(num_state_slots),
            int(mode), int(heads), int(head_dim)]
    rc = lib.seg_la_build_table(*args, ctypes.c_void_p(0), 0, ctypes.byref(desc))
    if rc != 0:
        raise SegAttnError("seg_la_build_table", rc)
    host = torch.zeros(max(1, (desc.table_bytes + 3) // 4), dtype=torch.int32, pin_memory=pin)
    rc = lib.seg_la_build_table(*args, ctypes.c_void_p(host.data_ptr()), int(desc.table_bytes),
                                ctypes.byref(desc))
    if rc != 0:
        raise SegAttnError("seg_la_build_table", rc)
    return host, desc


def seg_la_workspace_size(desc: seg_la_table_desc) -> int:
    return int(load_library().seg_la_workspace_size(ctypes.byref(desc)))


def seg_la_prefill(q, k, v, g, out, state_pool, dev_table, desc, scale, workspace=None,
                   stream=None) -> None:
    """Chunked simple-GLA prefill on ``stream`` (default: torch's current stream)."""
    lib = load_library()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.seg_la_prefill(_dptr(q), _dptr(k), _dptr(v), _dptr(g), _dptr(out), _dptr(state_pool),
                            _dptr(dev_table), ctypes.byref(desc), float(scale), _dptr(workspace),
                            int(ws_bytes), _stream_ptr(stream))
    if rc != 0:
        raise SegAttnError("seg_la_prefill", rc)


def seg_la_decode(q, k, v, g, out, state_pool, dev_table, desc, scale, stream=None) -> None:
    """One-token simple-GLA decode on ``stream`` (default: torch's current stream)."""
    lib = load_library()
    rc = lib.seg_la_decode(_dptr(q), _dptr(k), _dptr(v), _dptr(g), _dptr(out), _dptr(state_pool),
                           _dptr(dev_table), ctypes.byref(desc), float(scale), _stream_ptr(stream))
    if rc != 0:
        raise SegAttnError("seg_la_decode", rc)


@dataclass
class LATable:
    """A built linear-attention table: host copy, description, device copy."""
    host: torch.Tensor
    desc: seg_la_table_desc
    device: Optional[torch.Tensor] = None

    @classmethod
    def build(cls, q_lens, in_slot, out_slot, num_state_slots, mode, heads, head_dim, pin=False):
        host, desc = seg_la_build_table(q_lens, in_slot, out_slot, num_state_slots, mode, heads,
                                        head_dim, pin=pin)
        return cls(host=host, desc=desc)

    def to(self, device, non_blocking=False) -> "LATable":
        self.device = self.host.to(device, non_blocking=non_blocking)
        return self

    @property
    def workspace_bytes(self) -> int:
        return seg_la_workspace_size(self.desc)


# ------------------------------------------------- rotary positions and drafted tokens
# These calls check dtypes, shapes, strides and devices as well, and run on the
# tensors' device whichever is current (seg_draft.h has the rest of the contract).
# Their arguments travel as one packed block (csrc/bind.cpp): a decode step makes
# them with a handful of tokens, where converting 20 arguments one by one costs more
# than the kernel takes.
_ROPE_SCALES = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "wavelength": 4, "per_pair": 5}
_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


@dataclass
class RopeScaling:
    """Scaling of the rotary frequencies for contexts longer than the original one.

    ``kind``: "linear", "ntk", "yarn", "wavelength" or "per_pair" (formulas in seg_draft.h);
    ``amp`` 0 and ``low`` = ``high`` = 0 take the kind's own values; ``factors``: one per pair.
    """
    kind: str
    factor: float = 1.0
    original_len: float = 0.0
    low: float = 0.0
    high: float = 0.0
    amp: float = 0.0
    factors: Optional[Sequence[float]] = None


def _bad(fn: str, detail: str):
    raise SegAttnError(fn, STATUS["INVALID_ARG"], detail)


_packers = {}


def _packed(fn_name: str, n: int):
    """(entry point taking one packed block, packer of n 64-bit values) of a call."""
    got = _packers.get(fn_name)
    if got is None:
        fn = getattr(load_library(), fn_name + "_packed")
        fn.argtypes, fn.restype = [ctypes.c_char_p], ctypes.c_int
        got = _packers[fn_name] = fn, struct.Struct(f"={n}q").pack
    return got


def _invoke(fn_name: str, device: int, stream, args: tuple) -> None:
    """Call the entry point with ``args`` + the stream, with ``device`` current."""
    fn, pack = _packed(fn_name, len(args) + 1)
    if stream is None:
        raw = _current_raw_stream(device)
    elif stream.device.index != device:
        _bad(fn_name, f"stream on {stream.device}, tensors on cuda:{device}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == device:
        rc = fn(pack(*args, raw))
    else:
        with torch.cuda.device(device):
            rc = fn(pack(*args, raw))
    if rc != 0:
        raise SegAttnError(fn_name, rc)


# the stream as an integer, without making a Stream object (1 us) where torch has the call
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _ptr(fn: str, name: str, t: torch.Tensor, dtype, device: int, numel: int = -1) -> int:
    """Address of a dense tensor of the given dtype, device and element count (-1: any)."""
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous() or (
            numel >= 0 and t.numel() != numel):
        _bad(fn, f"{name}: a dense {dtype} tensor on cuda:{device}"
                 + (f" of {numel} values" if numel >= 0 else "")
                 + f", not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(fn: str, name: str, t: torch.Tensor, shape: tuple, device: int):
    """(address, token stride) of bf16 rows [n, heads, d] with dense heads."""
    s = t.stride()
    if (t.dtype is not _BF16 or t.get_device() != device or t.shape != shape
            or (s[2] != 1 and shape[2] > 1) or (s[1] != shape[2] and shape[1] > 1)):
        _bad(fn, f"{name}: bf16 {list(shape)} with dense heads on cuda:{device}, "
                 f"not {t.dtype} {tuple(t.shape)} strides {s} on {t.device}")
    return t.data_ptr(), s[0]


def _cuda_device(fn: str, name: str, t: torch.Tensor, dim: int) -> int:
    if not t.is_cuda or t.dim() != dim:
        _bad(fn, f"{name}: a {dim}-dimensional CUDA tensor, not {t.dim()}-dimensional on {t.device}")
    return t.get_device()


def seg_attn_rope_plan(rotary_dim: int, interleaved: bool = False, base: float = 10000.0,
                       scaling: Optional[RopeScaling] = None) -> seg_attn_rope_desc:
    """Plan of a rotation (host value, nothing to free).  Raises SegAttnError."""
    desc, arg, keep = seg_attn_rope_desc(), None, None
    if scaling is not None:
        if scaling.kind not in _ROPE_SCALES:
            _bad("seg_attn_rope_plan", f"scaling kind {scaling.kind!r}")
        if scaling.factors is not None:
            keep = np.ascontiguousarray(np.asarray(scaling.factors, dtype=np.float64).reshape(-1))
        arg = ctypes.byref(seg_attn_rope_scaling(
            _ROPE_SCALES[scaling.kind], keep.size if keep is not None else 0, scaling.factor,
            scaling.original_len, scaling.low, scaling.high, scaling.amp,
            keep.ctypes.data if keep is not None and keep.size else None))
    rc = load_library().seg_attn_rope_plan(int(rotary_dim), int(bool(interleaved)), float(base),
                                           arg, ctypes.byref(desc))
    if rc != 0:
        raise SegAttnError("seg_attn_rope_plan", rc)
    return desc


def seg_attn_rope(x, out, positions, rope: seg_attn_rope_desc, backward: bool = False,
                  stream=None) -> None:
    """Rotate x [n, heads, d] (bf16, dense heads, any token stride) into ``out`` (may be x) by
    the angles of ``positions`` (device int32 [n]); ``backward``: the transposed rotation."""
    fn = "seg_attn_rope"
    dev = _cuda_device(fn, "x", x, 3)
    shape = x.shape
    n, h, d = shape
    _invoke(fn, dev, stream, (*_rows(fn, "x", x, shape, dev), *_rows(fn, "out", out, shape, dev),
                              _ptr(fn, "positions", positions, _I32, dev, n), n, h, d,
                              ctypes.addressof(rope), 1 if backward else 0))


def _rope_append(fn, q, q_out, k_new, v_new, positions, slots, rope, scales, k_pool, v_pool,
                 stream):
    dev = _cuda_device(fn, "k_pool", k_pool, 3)
    S, hk, d = k_pool.shape
    n = k_new.shape[0]
    if (q is None) != (q_out is None):
        _bad(fn, "q and q_out: both or neither")
    hq = 0
    rows = (0, 0, 0, 0)
    if q is not None:
        if q.dim() != 3:
            _bad(fn, f"q: [n, heads, d], not {tuple(q.shape)}")
        hq = q.shape[1]
        shape = (n, hq, d)
        rows = (*_rows(fn, "q", q, shape, dev), *_rows(fn, "q_out", q_out, shape, dev))
    shape = (n, hk, d)
    kind = _BF16 if scales is None else _U8
    scale_ptrs = () if scales is None else tuple(
        _ptr(fn, "scales", t, _F32, dev, hk) for t in scales)
    _invoke(fn, dev, stream, (
        *rows, *_rows(fn, "k_new", k_new, shape, dev), *_rows(fn, "v_new", v_new, shape, dev),
        _ptr(fn, "positions", positions, _I32, dev, n), _ptr(fn, "slots", slots, _I32, dev, n),
        n, hq, hk, d, ctypes.addressof(rope), *scale_ptrs, _ptr(fn, "k_pool", k_pool, kind, dev),
        _ptr(fn, "v_pool", v_pool, kind, dev, S * hk * d), S))


def seg_attn_rope_append(q, q_out, k_new, v_new, positions, slots, rope: seg_attn_rope_desc,
                         k_pool, v_pool, stream=None) -> None:
    """q_out = rotated q; rotated k_new and v_new into their ``slots`` of the bf16 pools.  q, k_new
    and v_new [n, heads, d] may be parts of one projection; q and q_out may both be None."""
    _rope_append("seg_attn_rope_append", q, q_out, k_new, v_new, positions, slots, rope, None,
                 k_pool, v_pool, stream)


def seg_attn_rope_append_fp8(q, q_out, k_new, v_new, positions, slots, rope: seg_attn_rope_desc,
                             k_scale, v_scale, k_pool, v_pool, stream=None) -> None:
    """seg_attn_rope_append into E4M3 pools (uint8) with per-kv-head fp32 scales."""
    _rope_append("seg_attn_rope_append_fp8", q, q_out, k_new, v_new, positions, slots, rope,
                 (k_scale, v_scale), k_pool, v_pool, stream)


def seg_attn_build_tree_table(draft_lens, seg_counts, seg_starts, seg_lens, num_slots: int,
                              q_heads: int, kv_heads: int, head_dim: int, parents=None, mask=None,
                              pin: bool = False):
    """Returns (host table as an int32 torch tensor, seg_attn_tree_desc).  Raises SegAttnError."""
    fn = "seg_attn_build_tree_table"
    lib = load_library()
    dl, sc, ss, sl = _i32(draft_lens), _i32(seg_counts), _i32(seg_starts), _i32(seg_lens)
    if sc.size != dl.size or int(np.maximum(sc, 0).sum(dtype=np.int64)) != ss.size or ss.size != sl.size:
        _bad(fn, "seg_counts per request, seg_starts and seg_lens per segment")
    pa = _i32(parents) if parents is not None else None
    ma = None
    if mask is not None:
        ma = np.ascontiguousarray(np.asarray(mask).reshape(-1).astype(bool).view(np.uint8))
    t = np.maximum(dl.astype(np.int64), 0)
    if (pa is not None and pa.size != t.sum()) or (ma is not None and ma.size != (t * t).sum()):
        _bad(fn, "parents: one per drafted token; mask: draft_len^2 per request")
    desc = seg_attn_tree_desc()
    # an empty parents or mask array still says which form the trees have
    some = lambda a: None if a is None else ctypes.c_void_p(a.ctypes.data)
    args = [int(dl.size), _np_ptr(dl), some(pa), some(ma), _np_ptr(sc), _np_ptr(ss), _np_ptr(sl),
            int(num_slots), int(q_heads), int(kv_heads), int(head_dim)]
    rc = lib.seg_attn_build_tree_table(*args, None, 0, ctypes.byref(desc))
    if rc != 0:
        raise SegAttnError(fn, rc)
    host = torch.zeros(max(1, (desc.table_bytes + 3) // 4), dtype=torch.int32, pin_memory=pin)
    rc = lib.seg_attn_build_tree_table(*args, ctypes.c_void_p(host.data_ptr()),
                                       int(desc.table_bytes), ctypes.byref(desc))
    if rc != 0:
        raise SegAttnError(fn, rc)
    return host, desc


def seg_attn_tree_workspace_size(desc: seg_attn_tree_desc) -> int:
    return int(load_library().seg_attn_tree_workspace_size(ctypes.byref(desc)))


@dataclass
class TreeTable:
    """A built drafted-token table: host copy, description, device copy and workspace size."""
    host: torch.Tensor
    desc: seg_attn_tree_desc
    device: Optional[torch.Tensor] = None

    @classmethod
    def build(cls, draft_lens, seg_starts, seg_lens, num_slots, q_heads, kv_heads, head_dim,
              parents=None, mask=None, pin=False):
        """Per-request segment lists in; ``parents`` / ``mask`` flat, requests back to back."""
        host, desc = seg_attn_build_tree_table(
            draft_lens, [len(s) for s in seg_starts], [x for s in seg_starts for x in s],
            [x for s in seg_lens for x in s], num_slots, q_heads, kv_heads, head_dim,
            parents=parents, mask=mask, pin=pin)
        return cls(host=host, desc=desc)

    def to(self, device, non_blocking=False) -> "TreeTable":
        self.device = self.host.to(device, non_blocking=non_blocking)
        return self

    @property
    def workspace_bytes(self) -> int:
        return seg_attn_tree_workspace_size(self.desc)


# q_heads, kv_heads, head_dim, num_slots, total_q of the pass of a tree table
_tree_sizes = struct.Struct("=3i2q").unpack_from
_tree_sizes_at = seg_attn_tree_desc.pass_.offset + seg_attn_table_desc.q_heads.offset


def _tree(fn, q, k_pool, v_pool, scales, out, lse, dev_table, desc, softmax_scale, workspace,
          stream):
    dev = _cuda_device(fn, "q", q, 3)
    # read from the descriptor at every call: the caller may have refilled it
    hq, hk, d, slots, total_q = _tree_sizes(desc, _tree_sizes_at)
    nq, nl, pool = total_q * hq * d, total_q * hq, slots * hk * d
    kind = _BF16 if scales is None else _U8
    table = _ptr(fn, "dev_table", dev_table, _I32, dev)
    if dev_table.numel() * 4 < desc.table_bytes:
        _bad(fn, "dev_table is shorter than the table")
    scale_ptrs = () if scales is None else tuple(
        _ptr(fn, "scales", t, _F32, dev, hk) for t in scales)
    _invoke(fn, dev, stream, (
        _ptr(fn, "q", q, _BF16, dev, nq), _ptr(fn, "k_pool", k_pool, kind, dev, pool),
        _ptr(fn, "v_pool", v_pool, kind, dev, pool), *scale_ptrs,
        _ptr(fn, "out", out, _BF16, dev, nq),
        _ptr(fn, "lse", lse, _F32, dev, nl) if lse is not None else 0, table,
        ctypes.addressof(desc), _double_bits(softmax_scale),
        *((_ptr(fn, "workspace", workspace, workspace.dtype, dev), workspace.nbytes)
          if workspace is not None else (0, 0))))


def _double_bits(x: float) -> int:
    return _q_of(_of_d(x))[0]


_of_d, _q_of = struct.Struct("=d").pack, struct.Struct("=q").unpack


def seg_attn_tree(q, k_pool, v_pool, out, lse, dev_table, desc, softmax_scale, workspace=None,
                  stream=None) -> None:
    """Attention of drafted tokens (q, out bf16 [total, Hq, d]) over the bf16 pools; ``lse`` fp32
    [total, Hq] or None."""
    _tree("seg_attn_tree", q, k_pool, v_pool, None, out, lse, dev_table, desc, softmax_scale,
          workspace, stream)


def seg_attn_tree_fp8(q, k_pool, v_pool, k_scale, v_scale, out, lse, dev_table, desc,
                      softmax_scale, workspace=None, stream=None) -> None:
    """seg_attn_tree over E4M3 pools (uint8 [S, Hkv, d]) with per-kv-head fp32 scales."""
    _tree("seg_attn_tree_fp8", q, k_pool, v_pool, (k_scale, v_scale), out, lse, dev_table, desc,
          softmax_scale, workspace, stream)


def seg_attn_kv_move(k_pool, v_pool, src, dst, offsets=None, stream=None) -> None:
    """k_pool[dst[i]] = k_pool[src[i]], v_pool likewise (pools bf16 or uint8 [S, Hkv, d]; src, dst
    device int32), in order inside each group ``offsets[g] : offsets[g + 1]`` (device int32;
    None: every move on its own)."""
    fn = "seg_attn_kv_move"
    dev = _cuda_device(fn, "k_pool", k_pool, 3)
    S, hk, d = k_pool.shape
    kind = k_pool.dtype
    if kind is not _BF16 and kind is not _U8:
        _bad(fn, f"k_pool: bfloat16 or uint8, not {kind}")
    n = src.numel()
    offs = groups = 0
    if offsets is not None:
        offs, groups = _ptr(fn, "offsets", offsets, _I32, dev), offsets.numel() - 1
        if groups < 0:
            _bad(fn, "offsets: at least one value")
    _invoke(fn, dev, stream, (
        _ptr(fn, "k_pool", k_pool, kind, dev), _ptr(fn, "v_pool", v_pool, kind, dev, S * hk * d),
        _ptr(fn, "src", src, _I32, dev, n), _ptr(fn, "dst", dst, _I32, dev, n), n, offs, groups,
        hk, d, 2 if kind is _BF16 else 1, S))
