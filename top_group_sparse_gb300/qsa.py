"""Thin ctypes binding of libqsa (``include/qsa.h``, ``qsa_cache.h``, ``qsa_rows.h``) -- argument marshalling only.

Every function carries the name of the C entry point it calls and does
nothing but turn torch tensors (device memory) and plain Python values into
the C arguments; every step of the path runs in the library's CUDA kernels.
The library is loaded on first use; if it is missing or fails to load, the
call raises -- there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

__all__ = [
    "QsaError", "QsaDims", "QsaInputs", "QsaStats", "load", "library_path", "exported_symbols",
    "qsa_workspace_size", "qsa_score_stride", "qsa_row_capacity", "qsa_get_stats", "qsa_get_stats_pooled",
    "qsa_status_string", "qsa_workspace_init", "qsa_check_errors", "qsa_score_groups",
    "qsa_select", "qsa_gather", "qsa_attend", "qsa_gather_attend", "qsa_attend_state", "qsa_merge_states", "qsa_selftest_copy_timeout", "qsa_decode",
    "qsa_decode_profiled", "qsa_attend_noalloc", "qsa_pool_groups", "qsa_score_pooled",
    "qsa_decode_pooled", "qsa_score_groups_shared", "qsa_decode_shared", "qsa_probe_ffma",
    "make_dims",
    "DeviceBatch",
    "QSA_DEVERR_VISIBLE_RANGE", "QSA_DEVERR_SLOT_RANGE", "QSA_DEVERR_ROW_RANGE", "QSA_DEVERR_NOT_SHARED",
    "QSA_DEVERR_WAIT_TIMEOUT",
    "QsaCodedCache", "QsaHistory", "qsa_code_groups", "qsa_coded_workspace_size", "qsa_attend_coded",
    "qsa_decode_coded", "qsa_evict_select", "qsa_evict_compact", "QSA_CODE_E4M3", "QSA_CODE_INT8",
    "QSA_CODE_E2M1", "QSA_CODE_INT4", "code_bytes", "QsaProjection", "QsaRotation", "QsaNewTokens", "qsa_append_tokens",
    "qsa_read_groups", "QSA_ROWS_F32", "QSA_ROWS_BF16", "QSA_ROWS_F16", "QSA_PAIR_HALVES", "QSA_PAIR_NEIGHBOURS",
    "QSA_MAX_AXES", "QSA_ROWS_WORKSPACE_BYTES",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "_build", "libqsa.so")

QSA_OK = 0
QSA_ERR_DEVICE_FAULT = 5
QSA_DEVERR_VISIBLE_RANGE = 0x1
QSA_DEVERR_SLOT_RANGE = 0x2
QSA_DEVERR_ROW_RANGE = 0x4
QSA_DEVERR_WAIT_TIMEOUT = 0x8
QSA_DEVERR_NOT_SHARED = 0x10
QSA_CODE_E4M3 = 0
QSA_CODE_INT8 = 1
QSA_CODE_E2M1 = 4
QSA_CODE_INT4 = 5
QSA_ROWS_F32, QSA_ROWS_BF16, QSA_ROWS_F16 = 0, 1, 2
QSA_PAIR_HALVES, QSA_PAIR_NEIGHBOURS = 0, 1
QSA_MAX_AXES = 4
QSA_ROWS_WORKSPACE_BYTES = 256


class QsaError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: status {status}: {msg}")
        self.status = status


class QsaDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("idx_heads", ctypes.c_int32),
                ("idx_dim", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group", ctypes.c_int32), ("budget_groups", ctypes.c_int32),
                ("max_visible", ctypes.c_int32), ("scale", ctypes.c_float)]


class QsaInputs(ctypes.Structure):
    _fields_ = [("q_idx", ctypes.c_void_p), ("idx_keys", ctypes.c_void_p),
                ("key_offset", ctypes.c_void_p), ("visible", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p),
                ("v_cache", ctypes.c_void_p), ("num_slots", ctypes.c_int64),
                ("slot_map", ctypes.c_void_p), ("slot_offset", ctypes.c_void_p)]


class QsaStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "candidate_groups", "selected_groups", "selected_tokens", "raw_key_bytes", "kv_bytes",
        "pooled_key_bytes", "workspace_bytes", "total_bytes", "dense_mask_bytes")]

    def as_dict(self):
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


class QsaCodedCache(ctypes.Structure):
    """qsa_coded_cache (include/qsa_cache.h)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("block_map", ctypes.c_void_p), ("block_offset", ctypes.c_void_p), ("format", ctypes.c_int32)]

    @classmethod
    def of(cls, codes, scales, block_map, block_offset, fmt):
        """From tensors: codes [num_blocks, n_kv, code_bytes(fmt, d)] (uint8), scales [num_blocks, n_kv, 2]."""
        return cls(_ptr(codes), _ptr(scales), int(codes.shape[0]), _ptr(block_map), _ptr(block_offset), int(fmt))


class QsaHistory(ctypes.Structure):
    """qsa_history (include/qsa_cache.h)."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "idx_keys", "key_offset", "pooled", "pool_offset", "slot_map", "slot_offset", "block_map", "block_offset",
        "weights", "weight_offset", "visible")]

    @classmethod
    def of(cls, **members):
        """From tensors by member name; members left out are NULL."""
        return cls(**{k: _ptr(v) for k, v in members.items()})


class QsaProjection(ctypes.Structure):
    """qsa_projection (include/qsa_rows.h)."""
    _fields_ = [("rows", ctypes.c_void_p), ("stride", ctypes.c_int64), ("norm", ctypes.c_void_p)]


class QsaRotation(ctypes.Structure):
    """qsa_rotation (include/qsa_rows.h)."""
    _fields_ = [("freq", ctypes.c_void_p), ("dims", ctypes.c_int32), ("pairing", ctypes.c_int32)]


class QsaNewTokens(ctypes.Structure):
    """qsa_new_tokens (include/qsa_rows.h).  It holds pointers: the tensors it was made from have to live as
    long as it is used.  Made by `of`, it knows their sizes, and a call whose dims need more is refused."""
    _fields_ = ([(n, QsaProjection) for n in ("q", "k", "v", "q_idx", "idx_key")] +
                [("type", ctypes.c_int32), ("axes", ctypes.c_int32), ("positions", ctypes.c_void_p),
                 ("turn", QsaRotation), ("turn_idx", QsaRotation), ("eps", ctypes.c_float)])
    _sizes = None  # of the tensors that `of` was given
    _fits = None   # the dims that `check` has last found room for (a comparison costs a call 0.1 us, the check 1 us)

    @classmethod
    def of(cls, q=None, k=None, v=None, q_idx=None, idx_key=None, *, positions=None, freq=None, idx_freq=None,
           pairing=QSA_PAIR_HALVES, idx_pairing=None, q_norm=None, k_norm=None, q_idx_norm=None, idx_key_norm=None,
           eps=1e-6):
        """From tensors: the projections, one row per query with its heads side by side ([B, heads * width] or
        [B, heads, width], rows any stride apart), all of one type (float32, bfloat16, float16); positions
        [axes, B] or [B] int32; freq, idx_freq [axes, dims / 2] or [dims / 2] f32; norms [width] f32."""
        import torch
        given = {"q": (q, q_norm), "k": (k, k_norm), "v": (v, None), "q_idx": (q_idx, q_idx_norm),
                 "idx_key": (idx_key, idx_key_norm)}
        types = {torch.float32: QSA_ROWS_F32, torch.bfloat16: QSA_ROWS_BF16, torch.float16: QSA_ROWS_F16}
        dtypes = {x.dtype for x, _ in given.values() if x is not None}
        if len(dtypes) != 1 or not dtypes <= set(types):
            raise ValueError(f"the projections have one type of float32, bfloat16 and float16, not {dtypes or 'none'}")
        made, sizes = {}, {}
        for name, (x, norm) in given.items():
            if x is None:
                if norm is not None:
                    raise ValueError(f"{name}_norm without {name}")
                continue
            if not 2 <= x.dim() <= 3 or x.stride(-1) != 1 or (x.dim() == 3 and x.shape[1] > 1 and x.stride(1) != x.shape[2]):
                raise ValueError(f"{name}: one row per query, its heads side by side")
            # (the stride of a single row says nothing)
            width = x.shape[1] * (x.shape[2] if x.dim() == 3 else 1)
            made[name] = QsaProjection(_ptr(x), int(x.stride(0)) if x.shape[0] > 1 else width, _f32(name + "_norm", norm))
            sizes[name] = (int(x.shape[0]), int(width), None if norm is None else int(norm.numel()))
        axes = 1 if positions is None or positions.dim() == 1 else int(positions.shape[0])
        if positions is not None and (positions.dtype != torch.int32 or not positions.is_contiguous()):
            raise ValueError("positions: int32, contiguous")

        def rotation(name, f, pair):
            if f is None or f.numel() == 0:
                return QsaRotation(None, 0, int(pair))
            if (1 if f.dim() == 1 else f.shape[0]) != axes:
                raise ValueError(f"{name} has a row for each of the {axes} axes of positions")
            return QsaRotation(_f32(name, f), 2 * int(f.shape[-1]), int(pair))

        self = cls(type=types[dtypes.pop()], axes=axes, positions=_ptr(positions), eps=float(eps),
                   turn=rotation("freq", freq, pairing),
                   turn_idx=rotation("idx_freq", idx_freq, pairing if idx_pairing is None else idx_pairing), **made)
        self._sizes = sizes
        self._places = {n: (x.rows, x.norm) for n, x in made.items()}, self.positions
        self._position_row = None if positions is None else int(positions.shape[-1])
        return self

    def _turned(self):
        return bool((self.turn.dims and (self.q.rows or self.k.rows)) or
                    (self.turn_idx.dims and (self.q_idx.rows or self.idx_key.rows)))

    def check(self, dims):
        """Raises ValueError where a call with these dims would read past a tensor that `of` was given: fewer rows
        or positions than the batch has queries (of several axes also more positions, which would be read from the
        wrong places), rows shorter than their heads, norms shorter than a head.  A pointer that was put in the
        place of such a tensor's later is taken as it is."""
        if self._sizes is None:
            return
        batch, d, di = dims.batch, dims.head_dim, dims.idx_dim
        heads = {"q": dims.q_heads, "k": dims.kv_heads, "v": dims.kv_heads, "q_idx": dims.idx_heads, "idx_key": 1}
        places, positions = self._places
        for name, (rows, elements, norm) in self._sizes.items():
            now, width = getattr(self, name), di if "idx" in name else d
            same = now.rows == places[name][0]
            if same and rows < batch:
                raise ValueError(f"{name} has {rows} rows, the batch {batch} queries")
            if same and elements < heads[name] * width:
                raise ValueError(f"{name} has {elements} elements a row, not {heads[name]} heads of {width}")
            if now.rows and norm is not None and now.norm == places[name][1] and norm < width:
                raise ValueError(f"{name}_norm has {norm} weights, not {width}")
        n = self._position_row
        if n is not None and self.positions == positions and self._turned() and (n < batch or (self.axes > 1 and n != batch)):
            raise ValueError(f"positions have {n} entries an axis, the batch {batch} queries")
        self._fits = bytes(dims)


_lib = None
_P = ctypes.c_void_p
_NP = ctypes.POINTER(QsaNewTokens)
_CP = ctypes.POINTER(QsaCodedCache)
_HP = ctypes.POINTER(QsaHistory)
_DP = ctypes.POINTER(QsaDims)
_IP = ctypes.POINTER(QsaInputs)


def library_path() -> str:
    return _LIB_PATH


def load(path: str | None = None):
    """Load libqsa.so (raises if it is not built or cannot be loaded)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libqsa.so is not built ({p}); run __graft_entry__.build() first")
    L = ctypes.CDLL(p)
    L.qsa_workspace_size.argtypes = [_DP]
    L.qsa_workspace_size.restype = ctypes.c_size_t
    L.qsa_score_stride.argtypes = [_DP]
    L.qsa_score_stride.restype = ctypes.c_int64
    L.qsa_row_capacity.argtypes = [_DP]
    L.qsa_row_capacity.restype = ctypes.c_int32
    L.qsa_get_stats.argtypes = [_DP, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(QsaStats)]
    L.qsa_get_stats.restype = ctypes.c_int
    L.qsa_get_stats_pooled.argtypes = [_DP, ctypes.POINTER(ctypes.c_int32), ctypes.c_int64, ctypes.POINTER(QsaStats)]
    L.qsa_get_stats_pooled.restype = ctypes.c_int
    L.qsa_status_string.argtypes = [ctypes.c_int]
    L.qsa_status_string.restype = ctypes.c_char_p
    L.qsa_workspace_init.argtypes = [_P, ctypes.c_size_t, _P]
    L.qsa_workspace_init.restype = ctypes.c_int
    L.qsa_check_errors.argtypes = [_P, ctypes.c_size_t, _P, ctypes.POINTER(ctypes.c_uint32)]
    L.qsa_check_errors.restype = ctypes.c_int
    L.qsa_score_groups.argtypes = [_DP, _IP, _P, _P, ctypes.c_size_t, _P]
    L.qsa_score_groups.restype = ctypes.c_int
    L.qsa_select.argtypes = [_DP, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_select.restype = ctypes.c_int
    L.qsa_gather.argtypes = [_DP, _IP, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_gather.restype = ctypes.c_int
    L.qsa_attend.argtypes = [_DP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_attend.restype = ctypes.c_int
    L.qsa_gather_attend.argtypes = [_DP, _IP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_gather_attend.restype = ctypes.c_int
    L.qsa_attend_state.argtypes = [_DP, _IP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_attend_state.restype = ctypes.c_int
    L.qsa_merge_states.argtypes = [_DP, ctypes.c_int32, _P, _P, _P, _P, _P]
    L.qsa_selftest_copy_timeout.argtypes = [_DP, _IP, _P, _P, ctypes.c_size_t, ctypes.c_uint64, _P]
    L.qsa_selftest_copy_timeout.restype = ctypes.c_int
    L.qsa_merge_states.restype = ctypes.c_int
    L.qsa_decode.argtypes = [_DP, _IP, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_decode.restype = ctypes.c_int
    L.qsa_decode_profiled.argtypes = [_DP, _IP, _P, _P, _P, _P, ctypes.c_size_t, _P,
                                      ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32]
    L.qsa_decode_profiled.restype = ctypes.c_int
    L.qsa_attend_noalloc.argtypes = [_DP, _P, _P, _P, _P, _P, _P]
    L.qsa_attend_noalloc.restype = ctypes.c_int
    L.qsa_pool_groups.argtypes = [_DP, _IP, _P, _P, ctypes.c_int32, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_pool_groups.restype = ctypes.c_int
    L.qsa_score_pooled.argtypes = [_DP, _IP, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_score_pooled.restype = ctypes.c_int
    L.qsa_decode_pooled.argtypes = [_DP, _IP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_decode_pooled.restype = ctypes.c_int
    L.qsa_score_groups_shared.argtypes = [_DP, _IP, _P, _P, ctypes.c_size_t, _P]
    L.qsa_score_groups_shared.restype = ctypes.c_int
    L.qsa_decode_shared.argtypes = [_DP, _IP, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_decode_shared.restype = ctypes.c_int
    L.qsa_probe_ffma.argtypes = [ctypes.c_int32, ctypes.c_int32, _P, ctypes.POINTER(ctypes.c_int64), _P]
    L.qsa_probe_ffma.restype = ctypes.c_int
    L.qsa_coded_workspace_size.argtypes = [_DP, ctypes.c_int32, ctypes.c_int32]
    L.qsa_coded_workspace_size.restype = ctypes.c_size_t
    L.qsa_code_groups.argtypes = [_DP, _IP, _CP, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]
    L.qsa_code_groups.restype = ctypes.c_int
    L.qsa_attend_coded.argtypes = [_DP, _IP, _CP, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_attend_coded.restype = ctypes.c_int
    L.qsa_decode_coded.argtypes = [_DP, _IP, _CP, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
    L.qsa_decode_coded.restype = ctypes.c_int
    L.qsa_evict_select.argtypes = [_DP, _P, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P,
                                   ctypes.c_size_t, _P]
    L.qsa_evict_select.restype = ctypes.c_int
    L.qsa_evict_compact.argtypes = [_DP, ctypes.c_int32, _P, _P, _HP, _HP, _P, ctypes.c_size_t, _P]
    L.qsa_evict_compact.restype = ctypes.c_int
    L.qsa_append_tokens.argtypes = [_DP, _IP, _NP, _P, ctypes.c_size_t, _P]
    L.qsa_append_tokens.restype = ctypes.c_int
    L.qsa_read_groups.argtypes = [_DP, _IP, _CP, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]
    L.qsa_read_groups.restype = ctypes.c_int
    if path is None:
        _lib = L
    return L


def exported_symbols(header: str | None = None) -> list[str]:
    """Names of the functions include/qsa.h (or the given header) declares."""
    import re
    header = header or os.path.join(os.path.dirname(_PKG), "include", "qsa.h")
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(qsa_[a-z_]+)\s*\(", text)))


# ---- marshalling helpers ----------------------------------------------------

def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _f32(name, x) -> int | None:
    """Pointer of a contiguous float32 tensor (None: NULL)."""
    import torch
    if x is not None and (x.dtype != torch.float32 or not x.is_contiguous()):
        raise ValueError(f"{name}: float32, contiguous")
    return _ptr(x)


def _stream(stream) -> int | None:
    if stream is None:
        # the current stream's handle without a Stream object around it (0.3 us instead of 3 us), where
        # torch has that: it is not of its public interface
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return int(torch.cuda.current_stream().cuda_stream) if raw is None else raw(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _ws(ws):
    """(pointer, bytes) of a workspace given as a tensor or a (ptr, bytes) pair."""
    if isinstance(ws, tuple):
        return ws
    return _ptr(ws), ws.numel() * ws.element_size()


def _check(fn: str, st: int):
    if st != QSA_OK:
        raise QsaError(fn, st, load().qsa_status_string(st).decode())
    return st


def make_dims(batch, idx_heads, idx_dim, q_heads, kv_heads, head_dim, budget_groups=512,
              max_visible=0, scale=None, group=4) -> QsaDims:
    if scale is None:
        scale = float(np.float32(1.0 / np.sqrt(head_dim)))
    return QsaDims(int(batch), int(idx_heads), int(idx_dim), int(q_heads), int(kv_heads),
                   int(head_dim), int(group), int(budget_groups), int(max_visible), float(scale))


# ---- the C entry points -----------------------------------------------------

def qsa_workspace_size(dims: QsaDims) -> int:
    return int(load().qsa_workspace_size(ctypes.byref(dims)))


def qsa_score_stride(dims: QsaDims) -> int:
    return int(load().qsa_score_stride(ctypes.byref(dims)))


def qsa_row_capacity(dims: QsaDims) -> int:
    return int(load().qsa_row_capacity(ctypes.byref(dims)))


def qsa_get_stats(dims: QsaDims, visible_host) -> dict:
    vis = np.ascontiguousarray(np.asarray(visible_host, dtype=np.int32))
    st = QsaStats()
    _check("qsa_get_stats", load().qsa_get_stats(
        ctypes.byref(dims), vis.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), ctypes.byref(st)))
    return st.as_dict()


def qsa_get_stats_pooled(dims: QsaDims, visible_host, pooled_rows: int) -> dict:
    vis = np.ascontiguousarray(np.asarray(visible_host, dtype=np.int32))
    st = QsaStats()
    _check("qsa_get_stats_pooled", load().qsa_get_stats_pooled(
        ctypes.byref(dims), vis.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), int(pooled_rows),
        ctypes.byref(st)))
    return st.as_dict()


def qsa_status_string(status: int) -> str:
    return load().qsa_status_string(int(status)).decode()


def qsa_workspace_init(ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_workspace_init", load().qsa_workspace_init(p, n, _stream(stream)))


def qsa_check_errors(ws, stream=None) -> tuple[int, int]:
    """Returns (status, flags); does not raise on QSA_ERR_DEVICE_FAULT."""
    p, n = _ws(ws)
    flags = ctypes.c_uint32(0)
    st = load().qsa_check_errors(p, n, _stream(stream), ctypes.byref(flags))
    if st not in (QSA_OK, QSA_ERR_DEVICE_FAULT):
        _check("qsa_check_errors", st)
    return int(st), int(flags.value)


def qsa_score_groups(dims, inputs, scores, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_score_groups", load().qsa_score_groups(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(scores), p, n, _stream(stream)))


def qsa_select(dims, visible, scores, ids, n_ids, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_select", load().qsa_select(
        ctypes.byref(dims), _ptr(visible), _ptr(scores), _ptr(ids), _ptr(n_ids), p, n,
        _stream(stream)))


def qsa_gather(dims, inputs, ids, n_ids, k_scr, v_scr, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_gather", load().qsa_gather(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(ids), _ptr(n_ids), _ptr(k_scr),
        _ptr(v_scr), p, n, _stream(stream)))


def qsa_attend(dims, q, k_scr, v_scr, n_ids, out, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_attend", load().qsa_attend(
        ctypes.byref(dims), _ptr(q), _ptr(k_scr), _ptr(v_scr), _ptr(n_ids), _ptr(out), p, n,
        _stream(stream)))


def qsa_gather_attend(dims, inputs, ids, n_ids, k_scr, v_scr, out, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_gather_attend", load().qsa_gather_attend(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(ids), _ptr(n_ids), _ptr(k_scr), _ptr(v_scr),
        _ptr(out), p, n, _stream(stream)))


def qsa_attend_state(dims, inputs, ids, n_ids, acc, m, l, ws, stream=None) -> int:
    """Online-softmax state (acc [B, n_q, d], m [B, n_q], l [B, n_q]) of each
    query's rows ids[b, :n_ids[b]], resolved through the slot map."""
    p, n = _ws(ws)
    return _check("qsa_attend_state", load().qsa_attend_state(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(ids), _ptr(n_ids), _ptr(acc), _ptr(m), _ptr(l),
        p, n, _stream(stream)))


def qsa_selftest_copy_timeout(dims, inputs, scores, ws, wait_ns, stream=None) -> int:
    """The failure-detection self-test (include/qsa_selftest.h): the raw scorer
    with no copy issued, so that every CTA's bounded wait runs out after wait_ns."""
    p, n = _ws(ws)
    return _check("qsa_selftest_copy_timeout", load().qsa_selftest_copy_timeout(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(scores), p, n, int(wait_ns), _stream(stream)))


def qsa_merge_states(dims, n_parts, m, l, acc, out, stream=None) -> int:
    """Output [B, n_q, d] of rows whose consecutive slices' states are
    m, l [n_parts, B, n_q] and acc [n_parts, B, n_q, d], merged in slice order."""
    return _check("qsa_merge_states", load().qsa_merge_states(
        ctypes.byref(dims), int(n_parts), _ptr(m), _ptr(l), _ptr(acc), _ptr(out), _stream(stream)))


def qsa_decode(dims, inputs, ids, n_ids, out, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_decode", load().qsa_decode(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(ids), _ptr(n_ids), _ptr(out), p, n,
        _stream(stream)))


def qsa_decode_profiled(dims, inputs, ids, n_ids, out, ws, events, stream=None) -> int:
    """events: four torch.cuda.Event(enable_timing=True) (or raw cudaEvent_t ints)."""
    handles = []
    for e in events:
        if isinstance(e, int):
            handles.append(e)
        else:
            if not e.cuda_event:  # torch creates the CUDA event on first record
                e.record()
            handles.append(int(e.cuda_event))
    arr = (ctypes.c_void_p * len(handles))(*handles)
    p, n = _ws(ws)
    return _check("qsa_decode_profiled", load().qsa_decode_profiled(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(ids), _ptr(n_ids), _ptr(out), p, n,
        _stream(stream), arr, len(handles)))


def qsa_pool_groups(dims, inputs, group_begin, group_end, max_groups, pooled, pool_offset, ws,
                    stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_pool_groups", load().qsa_pool_groups(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(group_begin), _ptr(group_end), int(max_groups),
        _ptr(pooled), _ptr(pool_offset), p, n, _stream(stream)))


def qsa_score_pooled(dims, inputs, pooled, pool_offset, scores, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_score_pooled", load().qsa_score_pooled(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(pooled), _ptr(pool_offset), _ptr(scores), p, n,
        _stream(stream)))


def qsa_decode_pooled(dims, inputs, pooled, pool_offset, ids, n_ids, out, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_decode_pooled", load().qsa_decode_pooled(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(pooled), _ptr(pool_offset), _ptr(ids),
        _ptr(n_ids), _ptr(out), p, n, _stream(stream)))


def qsa_score_groups_shared(dims, inputs, scores, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_score_groups_shared", load().qsa_score_groups_shared(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(scores), p, n, _stream(stream)))


def qsa_decode_shared(dims, inputs, ids, n_ids, out, ws, stream=None) -> int:
    p, n = _ws(ws)
    return _check("qsa_decode_shared", load().qsa_decode_shared(
        ctypes.byref(dims), ctypes.byref(inputs), _ptr(ids), _ptr(n_ids), _ptr(out), p, n,
        _stream(stream)))


def qsa_probe_ffma(blocks_per_sm, iters, sink, stream=None) -> int:
    """Launches the FFMA throughput probe; returns the FMAs it performs."""
    count = ctypes.c_int64(0)
    _check("qsa_probe_ffma", load().qsa_probe_ffma(int(blocks_per_sm), int(iters), _ptr(sink),
                                                   ctypes.byref(count), _stream(stream)))
    return int(count.value)


def qsa_attend_noalloc(dims, q, k_scr, v_scr, n_ids, out, stream=None) -> int:
    """Attention stage with the library's fixed static scratch instead of a
    workspace, for callers that cannot allocate device memory."""
    return _check("qsa_attend_noalloc", load().qsa_attend_noalloc(
        ctypes.byref(dims), _ptr(q), _ptr(k_scr), _ptr(v_scr), _ptr(n_ids), _ptr(out),
        _stream(stream)))


# ---- the coded cache and the eviction (include/qsa_cache.h) ------------------

def qsa_coded_workspace_size(dims, whole_history=False, with_weights=False) -> int:
    return int(load().qsa_coded_workspace_size(ctypes.byref(dims), int(bool(whole_history)), int(bool(with_weights))))


def qsa_code_groups(dims, inputs, cache, group_begin, group_end, max_groups, ws, stream=None) -> int:
    """Codes groups [group_begin[b], group_end[b]) of every query into its blocks of the coded cache."""
    p, n = _ws(ws)
    return _check("qsa_code_groups", load().qsa_code_groups(
        ctypes.byref(dims), ctypes.byref(inputs), ctypes.byref(cache), _ptr(group_begin), _ptr(group_end),
        int(max_groups), p, n, _stream(stream)))


def qsa_attend_coded(dims, inputs, cache, ids, n_ids, out, ws, weights=None, weight_offset=None, stream=None) -> int:
    """Attention over the coded cache: over the rows ids[b, :n_ids[b]], or (ids = n_ids = None) over every
    visible token; weights: the accumulators that the groups' shares of attention are added to."""
    p, n = _ws(ws)
    return _check("qsa_attend_coded", load().qsa_attend_coded(
        ctypes.byref(dims), ctypes.byref(inputs), ctypes.byref(cache), _ptr(ids), _ptr(n_ids), _ptr(out),
        _ptr(weights), _ptr(weight_offset), p, n, _stream(stream)))


def qsa_decode_coded(dims, inputs, cache, ids, n_ids, out, ws, pooled=None, pool_offset=None, weights=None,
                     weight_offset=None, stream=None) -> int:
    """The whole path over a coded cache, scored from the pooled-key cache when `pooled` is given."""
    p, n = _ws(ws)
    return _check("qsa_decode_coded", load().qsa_decode_coded(
        ctypes.byref(dims), ctypes.byref(inputs), ctypes.byref(cache), _ptr(pooled), _ptr(pool_offset), _ptr(ids),
        _ptr(n_ids), _ptr(out), _ptr(weights), _ptr(weight_offset), p, n, _stream(stream)))


def qsa_evict_select(dims, visible, weights, weight_offset, keep_groups, sink_groups, recent_groups, kept, n_kept, ws,
                     evicted=None, stream=None) -> int:
    """The groups each history keeps: kept [B, keep_groups] ascending, n_kept [B]; evicted: the others."""
    p, n = _ws(ws)
    return _check("qsa_evict_select", load().qsa_evict_select(
        ctypes.byref(dims), _ptr(visible), _ptr(weights), _ptr(weight_offset), int(keep_groups), int(sink_groups),
        int(recent_groups), _ptr(kept), _ptr(n_kept), _ptr(evicted), p, n, _stream(stream)))


def qsa_evict_compact(dims, keep_groups, kept, n_kept, src, dst, ws, stream=None) -> int:
    """Moves the kept groups of the histories `src` to `dst` (QsaHistory each)."""
    p, n = _ws(ws)
    return _check("qsa_evict_compact", load().qsa_evict_compact(
        ctypes.byref(dims), int(keep_groups), _ptr(kept), _ptr(n_kept), ctypes.byref(src), ctypes.byref(dst), p, n,
        _stream(stream)))


# ---- rows into the caches and back (include/qsa_rows.h) ----------------------

def code_bytes(fmt: int, head_dim: int) -> int:
    """Bytes of one (group, KV head)'s codes in a coded cache."""
    return 9 * head_dim // 2 if fmt in (QSA_CODE_E2M1, QSA_CODE_INT4) else 8 * head_dim


def qsa_append_tokens(dims, inputs, tokens, ws, stream=None) -> int:
    """Normalises and rotates the new token (the last visible one) of every query and writes it where `inputs`
    points: q, q_idx, its row of idx_keys, its slot of k_cache / v_cache.  Tokens made of tensors that are too
    small for dims raise ValueError."""
    if tokens._fits != bytes(dims):
        tokens.check(dims)
    p, n = _ws(ws)
    return _check("qsa_append_tokens", load().qsa_append_tokens(
        ctypes.byref(dims), ctypes.byref(inputs), ctypes.byref(tokens), p, n, _stream(stream)))


def qsa_read_groups(dims, inputs, cache, group_begin, group_end, max_groups, ws, stream=None) -> int:
    """Writes groups [group_begin[b], group_end[b]) of every query from its blocks of the coded cache back to their
    rows of k_cache / v_cache."""
    p, n = _ws(ws)
    return _check("qsa_read_groups", load().qsa_read_groups(
        ctypes.byref(dims), ctypes.byref(inputs), ctypes.byref(cache), _ptr(group_begin), _ptr(group_end),
        int(max_groups), p, n, _stream(stream)))


# ---- device-resident batch (plumbing: torch owns the memory) ----------------

def _packed(arrays, device):
    """One uint8 device buffer holding the given (name, numpy array or
    (shape, dtype, fill)) items back to back, each on a 16-byte boundary;
    returns (buffer, {name: typed view})."""
    import torch
    items, off = [], 0
    for name, a in arrays:
        if isinstance(a, tuple):
            shape, dtype, fill = a
            nbytes = int(np.prod(shape)) * np.dtype(dtype).itemsize
        else:
            a = np.ascontiguousarray(a)
            shape, dtype, fill, nbytes = a.shape, a.dtype, None, a.nbytes
        off = (off + 15) // 16 * 16
        items.append((name, off, shape, dtype, fill, a))
        off += nbytes
    buf = torch.zeros(max(off, 16), dtype=torch.uint8, device=device)
    views = {}
    tdt = {np.dtype(np.float32): torch.float32, np.dtype(np.int32): torch.int32,
           np.dtype(np.int64): torch.int64}
    for name, o, shape, dtype, fill, a in items:
        n = int(np.prod(shape)) * np.dtype(dtype).itemsize
        v = buf[o:o + n].view(tdt[np.dtype(dtype)]).view(tuple(shape))
        if fill is None:
            v.copy_(torch.from_numpy(a))
        else:
            v.fill_(fill)
        views[name] = v
    return buf, views


class DeviceBatch:
    """The arrays of one workload copied into device memory, with the output
    buffers and the workspace the library needs, all allocated by torch.

    A decode step's own inputs (q_idx, q, visible, key_offset, slot_offset)
    share one buffer, `step_in`, and its outputs (ids, n_ids, out) another,
    `step_out`: a step driven from host memory is one copy in and one copy
    out (`step_host_buffers`, `decode_from_host`)."""

    def __init__(self, w, device="cuda", budget=None, queries=None):
        import torch
        self.w = w
        sel = np.arange(w.batch) if queries is None else np.asarray(queries, np.int64)
        dev = torch.device(device)

        def put(a):
            return torch.from_numpy(np.ascontiguousarray(a)).to(dev)

        self.step_in, v = _packed([("q_idx", w.q_idx[sel]), ("q", w.q[sel]),
                                   ("visible", w.visible[sel]), ("key_offset", w.key_offset[sel]),
                                   ("slot_offset", w.slot_offset[sel])], dev)
        self.q_idx, self.q, self.visible = v["q_idx"], v["q"], v["visible"]
        self.key_offset, self.slot_offset = v["key_offset"], v["slot_offset"]
        self.idx_keys = put(w.idx_keys)
        self.k_cache = put(w.k_cache)
        self.v_cache = put(w.v_cache)
        self.slot_map = put(w.slot_map)
        B = len(sel)
        mv = int(w.visible[sel].max(initial=0))
        self.dims = make_dims(B, w.idx_heads, w.idx_dim, w.q_heads, w.kv_heads, w.head_dim,
                              budget_groups=w.budget if budget is None else budget,
                              max_visible=max(mv, w.max_visible if queries is None else mv),
                              scale=w.scale)
        self.inputs = QsaInputs(
            _ptr(self.q_idx), _ptr(self.idx_keys), _ptr(self.key_offset), _ptr(self.visible),
            _ptr(self.q), _ptr(self.k_cache), _ptr(self.v_cache), int(w.num_slots),
            _ptr(self.slot_map), _ptr(self.slot_offset))
        self.row_cap = qsa_row_capacity(self.dims)
        self.score_stride = qsa_score_stride(self.dims)
        nbytes = qsa_workspace_size(self.dims)
        if nbytes == 0:
            raise ValueError("invalid dims")
        # zero-filled: the workspace header must start clean
        self.ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self.coded_ws = None  # of the calls over a coded cache (make_coded_cache)
        self.step_out, v = _packed([("ids", ((B, self.row_cap), np.int32, -1)),
                                    ("n_ids", ((B,), np.int32, -1)),
                                    ("out", ((B, w.q_heads, w.head_dim), np.float32, float("nan")))], dev)
        self.ids, self.n_ids, self.out = v["ids"], v["n_ids"], v["out"]
        self.scores = torch.full((B, self.score_stride), float("nan"), dtype=torch.float32, device=dev)
        self.k_scr = torch.zeros((B, self.row_cap, w.kv_heads, w.head_dim), dtype=torch.float32, device=dev)
        self.v_scr = torch.zeros_like(self.k_scr)

    # a decode step driven from host memory: one copy in, one copy out
    def step_host_buffers(self):
        """Pinned host buffers laid out like step_in (holding this batch's
        current step inputs) and step_out."""
        import torch
        h_in = torch.empty(self.step_in.shape, dtype=torch.uint8).pin_memory()
        h_in.copy_(self.step_in)
        h_out = torch.empty(self.step_out.shape, dtype=torch.uint8).pin_memory()
        return h_in, h_out

    def step_slot(self):
        """A second device buffer laid out like step_in (holding the same step
        inputs) and the QsaInputs that point into it -- the history, the K/V
        caches and the slot map stay shared -- so that two host-driven steps
        can be in flight at once: one step's inputs copied in while the other
        step's kernels run.  Returns (buffer, inputs)."""
        buf = self.step_in.clone()
        base = self.step_in.data_ptr()

        def at(t):
            return buf.data_ptr() + (t.data_ptr() - base)

        inp = QsaInputs(at(self.q_idx), _ptr(self.idx_keys), at(self.key_offset), at(self.visible), at(self.q),
                        _ptr(self.k_cache), _ptr(self.v_cache), int(self.inputs.num_slots), _ptr(self.slot_map),
                        at(self.slot_offset))
        return buf, inp

    def decode_from_host(self, h_in, h_out, stream=None):
        """One step on the current torch stream (or `stream`): the step's
        inputs from h_in, qsa_decode, the ID rows, counts and outputs to
        h_out (both copies asynchronous; synchronise before reading h_out)."""
        import torch
        s = stream if stream is not None else torch.cuda.current_stream()
        with torch.cuda.stream(s):
            self.step_in.copy_(h_in, non_blocking=True)
            self.decode(s)
            h_out.copy_(self.step_out, non_blocking=True)

    def decode_into_host(self, h_in, h_out, stream=None):
        """One step on the current torch stream (or `stream`): the step's
        inputs copied in from h_in, then qsa_decode with its ID rows, counts
        and outputs pointing straight into the pinned host buffer h_out (laid
        out like step_out): the last kernel stores them there, so no copy
        follows.  Synchronise before reading h_out."""
        import torch
        s = stream if stream is not None else torch.cuda.current_stream()
        hi, hn, ho = self.host_outputs(h_out)
        with torch.cuda.stream(s):
            self.step_in.copy_(h_in, non_blocking=True)
            qsa_decode(self.dims, self.inputs, hi, hn, ho, self.ws, s)

    def capture_decode_from_host(self, h_in, h_out, direct=False):
        """A CUDA graph of one host-driven step (copy in, qsa_decode, copy
        out), for a loop that repeats it: `g.replay()` on the current stream
        launches the whole step at once.  Run one eager step first (the
        library's one-time per-device setup must not happen during capture).
        The step reads the per-SM scorer weights from the workspace when it
        runs, so replays keep learning them."""
        import torch
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                if direct:
                    self.decode_into_host(h_in, h_out, s)
                else:
                    self.decode_from_host(h_in, h_out, s)
        torch.cuda.current_stream().wait_stream(s)
        return g

    def host_outputs(self, h_out):
        """(ids, n_ids, out) views of a host buffer laid out like step_out."""
        import torch
        res = []
        for t in (self.ids, self.n_ids, self.out):
            o = t.data_ptr() - self.step_out.data_ptr()
            n = t.numel() * t.element_size()
            res.append(h_out[o:o + n].view(t.dtype).view(t.shape))
        return tuple(res)

    # the four stages and the whole path, on this batch's buffers
    def score(self, stream=None):
        return qsa_score_groups(self.dims, self.inputs, self.scores, self.ws, stream)

    def select(self, stream=None):
        return qsa_select(self.dims, self.visible, self.scores, self.ids, self.n_ids, self.ws, stream)

    def gather(self, stream=None):
        return qsa_gather(self.dims, self.inputs, self.ids, self.n_ids, self.k_scr, self.v_scr,
                          self.ws, stream)

    def attend(self, stream=None):
        return qsa_attend(self.dims, self.q, self.k_scr, self.v_scr, self.n_ids, self.out,
                          self.ws, stream)

    def gather_attend(self, stream=None):
        return qsa_gather_attend(self.dims, self.inputs, self.ids, self.n_ids, self.k_scr,
                                 self.v_scr, self.out, self.ws, stream)

    def decode(self, stream=None):
        return qsa_decode(self.dims, self.inputs, self.ids, self.n_ids, self.out, self.ws, stream)

    def decode_profiled(self, events, stream=None):
        return qsa_decode_profiled(self.dims, self.inputs, self.ids, self.n_ids, self.out, self.ws,
                                   events, stream)

    # ---- the incremental form: a pooled-key cache -----------------------------
    def make_pooled_cache(self):
        """Allocates the pooled-key cache: one block of rows per distinct
        history (queries that share a history share its rows), room for the
        longest T over the queries of that history."""
        import torch
        ko = self.key_offset.cpu().numpy()
        T = self.visible.cpu().numpy()
        base, rows = {}, 0
        for k in sorted(set(ko.tolist())):
            base[k] = rows
            rows += int(T[ko == k].max()) // 4
        self.pool_offset = torch.from_numpy(np.array([base[k] for k in ko.tolist()], np.int64)).to(self.q.device)
        self.pooled = torch.zeros((max(rows, 1), self.w.idx_dim), dtype=torch.float32, device=self.q.device)
        # the query of each history with the longest T pools the history's groups
        owner = {}
        for b, k in enumerate(ko.tolist()):
            if k not in owner or T[b] > T[owner[k]]:
                owner[k] = b
        self._pool_owner = np.array([owner[k] == b for b, k in enumerate(ko.tolist())])
        return self.pooled

    def pool(self, group_begin, group_end, stream=None):
        """Appends groups [group_begin[b], group_end[b]) of every query (host arrays)."""
        import torch
        gb = np.asarray(group_begin, np.int32)
        ge = np.asarray(group_end, np.int32)
        mg = int((ge - gb).max(initial=0))
        dev = self.q.device
        self._pool_args = (torch.from_numpy(gb).to(dev), torch.from_numpy(ge).to(dev))
        return qsa_pool_groups(self.dims, self.inputs, self._pool_args[0], self._pool_args[1], max(mg, 0),
                               self.pooled, self.pool_offset, self.ws, stream)

    def pool_all(self, stream=None):
        """Pools every complete group of every history (once per history)."""
        G = (self.visible.cpu().numpy() // 4).astype(np.int32)
        ge = np.where(self._pool_owner, G, 0).astype(np.int32)
        return self.pool(np.zeros_like(ge), ge, stream)

    def score_pooled(self, stream=None):
        return qsa_score_pooled(self.dims, self.inputs, self.pooled, self.pool_offset, self.scores,
                                self.ws, stream)

    def decode_pooled(self, stream=None):
        return qsa_decode_pooled(self.dims, self.inputs, self.pooled, self.pool_offset, self.ids,
                                 self.n_ids, self.out, self.ws, stream)

    # ---- new tokens -------------------------------------------------------------
    def append(self, tokens, stream=None):
        """Writes the batch's new tokens (a QsaNewTokens) into q, q_idx, idx_keys and the K/V cache."""
        return qsa_append_tokens(self.dims, self.inputs, tokens, self.ws, stream)

    # ---- a K/V cache in 8 or 4 bits ---------------------------------------------
    def make_coded_cache(self, fmt=QSA_CODE_E4M3):
        """Allocates the coded cache: one block per complete group of each distinct
        history (in order), its accumulated weights (one per group and one for an
        incomplete one) and a workspace that serves every call on this batch.  Histories
        that are to grow are as long as they will be when this is called."""
        import torch
        ko = self.key_offset.cpu().numpy()
        T = self.visible.cpu().numpy()
        block, weight, blocks, weights, owner = {}, {}, 0, 0, {}
        for b, k in enumerate(ko.tolist()):
            if k not in owner or T[b] > T[owner[k]]:
                owner[k] = b
        for k in sorted(owner):
            block[k], weight[k] = blocks, weights
            blocks += int(T[owner[k]]) // 4
            weights += -(-int(T[owner[k]]) // 4)
        dev, w = self.q.device, self.w

        def put(rows):
            return torch.from_numpy(np.array([rows[k] for k in ko.tolist()], np.int64)).to(dev)

        self.block_offset, self.weight_offset = put(block), put(weight)
        self.block_map = torch.arange(max(blocks, 1), dtype=torch.int32, device=dev)
        self.codes = torch.zeros((max(blocks, 1), w.kv_heads, code_bytes(fmt, w.head_dim)), dtype=torch.uint8, device=dev)
        self.scales = torch.zeros((max(blocks, 1), w.kv_heads, 2), dtype=torch.float32, device=dev)
        self.weights = torch.zeros(max(weights, 1), dtype=torch.float32, device=dev)
        self.coded = QsaCodedCache.of(self.codes, self.scales, self.block_map, self.block_offset, fmt)
        self.coded_ws = torch.zeros(qsa_coded_workspace_size(self.dims, True, True), dtype=torch.uint8, device=dev)
        self._code_history = np.unique(ko, return_inverse=True)[1].reshape(-1)
        self._code_room = np.array([int(T[owner[k]]) // 4 for k in ko.tolist()], np.int32), self.coded
        return self.coded

    def _check_blocks(self, group_begin, group_end):
        """Refuses groups behind the last block of their history, whose entries of the block map are another's."""
        room, made = self._code_room
        if made is not self.coded:  # (a cache of the caller's own)
            return
        over = np.flatnonzero((group_end > group_begin) & (group_end > room))
        if len(over):
            b = int(over[0])
            raise ValueError(f"query {b}: groups up to {int(group_end[b])} of a history that had blocks for {int(room[b])} "
                             "when the cache was made")

    def _whole_histories(self):
        """Group ends per query that cover every complete group of each history once, as the batch stands: at the first
        of the queries that see most of it."""
        T, of = self.visible.cpu().numpy(), self._code_history
        order = np.lexsort((np.arange(len(T)), -T.astype(np.int64), of))
        first = order[np.r_[True, of[order][1:] != of[order][:-1]]] if len(T) else order
        ge = np.zeros(len(T), np.int32)
        ge[first] = T[first] // 4
        ge[T < 0] = -1  # (the call flags it)
        return ge

    def code(self, group_begin, group_end, stream=None):
        """Codes groups [group_begin[b], group_end[b]) of every query (host arrays, copied on `stream`:
        not for a capture, where qsa_code_groups takes device arrays)."""
        import torch
        gb, ge = np.asarray(group_begin, np.int32), np.asarray(group_end, np.int32)
        if gb.shape != (self.dims.batch,) or ge.shape != gb.shape:
            raise ValueError(f"group_begin and group_end have one entry per query ({self.dims.batch})")
        self._check_blocks(gb, ge)
        handle = _stream(stream)
        on = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
        with torch.cuda.stream(on):  # their memory is that stream's, until the next call there
            args = torch.from_numpy(np.stack([gb, ge])).to(self.q.device)
            return qsa_code_groups(self.dims, self.inputs, self.coded, args[0], args[1],
                                   max(int((ge - gb).max(initial=0)), 0), self.coded_ws, handle)

    def read_back(self, stream=None):
        """Writes every complete group of every history from its codes back to its rows of k_cache / v_cache."""
        import torch
        ge = self._whole_histories()
        self._check_blocks(np.zeros_like(ge), ge)
        handle = _stream(stream)
        on = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
        with torch.cuda.stream(on):
            args = torch.from_numpy(np.stack([np.zeros_like(ge), ge])).to(self.q.device)
            return qsa_read_groups(self.dims, self.inputs, self.coded, args[0], args[1], int(ge.max(initial=0)),
                                   self.coded_ws, handle)

    def code_all(self, stream=None):
        """Codes every complete group of every history (once per history)."""
        ge = self._whole_histories()
        return self.code(np.zeros_like(ge), ge, stream)

    def attend_coded(self, whole=False, weigh=False, stream=None):
        """Attention over the coded cache: the rows in ids / n_ids, or the whole histories."""
        return qsa_attend_coded(self.dims, self.inputs, self.coded, None if whole else self.ids,
                                None if whole else self.n_ids, self.out, self.coded_ws,
                                weights=self.weights if weigh else None,
                                weight_offset=self.weight_offset if weigh else None, stream=stream)

    def decode_coded(self, weigh=False, stream=None):
        """The whole path over the coded cache (scored from the raw index keys)."""
        return qsa_decode_coded(self.dims, self.inputs, self.coded, self.ids, self.n_ids, self.out, self.coded_ws,
                                weights=self.weights if weigh else None,
                                weight_offset=self.weight_offset if weigh else None, stream=stream)

    # ---- queries over one shared history ------------------------------------
    def score_shared(self, stream=None):
        return qsa_score_groups_shared(self.dims, self.inputs, self.scores, self.ws, stream)

    def decode_shared(self, stream=None):
        return qsa_decode_shared(self.dims, self.inputs, self.ids, self.n_ids, self.out, self.ws, stream)

    def check_errors(self, stream=None):
        """(status, flags) of every call on this batch since the last check, those over its coded cache included."""
        st, flags = qsa_check_errors(self.ws, stream)
        if self.coded_ws is not None:
            coded_st, coded_flags = qsa_check_errors(self.coded_ws, stream)
            st, flags = max(st, coded_st), flags | coded_flags
        return st, flags
