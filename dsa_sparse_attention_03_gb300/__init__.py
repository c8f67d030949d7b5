"""Python binding of libdsa (the DSA decode step for GB300, sm_103a).

Argument marshalling only: every step of the path runs in libdsa's CUDA
kernels, reached through its C ABI (``include/dsa.h``) with ctypes.  PyTorch
supplies device memory and streams.  There is no fallback: if the shared library
is missing this module raises at import.

Entry points mirror the C names::

    prob = Problem.from_tensors(...)          # sizes + device pointers
    ws = alloc_workspace(prob)                # caller-owned scratch
    dsa_index_scores(prob, scores, ws)
    dsa_topk(prob, scores, idx, nsel, ws)
    dsa_sparse_attn(prob, idx, nsel, out, lse, ws)
    dsa_decode_step(prob, idx, nsel, out, ws)
    dsa_read_device_status(ws)

and the indexer front end (``include/dsa_front_end.h``)::

    dsa_indexer_front_end(prob, d, x, wq, ww, q_idx, w_idx, ws_front, ...)

and dense attention (``include/dsa_dense.h``)::

    dp = DenseProblem.from_tensors(q=..., k=..., v=..., offsets=..., row_offsets=..., row_len=..., ...)
    dsa_dense_attn(dp, out, lse, alloc_dense_workspace(dp))

and linear attention with a decay for each head (``include/dsa_linear.h``)::

    lp = LinearProblem.from_tensors(q=..., k=..., v=..., log_decay=..., row_offsets=..., scale=...)
    dsa_linear_attn(lp, state_in, state_out, out, alloc_linear_workspace(lp))    # prompts
    dsa_linear_step(lp, state, state, out, ws)                                   # one token of each request

and norms with the position rotation (``include/dsa_rope.h``) and the paged cache held in
4 bits (``include/dsa_kv4.h``)::

    qk = QKProblem.from_tensors(q=..., k=..., v=..., positions=..., inv_freq=..., q_weight=..., k_weight=..., ...)
    dsa_qk_norm_rope(qk, q_out, k_out)
    cache = KV4Cache.from_tensors(pages=alloc_kv4_pages(...), table=..., page_size=64, D_k=128, D_v=128)
    dsa_kv4_append(cache, qk, q_out, alloc_kv4_workspace())
    kp = KV4Problem.from_tensors(cache=cache, q=q_out, row_offsets=..., row_len=..., softmax_scale=...)
    dsa_kv4_attn(kp, out, lse, alloc_kv4_workspace(kp))
    dsa_kv4_read(cache, row_offsets, positions, k_out, v_out, ws)
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libdsa.so")

DSA_OK = 0
DSA_ERR_INVALID_ARG = 1
DSA_ERR_UNSUPPORTED = 2
DSA_ERR_OVERFLOW_RISK = 3
DSA_ERR_CUDA = 4
DSA_ERR_TIMEOUT = 5
DSA_ERR_DEVICE_INDEX = 6
DSA_ERR_RANGE = 7

DSA_DEVICE_TIMEOUT = 0x1
DSA_DEVICE_BAD_INDEX = 0x2
DSA_DEVICE_CAPACITY = 0x4
DSA_DEVICE_RANGE = 0x8

DSA_INDEXER_AUTO = 0
DSA_INDEXER_DP4A = 1
DSA_INDEXER_TC = 2
DSA_FLAG_NO_RELU = 0x100
DSA_FLAG_KV_FP8 = 0x200
DSA_FLAG_FP16 = 0x400
DSA_FLAG_ROPE_ADJACENT = 0x800

INDEXERS = {"auto": DSA_INDEXER_AUTO, "dp4a": DSA_INDEXER_DP4A, "tc": DSA_INDEXER_TC}

# Symbols the header declares (checked by the ABI test).
EXPORTS = ("dsa_version", "dsa_last_error_string", "dsa_indexer_kind", "dsa_decode_step_kernels",
           "dsa_workspace_size",
           "dsa_index_scores",
           "dsa_topk", "dsa_topk_static", "dsa_sparse_attn", "dsa_decode_step",
           "dsa_read_device_status", "dsa_get_device_status", "dsa_check_bounds",
           # include/dsa_front_end.h
           "dsa_front_end_workspace_size", "dsa_indexer_front_end",
           # include/dsa_dense.h
           "dsa_dense_workspace_size", "dsa_dense_attn",
           # include/dsa_linear.h
           "dsa_linear_workspace_size", "dsa_linear_attn", "dsa_linear_step",
           # include/dsa_rope.h, include/dsa_kv4.h
           "dsa_qk_norm_rope", "dsa_kv4_block_bytes", "dsa_kv4_append", "dsa_kv4_read", "dsa_kv4_workspace_size",
           "dsa_kv4_attn",
           # include/dsa_testing.h
           "dsa_test_topk_missing_arrival", "dsa_test_attn_missing_gather",
           "dsa_test_indexer_missing_tile", "dsa_test_dense_missing_tile",
           "dsa_test_linear_missing_tile", "dsa_test_kv4_missing_stage")


class dsa_problem(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("B", ctypes.c_int32), ("H_i", ctypes.c_int32),
        ("D_i", ctypes.c_int32), ("H_q", ctypes.c_int32), ("D_k", ctypes.c_int32),
        ("D_v", ctypes.c_int32), ("k", ctypes.c_int32), ("L_max", ctypes.c_int32),
        ("flags", ctypes.c_int32), ("L_total", ctypes.c_int64),
        ("qk_abs_max", ctypes.c_int32), ("w_abs_max", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float), ("reserved0", ctypes.c_int32),
        ("q_idx", ctypes.c_void_p), ("w_idx", ctypes.c_void_p), ("k_idx", ctypes.c_void_p),
        ("q", ctypes.c_void_p), ("kv", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p), ("row_len", ctypes.c_void_p),
        ("kv_scale", ctypes.c_void_p),
    ]


class dsa_dense_problem(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("B", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
        ("D_k", ctypes.c_int32), ("D_v", ctypes.c_int32), ("L_max", ctypes.c_int32), ("rows_max", ctypes.c_int32),
        ("L_total", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("softmax_scale", ctypes.c_float), ("flags", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p), ("row_len", ctypes.c_void_p),
    ]


class dsa_linear_problem(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("D_k", ctypes.c_int32),
        ("D_v", ctypes.c_int32), ("rows_max", ctypes.c_int32), ("n_states", ctypes.c_int32),
        ("flags", ctypes.c_int32), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("scale", ctypes.c_float), ("reserved0", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("log_decay", ctypes.c_void_p),
        ("row_offsets", ctypes.c_void_p), ("state_idx", ctypes.c_void_p),
    ]


class dsa_qk_problem(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("B", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
        ("D_k", ctypes.c_int32), ("D_v", ctypes.c_int32), ("rot", ctypes.c_int32), ("rot_first", ctypes.c_int32),
        ("eps", ctypes.c_float), ("flags", ctypes.c_int32), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("row_offsets", ctypes.c_void_p),
    ]


class dsa_kv4_cache(ctypes.Structure):
    _fields_ = [
        ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("D_k", ctypes.c_int32),
        ("D_v", ctypes.c_int32), ("B", ctypes.c_int32), ("table_cols", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("pages", ctypes.c_void_p), ("table", ctypes.c_void_p),
    ]


class dsa_kv4_problem(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("H_q", ctypes.c_int32), ("L_max", ctypes.c_int32), ("rows_max", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float), ("flags", ctypes.c_int32), ("q_stride", ctypes.c_int64),
        ("q", ctypes.c_void_p), ("row_offsets", ctypes.c_void_p), ("row_len", ctypes.c_void_p),
    ]


class dsa_affine_weights(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p)]


class DsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libdsa status {status}: {message}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libdsa is not built ({LIB_PATH} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(dsa_problem)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.dsa_version.restype = ctypes.c_int
    lib.dsa_last_error_string.restype = ctypes.c_char_p
    lib.dsa_indexer_kind.restype = ctypes.c_int
    lib.dsa_indexer_kind.argtypes = [P]
    lib.dsa_decode_step_kernels.restype = ctypes.c_int
    lib.dsa_decode_step_kernels.argtypes = [P]
    lib.dsa_workspace_size.restype = sz
    lib.dsa_workspace_size.argtypes = [P]
    lib.dsa_front_end_workspace_size.restype = sz
    lib.dsa_front_end_workspace_size.argtypes = [P, ctypes.c_int32]
    W = ctypes.POINTER(dsa_affine_weights)
    DP = ctypes.POINTER(dsa_dense_problem)
    lib.dsa_dense_workspace_size.restype = sz
    lib.dsa_dense_workspace_size.argtypes = [DP]
    LP = ctypes.POINTER(dsa_linear_problem)
    lib.dsa_linear_workspace_size.restype = sz
    lib.dsa_linear_workspace_size.argtypes = [LP]
    QP, CP, KP = (ctypes.POINTER(x) for x in (dsa_qk_problem, dsa_kv4_cache, dsa_kv4_problem))
    lib.dsa_kv4_block_bytes.restype = sz
    lib.dsa_kv4_block_bytes.argtypes = [ctypes.c_int32] * 3
    lib.dsa_kv4_workspace_size.restype = sz
    lib.dsa_kv4_workspace_size.argtypes = [CP, KP]
    for name, args in (
        ("dsa_index_scores", [P, vp, vp, sz, vp]),
        ("dsa_topk", [P, vp, vp, vp, vp, sz, vp]),
        ("dsa_topk_static", [P, vp, vp, vp, vp]),
        ("dsa_sparse_attn", [P, vp, vp, vp, vp, vp, sz, vp]),
        ("dsa_decode_step", [P, vp, vp, vp, vp, sz, vp]),
        ("dsa_read_device_status", [vp, vp, ctypes.POINTER(ctypes.c_int32)]),
        ("dsa_get_device_status", [vp, vp]),
        ("dsa_check_bounds", [P, ctypes.c_int64, ctypes.c_int64, vp, sz, vp]),
        ("dsa_indexer_front_end", [P, ctypes.c_int32, vp, W, W, vp, vp, vp, vp, vp, vp, sz, vp]),
        ("dsa_dense_attn", [DP, vp, vp, vp, sz, vp]),
        ("dsa_linear_attn", [LP, vp, vp, vp, vp, sz, vp]),
        ("dsa_linear_step", [LP, vp, vp, vp, vp, sz, vp]),
        ("dsa_qk_norm_rope", [QP, vp, vp, vp]),
        ("dsa_kv4_append", [CP, QP, vp, vp, sz, vp]),
        ("dsa_kv4_read", [CP, ctypes.c_int32, vp, vp, ctypes.c_int32, vp, vp, vp, sz, vp]),
        ("dsa_kv4_attn", [CP, KP, vp, vp, vp, sz, vp]),
        ("dsa_test_kv4_missing_stage", [CP, KP, vp, vp, vp, sz, ctypes.c_int64, vp]),
        ("dsa_test_dense_missing_tile", [DP, vp, vp, vp, sz, ctypes.c_int64, vp]),
        ("dsa_test_linear_missing_tile", [LP, vp, vp, vp, vp, sz, ctypes.c_int64, vp]),
        ("dsa_test_topk_missing_arrival", [P, vp, vp, vp, vp, sz, ctypes.c_int, ctypes.c_int64, vp]),
        ("dsa_test_attn_missing_gather", [P, vp, vp, vp, vp, vp, sz, ctypes.c_int64, vp]),
        ("dsa_test_indexer_missing_tile", [P, vp, vp, sz, ctypes.c_int64, vp]),
    ):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = args
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def _check(status: int) -> None:
    if status != DSA_OK:
        raise DsaError(status, _lib.dsa_last_error_string().decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Problem:
    """Sizes plus device tensors of one decode-step problem (see include/dsa.h).

    The tensors are kept referenced for the lifetime of the object.  ``L_max``
    and ``L_total`` are host values; ``from_tensors`` computes them from
    ``row_len``/``offsets`` (a device read) unless given.
    """

    _struct = dsa_problem

    def __init__(self, **kw):
        self._keep = {}
        self._on = None      # device on which the tensors were found (_check_call)
        self._fits = False   # whether the tensors were found to fit the sizes (_check_fits)
        s = self._struct()
        for f, _ in self._struct._fields_:
            v = kw.get(f)
            if v is None:
                continue
            if hasattr(v, "data_ptr"):
                self._keep[f] = v
                setattr(s, f, v.data_ptr())
            else:
                setattr(s, f, v)
        self.c = s

    @classmethod
    def from_tensors(cls, *, q_idx, w_idx, k_idx, q, kv, offsets, row_offsets, row_len, k,
                     softmax_scale, D_v=0, L_max=None, L_total=None, indexer="auto", relu=True,
                     qk_abs_max=0, w_abs_max=0, kv_fp8=False, kv_scale=None):
        R = int(row_len.shape[0])
        B = int(offsets.shape[0]) - 1
        if L_max is None:
            L_max = int(row_len.max().item()) if R else 0
        if L_total is None:
            L_total = int(offsets[-1].item())
        flags = (INDEXERS[indexer] | (0 if relu else DSA_FLAG_NO_RELU)
                 | (DSA_FLAG_KV_FP8 if kv_fp8 else 0))
        H_i, D_i = (int(q_idx.shape[1]), int(q_idx.shape[2])) if q_idx is not None else (0, 0)
        H_q, D_k = (int(q.shape[1]), int(q.shape[2])) if q is not None else (0, 0)
        return cls(R=R, B=B, H_i=H_i, D_i=D_i, H_q=H_q, D_k=D_k, D_v=int(D_v), k=int(k),
                   L_max=int(L_max), flags=flags, L_total=int(L_total), qk_abs_max=qk_abs_max,
                   w_abs_max=w_abs_max, softmax_scale=float(softmax_scale), q_idx=q_idx,
                   w_idx=w_idx, k_idx=k_idx, q=q, kv=kv, offsets=offsets,
                   row_offsets=row_offsets, row_len=row_len, kv_scale=kv_scale)

    def set(self, **kw):
        """Changes fields: sizes, or tensors in the place of the problem's."""
        self._on = None
        self._fits = False
        for f, v in kw.items():
            if hasattr(v, "data_ptr"):
                self._keep[f] = v
                v = v.data_ptr()
            setattr(self.c, f, v)
        return self

    def __getattr__(self, name):
        if name in ("c", "_keep", "_on", "_fits", "_expect"):
            raise AttributeError(name)
        return getattr(self.c, name)


def upload_inputs(inp, device="cuda", indexer="auto", relu=True, qk_abs_max=0, w_abs_max=0):
    """Copy a host problem (numpy arrays named as in include/dsa.h: q_idx,
    w_idx, k_idx, q, kv, offsets, row_offsets, row_len, plus k, D_v,
    softmax_scale; an FP8 cache has ``kv_format == "e4m3"``, kv as uint8 codes
    and ``kv_scale`` float32 or None) to ``device``.  Returns (Problem, dict of
    device tensors)."""
    import numpy as np
    import torch

    def dev(a, dt):
        return torch.from_numpy(np.ascontiguousarray(a)).to(device=device, dtype=dt)

    fp8 = getattr(inp, "kv_format", "bf16") == "e4m3"
    t = dict(
        q_idx=dev(inp.q_idx, torch.int8), w_idx=dev(inp.w_idx, torch.int32),
        k_idx=dev(inp.k_idx, torch.int8),
        q=dev(np.asarray(inp.q).view(np.int16), torch.int16),
        kv=(dev(np.asarray(inp.kv, dtype=np.uint8), torch.uint8) if fp8
            else dev(np.asarray(inp.kv).view(np.int16), torch.int16)),
        offsets=dev(inp.offsets, torch.int32), row_offsets=dev(inp.row_offsets, torch.int32),
        row_len=dev(inp.row_len, torch.int32))
    sc = getattr(inp, "kv_scale", None) if fp8 else None
    t["kv_scale"] = None if sc is None else dev(np.asarray(sc, dtype=np.float32), torch.float32)
    L_max = int(np.max(inp.row_len)) if len(inp.row_len) else 0
    prob = Problem.from_tensors(k=inp.k, D_v=inp.D_v, softmax_scale=inp.softmax_scale,
                                L_max=L_max, L_total=int(inp.offsets[-1]), indexer=indexer,
                                relu=relu, qk_abs_max=qk_abs_max, w_abs_max=w_abs_max,
                                kv_fp8=fp8, **t)
    return prob, t


def dsa_decode_step_kernels(prob: Problem) -> int:
    """Kernels one dsa_decode_step launches for this problem (2 or 3)."""
    return _lib.dsa_decode_step_kernels(ctypes.byref(prob.c))


def dsa_indexer_kind(prob: Problem) -> int:
    return _lib.dsa_indexer_kind(ctypes.byref(prob.c))


def indexer_kind(prob: Problem) -> str:
    return {DSA_INDEXER_DP4A: "dp4a", DSA_INDEXER_TC: "tc"}.get(dsa_indexer_kind(prob), "invalid")


def dsa_version() -> int:
    return _lib.dsa_version()


def dsa_workspace_size(prob: Problem) -> int:
    n = _lib.dsa_workspace_size(ctypes.byref(prob.c))
    if n == 0:
        raise DsaError(DSA_ERR_INVALID_ARG, _lib.dsa_last_error_string().decode())
    return n


def alloc_workspace(prob: Problem, device="cuda"):
    import torch
    return torch.empty(dsa_workspace_size(prob), dtype=torch.uint8, device=device)


def dsa_index_scores(prob: Problem, scores, ws, stream=None) -> None:
    _check(_lib.dsa_index_scores(ctypes.byref(prob.c), _ptr(scores), _ptr(ws), ws.numel(),
                                 _stream(stream)))


def dsa_topk(prob: Problem, scores, idx, nsel, ws, stream=None) -> None:
    _check(_lib.dsa_topk(ctypes.byref(prob.c), _ptr(scores), _ptr(idx), _ptr(nsel), _ptr(ws),
                         ws.numel(), _stream(stream)))


def dsa_topk_static(prob: Problem, scores, idx, nsel, stream=None) -> None:
    """dsa_topk with the library's fixed 4 MiB scratch instead of a workspace
    (see include/dsa.h: calls must not overlap)."""
    _check(_lib.dsa_topk_static(ctypes.byref(prob.c), _ptr(scores), _ptr(idx), _ptr(nsel),
                                _stream(stream)))


def dsa_sparse_attn(prob: Problem, idx, nsel, out, lse, ws, stream=None) -> None:
    _check(_lib.dsa_sparse_attn(ctypes.byref(prob.c), _ptr(idx), _ptr(nsel), _ptr(out),
                                _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def dsa_decode_step(prob: Problem, idx, nsel, out, ws, stream=None) -> None:
    _check(_lib.dsa_decode_step(ctypes.byref(prob.c), _ptr(idx), _ptr(nsel), _ptr(out),
                                _ptr(ws), ws.numel(), _stream(stream)))


# Test hooks (include/dsa_testing.h): one bounded device wait made to run out.

def dsa_test_topk_missing_arrival(prob: Problem, scores, idx, nsel, ws, skip_cta, limit_ns,
                                  stream=None) -> None:
    _check(_lib.dsa_test_topk_missing_arrival(ctypes.byref(prob.c), _ptr(scores), _ptr(idx),
                                              _ptr(nsel), _ptr(ws), ws.numel(), int(skip_cta),
                                              int(limit_ns), _stream(stream)))


def dsa_test_attn_missing_gather(prob: Problem, idx, nsel, out, lse, ws, limit_ns,
                                 stream=None) -> None:
    _check(_lib.dsa_test_attn_missing_gather(ctypes.byref(prob.c), _ptr(idx), _ptr(nsel),
                                             _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                             int(limit_ns), _stream(stream)))


def dsa_test_indexer_missing_tile(prob: Problem, scores, ws, limit_ns, stream=None) -> None:
    _check(_lib.dsa_test_indexer_missing_tile(ctypes.byref(prob.c), _ptr(scores), _ptr(ws),
                                              ws.numel(), int(limit_ns), _stream(stream)))


def dsa_check_bounds(prob: Problem, ws, key_row0=0, key_rows=None, stream=None) -> None:
    """Device check of the declared bounds (include/dsa.h); read the result
    with dsa_read_device_status."""
    n = int(prob.c.L_total) - int(key_row0) if key_rows is None else int(key_rows)
    _check(_lib.dsa_check_bounds(ctypes.byref(prob.c), int(key_row0), n, _ptr(ws), ws.numel(),
                                 _stream(stream)))


def dsa_get_device_status(ws, stream=None) -> int:
    """Synchronises the stream; returns DSA_OK, DSA_ERR_TIMEOUT or
    DSA_ERR_DEVICE_INDEX from the device status word (raises on other errors)."""
    st = _lib.dsa_get_device_status(_ptr(ws), _stream(stream))
    if st not in (DSA_OK, DSA_ERR_TIMEOUT, DSA_ERR_DEVICE_INDEX, DSA_ERR_RANGE):
        _check(st)
    return st


def dsa_read_device_status(ws, stream=None) -> int:
    """Synchronises the stream and returns the device status bits (raises on
    TIMEOUT / BAD_INDEX with the bits in ``DsaError.status``)."""
    bits = ctypes.c_int32(0)
    st = _lib.dsa_read_device_status(_ptr(ws), _stream(stream), ctypes.byref(bits))
    if st not in (DSA_OK, DSA_ERR_TIMEOUT, DSA_ERR_DEVICE_INDEX, DSA_ERR_RANGE):
        _check(st)
    return bits.value


# Indexer front end (include/dsa_front_end.h).

def affine_weights(codes, scales, biases) -> dsa_affine_weights:
    """The three device tensors of one 8-bit affine weight matrix."""
    return dsa_affine_weights(codes.data_ptr(), scales.data_ptr(), biases.data_ptr())


def dsa_front_end_workspace_size(prob: Problem, d: int) -> int:
    n = _lib.dsa_front_end_workspace_size(ctypes.byref(prob.c), int(d))
    if n == 0:
        raise DsaError(DSA_ERR_INVALID_ARG, _lib.dsa_last_error_string().decode())
    return n


def dsa_indexer_front_end(prob: Problem, d: int, x, wq, ww, q_idx, w_idx, ws, q_scale=None,
                          w_scale=None, proj=None, stream=None) -> None:
    """``wq``/``ww``: (codes, scales, biases) device tensors or dsa_affine_weights."""
    if not isinstance(wq, dsa_affine_weights):
        wq = affine_weights(*wq)
    if not isinstance(ww, dsa_affine_weights):
        ww = affine_weights(*ww)
    _check(_lib.dsa_indexer_front_end(ctypes.byref(prob.c), int(d), _ptr(x), ctypes.byref(wq),
                                      ctypes.byref(ww), _ptr(q_idx), _ptr(w_idx), _ptr(q_scale),
                                      _ptr(w_scale), _ptr(proj), _ptr(ws), ws.numel(),
                                      _stream(stream)))


# Dense attention (include/dsa_dense.h).

def _head_tensor(name, t):
    """(heads, width, token stride) of a [tokens, heads, width] tensor whose heads are packed."""
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name} must be [tokens, heads, width] with packed heads (a token stride is allowed)")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1] * t.shape[2]:   # (expanded: stride 0 means packed in the struct)
        raise ValueError(f"{name}'s tokens overlap (stride {t.stride(0)} for {t.shape[1]} heads of {t.shape[2]})")
    return int(t.shape[1]), int(t.shape[2]), int(t.stride(0)) if t.shape[0] > 1 else 0


def _fp16_flag(**ts):
    import torch
    kinds = {t.dtype for t in ts.values()}
    if kinds == {torch.bfloat16}:
        return 0
    if kinds == {torch.float16}:
        return DSA_FLAG_FP16
    raise ValueError(f"{', '.join(ts)} must all be bfloat16 or all float16, got {sorted(map(str, kinds))}")


def _check_device(prob):
    """The current CUDA device, on which the problem's own tensors have to be: they are
    looked over once, until ``set`` changes one."""
    import torch
    if prob._on is not None:       # (CUDA is up)
        dev = torch._C._cuda_getDevice()
    else:
        dev = torch.cuda.current_device() if torch.cuda.is_initialized() or torch.cuda.is_available() else None
    if prob._on != dev or dev is None:
        for t in prob._keep.values():
            if t.get_device() != dev:
                raise ValueError(f"a tensor is on {t.device}, not on the current CUDA device")
        prob._on = dev
    return dev


def _check_call(prob, outputs, ws):
    """What a call checks of its tensors: each output (name, tensor, shape, dtype; the
    tensor may be None) and that everything is on the current CUDA device."""
    dev = _check_device(prob)
    _check_outputs(dev, outputs, ws)
    return dev


def _check_outputs(dev, outputs, ws):
    for name, t, shape, dtype in outputs:
        if t is None:
            continue
        if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                             f"got {t.dtype} {tuple(t.shape)}")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    if ws is not None and ws.get_device() != dev:
        raise ValueError(f"the workspace is on {ws.device}, not on the current CUDA device")


def _check_ints(n, **ts):
    import torch
    for name, t in ts.items():
        if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous()
                              or (n.get(name) is not None and t.shape[0] != n[name])):
            raise ValueError(f"{name} must be a contiguous int32 vector"
                             + (f" of {n[name]} entries" if n.get(name) is not None else ""))


def _check_fits(prob, heads, ints, fixed=()):
    """The problem's tensors against its sizes, which ``set`` may have changed apart: q, k and
    v (name: heads, width, token stride, tokens at least), vectors of int32 (name: entries at least)
    and others (name, dtype, shape)."""
    if prob._fits:
        return
    for name, (h, d, stride, n) in heads.items():
        t = prob._keep[name]
        got = _head_tensor(name, t)
        if got[:2] != (h, d) or t.shape[0] < n or (n > 1 and got[2] != (stride or h * d)):
            raise ValueError(f"{name} of shape {tuple(t.shape)} and token stride {t.stride(0)} does not fit the problem: "
                             f"{n} tokens of {h} heads of {d}, stride {stride or h * d}")
    if _fp16_flag(**{x: prob._keep[x] for x in heads}) != prob.c.flags & DSA_FLAG_FP16:
        raise ValueError(f"{', '.join(heads)} are not of the problem's type")
    for name, n in ints.items():
        t = prob._keep.get(name)
        if t is None or getattr(prob.c, name) is None:
            continue
        _check_ints({}, **{name: t})
        if t.shape[0] < n:
            raise ValueError(f"{name} has {t.shape[0]} entries, the problem needs {n}")
    for name, dtype, shape in fixed:
        t = prob._keep[name]
        if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
    prob._fits = True


class DenseProblem(Problem):
    """Sizes plus device tensors of one dense attention call (include/dsa_dense.h).

    q [R, H_q, D_k], k [L_total, H_kv, D_k] and v [L_total, H_kv, D_v] are bfloat16 or
    float16; they may be views with a token stride (slices of a fused projection).
    ``L_max``, ``L_total`` and ``rows_max`` are host values, read from the device
    tensors unless given.
    """

    _struct = dsa_dense_problem

    @classmethod
    def from_tensors(cls, *, q, k, v, offsets, row_offsets, row_len, softmax_scale, L_max=None, L_total=None,
                     rows_max=None):
        H_q, D_k, q_stride = _head_tensor("q", q)
        H_kv, D, k_stride = _head_tensor("k", k)
        H_v, D_v, v_stride = _head_tensor("v", v)
        if D != D_k or H_v != H_kv or k.shape[0] != v.shape[0]:
            raise ValueError("q and k must have one width, k and v the same tokens and heads")
        R = int(q.shape[0])
        B = int(offsets.shape[0]) - 1
        _check_ints(dict(offsets=B + 1, row_offsets=B + 1, row_len=R), offsets=offsets, row_offsets=row_offsets,
                    row_len=row_len)
        if L_max is None:
            L_max = int(row_len.max().item()) if R else 0
        if L_total is None:
            L_total = int(offsets[-1].item())
        if L_total > k.shape[0]:
            raise ValueError(f"L_total={L_total} but k and v have {k.shape[0]} tokens")
        if rows_max is None:
            rows_max = int((row_offsets[1:] - row_offsets[:-1]).max().item()) if R else 0
        prob = cls(R=R, B=B, H_q=H_q, H_kv=H_kv, D_k=D_k, D_v=D_v, L_max=int(L_max), rows_max=int(rows_max),
                   L_total=int(L_total), q_stride=q_stride, k_stride=k_stride, v_stride=v_stride,
                   softmax_scale=float(softmax_scale), flags=_fp16_flag(q=q, k=k, v=v), q=q, k=k, v=v,
                   offsets=offsets, row_offsets=row_offsets, row_len=row_len)
        prob._fits = True
        return prob


def dsa_dense_workspace_size(prob: DenseProblem) -> int:
    n = _lib.dsa_dense_workspace_size(ctypes.byref(prob.c))
    if n == 0:
        raise DsaError(DSA_ERR_INVALID_ARG, _lib.dsa_last_error_string().decode())
    return n


def alloc_dense_workspace(prob: DenseProblem, device="cuda"):
    import torch
    return torch.empty(dsa_dense_workspace_size(prob), dtype=torch.uint8, device=device)


def dsa_dense_attn(prob: DenseProblem, out, lse, ws, stream=None) -> None:
    """out [R, H_q, D_v] in the operands' type; lse [R, H_q] float32 or None."""
    import torch
    if prob._on is None:           # (new, or changed)
        c = prob.c
        _check_fits(prob, dict(q=(c.H_q, c.D_k, c.q_stride, c.R), k=(c.H_kv, c.D_k, c.k_stride, c.L_total),
                               v=(c.H_kv, c.D_v, c.v_stride, c.L_total)),
                    dict(offsets=c.B + 1, row_offsets=c.B + 1, row_len=c.R))
        prob._expect = (ctypes.byref(c), (c.R, c.H_q, c.D_v), prob._keep["q"].dtype, (c.R, c.H_q))
    ref, shape, dtype, rows = prob._expect
    dev = _check_call(prob, (("out", out, shape, dtype), ("lse", lse, rows, torch.float32)), ws)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    _check(_lib.dsa_dense_attn(ref, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


# Linear attention with a decay for each head (include/dsa_linear.h).

class LinearProblem(Problem):
    """Sizes plus device tensors of one linear attention call (include/dsa_linear.h).

    q, k [R, H, D_k] and v [R, H, D_v] are bfloat16 or float16 (views with a token
    stride are fine), log_decay is float32 [H].  ``row_offsets`` is None for
    dsa_linear_step alone: one token of each request.  ``rows_max`` is a host value,
    read from ``row_offsets`` unless given; ``n_states`` is the number of places of
    the state arrays (the requests, unless ``state_idx`` names places).
    """

    _struct = dsa_linear_problem

    @classmethod
    def from_tensors(cls, *, q, k, v, log_decay, row_offsets=None, scale, rows_max=None, state_idx=None,
                     n_states=None):
        import torch
        H, D_k, q_stride = _head_tensor("q", q)
        H_k, D, k_stride = _head_tensor("k", k)
        H_v, D_v, v_stride = _head_tensor("v", v)
        if D != D_k or H_k != H or H_v != H or not q.shape[0] == k.shape[0] == v.shape[0]:
            raise ValueError("q, k and v must have the same tokens and heads, q and k one width")
        if log_decay.dtype != torch.float32 or tuple(log_decay.shape) != (H,) or not log_decay.is_contiguous():
            raise ValueError(f"log_decay must be a contiguous float32 vector of {H} entries")
        R = int(q.shape[0])
        B = R if row_offsets is None else int(row_offsets.shape[0]) - 1
        _check_ints(dict(row_offsets=B + 1, state_idx=B), row_offsets=row_offsets, state_idx=state_idx)
        if rows_max is None:
            rows_max = 1 if row_offsets is None else int((row_offsets[1:] - row_offsets[:-1]).max().item())
        if n_states is None:
            if state_idx is not None:
                raise ValueError("state_idx needs n_states")
            n_states = B
        prob = cls(R=R, B=B, H=H, D_k=D_k, D_v=D_v, rows_max=int(rows_max), n_states=int(n_states),
                   flags=_fp16_flag(q=q, k=k, v=v), q_stride=q_stride, k_stride=k_stride, v_stride=v_stride,
                   scale=float(scale), q=q, k=k, v=v, log_decay=log_decay, row_offsets=row_offsets,
                   state_idx=state_idx)
        prob._fits = True
        return prob


def dsa_linear_workspace_size(prob: LinearProblem) -> int:
    n = _lib.dsa_linear_workspace_size(ctypes.byref(prob.c))
    if n == 0:
        raise DsaError(DSA_ERR_INVALID_ARG, _lib.dsa_last_error_string().decode())
    return n


def alloc_linear_workspace(prob: LinearProblem, device="cuda"):
    import torch
    return torch.empty(dsa_linear_workspace_size(prob), dtype=torch.uint8, device=device)


def _linear_call(fn, prob, state_in, state_out, out, ws, stream):
    import torch
    if prob._on is None:           # (new, or changed)
        c = prob.c
        _check_fits(prob, dict(q=(c.H, c.D_k, c.q_stride, c.R), k=(c.H, c.D_k, c.k_stride, c.R),
                               v=(c.H, c.D_v, c.v_stride, c.R)),
                    dict(row_offsets=c.B + 1, state_idx=c.B), (("log_decay", torch.float32, (c.H,)),))
        prob._expect = (ctypes.byref(c), (c.R, c.H, c.D_v), prob._keep["q"].dtype, (c.n_states, c.H, c.D_k, c.D_v))
    ref, shape, dtype, states = prob._expect
    dev = _check_call(prob, (("out", out, shape, dtype), ("state_in", state_in, states, torch.float32),
                             ("state_out", state_out, states, torch.float32)), ws)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    _check(fn(ref, _ptr(state_in), _ptr(state_out), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))


def dsa_linear_attn(prob: LinearProblem, state_in, state_out, out, ws, stream=None) -> None:
    """Prompts.  state_in (None: zeros) and state_out (None: not wanted) are float32
    [n_states, H, D_k, D_v], and may be one tensor; out [R, H, D_v] in the operands' type."""
    _linear_call(_lib.dsa_linear_attn, prob, state_in, state_out, out, ws, stream)


def dsa_linear_step(prob: LinearProblem, state_in, state_out, out, ws, stream=None) -> None:
    """One token of each request; arguments as dsa_linear_attn."""
    _linear_call(_lib.dsa_linear_step, prob, state_in, state_out, out, ws, stream)


# Norms and the position rotation (include/dsa_rope.h), the 4-bit cache (include/dsa_kv4.h).

class QKProblem(Problem):
    """Sizes plus device tensors of dsa_qk_norm_rope and dsa_kv4_append (include/dsa_rope.h).

    q [R, H_q, D_k], k [R, H_kv, D_k] and v [R, H_kv, D_v] (any may be None; dsa_kv4_append
    needs k, v and ``row_offsets``) are bfloat16 or float16 and may be views with a token stride.
    ``inv_freq`` is float64 [rot / 2], radians a position (None: no rotation), of the columns
    from ``rot_first`` on; ``interleaved`` pairs adjacent columns, otherwise halves.
    ``q_weight`` and ``k_weight`` [D_k] are the norms' weights in the operands' type (None: not
    normed).  A negative position skips its row.
    """

    _struct = dsa_qk_problem

    @classmethod
    def from_tensors(cls, *, q=None, k=None, v=None, positions, inv_freq=None, rot_first=0, interleaved=False,
                     q_weight=None, k_weight=None, eps=1e-6, row_offsets=None):
        heads = {n: t for n, t in (("q", q), ("k", k), ("v", v)) if t is not None}
        if q is None and k is None:
            raise ValueError("q or k must be given")
        size = {n: _head_tensor(n, t) for n, t in heads.items()}
        R = int(next(iter(heads.values())).shape[0])
        D_k = size["q" if q is not None else "k"][1]
        H_kv = size["k"][0] if k is not None else 0
        if any(t.shape[0] != R for t in heads.values()):
            raise ValueError(f"{', '.join(heads)} must have the same tokens")
        if k is not None and size["k"][1] != D_k or v is not None and (k is None or size["v"][0] != H_kv):
            raise ValueError("q and k must have one width, k and v the same heads")
        rot = 0 if inv_freq is None else 2 * int(inv_freq.shape[0])
        flags = _fp16_flag(**heads) | (DSA_FLAG_ROPE_ADJACENT if interleaved else 0)
        prob = cls(R=R, B=0 if row_offsets is None else int(row_offsets.shape[0]) - 1, H_q=size["q"][0] if q is not None else 0,
                   H_kv=H_kv, D_k=D_k, D_v=size["v"][1] if v is not None else 0, rot=rot, rot_first=int(rot_first),
                   eps=float(eps), flags=flags, **{n + "_stride": s[2] for n, s in size.items()}, **heads,
                   positions=positions, inv_freq=inv_freq, q_weight=q_weight, k_weight=k_weight, row_offsets=row_offsets)
        prob._look()
        return prob

    def _look(self):
        """The tensors against the sizes (see _check_fits)."""
        import torch
        c, keep = self.c, self._keep
        heads = {n: s for n, s in (("q", (c.H_q, c.D_k, c.q_stride, c.R)), ("k", (c.H_kv, c.D_k, c.k_stride, c.R)),
                                   ("v", (c.H_kv, c.D_v, c.v_stride, c.R))) if getattr(c, n) is not None}
        dtype = keep[next(iter(heads))].dtype if heads else None
        fixed = [(n, d, s) for n, d, s in (("q_weight", dtype, (c.D_k,)), ("k_weight", dtype, (c.D_k,)),
                                           ("inv_freq", torch.float64, (c.rot // 2,))) if getattr(c, n) is not None]
        _check_fits(self, heads, dict(positions=c.R, row_offsets=c.B + 1), fixed)
        self._expect = (ctypes.byref(c), dtype, {"q": (c.q, (c.R, c.H_q, c.D_k)), "k": (c.k, (c.R, c.H_kv, c.D_k))})

    def _output(self, name, t, dev):
        """Checks an output: packed, or the input itself."""
        ptr, shape = self._expect[2][name]
        if ptr is None:
            return None
        if t is None:
            raise ValueError(f"{name}_out must be given where {name} is")
        at = t.data_ptr()
        if at == ptr and shape[0] > 0:
            x = self._keep[name]
            if t.shape != x.shape or t.stride() != x.stride() or t.dtype != x.dtype:
                raise ValueError(f"{name}_out begins where {name} does, but is not the same tensor")
        else:
            _check_outputs(dev, ((name + "_out", t, shape, self._expect[1]),), None)
        return at


def dsa_qk_norm_rope(prob: QKProblem, q_out, k_out, stream=None) -> None:
    """q_out [R, H_q, D_k] and k_out [R, H_kv, D_k], packed, or q and k themselves; None
    where the problem has no q (k)."""
    import torch
    if prob._on is None:
        prob._look()
    dev = _check_device(prob)
    q, k = prob._output("q", q_out, dev), prob._output("k", k_out, dev)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    _check(_lib.dsa_qk_norm_rope(prob._expect[0], q, k, _stream(stream)))


def dsa_kv4_block_bytes(D_k: int, D_v: int, page_size: int) -> int:
    """Bytes of one page of one K/V head."""
    n = _lib.dsa_kv4_block_bytes(int(D_k), int(D_v), int(page_size))
    if n == 0:
        raise DsaError(DSA_ERR_UNSUPPORTED, f"no 4-bit cache of D_k={D_k}, D_v={D_v}, page_size={page_size}")
    return n


def alloc_kv4_pages(n_pages, H_kv, D_k, D_v, page_size, device="cuda"):
    """A pool of pages (not cleared)."""
    import torch
    return torch.empty(n_pages, H_kv, dsa_kv4_block_bytes(D_k, D_v, page_size), dtype=torch.uint8, device=device)


class KV4Cache(Problem):
    """A pool of pages and the table of its requests (include/dsa_kv4.h): ``pages`` uint8 [n_pages,
    H_kv, block], ``table`` int32 [B, pages of a request]."""

    _struct = dsa_kv4_cache
    revision = 0     # of the fields: a problem looks the cache over again when it has changed

    def set(self, **kw):
        self.revision += 1
        return super().set(**kw)

    @classmethod
    def from_tensors(cls, *, pages, table, page_size, D_k, D_v):
        if pages.dim() != 3 or table.dim() != 2:
            raise ValueError("pages must be [n_pages, H_kv, block] and table [B, pages of a request]")
        cache = cls(n_pages=int(pages.shape[0]), page_size=int(page_size), H_kv=int(pages.shape[1]), D_k=int(D_k),
                    D_v=int(D_v), B=int(table.shape[0]), table_cols=int(table.shape[1]), pages=pages, table=table)
        cache._look()
        return cache

    def _look(self):
        import torch
        c, keep = self.c, self._keep
        block = dsa_kv4_block_bytes(c.D_k, c.D_v, c.page_size)
        for name, dtype, shape in (("pages", torch.uint8, (c.n_pages, c.H_kv, block)),
                                   ("table", torch.int32, (c.B, c.table_cols))):
            t = keep[name]
            if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}, got {t.dtype} {tuple(t.shape)}")
        self._expect = (ctypes.byref(c), c.B + 1, c.H_kv, c.D_k, c.D_v)


def _check_cache(cache):
    """Looks the cache's tensors over; the current device."""
    if cache._on is None:
        cache._look()
    return _check_device(cache)


def dsa_kv4_append(cache: KV4Cache, prob: QKProblem, q_out, ws, stream=None) -> None:
    """Rows into the cache; q_out as in dsa_qk_norm_rope (None where the problem has no q)."""
    import torch
    if prob._on is None:
        prob._look()
    dev = _check_cache(cache)
    _check_device(prob)
    q = prob._output("q", q_out, dev)
    _check_outputs(dev, (), ws)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    _check(_lib.dsa_kv4_append(cache._expect[0], prob._expect[0], q, _ptr(ws), ws.numel(), _stream(stream)))


def dsa_kv4_read(cache: KV4Cache, row_offsets, positions, k_out, v_out, ws, stream=None) -> None:
    """k_out [R, H_kv, D_k] and v_out [R, H_kv, D_v] (either may be None), bfloat16 or float16: what the
    cache holds at positions[r] of row r's request."""
    import torch
    dev = _check_cache(cache)
    ref, n, H_kv, D_k, D_v = cache._expect
    R = positions.shape[0]
    dtype = torch.bfloat16 if k_out is None and v_out is None else (v_out if k_out is None else k_out).dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError(f"k_out and v_out must be bfloat16 or float16, got {dtype}")
    flags = DSA_FLAG_FP16 if dtype is torch.float16 else 0
    _check_outputs(dev, (("k_out", k_out, (R, H_kv, D_k), dtype), ("v_out", v_out, (R, H_kv, D_v), dtype),
                         ("row_offsets", row_offsets, (n,), torch.int32), ("positions", positions, (R,), torch.int32)), ws)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    _check(_lib.dsa_kv4_read(ref, R, _ptr(row_offsets), _ptr(positions), flags, _ptr(k_out), _ptr(v_out), _ptr(ws),
                             ws.numel(), _stream(stream)))


class KV4Problem(Problem):
    """Sizes plus device tensors of one attention call over a KV4Cache (include/dsa_kv4.h).

    q [R, H_q, D_k] is bfloat16 or float16 and may be a view with a token stride.  ``L_max`` and
    ``rows_max`` are host values, read from the device tensors unless given.
    """

    _struct = dsa_kv4_problem

    @classmethod
    def from_tensors(cls, *, cache, q, row_offsets, row_len, softmax_scale, L_max=None, rows_max=None):
        H_q, D, stride = _head_tensor("q", q)
        R = int(q.shape[0])
        _check_ints(dict(row_offsets=cache.c.B + 1, row_len=R), row_offsets=row_offsets, row_len=row_len)
        if L_max is None:
            L_max = int(row_len.max().item()) if R else 0
        if rows_max is None:
            rows_max = int((row_offsets[1:] - row_offsets[:-1]).max().item()) if R else 0
        prob = cls(R=R, H_q=H_q, L_max=int(L_max), rows_max=int(rows_max), softmax_scale=float(softmax_scale),
                   flags=_fp16_flag(q=q), q_stride=stride, q=q, row_offsets=row_offsets, row_len=row_len)
        prob._keep_cache = cache
        if D != cache.c.D_k:
            raise ValueError(f"q is {D} wide, the cache's keys {cache.c.D_k}")
        prob._look()
        return prob

    def _look(self):
        c, cache = self.c, self._keep_cache.c
        self._fits = False
        _check_fits(self, dict(q=(c.H_q, cache.D_k, c.q_stride, c.R)), dict(row_offsets=cache.B + 1, row_len=c.R))
        self._revision = self._keep_cache.revision
        self._expect = (ctypes.byref(c), (c.R, c.H_q, cache.D_v), self._keep["q"].dtype, (c.R, c.H_q))

    def __getattr__(self, name):
        if name in ("_keep_cache", "_revision"):
            raise AttributeError(name)
        return Problem.__getattr__(self, name)


def dsa_kv4_workspace_size(prob: KV4Problem) -> int:
    n = _lib.dsa_kv4_workspace_size(ctypes.byref(prob._keep_cache.c), ctypes.byref(prob.c))
    if n == 0:
        raise DsaError(DSA_ERR_INVALID_ARG, _lib.dsa_last_error_string().decode())
    return n


def alloc_kv4_workspace(prob: Optional[KV4Problem] = None, device="cuda"):
    """For dsa_kv4_attn on ``prob``; without one, for dsa_kv4_append and dsa_kv4_read."""
    import torch
    return torch.empty(256 if prob is None else dsa_kv4_workspace_size(prob), dtype=torch.uint8, device=device)


def _kv4_call(prob, out, lse, ws):
    import torch
    cache = prob._keep_cache
    if prob._on is None or prob._revision != cache.revision:
        cache._look()
        prob._look()
    ref, shape, dtype, rows = prob._expect
    dev = _check_cache(cache)
    _check_call(prob, (("out", out, shape, dtype), ("lse", lse, rows, torch.float32)), ws)
    return cache._expect[0], ref, dev


def dsa_kv4_attn(prob: KV4Problem, out, lse, ws, stream=None) -> None:
    """out [R, H_q, D_v] in the queries' type; lse [R, H_q] float32 or None."""
    import torch
    cache, ref, dev = _kv4_call(prob, out, lse, ws)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    _check(_lib.dsa_kv4_attn(cache, ref, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


# Test hooks of these calls (include/dsa_testing.h).

def dsa_test_kv4_missing_stage(prob: KV4Problem, out, lse, ws, limit_ns, stream=None) -> None:
    cache, ref, _ = _kv4_call(prob, out, lse, ws)
    _check(_lib.dsa_test_kv4_missing_stage(cache, ref, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), int(limit_ns),
                                           _stream(stream)))


def dsa_test_dense_missing_tile(prob: DenseProblem, out, lse, ws, limit_ns, stream=None) -> None:
    _check(_lib.dsa_test_dense_missing_tile(ctypes.byref(prob.c), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                            int(limit_ns), _stream(stream)))


def dsa_test_linear_missing_tile(prob: LinearProblem, state_in, state_out, out, ws, limit_ns, stream=None) -> None:
    _check(_lib.dsa_test_linear_missing_tile(ctypes.byref(prob.c), _ptr(state_in), _ptr(state_out), _ptr(out),
                                             _ptr(ws), ws.numel(), int(limit_ns), _stream(stream)))
