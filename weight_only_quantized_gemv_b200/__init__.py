"""Python binding of ``libqlinear.so``: the weight-only-quantized linear layer on B200.

Argument marshalling only.  Every function here forwards to the C entry point of
the same name in ``include/qlinear.h``; device arguments are ``torch.Tensor``
objects on the current CUDA device (their ``data_ptr()`` is passed), host
arguments of the packers are NumPy arrays.  A non-OK status raises
``QLinearError``.  There is no fallback: if the shared library is missing, the
import fails.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libqlinear.so")

if not os.path.exists(LIBRARY_PATH):
    raise ImportError(
        f"{LIBRARY_PATH} is missing: build it with "
        "`python -c 'import __graft_entry__ as g; g.build()'` or "
        "`python weight_only_quantized_gemv_b200/build.py`")

_lib = ctypes.CDLL(LIBRARY_PATH)

QL_FMT_W2, QL_FMT_W3, QL_FMT_W4, QL_FMT_W8, QL_FMT_LUT4 = 2, 3, 4, 8, 16
QL_FMT_CB = 32  # the codebook in the tensor-core layout (workspace and plan queries)
FORMATS = {"w2": QL_FMT_W2, "w3": QL_FMT_W3, "w4": QL_FMT_W4, "w8": QL_FMT_W8,
           "lut4": QL_FMT_LUT4}
STATUS = {0: "QL_OK", 1: "QL_ERR_NULL", 2: "QL_ERR_SHAPE", 3: "QL_ERR_ALIGN",
          4: "QL_ERR_UNSUPPORTED", 5: "QL_ERR_WORKSPACE", 6: "QL_ERR_CUDA",
          7: "QL_ERR_LIBRARY", 8: "QL_ERR_ALIAS"}
QL_ERR_WORKSPACE = 5
TYPES = {"float16": 0, "bfloat16": 1}  # ql_type
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}  # ql_act

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_LL = ctypes.c_longlong


class ql_policy_entry(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("m_lo", ctypes.c_int), ("m_hi", ctypes.c_int), ("strategy", ctypes.c_int),
                ("warps_per_unit", ctypes.c_int), ("ctas", ctypes.c_int)]


QL_STRATEGY_GEMV, QL_STRATEGY_PREFILL = 0, 1


class ql_plan(ctypes.Structure):
    _fields_ = [("ctas", ctypes.c_int), ("warps", ctypes.c_int), ("tiles_per_warp", ctypes.c_int),
                ("units", ctypes.c_longlong), ("m_bucket", ctypes.c_int),
                ("warps_per_unit", ctypes.c_int)]


_SIGS = {
    "ql_status_str": (ctypes.c_char_p, [_I]),
    "qlinear_packed_bytes": (_SZ, [_I, _I, _I]),
    "qlinear_params_bytes": (_SZ, [_I, _I, _I]),
    "qlinear_pack": (_I, [_I, _P, _P, _I, _I]),
    "qlinear_pack_params": (_I, [_I, _P, _P, _I, _I]),
    "qlinear_params_bytes_grouped": (_SZ, [_I, _I, _I, _I]),
    "qlinear_pack_params_grouped": (_I, [_I, _I, _P, _P, _I, _I]),
    "qlinear_pack_tilecoo": (_I, [_P, _P, _P, _I, _I, _P, _P, _P]),
    "qlinear_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "qlinear_w4a16": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_w2a16": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_w8a16": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_w3a16": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_lut4": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_w4a16_outlier": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_debug_unpack": (_I, [_I, _P, _P, _I, _I, _P]),
    "qlinear_debug_dequant": (_I, [_I, _P, _P, _P, _P, _I, _I, _P]),
    "qlinear_plan": (_I, [_I, _I, _I, _I, ctypes.POINTER(ql_plan)]),
    "qlinear_read_error": (_I, [_P, ctypes.POINTER(ctypes.c_uint32), _P]),
    "qlinear_debug_wait_test": (_I, [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32]),
    "qlinear_w4a16_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "qlinear_w4a16_noalloc_read_error": (_I, [ctypes.POINTER(ctypes.c_uint32), _P]),
    "qlinear_dequant_fp16": (_I, [_I, _P, _P, _P, _P, _I, _I, _P]),
    "qlinear_prefill": (_I, [_I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "qlinear_prefill_fused": (_I, [_I, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_prefill_workspace_bytes": (_SZ, [_I, _I, _I]),
    "qlinear_prefill_read_error": (_I, [ctypes.POINTER(ctypes.c_uint32), _P]),
    "qlinear_policy_set": (_I, [ctypes.POINTER(ql_policy_entry), _I]),
    "qlinear_policy_size": (_I, []),
    "qlinear_policy_lookup": (_I, [_I, _I, _I, _I, ctypes.POINTER(ql_policy_entry),
                                   ctypes.POINTER(_I)]),
    "qlinear_matmul": (_I, [_I, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P, _P]),
    "qlinear_pack_codebook": (_I, [_P, _P, _I, _I]),
    "qlinear_pack_codebook_scales": (_I, [_P, _P, _I, _I]),
    "qlinear_codebook_workspace_bytes": (_SZ, [_I, _I, _I]),
    "qlinear_codebook": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_pack_codebook_tc": (_I, [_P, _P, _I, _I]),
    "qlinear_codebook_tc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_fused_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "qlinear_linear": (_I, [_I, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_linear_backward": (_I, [_I, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P, _SZ,
                                     _P]),
    "qlinear_gated": (_I, [_I, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_gated_backward": (_I, [_I, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P, _SZ,
                                    _P]),
    "qlinear_pack_gated": (_I, [_I, _P, _P, _P, _I, _I]),
    "qlinear_pack_params_gated": (_I, [_I, _P, _P, _P, _I, _I]),
    "qlinear_fp8_quantize": (_I, [_I, _P, _LL, _P, _P, _I, _I, _P]),
    "qlinear_fp8_quantize_weights": (_I, [_I, _P, _P, _P, _I, _I, _I, _P]),
    "qlinear_fp8_gated": (_I, [_I, _I, _P, _P, _P, _I, _I, _P]),
    "qlinear_fp8_gated_backward": (_I, [_I, _I, _P, _P, _P, _P, _I, _I, _P]),
    "qlinear_rmsnorm": (_I, [_I, _P, _LL, _P, _P, ctypes.c_float, _P, _P, _P, _P, _P, _I, _I,
                             _P]),
    "qlinear_rmsnorm_backward": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _SZ, _P]),
    "qlinear_rmsnorm_backward_grouped": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P,
                                              _SZ, _P]),
    "qlinear_rmsnorm_workspace_bytes": (_SZ, [_I, _I]),
    "qlinear_fp8_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "qlinear_fp8_linear": (_I, [_I, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_fp8_linear_backward": (_I, [_I, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_fp8_grouped": (_I, [_I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "qlinear_fp8_grouped_backward": (_I, [_I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ,
                                          _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


class QLinearError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.ql_status_str(status).decode()
        super().__init__(f"{where}: {STATUS.get(status, status)} ({msg})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != 0:
        raise QLinearError(status, where)


def _ptr(t) -> Optional[int]:
    """Device pointer of a torch tensor, or None."""
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _np_ptr(a: np.ndarray) -> int:
    assert a.flags["C_CONTIGUOUS"]
    return a.ctypes.data


# ---------------------------------------------------------------------------
# host packer (NumPy in, NumPy out)


def qlinear_packed_bytes(fmt: int, N: int, K: int) -> int:
    return int(_lib.qlinear_packed_bytes(fmt, N, K))


def qlinear_params_bytes(fmt: int, N: int, K: int) -> int:
    return int(_lib.qlinear_params_bytes(fmt, N, K))


def qlinear_pack(fmt: int, canonical: np.ndarray, N: int, K: int) -> np.ndarray:
    canonical = np.ascontiguousarray(canonical)
    out = np.empty(qlinear_packed_bytes(fmt, N, K), dtype=np.uint8)
    if out.size != canonical.nbytes:
        raise QLinearError(2, "qlinear_pack")
    _check(_lib.qlinear_pack(fmt, _np_ptr(canonical), _np_ptr(out), N, K), "qlinear_pack")
    return out


def qlinear_pack_params(fmt: int, canonical: np.ndarray, N: int, K: int) -> np.ndarray:
    canonical = np.ascontiguousarray(canonical)
    out = np.empty(canonical.shape, dtype=canonical.dtype)
    if canonical.nbytes != qlinear_params_bytes(fmt, N, K):
        raise QLinearError(2, "qlinear_pack_params")
    _check(_lib.qlinear_pack_params(fmt, _np_ptr(canonical), _np_ptr(out), N, K),
           "qlinear_pack_params")
    return out


def qlinear_params_bytes_grouped(fmt: int, group: int, N: int, K: int) -> int:
    return int(_lib.qlinear_params_bytes_grouped(fmt, group, N, K))


def qlinear_pack_params_grouped(fmt: int, group: int, canonical: np.ndarray, N: int,
                                K: int) -> np.ndarray:
    """fp16 [K / group, N] (or [1, N] for group = K) -> the kernel layout for that group."""
    canonical = np.ascontiguousarray(canonical, dtype=np.float16)
    rows = 1 if group == K else K // group
    if canonical.shape != (rows, N):
        raise QLinearError(2, "qlinear_pack_params_grouped")
    nbytes = qlinear_params_bytes_grouped(fmt, group, N, K)
    if nbytes == 0:
        raise QLinearError(2, "qlinear_pack_params_grouped")
    out = np.empty(nbytes // 2, dtype=np.float16)
    _check(_lib.qlinear_pack_params_grouped(fmt, group, _np_ptr(canonical), _np_ptr(out), N, K),
           "qlinear_pack_params_grouped")
    return out


def qlinear_pack_tilecoo(offsets: np.ndarray, rc: np.ndarray, vals: np.ndarray, N: int, K: int):
    offsets = np.ascontiguousarray(offsets, dtype=np.uint32)
    rc = np.ascontiguousarray(rc, dtype=np.uint8)
    vals = np.ascontiguousarray(vals).view(np.uint16)
    o2, r2, v2 = np.empty_like(offsets), np.empty_like(rc), np.empty_like(vals)
    _check(_lib.qlinear_pack_tilecoo(_np_ptr(offsets), _np_ptr(rc), _np_ptr(vals), N, K,
                                     _np_ptr(o2), _np_ptr(r2), _np_ptr(v2)), "qlinear_pack_tilecoo")
    return o2, r2, v2.view(np.float16)


# ---------------------------------------------------------------------------
# workspace / plan


def qlinear_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(_lib.qlinear_workspace_bytes(fmt, M, N, K))


def qlinear_plan(fmt: int, M: int, N: int, K: int) -> ql_plan:
    p = ql_plan()
    _check(_lib.qlinear_plan(fmt, M, N, K, ctypes.byref(p)), "qlinear_plan")
    return p


def qlinear_debug_wait_test(wait_limit=0, producer_delay_us=0, consumer_hold_us=0) -> None:
    """Settings for tests of the bounded device waits; no arguments restores the defaults."""
    _check(_lib.qlinear_debug_wait_test(wait_limit, producer_delay_us, consumer_hold_us),
           "qlinear_debug_wait_test")


def qlinear_read_error(workspace, stream=None) -> int:
    """Sticky error flags of the calls that used `workspace` (then cleared); 0 = none."""
    flags = ctypes.c_uint32(0)
    _check(_lib.qlinear_read_error(_ptr(workspace), ctypes.byref(flags), _stream(stream)),
           "qlinear_read_error")
    return int(flags.value)


# ---------------------------------------------------------------------------
# hot path (torch tensors on the current device)


def _uniform(name, x, qweight, scales, zeros, y, M, N, K, workspace, stream, group=128):
    st = getattr(_lib, name)(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(y), M, N, K,
                             group, _ptr(workspace), workspace.numel() * workspace.element_size()
                             if workspace is not None else 0, _stream(stream))
    _check(st, name)
    return y


def qlinear_w4a16(x, qweight, scales, zeros, y, M, N, K, workspace, stream=None, group=128):
    return _uniform("qlinear_w4a16", x, qweight, scales, zeros, y, M, N, K, workspace, stream, group)


def qlinear_w2a16(x, qweight, scales, zeros, y, M, N, K, workspace, stream=None, group=128):
    return _uniform("qlinear_w2a16", x, qweight, scales, zeros, y, M, N, K, workspace, stream, group)


def qlinear_w8a16(x, qweight, scales, zeros, y, M, N, K, workspace, stream=None, group=128):
    return _uniform("qlinear_w8a16", x, qweight, scales, zeros, y, M, N, K, workspace, stream, group)


def qlinear_w3a16(x, qweight, scales, zeros, y, M, N, K, workspace, stream=None, group=128):
    return _uniform("qlinear_w3a16", x, qweight, scales, zeros, y, M, N, K, workspace, stream, group)


def qlinear_w4a16_noalloc(x, qweight, scales, zeros, y, M, N, K, stream=None, group=128):
    """qlinear_w4a16 with the library's fixed device scratch instead of a workspace."""
    _check(_lib.qlinear_w4a16_noalloc(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(y),
                                      M, N, K, group, _stream(stream)), "qlinear_w4a16_noalloc")
    return y


def qlinear_w4a16_noalloc_read_error(stream=None) -> int:
    """Sticky error flags of qlinear_w4a16_noalloc's scratch on the current device (then
    cleared); 0 = none."""
    flags = ctypes.c_uint32(0)
    _check(_lib.qlinear_w4a16_noalloc_read_error(ctypes.byref(flags), _stream(stream)),
           "qlinear_w4a16_noalloc_read_error")
    return int(flags.value)


def qlinear_lut4(x, codes, lut16, absmax, y, M, N, K, workspace, stream=None, block=64):
    st = _lib.qlinear_lut4(_ptr(x), _ptr(codes), _ptr(lut16), _ptr(absmax), _ptr(y), M, N, K, block,
                           _ptr(workspace), workspace.numel() * workspace.element_size()
                           if workspace is not None else 0, _stream(stream))
    _check(st, "qlinear_lut4")
    return y


def qlinear_w4a16_outlier(x, qweight, scales, zeros, tile_offsets, tile_rc, tile_vals, y, M, N, K,
                          workspace, stream=None, group=128):
    st = _lib.qlinear_w4a16_outlier(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros),
                                    _ptr(tile_offsets), _ptr(tile_rc), _ptr(tile_vals), _ptr(y),
                                    M, N, K, group, _ptr(workspace),
                                    workspace.numel() * workspace.element_size()
                                    if workspace is not None else 0, _stream(stream))
    _check(st, "qlinear_w4a16_outlier")
    return y


def qlinear_debug_unpack(fmt, packed, codes, N, K, stream=None):
    _check(_lib.qlinear_debug_unpack(fmt, _ptr(packed), _ptr(codes), N, K, _stream(stream)),
           "qlinear_debug_unpack")
    return codes


def qlinear_debug_dequant(fmt, packed, p0, p1, w, N, K, stream=None):
    _check(_lib.qlinear_debug_dequant(fmt, _ptr(packed), _ptr(p0), _ptr(p1), _ptr(w), N, K,
                                      _stream(stream)), "qlinear_debug_dequant")
    return w


def qlinear_dequant_fp16(fmt, packed, p0, p1, w, N, K, stream=None):
    """Packed weights -> dense fp16 ``w[N, K]`` (see the C declaration for p0 / p1)."""
    _check(_lib.qlinear_dequant_fp16(fmt, _ptr(packed), _ptr(p0), _ptr(p1), _ptr(w), N, K,
                                     _stream(stream)), "qlinear_dequant_fp16")
    return w


def qlinear_prefill(fmt, x, packed, p0, p1, w_fp16, y, M, N, K, stream=None):
    """``y[M, N] = x[M, K] @ w_fp16[N, K]^T`` after dequantizing into ``w_fp16``."""
    _check(_lib.qlinear_prefill(fmt, _ptr(x), _ptr(packed), _ptr(p0), _ptr(p1), _ptr(w_fp16),
                                _ptr(y), M, N, K, _stream(stream)), "qlinear_prefill")
    return y


def qlinear_prefill_fused(fmt, x, packed, p0, p1, y, M, N, K, workspace=None, stream=None):
    """``y[M, N] = x[M, K] @ W^T`` with the weights dequantized inside the tensor-core GEMM;
    with a (zero-filled) workspace the k-blocks are shared out over the SMs (stream-K)."""
    _check(_lib.qlinear_prefill_fused(fmt, _ptr(x), _ptr(packed), _ptr(p0), _ptr(p1), _ptr(y),
                                      M, N, K, _ptr(workspace),
                                      workspace.numel() * workspace.element_size()
                                      if workspace is not None else 0, _stream(stream)),
           "qlinear_prefill_fused")
    return y


def qlinear_prefill_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.qlinear_prefill_workspace_bytes(M, N, K))


def qlinear_prefill_read_error(stream=None) -> int:
    """Sticky wait-timeout flags of the prefill GEMM kernels on the current device (then
    cleared); 0 = none."""
    flags = ctypes.c_uint32(0)
    _check(_lib.qlinear_prefill_read_error(ctypes.byref(flags), _stream(stream)),
           "qlinear_prefill_read_error")
    return int(flags.value)


# ---------------------------------------------------------------------------
# measured policy map and dispatcher


_ENTRY_KEYS = ("fmt", "N", "K", "m_lo", "m_hi", "strategy", "warps_per_unit", "ctas")


def qlinear_policy_set(entries) -> None:
    """Install a policy table: a sequence of dicts (or ql_policy_entry) with the entry's
    fields; an empty sequence clears it."""
    arr = (ql_policy_entry * max(len(entries), 1))()
    for i, e in enumerate(entries):
        arr[i] = e if isinstance(e, ql_policy_entry) else \
            ql_policy_entry(*[int(e.get(k, 0)) for k in _ENTRY_KEYS])
    _check(_lib.qlinear_policy_set(arr, len(entries)), "qlinear_policy_set")


def qlinear_policy_size() -> int:
    return int(_lib.qlinear_policy_size())


def qlinear_policy_lookup(fmt: int, M: int, N: int, K: int):
    """(decision as a dict, whether it came from the table)."""
    e = ql_policy_entry()
    ft = _I(0)
    _check(_lib.qlinear_policy_lookup(fmt, M, N, K, ctypes.byref(e), ctypes.byref(ft)),
           "qlinear_policy_lookup")
    return {k: getattr(e, k) for k in _ENTRY_KEYS}, bool(ft.value)


def default_policy_path() -> str:
    """The table measured on B200 for the Llama-shaped layers (the package's policy_b200.json,
    written by the tune module)."""
    return os.path.join(_HERE, "policy_b200.json")


def load_policy(path: Optional[str] = None) -> int:
    """Install the table of a JSON file written by the tune module (default: the B200 table);
    returns its size."""
    import json
    with open(path or default_policy_path()) as f:
        table = json.load(f)
    qlinear_policy_set(table["entries"])
    return qlinear_policy_size()


def qlinear_matmul(fmt, x, packed, p0, p1, y, M, N, K, workspace, w_fp16=None, stream=None):
    """y[M, N] = x[M, K] . W for any M, by the policy map (GEMV slices or prefill)."""
    st = _lib.qlinear_matmul(fmt, _ptr(x), _ptr(packed), _ptr(p0), _ptr(p1), _ptr(y), M, N, K,
                             _ptr(workspace), workspace.numel() * workspace.element_size()
                             if workspace is not None else 0, _ptr(w_fp16), _stream(stream))
    _check(st, "qlinear_matmul")
    return y


# ---------------------------------------------------------------------------
# codebook GEMV (Psumbook)


def qlinear_pack_codebook(codes: np.ndarray, N: int, K: int) -> np.ndarray:
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    if codes.size != K // 4 * N:
        raise QLinearError(2, "qlinear_pack_codebook")
    out = np.empty(codes.size, dtype=np.uint8)
    _check(_lib.qlinear_pack_codebook(_np_ptr(codes), _np_ptr(out), N, K), "qlinear_pack_codebook")
    return out


def qlinear_pack_codebook_scales(scales: np.ndarray, N: int, K: int) -> np.ndarray:
    scales = np.ascontiguousarray(scales).view(np.uint16)
    if scales.size != K // 128 * N:
        raise QLinearError(2, "qlinear_pack_codebook_scales")
    out = np.empty(scales.size, dtype=np.uint16)
    _check(_lib.qlinear_pack_codebook_scales(_np_ptr(scales), _np_ptr(out), N, K),
           "qlinear_pack_codebook_scales")
    return out


def qlinear_codebook_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(_lib.qlinear_codebook_workspace_bytes(M, N, K))


def qlinear_codebook(x, codes, scales, codebook, y, M, N, K, workspace, stream=None):
    st = _lib.qlinear_codebook(_ptr(x), _ptr(codes), _ptr(scales), _ptr(codebook), _ptr(y), M, N,
                               K, _ptr(workspace), workspace.numel() * workspace.element_size()
                               if workspace is not None else 0, _stream(stream))
    _check(st, "qlinear_codebook")
    return y


# codebook GEMV on the tensor cores (the GEMV kernel, codebook lookups as A fragments)


def qlinear_pack_codebook_tc(codes: np.ndarray, N: int, K: int) -> np.ndarray:
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    if codes.size != K // 4 * N:
        raise QLinearError(2, "qlinear_pack_codebook_tc")
    out = np.empty(codes.size, dtype=np.uint8)
    _check(_lib.qlinear_pack_codebook_tc(_np_ptr(codes), _np_ptr(out), N, K),
           "qlinear_pack_codebook_tc")
    return out


def qlinear_codebook_tc(x, codes, scales, codebook, y, M, N, K, workspace, stream=None):
    st = _lib.qlinear_codebook_tc(_ptr(x), _ptr(codes), _ptr(scales), _ptr(codebook), _ptr(y), M,
                                  N, K, _ptr(workspace), workspace.numel() * workspace.element_size()
                                  if workspace is not None else 0, _stream(stream))
    _check(st, "qlinear_codebook_tc")
    return y


# ---------------------------------------------------------------------------
# fused linear layers: bias, activation and residual in the epilogue, the gated projection,
# and their backward passes.  act: a key of ACTS, or a ql_act value.


def _act(act) -> int:
    if isinstance(act, str):
        if act not in ACTS:
            raise QLinearError(4, f"activation {act!r}")
        return ACTS[act]
    return int(act)


def _ws(workspace):
    return _ptr(workspace), (workspace.numel() * workspace.element_size()
                             if workspace is not None else 0)


def qlinear_fused_workspace_bytes(fmt: int, M: int, N: int, K: int, backward: bool = True) -> int:
    return int(_lib.qlinear_fused_workspace_bytes(fmt, M, N, K, int(backward)))


def qlinear_linear(fmt, x, packed, p0, p1, y, M, N, K, workspace, bias=None, residual=None,
                   act="none", z=None, stream=None):
    """``y[M, N] = act(x . W + bias) + residual``; z, when given, receives x . W + bias."""
    _check(_lib.qlinear_linear(fmt, _ptr(x), _ptr(packed), _ptr(p0), _ptr(p1), _ptr(bias),
                               _ptr(residual), _act(act), _ptr(y), _ptr(z), M, N, K,
                               *_ws(workspace), _stream(stream)), "qlinear_linear")
    return y


def qlinear_linear_backward(fmt, dy, z, packed, p0, p1, dx, M, N, K, workspace, act="none",
                            dbias=None, stream=None):
    """``dx[M, K] = (dy * act'(z)) . W^T``; dbias (fp32 [N]), when given, the column sums."""
    _check(_lib.qlinear_linear_backward(fmt, _ptr(dy), _ptr(z), _ptr(packed), _ptr(p0), _ptr(p1),
                                        _act(act), _ptr(dx), _ptr(dbias), M, N, K,
                                        *_ws(workspace), _stream(stream)),
           "qlinear_linear_backward")
    return dx


def qlinear_gated(fmt, x, packed, p0, p1, h, M, F, K, workspace, bias=None, act="silu", gu=None,
                  stream=None):
    """``h[M, F] = act(x . Wg + bias[0]) * (x . Wu + bias[1])``; gu [M, 2, F], when given,
    receives the two factors before the activation."""
    _check(_lib.qlinear_gated(fmt, _ptr(x), _ptr(packed), _ptr(p0), _ptr(p1), _ptr(bias),
                              _act(act), _ptr(h), _ptr(gu), M, F, K, *_ws(workspace),
                              _stream(stream)), "qlinear_gated")
    return h


def qlinear_gated_backward(fmt, dh, gu, packed, p0, p1, dx, M, F, K, workspace, act="silu",
                           dbias=None, stream=None):
    """``dx[M, K]`` of qlinear_gated from dh and the kept gu; dbias fp32 [2, F]."""
    _check(_lib.qlinear_gated_backward(fmt, _ptr(dh), _ptr(gu), _ptr(packed), _ptr(p0), _ptr(p1),
                                       _act(act), _ptr(dx), _ptr(dbias), M, F, K,
                                       *_ws(workspace), _stream(stream)),
           "qlinear_gated_backward")
    return dx


def qlinear_pack_gated(fmt: int, gate: np.ndarray, up: np.ndarray, F: int, K: int) -> np.ndarray:
    """Canonical codes of the gate and up projections -> one packed matrix of 2 F columns."""
    gate, up = np.ascontiguousarray(gate), np.ascontiguousarray(up)
    out = np.empty(qlinear_packed_bytes(fmt, 2 * F, K), dtype=np.uint8)
    if out.size == 0 or 2 * gate.nbytes != out.size or 2 * up.nbytes != out.size:
        raise QLinearError(2, "qlinear_pack_gated")
    _check(_lib.qlinear_pack_gated(fmt, _np_ptr(gate), _np_ptr(up), _np_ptr(out), F, K),
           "qlinear_pack_gated")
    return out


def qlinear_pack_params_gated(fmt: int, gate: np.ndarray, up: np.ndarray, F: int,
                              K: int) -> np.ndarray:
    """One parameter array of each projection (fp16 [K / 128, F], or LUT4's fp32 absmax
    [K / 64, F]) -> the kernel layout of the 2 F columns."""
    dtype = np.float32 if fmt == QL_FMT_LUT4 else np.float16
    gate, up = np.ascontiguousarray(gate, dtype=dtype), np.ascontiguousarray(up, dtype=dtype)
    nbytes = qlinear_params_bytes(fmt, 2 * F, K)
    if nbytes == 0 or 2 * gate.nbytes != nbytes or 2 * up.nbytes != nbytes:
        raise QLinearError(2, "qlinear_pack_params_gated")
    out = np.empty(nbytes // dtype().itemsize, dtype=dtype)
    _check(_lib.qlinear_pack_params_gated(fmt, _np_ptr(gate), _np_ptr(up), _np_ptr(out), F, K),
           "qlinear_pack_params_gated")
    return out


# ---------------------------------------------------------------------------
# 8-bit floating-point layers: e4m3 codes with a scale per 128.  type: a key of TYPES (a torch
# dtype's name), or a ql_type value.


def _type(type_) -> int:
    if isinstance(type_, str):
        if type_ not in TYPES:
            raise QLinearError(4, f"type {type_!r}")
        return TYPES[type_]
    return int(type_)


def qlinear_fp8_quantize(type_, x, q, scales, M, K, ldx=None, stream=None):
    """Codes ``q[M, K]`` and scales ``[M, ceil(K / 128)]`` of the rows of x, ldx elements apart."""
    _check(_lib.qlinear_fp8_quantize(_type(type_), _ptr(x), K if ldx is None else ldx, _ptr(q),
                                     _ptr(scales), M, K, _stream(stream)), "qlinear_fp8_quantize")
    return q


def qlinear_fp8_quantize_weights(type_, w, q, scales, E, N, K, stream=None):
    """Codes ``q[E, N, K]`` and scales ``[E, ceil(N / 128), ceil(K / 128)]`` of w."""
    _check(_lib.qlinear_fp8_quantize_weights(_type(type_), _ptr(w), _ptr(q), _ptr(scales), E, N,
                                             K, _stream(stream)), "qlinear_fp8_quantize_weights")
    return q


def qlinear_fp8_gated(type_, gu, q, scales, M, F, act="silu", stream=None):
    """Codes ``q[M, F]`` and scales of ``act(g) * u``, gu[M, 2 F] = (g, u)."""
    _check(_lib.qlinear_fp8_gated(_type(type_), _act(act), _ptr(gu), _ptr(q), _ptr(scales), M, F,
                                  _stream(stream)), "qlinear_fp8_gated")
    return q


def qlinear_fp8_gated_backward(type_, dh, gu, q, scales, M, F, act="silu", stream=None):
    """Codes ``q[M, 2 F]`` and scales of the gradients (dg, du)."""
    _check(_lib.qlinear_fp8_gated_backward(_type(type_), _act(act), _ptr(dh), _ptr(gu), _ptr(q),
                                           _ptr(scales), M, F, _stream(stream)),
           "qlinear_fp8_gated_backward")
    return q


def qlinear_rmsnorm(type_, x, weight, eps, M, K, residual=None, total=None, y=None, q=None,
                    scales=None, rstd=None, ldx=None, stream=None):
    """RMS norm of x (+ residual) into those of total, y, q with scales, and rstd that are given."""
    _check(_lib.qlinear_rmsnorm(_type(type_), _ptr(x), K if ldx is None else ldx, _ptr(residual),
                                _ptr(weight), eps, _ptr(total), _ptr(y), _ptr(q), _ptr(scales),
                                _ptr(rstd), M, K, _stream(stream)), "qlinear_rmsnorm")


def qlinear_rmsnorm_workspace_bytes(M: int, K: int) -> int:
    return int(_lib.qlinear_rmsnorm_workspace_bytes(M, K))


def qlinear_rmsnorm_backward(type_, dy, total, rstd, weight, dx, M, K, dtotal=None, dweight=None,
                             workspace=None, stream=None):
    """``dx[M, K]`` of qlinear_rmsnorm; dweight (fp32 [K]), when given, the weight's gradient."""
    _check(_lib.qlinear_rmsnorm_backward(_type(type_), _ptr(dy), _ptr(total), _ptr(rstd),
                                         _ptr(weight), _ptr(dtotal), _ptr(dx), _ptr(dweight), M,
                                         K, *_ws(workspace), _stream(stream)),
           "qlinear_rmsnorm_backward")
    return dx


def qlinear_rmsnorm_backward_grouped(type_, dy, total, rstd, weight, offsets, dx, M, E, K,
                                     dtotal=None, dweight=None, workspace=None, stream=None):
    """qlinear_rmsnorm_backward where only the rows offsets[0] .. offsets[E] - 1 have a dy; offsets
    int32 [E + 1] on the device."""
    _check(_lib.qlinear_rmsnorm_backward_grouped(_type(type_), _ptr(dy), _ptr(total), _ptr(rstd),
                                                 _ptr(weight), _ptr(dtotal), _ptr(offsets),
                                                 _ptr(dx), _ptr(dweight), M, E, K,
                                                 *_ws(workspace), _stream(stream)),
           "qlinear_rmsnorm_backward_grouped")
    return dx


def qlinear_fp8_workspace_bytes(M: int, E: int, N: int, K: int) -> int:
    return int(_lib.qlinear_fp8_workspace_bytes(M, E, N, K))


def qlinear_fp8_linear(type_, q, scales, w, wscales, y, M, N, K, workspace, stream=None):
    """``y[M, N] = x . W^T`` from the codes and scales of x [M, K] and W [N, K]."""
    _check(_lib.qlinear_fp8_linear(_type(type_), _ptr(q), _ptr(scales), _ptr(w), _ptr(wscales),
                                   _ptr(y), M, N, K, *_ws(workspace), _stream(stream)),
           "qlinear_fp8_linear")
    return y


def qlinear_fp8_linear_backward(type_, q, scales, w, wscales, dx, M, N, K, workspace,
                                stream=None):
    """``dx[M, K] = dy . W`` from the codes and scales of dy [M, N] and W [N, K]."""
    _check(_lib.qlinear_fp8_linear_backward(_type(type_), _ptr(q), _ptr(scales), _ptr(w),
                                            _ptr(wscales), _ptr(dx), M, N, K, *_ws(workspace),
                                            _stream(stream)), "qlinear_fp8_linear_backward")
    return dx


def qlinear_fp8_grouped(type_, q, scales, offsets, w, wscales, y, M, E, N, K, workspace,
                        stream=None):
    """qlinear_fp8_linear with rows offsets[e] .. offsets[e + 1] by W[e]; offsets int32 [E + 1] on
    the device."""
    _check(_lib.qlinear_fp8_grouped(_type(type_), _ptr(q), _ptr(scales), _ptr(offsets), _ptr(w),
                                    _ptr(wscales), _ptr(y), M, E, N, K, *_ws(workspace),
                                    _stream(stream)), "qlinear_fp8_grouped")
    return y


def qlinear_fp8_grouped_backward(type_, q, scales, offsets, w, wscales, dx, M, E, N, K, workspace,
                                 stream=None):
    """qlinear_fp8_linear_backward with rows offsets[e] .. offsets[e + 1] by W[e]."""
    _check(_lib.qlinear_fp8_grouped_backward(_type(type_), _ptr(q), _ptr(scales), _ptr(offsets),
                                             _ptr(w), _ptr(wscales), _ptr(dx), M, E, N, K,
                                             *_ws(workspace), _stream(stream)),
           "qlinear_fp8_grouped_backward")
    return dx
