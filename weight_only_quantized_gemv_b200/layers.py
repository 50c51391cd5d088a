"""Device-resident quantized linear layers.

A layer takes the canonical arrays of one weight matrix (NumPy, host), packs them
with the library's host packer, uploads the packed arrays once, and owns a
zero-filled workspace.  ``forward`` enqueues the entry point on a stream.  The
class only moves and marshals data; every operation runs in ``libqlinear.so``.
"""
from __future__ import annotations

import threading
from types import SimpleNamespace
from typing import Optional

import numpy as np
import torch
from torch.autograd import forward_ad

from . import (QL_ERR_WORKSPACE, QL_FMT_CB, QL_FMT_LUT4, QL_FMT_W2, QL_FMT_W3, QL_FMT_W4, QL_FMT_W8,
               qlinear_codebook, qlinear_codebook_tc, qlinear_codebook_workspace_bytes,
               qlinear_debug_dequant, qlinear_pack_codebook, qlinear_pack_codebook_scales,
               qlinear_pack_codebook_tc,
               qlinear_debug_unpack, qlinear_dequant_fp16, qlinear_lut4, qlinear_pack,
               qlinear_matmul, qlinear_pack_params, qlinear_pack_params_grouped,
               qlinear_prefill, qlinear_prefill_fused, qlinear_prefill_workspace_bytes,
               qlinear_fused_workspace_bytes, qlinear_pack_gated, qlinear_pack_params_gated,
               qlinear_read_error,
               qlinear_pack_tilecoo, qlinear_w2a16, qlinear_w3a16, qlinear_w4a16,
               qlinear_w4a16_outlier,
               qlinear_fp8_quantize_weights, qlinear_fp8_workspace_bytes,
               qlinear_rmsnorm_workspace_bytes,
               qlinear_w8a16, qlinear_workspace_bytes, _act, _check, _lib)

_ENTRY = {QL_FMT_W2: qlinear_w2a16, QL_FMT_W3: qlinear_w3a16, QL_FMT_W4: qlinear_w4a16,
          QL_FMT_W8: qlinear_w8a16}


def _dev(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


def _lut16(table) -> np.ndarray:
    """A LUT4 table as fp16; the kernels read 16 entries."""
    table = np.asarray(table, dtype=np.float16)
    if table.size < 16:
        raise ValueError(f"a LUT4 table has 16 entries, not {table.size}")
    return table


_FUSED_FORMATS = (QL_FMT_W2, QL_FMT_W4, QL_FMT_W8, QL_FMT_LUT4)
_F16, _F32 = torch.float16, torch.float32
_MAX_ROWS = 1 << 24  # of a fused call
# (the handle alone, without a Stream object around it, where torch offers that)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)
# (outside of a dual level no tensor has a tangent, and asking takes as long as its other checks)
_levels = forward_ad if hasattr(forward_ad, "_current_level") else SimpleNamespace(_current_level=0)


def _as_stream(stream, index: int) -> torch.cuda.Stream:
    """A torch stream, a raw cudaStream_t or None (the current one) as a torch stream."""
    if stream is None:
        return torch.cuda.current_stream(index)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    device = torch.device("cuda", index)
    return (torch.cuda.ExternalStream(stream, device=device) if stream
            else torch.cuda.default_stream(device))


def _dual(t: torch.Tensor) -> bool:
    """Whether forward-mode differentiation follows `t` (not inside an autograd.Function)."""
    return forward_ad.unpack_dual(t).tangent is not None


def _fused_ptr(t, shape: tuple, index: int, name: str, dtype=_F16) -> Optional[int]:
    """The data pointer of `t` once checked (None for None): `shape`, `dtype`, contiguous, on
    CUDA device `index`, and nothing that autograd would have to follow."""
    if t is None:
        return None
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which autograd does not carry through the "
                         "fused layers: call them under torch.no_grad() (as inside an "
                         "autograd.Function) and their backward methods for the gradient")
    if _levels._current_level >= 0 and _dual(t):
        raise ValueError(f"{name} has a tangent, which forward-mode differentiation does not carry "
                         "through the fused layers: call them inside an autograd.Function")
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != index):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on "
                         f"cuda:{index}, not {t.dtype} {tuple(t.shape)} with strides "
                         f"{t.stride()} on {t.device}")
    return t.data_ptr()


class _FusedWorkspace:
    """What the fused entries (bias / activation / residual, gated, backward) of a layer share:
    argument checks and the workspace.

    The workspace is one zero-filled buffer, made by ``reserve`` for the rows asked for, or by the
    first call that needs it, then for the next power of two of rows: buffers that were outgrown
    stay alive with the layer, since a captured graph may still use them, and lengths that rise
    step by step must not leave one each.  All layers lay a workspace out alike, so one that is
    large enough for the largest of a model's layers can be passed to the calls of all of them
    that follow one another (``workspace=``), instead of one in each.

    Calls of one layer run one after the other, whichever host threads they come from: a call's
    launches are enqueued under the layer's lock, and an eager call on another stream than the
    last waits for that stream's work.  Work that overlaps in time - graphs captured from one
    layer and replayed at the same time - needs a workspace of its own:
    ``workspace=layer.new_workspace(rows)``.  Tensors a call makes are made on its stream.  A
    stream given as a raw handle must live until the layer's next call on another stream, which
    waits for it.
    """

    def __getstate__(self):  # a copied or unpickled layer has a lock and workspaces of its own
        own = ("_fused_lock", "_fused_ws", "_fused_last")
        return {k: v for k, v in self.__dict__.items() if k not in own}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._fused_lock = threading.RLock()

    _fused_ws: tuple = ()    # buffers, the one in use last
    _fused_last = None       # stream of the last eager call: (raw handle, torch stream)

    def _fused_setup(self):
        """(fmt, N, K, device index) of the packed matrix, checked at the first call."""
        fmt, N, K = self._fused_matrix()
        if fmt not in _FUSED_FORMATS:
            raise ValueError("the fused layers cover W2, W4, W8 (group 128) and LUT4")
        self._fused = (fmt, N, K, self.qweight.get_device())
        return self._fused

    def _fused_weights(self) -> tuple:
        return self.qweight.data_ptr(), self.p0.data_ptr(), self.p1.data_ptr()

    _fused = None

    def _fused_bytes(self, rows: int, backward: bool) -> int:
        fmt, N, K, index = self._fused or self._fused_setup()
        with torch.cuda.device(index):
            need = qlinear_fused_workspace_bytes(fmt, rows, N, K, backward)
        if need == 0:
            raise ValueError(f"no fused product for {rows} rows, N={N}, K={K}")
        return need

    def new_workspace(self, rows: int, backward: bool = True) -> torch.Tensor:
        """A zero-filled workspace for calls of up to `rows` rows."""
        need = self._fused_bytes(rows, backward)
        with torch.cuda.device(self._fused[3]):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("reserve(rows) the workspace before capturing a graph")
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()  # the zero fill has landed, whichever stream uses it
        return ws

    def reserve(self, rows: int, backward: bool = True) -> None:
        """Make the layer's own workspace large enough for calls of up to `rows` rows (a call
        that needs more does this itself, except while a graph is being captured)."""
        with self._fused_lock:
            if (not self._fused_ws
                    or self._fused_ws[-1].numel() < self._fused_bytes(rows, backward)):
                self._fused_ws = self._fused_ws + (self.new_workspace(rows, backward),)

    def _fused_call(self, entry, name: str, head: tuple, rows: int, backward: bool, workspace,
                    stream):
        """entry(*head, workspace, bytes, stream), the layer's device being current.  The
        layer's own workspace is grown when the entry finds it too small."""
        index = self._fused[3]
        if stream is None:
            raw = _current_stream(index)
        else:
            raw = getattr(stream, "cuda_stream", stream)
        if workspace is not None:
            if workspace.get_device() != index or not workspace.is_contiguous():
                raise ValueError(f"the workspace must be a contiguous tensor on cuda:{index}")
            _check(entry(*head, workspace.data_ptr(),
                         workspace.numel() * workspace.element_size(), raw), name)
            return
        # the whole of a call's enqueueing: a second thread's stream must wait for all of it, and
        # on the same stream its launches must not come between these
        self._fused_lock.acquire()
        try:
            if self._fused_last is None or self._fused_last[0] != raw:
                self._fused_switch(raw, stream)
            if self._fused_ws:
                ws = self._fused_ws[-1]
                status = entry(*head, ws.data_ptr(), ws.numel(), raw)
                if status != QL_ERR_WORKSPACE:
                    _check(status, name)
                    return
            try:
                self.reserve(max(rows, min(1 << (rows - 1).bit_length(), _MAX_ROWS)), backward)
            except torch.OutOfMemoryError:
                self.reserve(rows, backward)
            ws = self._fused_ws[-1]
            _check(entry(*head, ws.data_ptr(), ws.numel(), raw), name)
        finally:
            self._fused_lock.release()

    def _fused_switch(self, raw: int, stream) -> None:
        """The layer's workspace moves to another stream: that one waits for the last."""
        stream = _as_stream(stream, self._fused[3])
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
        if self._fused_last is not None:
            stream.wait_stream(self._fused_last[1])
        self._fused_last = (raw, stream)

    @staticmethod
    def _fused_new(like: torch.Tensor, shape: tuple, index: int, stream) -> torch.Tensor:
        """A new tensor of an (already checked) input's type and device, made on the call's
        stream."""
        if stream is None:
            return like.new_empty(shape)
        with torch.cuda.stream(_as_stream(stream, index)):
            return like.new_empty(shape)

    def _fused_elsewhere(self, method, *args, **kw):
        """method(*args, **kw) with the layer's device current, if another one is now."""
        with torch.cuda.device(self._fused[3]):
            return method(*args, **kw)

    def fused_read_error(self, workspace=None, stream=None) -> int:
        """Sticky error flags of the calls that used the workspace (then cleared), or without
        one any of the layer's own, outgrown buffers included; 0 = every device wait completed.
        The device is synchronized first, whichever streams the calls ran on; `stream` carries
        the reading.  After a flag the workspace is zero-filled again: a call that gave up
        leaves arrivals in its counters."""
        with self._fused_lock:
            buffers = self._fused_ws if workspace is None else (workspace,)
            flags = 0
            for ws in buffers:
                with torch.cuda.device(ws.device):
                    torch.cuda.synchronize()
                    found = qlinear_read_error(ws, stream)
                    if found:
                        ws.zero_()
                        torch.cuda.synchronize()
                    flags |= found
            return flags


class QuantLinear(_FusedWorkspace):
    """One quantized weight matrix [K, N] resident on a CUDA device."""

    def __init__(self, fmt: int, K: int, N: int, canonical_codes: np.ndarray,
                 p0: np.ndarray, p1: Optional[np.ndarray] = None,
                 tilecoo: Optional[tuple] = None, device="cuda", max_m: int = 16,
                 group: int = 128):
        self.fmt, self.K, self.N, self.group = fmt, K, N, group
        self.device = torch.device(device)
        self._fused_lock = threading.RLock()
        packed = qlinear_pack(fmt, canonical_codes, N, K)
        self.qweight = _dev(packed, self.device)
        if fmt == QL_FMT_LUT4:
            self.p0 = _dev(_lut16(p0).view(np.uint16), self.device)
            self.p1 = _dev(qlinear_pack_params(fmt, np.asarray(p1, dtype=np.float32), N, K),
                           self.device)  # absmax
        elif group != 128:
            self.p0 = _dev(qlinear_pack_params_grouped(fmt, group, p0, N, K).view(np.uint16),
                           self.device)  # scales, one per (sub-group, column)
            self.p1 = _dev(qlinear_pack_params_grouped(fmt, group, p1, N, K).view(np.uint16),
                           self.device)  # zeros
        else:
            self.p0 = _dev(qlinear_pack_params(fmt, np.asarray(p0, dtype=np.float16), N, K)
                           .view(np.uint16), self.device)  # scales
            self.p1 = _dev(qlinear_pack_params(fmt, np.asarray(p1, dtype=np.float16), N, K)
                           .view(np.uint16), self.device)  # zeros
        self.tile = None
        if tilecoo is not None:
            off, rc, vals = qlinear_pack_tilecoo(*tilecoo, N, K)
            self.tile = (_dev(off, self.device), _dev(rc, self.device),
                         _dev(vals.view(np.uint16), self.device))
        ws = max(qlinear_workspace_bytes(fmt, m, N, K) for m in (1, max_m))
        self.workspace = torch.zeros(max(ws, 256) // 4 + 64, dtype=torch.int32, device=self.device)

    @property
    def weight_bytes(self) -> int:
        b = self.qweight.numel() + self.p0.numel() * self.p0.element_size() + \
            self.p1.numel() * self.p1.element_size()
        if self.tile is not None:
            b += sum(t.numel() * t.element_size() for t in self.tile)
        return b

    def forward(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """y[M, N] (fp16) = x[M, K] (fp16) . W."""
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float16, device=self.device)
        xv = x.view(torch.int16)
        yv = y.view(torch.int16)
        if self.tile is not None:
            qlinear_w4a16_outlier(xv, self.qweight, self.p0, self.p1, *self.tile, yv, M, self.N,
                                  self.K, self.workspace, stream)
        elif self.fmt == QL_FMT_LUT4:
            qlinear_lut4(xv, self.qweight, self.p0, self.p1, yv, M, self.N, self.K,
                         self.workspace, stream)
        else:
            _ENTRY[self.fmt](xv, self.qweight, self.p0, self.p1, yv, M, self.N, self.K,
                             self.workspace, stream, group=self.group)
        return y

    def read_error(self, stream=None) -> int:
        """Sticky error flags of the calls that used this layer's workspace (then cleared);
        0 = every device wait completed."""
        return qlinear_read_error(self.workspace, stream)

    def _group128(self, what: str) -> None:
        if self.group != 128:
            raise ValueError(f"{what} reads parameters packed for group 128")

    def dequant_fp16(self, w: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The dense fp16 weights, ``w[N, K]`` (one row per output column)."""
        self._group128("dequant_fp16")
        if w is None:
            w = torch.empty((self.N, self.K), dtype=torch.float16, device=self.device)
        qlinear_dequant_fp16(self.fmt, self.qweight, self.p0, self.p1, w.view(torch.int16),
                             self.N, self.K, stream)
        return w

    def prefill(self, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                w_fp16: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """y[M, N] = x[M, K] . W for any M: dequantize into ``w_fp16`` ([N, K] fp16, kept
        by the layer when not given), then one dense GEMM.  Dense part only (no outliers)."""
        if self.tile is not None:
            raise ValueError("prefill covers the dense formats; the outlier layer has none")
        self._group128("prefill")
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float16, device=self.device)
        if w_fp16 is None:
            if getattr(self, "_w_fp16", None) is None:
                self._w_fp16 = torch.empty((self.N, self.K), dtype=torch.float16,
                                           device=self.device)
            w_fp16 = self._w_fp16
        qlinear_prefill(self.fmt, x.view(torch.int16), self.qweight, self.p0, self.p1,
                        w_fp16.view(torch.int16), y.view(torch.int16), M, self.N, self.K, stream)
        return y

    def prefill_fused(self, x: torch.Tensor, y: Optional[torch.Tensor] = None,
                      stream=None, stream_k: bool = True) -> torch.Tensor:
        """y[M, N] = x[M, K] . W for any M, the weights dequantized inside the tensor-core
        GEMM (no fp16 weight matrix); stream_k shares the k-blocks out over the SMs through a
        workspace the layer keeps.  Dense part only (no outliers)."""
        if self.tile is not None:
            raise ValueError("prefill covers the dense formats; the outlier layer has none")
        self._group128("prefill")
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float16, device=self.device)
        ws = self._prefill_workspace(M) if stream_k else None
        qlinear_prefill_fused(self.fmt, x.view(torch.int16), self.qweight, self.p0, self.p1,
                              y.view(torch.int16), M, self.N, self.K, ws, stream)
        return y

    def _prefill_workspace(self, M: int) -> torch.Tensor:
        """The zero-filled stream-K workspace of the fused prefill, grown as M needs."""
        need = qlinear_prefill_workspace_bytes(M, self.N, self.K)
        ws = getattr(self, "_pf_ws", None)
        if ws is None or ws.numel() * 4 < need:
            ws = torch.zeros(need // 4 + 64, dtype=torch.int32, device=self.device)
            self._pf_ws = ws
        return ws

    def matmul(self, x: torch.Tensor, y: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
        """y[M, N] = x[M, K] . W for any M, dispatched by the library's policy map (the fused
        GEMV, over 16-row slices when M > 16, or the tensor-core prefill GEMM with the
        dequantization fused in)."""
        if self.tile is not None:
            raise ValueError("the policy map covers the dense formats")
        self._group128("matmul")
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float16, device=self.device)
        qlinear_matmul(self.fmt, x.view(torch.int16), self.qweight, self.p0, self.p1,
                       y.view(torch.int16), M, self.N, self.K, self.workspace, None, stream)
        return y

    def _fused_matrix(self) -> tuple:
        if self.tile is not None:
            raise ValueError("the fused layers cover the dense formats")
        self._group128("the fused layer")
        return self.fmt, self.N, self.K

    def linear(self, x: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, act: str = "none",
               y: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """y[M, N] = act(x[M, K] . W + bias[N]) + residual[M, N] in one kernel, for any M.  act:
        "none", "relu", "gelu", "gelu_tanh" or "silu".  z ([M, N] fp16), when given, receives
        x . W + bias for ``linear_backward``.  y may be the residual itself.  Autograd does not
        see the call: tensors that require a gradient are refused where it records."""
        fmt, N, K, index = self._fused or self._fused_setup()
        if torch.cuda.current_device() != index:
            return self._fused_elsewhere(self.linear, x, bias, residual, act, y, z, workspace,
                                         stream)
        M = x.shape[0]
        px = _fused_ptr(x, (M, K), index, "x")
        if y is None:
            y = self._fused_new(x, (M, N), index, stream)
        head = (fmt, px, *self._fused_weights(), _fused_ptr(bias, (N,), index, "bias"),
                _fused_ptr(residual, (M, N), index, "residual"), _act(act),
                _fused_ptr(y, (M, N), index, "y"), _fused_ptr(z, (M, N), index, "z"), M, N, K)
        if M:
            self._fused_call(_lib.qlinear_linear, "qlinear_linear", head, M, False, workspace,
                             stream)
        return y

    def linear_backward(self, dy: torch.Tensor, z: Optional[torch.Tensor] = None,
                        act: str = "none", dx: Optional[torch.Tensor] = None,
                        dbias: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The gradient of ``linear`` through the frozen weights: dx[M, K] = dz . W^T with
        dz = dy * act'(z), z as kept by ``linear`` (None with act "none").  dbias (fp32 [N]),
        when given, receives the column sums of dz.  The residual's gradient is dy."""
        fmt, N, K, index = self._fused or self._fused_setup()
        if torch.cuda.current_device() != index:
            return self._fused_elsewhere(self.linear_backward, dy, z, act, dx, dbias, workspace,
                                         stream)
        M = dy.shape[0]
        pdy = _fused_ptr(dy, (M, N), index, "dy")
        if dx is None:
            dx = self._fused_new(dy, (M, K), index, stream)
        head = (fmt, pdy, _fused_ptr(z, (M, N), index, "z"), *self._fused_weights(), _act(act),
                _fused_ptr(dx, (M, K), index, "dx"),
                _fused_ptr(dbias, (N,), index, "dbias", _F32), M, N, K)
        if M:
            self._fused_call(_lib.qlinear_linear_backward, "qlinear_linear_backward", head, M,
                             True, workspace, stream)
        elif dbias is not None:
            with torch.cuda.stream(_as_stream(stream, index)):
                dbias.zero_()
        return dx

    def debug_unpack(self, stream=None) -> torch.Tensor:
        codes = torch.empty((self.K, self.N), dtype=torch.uint8, device=self.device)
        qlinear_debug_unpack(self.fmt, self.qweight, codes, self.N, self.K, stream)
        return codes

    def debug_dequant(self, stream=None) -> torch.Tensor:
        self._group128("debug_dequant")
        w = torch.empty((self.K, self.N), dtype=torch.float32, device=self.device)
        qlinear_debug_dequant(self.fmt, self.qweight, self.p0, self.p1, w, self.N, self.K, stream)
        return w


class GatedLinear(_FusedWorkspace):
    """The gate and up projections of a gated feed-forward block as one packed matrix
    [K, 2 F] on the device: gate and up are (codes, p0, p1) of two [K, F] matrices in the
    canonical layouts (p0, p1: scales and zeros of group 128, or for LUT4 the table, which
    must be the same for both, and the absmax)."""

    def __init__(self, fmt: int, K: int, F: int, gate: tuple, up: tuple, device="cuda"):
        if fmt not in _FUSED_FORMATS:
            raise ValueError("the gated layer covers W2, W4, W8 (group 128) and LUT4")
        self.fmt, self.K, self.F, self.device = fmt, K, F, torch.device(device)
        self._fused_lock = threading.RLock()
        self.qweight = _dev(qlinear_pack_gated(fmt, gate[0], up[0], F, K), self.device)
        if fmt == QL_FMT_LUT4:
            tables = [_lut16(m[1]) for m in (gate, up)]
            if not np.array_equal(*tables):
                raise ValueError("gate and up share one LUT4 table")
            self.p0 = _dev(tables[0].view(np.uint16), self.device)
        else:
            self.p0 = _dev(qlinear_pack_params_gated(fmt, gate[1], up[1], F, K)
                           .view(np.uint16), self.device)
        p1 = qlinear_pack_params_gated(fmt, gate[2], up[2], F, K)
        self.p1 = _dev(p1 if fmt == QL_FMT_LUT4 else p1.view(np.uint16), self.device)

    def _fused_matrix(self) -> tuple:
        return self.fmt, 2 * self.F, self.K

    def forward(self, x: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "silu",
                h: Optional[torch.Tensor] = None, gu: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """h[M, F] = act(g) * u, g = x . Wg + bias[0], u = x . Wu + bias[1], in one kernel, for
        any M.  bias: [2, F] or None.  gu ([M, 2, F] fp16), when given, receives g and u for
        ``backward``."""
        fmt, _, K, index = self._fused or self._fused_setup()
        if torch.cuda.current_device() != index:
            return self._fused_elsewhere(self.forward, x, bias, act, h, gu, workspace, stream)
        M, F = x.shape[0], self.F
        px = _fused_ptr(x, (M, K), index, "x")
        if h is None:
            h = self._fused_new(x, (M, F), index, stream)
        head = (fmt, px, *self._fused_weights(), _fused_ptr(bias, (2, F), index, "bias"), _act(act),
                _fused_ptr(h, (M, F), index, "h"), _fused_ptr(gu, (M, 2, F), index, "gu"), M, F,
                K)
        if M:
            self._fused_call(_lib.qlinear_gated, "qlinear_gated", head, M, False, workspace,
                             stream)
        return h

    def backward(self, dh: torch.Tensor, gu: torch.Tensor, act: str = "silu",
                 dx: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """dx[M, K] of ``forward`` through the frozen weights, from dh and the kept gu; dbias
        (fp32 [2, F]), when given, receives the column sums of the gradients of g and u."""
        fmt, _, K, index = self._fused or self._fused_setup()
        if torch.cuda.current_device() != index:
            return self._fused_elsewhere(self.backward, dh, gu, act, dx, dbias, workspace,
                                         stream)
        M, F = dh.shape[0], self.F
        pdh = _fused_ptr(dh, (M, F), index, "dh")
        if dx is None:
            dx = self._fused_new(dh, (M, K), index, stream)
        head = (fmt, pdh, _fused_ptr(gu, (M, 2, F), index, "gu"), *self._fused_weights(), _act(act),
                _fused_ptr(dx, (M, K), index, "dx"),
                _fused_ptr(dbias, (2, F), index, "dbias", _F32), M, F, K)
        if M:
            self._fused_call(_lib.qlinear_gated_backward, "qlinear_gated_backward", head, M,
                             True, workspace, stream)
        elif dbias is not None:
            with torch.cuda.stream(_as_stream(stream, index)):
                dbias.zero_()
        return dx


class GatedMLP:
    """A gated feed-forward block: y = (act(x Wg + bias[0]) * (x Wu + bias[1])) Wd + down_bias +
    residual, two kernels forward; backward through the frozen weights from the kept gate and up
    values.  Both products of a call may share one workspace (``new_workspace``), which graphs
    that are replayed at the same time need one each of."""

    def __init__(self, gate_up: GatedLinear, down: QuantLinear, act: str = "silu"):
        if gate_up.F != down.K or gate_up.K != down.N:
            raise ValueError("the down projection is [F, K] for a gate and up of [K, F]")
        self.gate_up, self.down, self.act = gate_up, down, act

    def reserve(self, rows: int, backward: bool = True) -> None:
        self.gate_up.reserve(rows, backward)
        self.down.reserve(rows, backward)

    def new_workspace(self, rows: int, backward: bool = True) -> torch.Tensor:
        """A zero-filled workspace for calls of up to `rows` rows."""
        return max((lay.new_workspace(rows, backward) for lay in (self.gate_up, self.down)),
                   key=lambda ws: ws.numel())

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                gu: Optional[torch.Tensor] = None, stream=None,
                bias: Optional[torch.Tensor] = None, down_bias: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """y[M, N] from x[M, K]; bias [2, F] and down_bias [N]; gu ([M, 2, F] fp16), when given,
        is kept for ``backward``.  y may be the residual itself."""
        h = self.gate_up.forward(x, bias=bias, act=self.act, gu=gu, workspace=workspace,
                                 stream=stream)
        return self.down.linear(h, bias=down_bias, residual=residual, y=y, workspace=workspace,
                                stream=stream)

    def backward(self, dy: torch.Tensor, gu: torch.Tensor, stream=None,
                 dx: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                 ddown_bias: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
        """dx from dy and the gu that ``forward`` kept (the residual's gradient is dy); dbias
        (fp32 [2, F]) and ddown_bias (fp32 [N]), when given, receive the biases' gradients."""
        dh = self.down.linear_backward(dy, dbias=ddown_bias, workspace=workspace, stream=stream)
        return self.gate_up.backward(dh, gu, act=self.act, dx=dx, dbias=dbias,
                                     workspace=workspace, stream=stream)


def from_uniform(layer, device="cuda", max_m: int = 16) -> QuantLinear:
    """From a ``synth.gen.UniformLayer``-like object (bits, K, N, qweight, scales, zeros and,
    optionally, group)."""
    return QuantLinear(layer.bits, layer.K, layer.N, layer.qweight, layer.scales, layer.zeros,
                       device=device, max_m=max_m, group=getattr(layer, "group", 128))


def from_lut4(layer, device="cuda", max_m: int = 16) -> QuantLinear:
    return QuantLinear(QL_FMT_LUT4, layer.K, layer.N, layer.qbytes, layer.lut, layer.absmax,
                       device=device, max_m=max_m)


def from_outlier(layer, device="cuda", max_m: int = 16) -> QuantLinear:
    d = layer.dense
    return QuantLinear(QL_FMT_W4, d.K, d.N, d.qweight, d.scales, d.zeros,
                       tilecoo=(layer.tile_offsets, layer.tile_rc, layer.tile_vals),
                       device=device, max_m=max_m)


class CodebookLinear:
    """A codebook-quantized weight matrix (m1v4g128: codes uint8 [K / 4][N], scales fp16
    [K / 128][N], codebook fp16 [256][4]) on the device, packed for both GEMV forms: the
    Psumbook form (``qlinear_codebook``, M <= 4, N % 32 == 0) and the tensor-core form
    (``qlinear_codebook_tc``, M <= 16, N % 16 == 0)."""

    def __init__(self, K: int, N: int, codes: np.ndarray, scales: np.ndarray,
                 codebook: np.ndarray, device="cuda", max_m: int = 16):
        self.K, self.N, self.device, self.max_m = K, N, torch.device(device), max_m
        scales16 = np.ascontiguousarray(scales).view(np.uint16)
        self.codebook = _dev(np.ascontiguousarray(codebook).view(np.int16), self.device)
        self.codes_tc = _dev(qlinear_pack_codebook_tc(codes, N, K), self.device)
        self.scales_tc = _dev(qlinear_pack_params(QL_FMT_W4, scales16, N, K).view(np.int16),
                              self.device)
        ws = max(qlinear_workspace_bytes(QL_FMT_CB, m, N, K) for m in (1, max_m))
        self.ws_tc = torch.zeros(max(ws, 256) // 4 + 64, dtype=torch.int32, device=self.device)
        self.psum_ok = N % 32 == 0
        if self.psum_ok:
            self.codes_ps = _dev(qlinear_pack_codebook(codes, N, K), self.device)
            self.scales_ps = _dev(qlinear_pack_codebook_scales(scales16, N, K).view(np.int16),
                                  self.device)
            ws = max(qlinear_codebook_workspace_bytes(m, N, K) for m in range(1, 5))
            self.ws_ps = torch.zeros(max(ws, 256) // 4 + 64, dtype=torch.int32,
                                     device=self.device)

    def forward(self, x: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None,
                form: str = "tc") -> torch.Tensor:
        """y[M, N] (fp16) = x[M, K] (fp16) . W; form "tc" (tensor cores) or "psumbook"."""
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, self.N), dtype=torch.float16, device=self.device)
        xv, yv = x.view(torch.int16), y.view(torch.int16)
        if form == "tc":
            qlinear_codebook_tc(xv, self.codes_tc, self.scales_tc, self.codebook, yv, M, self.N,
                                self.K, self.ws_tc, stream)
        elif form == "psumbook":
            if not self.psum_ok:
                raise ValueError("the Psumbook form needs N % 32 == 0")
            qlinear_codebook(xv, self.codes_ps, self.scales_ps, self.codebook, yv, M, self.N,
                             self.K, self.ws_ps, stream)
        else:
            raise ValueError(f"unknown form {form!r}")
        return y

    def read_error(self, stream=None) -> int:
        """Sticky error flags of the tensor-core form's device waits (then cleared)."""
        return qlinear_read_error(self.ws_tc, stream)


def from_codebook(layer, device="cuda", max_m: int = 16) -> CodebookLinear:
    """From a ``synth.gen.CodebookLayer``-like object (K, N, codes, scales, codebook)."""
    return CodebookLinear(layer.K, layer.N, layer.codes, layer.scales, layer.codebook,
                          device=device, max_m=max_m)


# ---------------------------------------------------------------------------
# 8-bit floating-point layers: e4m3 codes with an fp32 scale per 128, for both operands

_F8, _I32 = torch.float8_e4m3fn, torch.int32
_TYPE_OF = {torch.float16: 0, torch.bfloat16: 1}  # ql_type


_MAX_COLUMNS = 1 << 30
_MAX_EXPERTS = 1024


def _blocks(columns: int) -> int:
    return (columns + 127) // 128


def _check_size(rows: int, columns: int) -> None:
    """(The library counts in 32 bits and checks what it is given, which larger numbers are not.)"""
    if rows > _MAX_ROWS or columns > _MAX_COLUMNS:
        raise ValueError(f"{rows} rows of {columns} columns: up to 2^24 and 2^30 are supported")


def _matrix(t: torch.Tensor, name: str) -> tuple:
    """(ql_type, device index, rows, columns) of a 16-bit matrix."""
    kind = _TYPE_OF.get(t.dtype)
    index = t.get_device()
    if kind is None or t.dim() != 2 or index < 0:
        raise ValueError(f"{name} must be a float16 or bfloat16 matrix on a CUDA device, not "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    M, C = t.shape
    _check_size(M, C)
    return kind, index, M, C


def _row_ptr(x: torch.Tensor, index: int, name: str) -> tuple:
    """(data pointer, elements between rows) of a matrix whose rows are contiguous, once checked
    like ``_fused_ptr``'s."""
    M, K = x.shape
    dual = _levels._current_level >= 0 and _dual(x)
    if x.is_contiguous() and not x.requires_grad and not dual:
        return x.data_ptr(), K
    ld = x.stride(0) if M > 1 else K
    if (dual or x.requires_grad and torch.is_grad_enabled() or x.stride(1) != 1 and K > 1
            or ld < K):
        _fused_ptr(x, (M, K), index, name, x.dtype)  # says why not
    return x.data_ptr(), ld


def _raw_stream(stream, index: int):
    return _current_stream(index) if stream is None else getattr(stream, "cuda_stream", stream)


# an empty tensor for each type and device index, from which new ones are quickest made
_empties: dict = {dtype: {} for dtype in (_F8, _F32, *_TYPE_OF)}


def _new(dtype, index: int, stream, *shape) -> torch.Tensor:
    """A new tensor on the call's stream."""
    like = _empties[dtype].get(index)
    if like is None:
        like = _empties[dtype][index] = torch.empty(0, dtype=dtype, device=f"cuda:{index}")
    if stream is None:
        return like.new_empty(*shape)  # (quicker than with a tuple)
    with torch.cuda.stream(_as_stream(stream, index)):
        return like.new_empty(*shape)


def _codes_out(q, scales, M: int, C: int, index: int, stream) -> tuple:
    """Codes [M, C] and scales, made where they are not given, and their data pointers."""
    if q is None:
        q = _new(_F8, index, stream, M, C)
        pq = q.data_ptr()
    else:
        pq = _fused_ptr(q, (M, C), index, "q", _F8)
    if scales is None:
        scales = _new(_F32, index, stream, M, (C + 127) // 128)
        return q, scales, pq, scales.data_ptr()
    return q, scales, pq, _fused_ptr(scales, (M, (C + 127) // 128), index, "scales", _F32)


def _on_device(index: int, method, *args):
    """method(*args) with the device current, if another one is now."""
    with torch.cuda.device(index):
        return method(*args)


def fp8_quantize(x: torch.Tensor, q: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """(q, scales): e4m3 codes [M, K] of x[M, K] (fp16 or bf16, K a multiple of 16; its rows may lie
    apart, by a multiple of 8) and an fp32 scale for every 128 columns, [M, ceil(K / 128)]; x is
    about q * scale."""
    kind, index, M, K = _matrix(x, "x")
    if torch.cuda.current_device() != index:
        return _on_device(index, fp8_quantize, x, q, scales, stream)
    px, ldx = _row_ptr(x, index, "x")
    q, scales, pq, ps = _codes_out(q, scales, M, K, index, stream)
    if M:
        _check(_lib.qlinear_fp8_quantize(kind, px, ldx, pq, ps, M, K, _raw_stream(stream, index)),
               "qlinear_fp8_quantize")
    return q, scales


def fp8_gated(gu: torch.Tensor, act: str = "silu", q: Optional[torch.Tensor] = None,
              scales: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """(q, scales): codes [M, F] and scales of act(g) * u, where gu[M, 2 F] = (g, u) (fp16 or
    bf16) is the output of a product with the gate's and the up projection's rows."""
    kind, index, M, C = _matrix(gu, "gu")
    if torch.cuda.current_device() != index:
        return _on_device(index, fp8_gated, gu, act, q, scales, stream)
    if C % 2:
        raise ValueError("gu holds gate and up values, 2 F columns")
    pgu = _fused_ptr(gu, (M, C), index, "gu", gu.dtype)
    q, scales, pq, ps = _codes_out(q, scales, M, C // 2, index, stream)
    if M:
        _check(_lib.qlinear_fp8_gated(kind, _act(act), pgu, pq, ps, M, C // 2,
                                      _raw_stream(stream, index)), "qlinear_fp8_gated")
    return q, scales


def fp8_gated_backward(dh: torch.Tensor, gu: torch.Tensor, act: str = "silu",
                       q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                       stream=None) -> tuple:
    """(q, scales): codes [M, 2 F] and scales of the gradients of g and u, from dh[M, F] and the gu
    that ``fp8_gated`` read."""
    kind, index, M, C = _matrix(gu, "gu")
    if torch.cuda.current_device() != index:
        return _on_device(index, fp8_gated_backward, dh, gu, act, q, scales, stream)
    if C % 2:
        raise ValueError("gu holds gate and up values, 2 F columns")
    pgu = _fused_ptr(gu, (M, C), index, "gu", gu.dtype)
    pdh = _fused_ptr(dh, (M, C // 2), index, "dh", gu.dtype)
    q, scales, pq, ps = _codes_out(q, scales, M, C, index, stream)
    if M:
        _check(_lib.qlinear_fp8_gated_backward(kind, _act(act), pdh, pgu, pq, ps, M, C // 2,
                                               _raw_stream(stream, index)),
               "qlinear_fp8_gated_backward")
    return q, scales


def fp8_quantize_weights(w: torch.Tensor, stream=None) -> tuple:
    """(codes, scales) of w[N, K] or w[E, N, K] (fp16 or bf16, contiguous, N and K multiples of
    16): e4m3 codes of the same shape and an fp32 scale per 128 x 128 block, for ``Fp8Linear`` and
    ``Fp8Experts``."""
    kind, index = _TYPE_OF.get(w.dtype), w.get_device()
    if kind is None or w.dim() not in (2, 3) or index < 0:
        raise ValueError("w must be a float16 or bfloat16 [N, K] or [E, N, K] on a CUDA device")
    *lead, N, K = w.shape
    with torch.cuda.device(index):
        _fused_ptr(w, w.shape, index, "w", w.dtype)
        codes = _new(_F8, index, stream, *w.shape)
        scales = _new(_F32, index, stream, *lead, _blocks(N), _blocks(K))
        qlinear_fp8_quantize_weights(kind, w, codes, scales, lead[0] if lead else 1, N, K, stream)
    return codes, scales


class RMSNorm(_FusedWorkspace):
    """RMS norm with the residual's addition and e4m3 output: weight [K] (fp16 or bf16, the type of
    the stream) on a CUDA device.  The weight stays the caller's tensor, and a call uses the values
    that the stream's earlier work leaves in it."""

    def __init__(self, weight: torch.Tensor, eps: float = 1e-6):
        weight = weight.detach()
        if (weight.dtype not in _TYPE_OF or weight.dim() != 1 or not weight.is_cuda
                or not weight.is_contiguous()):
            raise ValueError("the weight is a contiguous float16 or bfloat16 vector on a CUDA "
                             "device")
        self.weight, self.eps, self.K = weight, eps, weight.shape[0]
        if self.K % 16 or not 16 <= self.K <= 32768:
            raise ValueError(f"a norm has a multiple of 16 columns up to 32768, not {self.K}")
        self._fused_lock = threading.RLock()
        self._fused = (None, self.K, self.K, weight.get_device())

    def _fused_bytes(self, rows: int, backward: bool) -> int:
        with torch.cuda.device(self._fused[3]):
            need = qlinear_rmsnorm_workspace_bytes(rows, self.K)
        if need == 0:
            raise ValueError(f"no RMS norm of {rows} rows, K={self.K}")
        return need

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                total: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                rstd: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                scales: Optional[torch.Tensor] = None, stream=None) -> tuple:
        """(q, scales): e4m3 codes [M, K] and fp32 scales [M, ceil(K / 128)] of the norm of
        t = x + residual (t = x without a residual).  total, y ([M, K], the type of x) and rstd
        (fp32 [M]), when given, receive t, the norm's values in 16 bits and 1 / sqrt(mean(t^2) +
        eps); ``backward`` needs total (or x) and rstd.  total may be x or the residual itself.
        The rows of x may lie apart.  Autograd does not see the call: tensors that require a
        gradient are refused where it records."""
        weight, (_, _, K, index) = self.weight, self._fused
        if torch.cuda.current_device() != index:
            return self._fused_elsewhere(self.forward, x, residual, total, y, rstd, q, scales,
                                         stream)
        dtype, M = weight.dtype, x.shape[0]
        shape = (M, K)
        _check_size(M, K)
        if x.dtype is not dtype or x.shape != shape or x.get_device() != index:
            _fused_ptr(x, shape, index, "x", dtype)  # says why not
        px, ldx = _row_ptr(x, index, "x")
        if residual is not None:
            residual = _fused_ptr(residual, shape, index, "residual", dtype)
        if total is not None:
            total = _fused_ptr(total, shape, index, "total", dtype)
        if y is not None:
            y = _fused_ptr(y, shape, index, "y", dtype)
        if rstd is not None:
            rstd = _fused_ptr(rstd, (M,), index, "rstd", _F32)
        q, scales, pq, ps = _codes_out(q, scales, M, K, index, stream)
        if M:
            status = _lib.qlinear_rmsnorm(
                _TYPE_OF[dtype], px, ldx, residual, weight.data_ptr(), self.eps, total, y, pq, ps,
                rstd, M, K, _raw_stream(stream, index))
            if status:
                _check(status, "qlinear_rmsnorm")
        return q, scales

    def backward(self, dy: torch.Tensor, total: torch.Tensor, rstd: torch.Tensor,
                 dtotal: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                 dweight: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None,
                 offsets: Optional[torch.Tensor] = None) -> torch.Tensor:
        """dx[M, K], the gradient of x and of the residual, from the gradient dy of the norm's
        values (the quantization has the identity's), the kept total and rstd, and dtotal, the
        gradient that comes to total from elsewhere (dx may be dtotal itself).  dweight (fp32
        [K]), when given, receives the weight's.  offsets: those of the ``Fp8Experts`` call that dy
        comes from, where they leave rows out.  These have no dy: they add nothing to dweight, and
        their dx is dtotal, or 0 without one."""
        weight, (_, _, K, index) = self.weight, self._fused
        if torch.cuda.current_device() != index:
            return self._fused_elsewhere(self.backward, dy, total, rstd, dtotal, dx, dweight,
                                         workspace, stream, offsets)
        dtype, M = weight.dtype, dy.shape[0]
        _check_size(M, K)
        pdy = _fused_ptr(dy, (M, K), index, "dy", dtype)
        if dx is None:
            dx = self._fused_new(dy, (M, K), index, stream)
        pdw = _fused_ptr(dweight, (K,), index, "dweight", _F32)
        head = (_TYPE_OF[dtype], pdy, _fused_ptr(total, (M, K), index, "total", dtype),
                _fused_ptr(rstd, (M,), index, "rstd", _F32), weight.data_ptr(),
                _fused_ptr(dtotal, (M, K), index, "dtotal", dtype))
        pdx = _fused_ptr(dx, (M, K), index, "dx", dtype)
        if offsets is None:
            entry, name = _lib.qlinear_rmsnorm_backward, "qlinear_rmsnorm_backward"
            head = (*head, pdx, pdw, M, K)
        else:
            E = offsets.numel() - 1
            if not 1 <= E <= _MAX_EXPERTS:
                raise ValueError(f"offsets are those of 1 to {_MAX_EXPERTS} experts, not {E}")
            entry = _lib.qlinear_rmsnorm_backward_grouped
            name = "qlinear_rmsnorm_backward_grouped"
            head = (*head, _fused_ptr(offsets, (E + 1,), index, "offsets", _I32), pdx, pdw, M, E, K)
        if M and dweight is None:
            _check(entry(*head, None, 0, _raw_stream(stream, index)), name)
        elif M:
            self._fused_call(entry, name, head, M, True, workspace, stream)
        elif dweight is not None:
            with torch.cuda.stream(_as_stream(stream, index)):
                dweight.zero_()
        return dx


class _Fp8Weights(_FusedWorkspace):
    """e4m3 codes [..., N, K] and scales [..., ceil(N / 128), ceil(K / 128)] on a CUDA device; a
    workspace as in the fused layers, which any of these layers' calls that follow one another may
    share.  The constructor waits for the current stream (so that it cannot be part of a graph): the
    products read codes and scales before the work ahead of them on the stream has ended.  Whoever
    writes them later waits for that before the next call."""

    def _fp8_setup(self, codes, scales, dims: int, device) -> None:
        codes = torch.as_tensor(codes).detach()
        scales = torch.as_tensor(scales).detach()
        if codes.dtype is torch.uint8:
            codes = codes.view(_F8)
        if device is None:
            device = codes.device if codes.is_cuda else "cuda"
        if codes.dtype is not _F8 or codes.dim() != dims or scales.dtype is not _F32:
            raise ValueError(f"the weights are {dims}-dimensional e4m3 codes (float8_e4m3fn, or "
                             f"their bytes) and fp32 scales, not {codes.dtype} "
                             f"{tuple(codes.shape)} and {scales.dtype}")
        *lead, N, K = codes.shape
        if N % 16 or K % 16 or not (16 <= N <= _MAX_COLUMNS and 16 <= K <= _MAX_COLUMNS) or (
                lead and not 1 <= lead[0] <= _MAX_EXPERTS):
            raise ValueError(f"codes {tuple(codes.shape)}: N and K are multiples of 16 up to 2^30, "
                             "with 1 to 1024 experts")
        if tuple(scales.shape) != (*lead, _blocks(N), _blocks(K)):
            raise ValueError(f"codes {tuple(codes.shape)} have a scale per 128 x 128 block: "
                             f"{(*lead, _blocks(N), _blocks(K))}, not {tuple(scales.shape)}")
        self.codes = codes.to(device).contiguous()
        self.scales = scales.to(device).contiguous()
        self.device, self.N, self.K = self.codes.device, N, K
        self.E = lead[0] if lead else 1
        if self.device.type == "cuda":
            # the products read weights before the kernels ahead of them have ended
            torch.cuda.current_stream(self.device).synchronize()
        self._fused_lock = threading.RLock()
        self._fused = (None, N, K, self.codes.get_device())

    @property
    def weight_bytes(self) -> int:
        return self.codes.numel() + 4 * self.scales.numel()

    def _fused_bytes(self, rows: int, backward: bool) -> int:
        _, N, K, index = self._fused
        with torch.cuda.device(index):
            need = qlinear_fp8_workspace_bytes(rows, self.E, N, K)
        if need == 0:
            raise ValueError(f"no e4m3 product for {rows} rows, E={self.E}, N={N}, K={K}")
        return need

    def _product(self, entry, name, what, q, scales, offsets, out, C, R, dtype, backward,
                 workspace, stream):
        index = self._fused[3]
        M = q.shape[0]
        _check_size(M, C)
        pq = _fused_ptr(q, (M, C), index, "q", _F8)
        if out is not None:
            dtype = out.dtype
        kind = _TYPE_OF.get(dtype)
        if kind is None:
            raise ValueError(f"{what} is a float16 or bfloat16 tensor, not {dtype}")
        if out is None:
            out = _new(dtype, index, stream, M, R)
            pout = out.data_ptr()
        else:
            pout = _fused_ptr(out, (M, R), index, what, dtype)
        ps = _fused_ptr(scales, (M, (C + 127) // 128), index, "scales", _F32)
        if offsets:
            head = (kind, pq, ps, *offsets, self.codes.data_ptr(), self.scales.data_ptr(), pout, M,
                    self.E, self.N, self.K)
        else:
            head = (kind, pq, ps, self.codes.data_ptr(), self.scales.data_ptr(), pout, M, self.N,
                    self.K)
        if M:
            self._fused_call(entry, name, head, M, backward, workspace, stream)
        return out


class Fp8Linear(_Fp8Weights):
    """One weight matrix in e4m3: codes [N, K] (float8_e4m3fn or uint8, a tensor or an array; N and
    K multiples of 16) and an fp32 scale per 128 x 128 block, [ceil(N / 128), ceil(K / 128)]
    (``fp8_quantize_weights`` makes both)."""

    def __init__(self, codes, scales, device=None):
        self._fp8_setup(codes, scales, 2, device)

    def forward(self, q: torch.Tensor, scales: torch.Tensor, y: Optional[torch.Tensor] = None,
                dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """y[M, N] (dtype: float16 or bfloat16, or that of y when given) = x . W^T for any M, from
        the codes q[M, K] and scales of x (``RMSNorm.forward``, ``fp8_gated``,
        ``fp8_quantize``)."""
        if torch.cuda.current_device() != self._fused[3]:
            return self._fused_elsewhere(self.forward, q, scales, y, dtype, workspace, stream)
        return self._product(_lib.qlinear_fp8_linear, "qlinear_fp8_linear", "y", q, scales, (), y,
                             self.K, self.N, dtype, False, workspace, stream)

    def backward(self, q: torch.Tensor, scales: torch.Tensor, dx: Optional[torch.Tensor] = None,
                 dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        """dx[M, K] = dy . W through the frozen weights, from the codes q[M, N] and scales of dy
        (``fp8_quantize``, ``fp8_gated_backward``)."""
        if torch.cuda.current_device() != self._fused[3]:
            return self._fused_elsewhere(self.backward, q, scales, dx, dtype, workspace, stream)
        return self._product(_lib.qlinear_fp8_linear_backward, "qlinear_fp8_linear_backward", "dx",
                             q, scales, (), dx, self.N, self.K, dtype, True, workspace, stream)


class Fp8Experts(_Fp8Weights):
    """One weight matrix per expert in e4m3: codes [E, N, K] and scales [E, ceil(N / 128),
    ceil(K / 128)] as in ``Fp8Linear``, up to 1024 experts.  The rows of a call are in the order of
    the experts: rows offsets[e] .. offsets[e + 1] - 1 are expert e's, any number of them, none
    included.  offsets (int32 [E + 1], on the device) is read by the kernel alone.  Rows before the
    first and behind the last offset are neither read nor written.  The tiles' width goes by the
    call's rows over all E experts: many rows on few of many experts cost more than they need to."""

    def __init__(self, codes, scales, device=None):
        self._fp8_setup(codes, scales, 3, device)

    def _offsets(self, offsets: torch.Tensor) -> tuple:
        return (_fused_ptr(offsets, (self.E + 1,), self._fused[3], "offsets", _I32),)

    def forward(self, q: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                y: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """y[T, N]: each row of x (codes q[T, K], scales) by its expert's W^T."""
        if torch.cuda.current_device() != self._fused[3]:
            return self._fused_elsewhere(self.forward, q, scales, offsets, y, dtype, workspace,
                                         stream)
        return self._product(_lib.qlinear_fp8_grouped, "qlinear_fp8_grouped", "y", q, scales,
                             self._offsets(offsets), y, self.K, self.N, dtype, False, workspace,
                             stream)

    def backward(self, q: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                 dx: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """dx[T, K]: each row of dy (codes q[T, N], scales) by its expert's W."""
        if torch.cuda.current_device() != self._fused[3]:
            return self._fused_elsewhere(self.backward, q, scales, offsets, dx, dtype, workspace,
                                         stream)
        return self._product(_lib.qlinear_fp8_grouped_backward, "qlinear_fp8_grouped_backward",
                             "dx", q, scales, self._offsets(offsets), dx, self.N, self.K, dtype,
                             True, workspace, stream)


class Fp8GatedMLP:
    """A gated feed-forward block whose products have both operands in e4m3: y = (act(g) * u) Wd^T,
    (g, u) = v Wgu^T, where v is the RMS norm of x + residual (with a norm) or x itself.  gate_up
    holds the gate's rows before the up projection's.  Both may be ``Fp8Linear``, or both
    ``Fp8Experts``, whose calls take offsets and rows in the order of the experts.  backward goes
    through the frozen weights from what forward was given to keep.

    Rows of no expert (before the first and behind the last offset): forward writes total and rstd
    for them, but neither gu nor y.  What those and dy hold there goes into nothing.  In backward
    they add nothing to dweight; their dx is dtotal, or 0 without one, and without a norm it is not
    written."""

    def __init__(self, gate_up, down, norm: Optional[RMSNorm] = None, act: str = "silu"):
        if type(gate_up) is not type(down) or gate_up.E != down.E:
            raise ValueError("gate_up and down are both Fp8Linear or both Fp8Experts")
        if gate_up.N != 2 * down.K or (norm is not None and norm.K != gate_up.K):
            raise ValueError("gate_up is [2 F, K], down [N, F] and the norm [K]")
        self.gate_up, self.down, self.norm, self.act = gate_up, down, norm, act
        self._grouped = isinstance(gate_up, Fp8Experts)

    def reserve(self, rows: int, backward: bool = True) -> None:
        for layer in (self.gate_up, self.down, self.norm):
            if layer is not None:
                layer.reserve(rows, backward)

    def new_workspace(self, rows: int, backward: bool = True) -> torch.Tensor:
        """A zero-filled workspace for calls of up to `rows` rows."""
        layers = [self.gate_up, self.down] + ([self.norm] if self.norm is not None else [])
        return max((lay.new_workspace(rows, backward) for lay in layers),
                   key=lambda ws: ws.numel())

    def _rows(self, offsets) -> tuple:
        if (offsets is not None) != self._grouped:
            raise ValueError("offsets go with Fp8Experts")
        return (offsets,) if self._grouped else ()

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                offsets: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
                rstd: Optional[torch.Tensor] = None, gu: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """y[M, N] from x[M, K].  total and rstd (see ``RMSNorm.forward``) and gu ([M, 2 F]), when
        given, are kept for ``backward``; y's residual is total."""
        rows = self._rows(offsets)
        if self.norm is not None:
            q, scales = self.norm.forward(x, residual, total=total, rstd=rstd, stream=stream)
        elif residual is not None or total is not None or rstd is not None:
            raise ValueError("residual, total and rstd go with a norm")
        else:
            q, scales = fp8_quantize(x, stream=stream)
        gu = self.gate_up.forward(q, scales, *rows, y=gu, dtype=x.dtype, workspace=workspace,
                                  stream=stream)
        q, scales = fp8_gated(gu, self.act, stream=stream)
        return self.down.forward(q, scales, *rows, y=y, dtype=x.dtype, workspace=workspace,
                                 stream=stream)

    def backward(self, dy: torch.Tensor, gu: torch.Tensor, total: Optional[torch.Tensor] = None,
                 rstd: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                 dtotal: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                 dweight: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """dx from dy and what ``forward`` kept; with a norm, from total (or x) and rstd too, dtotal
        being the gradient that total gets from elsewhere and dweight (fp32 [K]), when given, the
        norm weight's."""
        rows = self._rows(offsets)
        if self.norm is None and not (total is rstd is dtotal is dweight is None):
            raise ValueError("total, rstd, dtotal and dweight go with a norm")
        q, scales = fp8_quantize(dy, stream=stream)
        dh = self.down.backward(q, scales, *rows, dtype=dy.dtype, workspace=workspace,
                                stream=stream)
        q, scales = fp8_gated_backward(dh, gu, self.act, stream=stream)
        if self.norm is None:
            return self.gate_up.backward(q, scales, *rows, dx=dx, dtype=dy.dtype,
                                         workspace=workspace, stream=stream)
        dv = self.gate_up.backward(q, scales, *rows, dtype=dy.dtype, workspace=workspace,
                                   stream=stream)
        return self.norm.backward(dv, total, rstd, dtotal=dtotal, dx=dx, dweight=dweight,
                                  workspace=workspace, stream=stream, offsets=offsets)
