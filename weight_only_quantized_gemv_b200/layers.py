"""Device-resident quantized linear layers.

A layer takes the canonical arrays of one weight matrix (NumPy, host), packs them
with the library's host packer, uploads the packed arrays once, and owns a
zero-filled workspace.  ``forward`` enqueues the entry point on a stream.  The
class only moves and marshals data; every operation runs in ``libqlinear.so``.
"""
from __future__ import annotations

import threading
from typing import Optional

import numpy as np
import torch

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


def _as_stream(stream, index: int) -> torch.cuda.Stream:
    """A torch stream, a raw cudaStream_t or None (the current one) as a torch stream."""
    if stream is None:
        return torch.cuda.current_stream(index)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    device = torch.device("cuda", index)
    return (torch.cuda.ExternalStream(stream, device=device) if stream
            else torch.cuda.default_stream(device))


def _fused_ptr(t, shape: tuple, index: int, name: str, dtype=_F16) -> Optional[int]:
    """The data pointer of `t` once checked (None for None): `shape`, `dtype`, contiguous, on
    CUDA device `index`, and nothing that autograd would have to follow."""
    if t is None:
        return None
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which autograd does not carry through the "
                         "fused layers: call them under torch.no_grad() (as inside an "
                         "autograd.Function) and their backward methods for the gradient")
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
