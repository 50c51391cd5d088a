"""Device-resident quantized linear layers.

A layer takes the canonical arrays of one weight matrix (NumPy, host), packs them
with the library's host packer, uploads the packed arrays once, and owns a
zero-filled workspace.  ``forward`` enqueues the entry point on a stream.  The
class only moves and marshals data; every operation runs in ``libqlinear.so``.
"""
from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import (QL_FMT_CB, QL_FMT_LUT4, QL_FMT_W2, QL_FMT_W3, QL_FMT_W4, QL_FMT_W8,
               qlinear_codebook, qlinear_codebook_tc, qlinear_codebook_workspace_bytes,
               qlinear_debug_dequant, qlinear_pack_codebook, qlinear_pack_codebook_scales,
               qlinear_pack_codebook_tc,
               qlinear_debug_unpack, qlinear_dequant_fp16, qlinear_lut4, qlinear_pack,
               qlinear_matmul, qlinear_pack_params, qlinear_pack_params_grouped,
               qlinear_prefill, qlinear_prefill_fused, qlinear_prefill_workspace_bytes,
               qlinear_fused_workspace_bytes, qlinear_gated, qlinear_gated_backward,
               qlinear_linear, qlinear_linear_backward, qlinear_pack_gated,
               qlinear_pack_params_gated,
               qlinear_read_error,
               qlinear_pack_tilecoo, qlinear_w2a16, qlinear_w3a16, qlinear_w4a16,
               qlinear_w4a16_outlier,
               qlinear_w8a16, qlinear_workspace_bytes)

_ENTRY = {QL_FMT_W2: qlinear_w2a16, QL_FMT_W3: qlinear_w3a16, QL_FMT_W4: qlinear_w4a16,
          QL_FMT_W8: qlinear_w8a16}


def _dev(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


def _as_stream(stream, device) -> torch.cuda.Stream:
    """A torch stream, a raw cudaStream_t or None (the current one) as a torch stream."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return (torch.cuda.ExternalStream(stream, device=device) if stream
            else torch.cuda.default_stream(device))


_FUSED_FORMATS = (QL_FMT_W2, QL_FMT_W4, QL_FMT_W8, QL_FMT_LUT4)


class _FusedWorkspace:
    """What the fused entries (bias / activation / residual, gated, backward) of a layer share:
    argument checks and the workspace.

    The workspace is one zero-filled buffer, grown by ``reserve`` as more rows are asked for;
    buffers that were outgrown stay alive with the layer, since a captured graph may still use
    them.  Calls of one layer run one after the other: an eager call on another stream than
    the last waits for that stream's work.  Work that overlaps in time - graphs captured from
    one layer and replayed at the same time - needs a workspace of its own:
    ``workspace=layer.new_workspace(rows)``.  Tensors a call makes are made on its stream.
    """

    _fused_shape: tuple  # (fmt, N, K) of the packed matrix

    def _fused_bytes(self, rows: int, backward: bool) -> int:
        fmt, N, K = self._fused_shape
        if fmt not in _FUSED_FORMATS:
            raise ValueError("the fused layers cover W2, W4, W8 (group 128) and LUT4")
        need = qlinear_fused_workspace_bytes(fmt, rows, N, K, backward)
        if need == 0:
            raise ValueError(f"no fused product for {rows} rows, N={N}, K={K}")
        return need

    def new_workspace(self, rows: int, backward: bool = True) -> torch.Tensor:
        """A zero-filled workspace for calls of up to `rows` rows."""
        device = self.qweight.device
        with torch.cuda.device(device):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("reserve(rows) the workspace before capturing a graph")
            ws = torch.zeros(self._fused_bytes(rows, backward), dtype=torch.uint8, device=device)
            torch.cuda.synchronize()  # the zero fill has landed, whichever stream uses it
        return ws

    def reserve(self, rows: int, backward: bool = True) -> None:
        """Make the layer's own workspace large enough for calls of up to `rows` rows (a call
        that needs more does this itself, except while a graph is being captured)."""
        held = self.__dict__.setdefault("_fused_ws", [])
        with torch.cuda.device(self.qweight.device):
            need = self._fused_bytes(rows, backward)
        if not held or held[-1].numel() < need:
            held.append(self.new_workspace(rows, backward))

    def _fused_call(self, fn, rows: int, backward: bool, workspace, stream):
        """fn(workspace, stream) with the layer's device current."""
        device = self.qweight.device
        with torch.cuda.device(device):
            stream = _as_stream(stream, device)
            if workspace is None:
                self.reserve(rows, backward)
                workspace = self._fused_ws[-1]
                with torch.cuda.stream(stream):
                    capturing = torch.cuda.is_current_stream_capturing()
                if not capturing:
                    last = self.__dict__.get("_fused_stream")
                    if last is not None and last.cuda_stream != stream.cuda_stream:
                        stream.wait_stream(last)
                    self._fused_stream = stream
            elif workspace.device != device or not workspace.is_contiguous():
                raise ValueError(f"the workspace must be a contiguous tensor on {device}")
            fn(workspace, stream)

    def _fused_tensor(self, t, shape, name, dtype=torch.float16, make=False, stream=None):
        """`t` checked (or, with make, a new tensor when None)."""
        device = self.qweight.device
        if t is None:
            if not make:
                return None
            with torch.cuda.device(device), torch.cuda.stream(_as_stream(stream, device)):
                return torch.empty(shape, dtype=dtype, device=device)
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the layer on {device}")
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape "
                             f"{tuple(shape)}, not {t.dtype} {tuple(t.shape)} with strides "
                             f"{t.stride()}")
        return t

    def fused_read_error(self, workspace=None, stream=None) -> int:
        """Sticky error flags of the calls that used the workspace (then cleared); 0 = every
        device wait completed."""
        if workspace is None:
            if not self.__dict__.get("_fused_ws"):
                return 0
            workspace = self._fused_ws[-1]
        with torch.cuda.device(self.qweight.device):
            return qlinear_read_error(workspace, stream)


class QuantLinear(_FusedWorkspace):
    """One quantized weight matrix [K, N] resident on a CUDA device."""

    def __init__(self, fmt: int, K: int, N: int, canonical_codes: np.ndarray,
                 p0: np.ndarray, p1: Optional[np.ndarray] = None,
                 tilecoo: Optional[tuple] = None, device="cuda", max_m: int = 16,
                 group: int = 128):
        self.fmt, self.K, self.N, self.group = fmt, K, N, group
        self.device = torch.device(device)
        packed = qlinear_pack(fmt, canonical_codes, N, K)
        self.qweight = _dev(packed, self.device)
        if fmt == QL_FMT_LUT4:
            self.p0 = _dev(np.asarray(p0, dtype=np.float16).view(np.uint16), self.device)  # lut16
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

    @property
    def _fused_shape(self) -> tuple:
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
        x . W + bias for ``linear_backward``.  y may be the residual itself."""
        fmt, N, K = self._fused_shape
        M = x.shape[0]
        self._fused_tensor(x, (M, K), "x")
        self._fused_tensor(bias, (N,), "bias")
        self._fused_tensor(residual, (M, N), "residual")
        self._fused_tensor(z, (M, N), "z")
        y = self._fused_tensor(y, (M, N), "y", make=True, stream=stream)
        if M:
            self._fused_call(lambda ws, st: qlinear_linear(
                fmt, x, self.qweight, self.p0, self.p1, y, M, N, K, ws, bias, residual, act, z,
                st), M, False, workspace, stream)
        return y

    def linear_backward(self, dy: torch.Tensor, z: Optional[torch.Tensor] = None,
                        act: str = "none", dx: Optional[torch.Tensor] = None,
                        dbias: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The gradient of ``linear`` through the frozen weights: dx[M, K] = dz . W^T with
        dz = dy * act'(z), z as kept by ``linear`` (None with act "none").  dbias (fp32 [N]),
        when given, receives the column sums of dz.  The residual's gradient is dy."""
        fmt, N, K = self._fused_shape
        M = dy.shape[0]
        self._fused_tensor(dy, (M, N), "dy")
        self._fused_tensor(z, (M, N), "z")
        self._fused_tensor(dbias, (N,), "dbias", torch.float32)
        dx = self._fused_tensor(dx, (M, K), "dx", make=True, stream=stream)
        if M:
            self._fused_call(lambda ws, st: qlinear_linear_backward(
                fmt, dy, z, self.qweight, self.p0, self.p1, dx, M, N, K, ws, act, dbias, st),
                M, True, workspace, stream)
        elif dbias is not None:
            with torch.cuda.stream(_as_stream(stream, dbias.device)):
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
        self.qweight = _dev(qlinear_pack_gated(fmt, gate[0], up[0], F, K), self.device)
        if fmt == QL_FMT_LUT4:
            tables = [np.asarray(m[1], dtype=np.float16) for m in (gate, up)]
            if not np.array_equal(*tables):
                raise ValueError("gate and up share one LUT4 table")
            self.p0 = _dev(tables[0].view(np.uint16), self.device)
        else:
            self.p0 = _dev(qlinear_pack_params_gated(fmt, gate[1], up[1], F, K)
                           .view(np.uint16), self.device)
        p1 = qlinear_pack_params_gated(fmt, gate[2], up[2], F, K)
        self.p1 = _dev(p1 if fmt == QL_FMT_LUT4 else p1.view(np.uint16), self.device)
        self._fused_shape = (fmt, 2 * F, K)

    def forward(self, x: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "silu",
                h: Optional[torch.Tensor] = None, gu: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """h[M, F] = act(g) * u, g = x . Wg + bias[0], u = x . Wu + bias[1], in one kernel, for
        any M.  bias: [2, F] or None.  gu ([M, 2, F] fp16), when given, receives g and u for
        ``backward``."""
        M = x.shape[0]
        self._fused_tensor(x, (M, self.K), "x")
        self._fused_tensor(bias, (2, self.F), "bias")
        self._fused_tensor(gu, (M, 2, self.F), "gu")
        h = self._fused_tensor(h, (M, self.F), "h", make=True, stream=stream)
        if M:
            self._fused_call(lambda ws, st: qlinear_gated(
                self.fmt, x, self.qweight, self.p0, self.p1, h, M, self.F, self.K, ws, bias,
                act, gu, st), M, False, workspace, stream)
        return h

    def backward(self, dh: torch.Tensor, gu: torch.Tensor, act: str = "silu",
                 dx: Optional[torch.Tensor] = None, dbias: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """dx[M, K] of ``forward`` through the frozen weights, from dh and the kept gu; dbias
        (fp32 [2, F]), when given, receives the column sums of the gradients of g and u."""
        M = dh.shape[0]
        self._fused_tensor(dh, (M, self.F), "dh")
        self._fused_tensor(gu, (M, 2, self.F), "gu")
        self._fused_tensor(dbias, (2, self.F), "dbias", torch.float32)
        dx = self._fused_tensor(dx, (M, self.K), "dx", make=True, stream=stream)
        if M:
            self._fused_call(lambda ws, st: qlinear_gated_backward(
                self.fmt, dh, gu, self.qweight, self.p0, self.p1, dx, M, self.F, self.K, ws,
                act, dbias, st), M, True, workspace, stream)
        elif dbias is not None:
            with torch.cuda.stream(_as_stream(stream, dbias.device)):
                dbias.zero_()
        return dx


class GatedMLP:
    """A gated feed-forward block: y = (act(x Wg) * (x Wu)) Wd + residual, two kernels forward;
    backward through the frozen weights from the kept gate and up values."""

    def __init__(self, gate_up: GatedLinear, down: QuantLinear, act: str = "silu"):
        if gate_up.F != down.K or gate_up.K != down.N:
            raise ValueError("the down projection is [F, K] for a gate and up of [K, F]")
        self.gate_up, self.down, self.act = gate_up, down, act

    def reserve(self, rows: int, backward: bool = True) -> None:
        self.gate_up.reserve(rows, backward)
        self.down.reserve(rows, backward)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                gu: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        h = self.gate_up.forward(x, act=self.act, gu=gu, stream=stream)
        return self.down.linear(h, residual=residual, stream=stream)

    def backward(self, dy: torch.Tensor, gu: torch.Tensor, stream=None) -> torch.Tensor:
        """dx from dy and the gu that ``forward`` kept (the residual's gradient is dy)."""
        dh = self.down.linear_backward(dy, stream=stream)
        return self.gate_up.backward(dh, gu, act=self.act, stream=stream)


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
