"""The experts' products between dispatch and combine (include/moe_experts.h).

``ExpertRows`` holds what the calls on one set of packed rows share (the
layout's offsets and a workspace) and has the products as methods;
``ExpertFFN`` is the two-layer expert network made of them, with its hidden
layer saved in 8 bits between the passes.  Every method checks its arguments
on the host, allocates the outputs it is not given (through PyTorch) and
enqueues the library's kernels on the handle's stream: the plan's for the rows
of a plan, else the current one.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import abi

ACTIVATIONS = {"none": abi.MOE_ACT_NONE, "silu": abi.MOE_ACT_SILU, "gelu": abi.MOE_ACT_GELU,
               "swiglu": abi.MOE_ACT_SWIGLU}
SAVED_BLOCK = 32  # columns that share one scale byte
_STATUS_BYTES = 8192
_INT_MAX = (1 << 31) - 1  # the library refuses what is too large for it; ctypes passes the low 32 bits of more


@dataclass
class SavedLayer:
    """A layer's activation inputs in 8 bits: e4m3 ``codes`` [rows, N] and
    one scale byte per 32 columns, ``scales`` [rows, N / 32]; a value is
    e4m3(code) * 2^(byte - 127).  Byte 255 marks a block that held a NaN or
    an infinity."""
    codes: torch.Tensor
    scales: torch.Tensor

    @staticmethod
    def empty(rows: int, N: int, device="cuda") -> "SavedLayer":
        if N % SAVED_BLOCK:
            raise ValueError(f"a saved layer's columns are a multiple of {SAVED_BLOCK}, got {N}")
        return SavedLayer(torch.empty((rows, N), dtype=torch.uint8, device=device),
                          torch.empty((rows, N // SAVED_BLOCK), dtype=torch.uint8, device=device))


def _act(name: str) -> int:
    try:
        return ACTIVATIONS[name]
    except KeyError:
        raise ValueError(f"act: one of {', '.join(ACTIVATIONS)}, got {name!r}") from None


def _columns(n: int, name: str) -> int:
    if n > _INT_MAX:
        raise ValueError(f"{name}: {n} columns are too many")
    return n


def _refuse(t, dtype, shape, name, device):
    """Say what is wrong with a tensor that _check turned down."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the rows are on {device}")
    raise ValueError(f"{name}: must be contiguous")


def _check(t, dtype, shape, name, device):
    """A contiguous tensor of exactly this type, shape and device; its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, shape, name, device)


def _check_rows(t, dtype, rows, cols, name, device):
    """A contiguous [at least `rows`, cols] tensor of this type and device; its address."""
    try:
        shape = t.shape
        if (t.dtype is dtype and len(shape) == 2 and shape[0] >= rows and shape[1] == cols and t.device == device
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and (t.dim() != 2 or t.shape[1] != cols or t.shape[0] < rows):
        raise ValueError(f"{name}: expected shape ({rows}, {cols}) or more rows, got {tuple(t.shape)}")
    _refuse(t, dtype, getattr(t, "shape", None), name, device)


def quantize_weights(w: torch.Tensor):
    """Weights [E, N, K] (or [N, K]) in e4m3 for products with e4m3 rows, once
    when a model is loaded: codes (uint8) and (scale, sum) [.., N, 2] fp32 with
    scale = max |w| / 448 of each output column (1 for a column of zeros) and
    sum the sum over k of scale * code."""
    codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    scales = torch.empty((*w.shape[:-1], 2), dtype=torch.float32, device=w.device)
    for c, s, v in zip(codes.view(-1, *w.shape[-2:]), scales.view(-1, w.shape[-2], 2), w.view(-1, *w.shape[-2:])):
        v = v.float()
        top = v.abs().amax(1)
        scale = torch.where(top > 0, top / 448.0, 1.0)
        q = (v / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        c.copy_(q.view(torch.uint8))
        s[:, 0] = scale
        s[:, 1] = (q.double().sum(1) * scale.double()).float()
    return codes, scales


class ExpertRows:
    """The packed rows of a layout: expert e has rows offsets[e] ..
    offsets[e+1]-1 of buffers that hold ``rows`` rows (or more: those past
    ``rows`` are left alone).

    ``offsets`` is the layout's device tensor (int32 [E+1]); None makes all
    rows one group, for the shared experts' plain products (weights then
    lack the expert axis: [N, K], bias [N]).  ``ws`` is a workspace whose
    status word takes device-detected problems; one is made if none is
    given.

    With a ``stream`` every call runs on it, whatever the current stream is,
    as a RoutePlan's calls do, and the outputs that the handle allocates
    belong to it: other streams that use them wait for it.  Without one a
    call runs on the stream that is current then.  The rows' device is the
    current one at every call."""

    def __init__(self, offsets: torch.Tensor | None = None, *, rows: int, device="cuda", ws=None, stream=None):
        if not 0 <= rows <= _INT_MAX:
            raise ValueError(f"rows: {rows}")
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.grouped = offsets is not None
        self.E = 1
        if offsets is not None:
            if offsets.dim() != 1 or not 2 <= offsets.numel() <= abi.MOE_MAX_EXPERTS + 1:
                raise ValueError(f"offsets: expected [E + 1] with E in 1..{abi.MOE_MAX_EXPERTS}, "
                                 f"got {tuple(offsets.shape)}")
            self.E = offsets.numel() - 1
            _check(offsets, torch.int32, offsets.shape, "offsets", self.device)
        self.rows, self.offsets = rows, offsets
        self.stream = stream
        if ws is None:
            with self._owner():
                ws = torch.zeros(_STATUS_BYTES, dtype=torch.uint8, device=self.device)
        elif ws.numel() * ws.element_size() < _STATUS_BYTES or ws.device != self.device:
            raise ValueError(f"ws: a workspace of at least {_STATUS_BYTES} bytes on {self.device}")
        self.ws = ws
        self._c = abi.moe_rows(rows, self.E, None if offsets is None else offsets.data_ptr(), ws.data_ptr())
        self._ref = ctypes.byref(self._c)
        self._lib = abi.lib()

    @staticmethod
    def of(plan) -> "ExpertRows":
        """The packed rows of a RoutePlan, on its stream, where its dispatch
        writes them and its combine reads what the experts make of them;
        problems are recorded in its workspace."""
        return ExpertRows(plan.layout.offsets, rows=plan.r_max, device=plan.layout.offsets.device, ws=plan.ws,
                          stream=plan.stream)

    def status(self) -> int:
        """Synchronise, return and clear the device status."""
        self._stream()  # the device is the current one
        return abi.moe_get_status(self.ws, self.stream)

    def cut(self, product: str, N: int, K: int, e4m3: bool = False):
        """(SMs of a tile, rows per tile, blocks that share its sums) of
        "linear", "dgrad" or "wgrad" with weights [N, K] on the current
        device, for tests and tuning."""
        c = (ctypes.c_int32 * 3)()
        abi._check(self._lib.moe_expert_cut(("linear", "dgrad", "wgrad").index(product), int(e4m3), self.rows, self.E,
                                            _columns(K, "w"), _columns(N, "w"), c), "moe_expert_cut")
        return tuple(c)

    def new_saved(self, N: int) -> SavedLayer:
        with self._owner():
            return SavedLayer.empty(self.rows, N, self.device)

    # ------------------------------------------------------------------
    def _stream(self):
        if self.device.type != "cuda":
            raise ValueError(f"the rows are on {self.device}: a CUDA device is needed")
        # a launch goes to the current device, whatever the stream handle was asked of
        if torch._C._cuda_getDevice() != self.device.index:
            raise ValueError(f"the rows are on {self.device}, the current device is "
                             f"cuda:{torch._C._cuda_getDevice()}: make theirs current (torch.cuda.device)")
        if self.stream is not None:
            return self.stream.cuda_stream
        # the current stream's handle, without the Stream object around it
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def _owner(self):
        """Where memory is allocated: on the handle's stream, which uses it."""
        if self.stream is None or torch._C._cuda_getCurrentRawStream(self.device.index) == self.stream.cuda_stream:
            return contextlib.nullcontext()
        return torch.cuda.stream(self.stream)

    def _new(self, shape, dtype=torch.bfloat16):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with self._owner():
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _weights(self, w, dtype):
        """(N, K, address) of weights [E, N, K], or [N, K] for one plain group."""
        shape = w.shape if isinstance(w, torch.Tensor) else ()
        if len(shape) != (3 if self.grouped else 2):
            raise ValueError("w: expected a tensor of " + ("[E, N, K]" if self.grouped else "[N, K]"))
        if self.grouped and shape[0] != self.E:
            raise ValueError(f"w: {shape[0]} experts, the rows have {self.E}")
        N, K = shape[-2:]
        if N > _INT_MAX or K > _INT_MAX:
            raise ValueError(f"w: {max(N, K)} columns are too many")
        return N, K, _check(w, dtype, shape, "w", self.device)

    def _per_expert(self, *shape):
        return (self.E, *shape) if self.grouped else shape

    def _opt(self, t, dtype, shape, name):
        return None if t is None else _check(t, dtype, shape, name, self.device)

    def _out(self, t, dtype, shape, name):
        if t is None:
            t = self._new(shape, dtype)
            return t, t.data_ptr()
        return t, _check(t, dtype, shape, name, self.device)

    def _out_rows(self, t, cols, name):
        if t is None:
            t = self._new((self.rows, cols))
            return t, t.data_ptr()
        return t, _check_rows(t, torch.bfloat16, self.rows, cols, name, self.device)

    def _saved(self, saved, N):
        return (_check_rows(saved.codes, torch.uint8, self.rows, N, "saved.codes", self.device),
                _check_rows(saved.scales, torch.uint8, self.rows, N // SAVED_BLOCK, "saved.scales", self.device))

    # ------------------------------------------------------------------
    def linear(self, x, w, *, bias=None, act: str = "none", residual=None, saved: SavedLayer | None = None,
               x_scales=None, w_scales=None, out=None):
        """act(x w^T + bias) + residual for each expert's rows -> [rows, N]
        ([rows, N / 2] for swiglu, whose columns are gates, then ups).

        x [rows, K] and w [E, N, K] are bf16, or e4m3 codes (uint8) with
        x_scales [rows, 2] (scale, zero) and w_scales [E, N, 2] (scale, sum).
        ``saved`` receives the activation's inputs in 8 bits."""
        a, dev, rows = _act(act), self.device, self.rows
        dtype = torch.bfloat16
        xs = ws = bp = rp = sc = ss = None
        if x_scales is not None or w_scales is not None:
            if x_scales is None or w_scales is None:
                raise ValueError("x_scales and w_scales go together")
            dtype = torch.uint8
        N, K, wp = self._weights(w, dtype)
        xp = _check_rows(x, dtype, rows, K, "x", dev)
        if x_scales is not None:
            xs = _check_rows(x_scales, torch.float32, rows, 2, "x_scales", dev)
            ws = _check(w_scales, torch.float32, self._per_expert(N, 2), "w_scales", dev)
        if bias is not None:
            bp = _check(bias, torch.bfloat16, self._per_expert(N), "bias", dev)
        cols = N // 2 if a == abi.MOE_ACT_SWIGLU else N
        if residual is not None:
            rp = _check_rows(residual, torch.bfloat16, rows, cols, "residual", dev)
        if saved is not None:
            sc, ss = self._saved(saved, N)
        if out is None:
            out = self._new((rows, cols))
            op = out.data_ptr()
        else:
            op = _check_rows(out, torch.bfloat16, rows, cols, "out", dev)
        st = self._lib.moe_expert_linear(self._ref, xp, xs, K, wp, ws, N, bp, a, rp, op, sc, ss, self._stream())
        if st:
            abi._check(st, "moe_expert_linear")
        return out

    def dgrad(self, dy, w, *, act: str = "none", saved: SavedLayer | None = None, out=None, a=None):
        """dy w -> [rows, K]; with ``act`` and the ``saved`` input of the
        activation that made this product's rows, the gradient with respect
        to that input ([rows, K], swiglu: [rows, 2K]).  ``a`` [rows, K], if
        given, receives act(saved)."""
        code = _act(act)
        N, K, wp = self._weights(w, torch.bfloat16)
        if (saved is None) != (code == abi.MOE_ACT_NONE):
            raise ValueError("act and saved go together")
        if a is not None and saved is None:
            raise ValueError("a: only with a saved layer")
        cols = 2 * K if code == abi.MOE_ACT_SWIGLU else K
        dp = _check_rows(dy, torch.bfloat16, self.rows, N, "dy", self.device)
        sc = ss = ap = None
        if saved is not None:
            sc, ss = self._saved(saved, cols)
            if a is not None:
                ap = _check_rows(a, torch.bfloat16, self.rows, K, "a", self.device)
        out, op = self._out_rows(out, cols, "out")
        st = self._lib.moe_expert_dgrad(self._ref, dp, N, wp, K, code, sc, ss, op, ap, self._stream())
        if st:
            abi._check(st, "moe_expert_dgrad")
        return out

    def wgrad(self, dy, x, *, bias: bool = False, dtype=torch.bfloat16, out=None, out_bias=None):
        """(dw [E, N, K], db [E, N] or None) = sums of dy^T x and of dy over
        each expert's rows; zeros for an expert without rows.  ``dtype`` is
        bf16 or fp32."""
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"dtype: bfloat16 or float32, got {dtype}")
        if dy.dim() != 2 or x.dim() != 2:
            raise ValueError("dy and x: expected [rows, columns]")
        N, K = _columns(dy.shape[1], "dy"), _columns(x.shape[1], "x")
        dp = _check_rows(dy, torch.bfloat16, self.rows, N, "dy", self.device)
        xp = _check_rows(x, torch.bfloat16, self.rows, K, "x", self.device)
        out, op = self._out(out, dtype, self._per_expert(N, K), "out")
        bp = None
        if bias or out_bias is not None:
            out_bias, bp = self._out(out_bias, dtype, self._per_expert(N), "out_bias")
        abi._check(self._lib.moe_expert_wgrad(self._ref, dp, N, xp, K, op, bp, int(dtype == torch.float32),
                                              self._stream()), "moe_expert_wgrad")
        return out, out_bias

    def act_backward(self, dy, *, act: str, saved: SavedLayer, out=None, a=None):
        """The gradient through an activation whose input was saved:
        dy * act'(saved) -> [rows, N].  ``a``, if given, receives act(saved)."""
        code = _act(act)
        if code == abi.MOE_ACT_NONE:
            raise ValueError("act: 'none' has no backward pass")
        N = _columns(saved.codes.shape[-1], "saved.codes")
        cols = N // 2 if code == abi.MOE_ACT_SWIGLU else N
        dp = _check_rows(dy, torch.bfloat16, self.rows, cols, "dy", self.device)
        sc, ss = self._saved(saved, N)
        ap = None if a is None else _check_rows(a, torch.bfloat16, self.rows, cols, "a", self.device)
        out, op = self._out_rows(out, N, "out")
        abi._check(self._lib.moe_act_backward(self._ref, dp, N, code, sc, ss, op, ap, self._stream()),
                   "moe_act_backward")
        return out

    def linear_backward(self, dy, x, w, *, act: str = "none", saved: SavedLayer | None = None, bias: bool = False,
                        dtype=torch.bfloat16):
        """(dx, dw, db) of ``linear``; with an activation, through the layer
        it saved.  The residual's gradient is dy."""
        if (saved is None) != (_act(act) == abi.MOE_ACT_NONE):
            raise ValueError("act and saved go together")
        du = dy if saved is None else self.act_backward(dy, act=act, saved=saved)
        dx = self.dgrad(du, w)
        dw, db = self.wgrad(du, x, bias=bias, dtype=dtype)
        return dx, dw, db


@dataclass
class FFNGrads:
    dx: torch.Tensor
    dw1: torch.Tensor
    dw2: torch.Tensor
    db1: torch.Tensor | None = None
    db2: torch.Tensor | None = None


class ExpertFFN:
    """The experts' network y = act(x w1^T + b1) w2^T + b2 over packed rows.

    Between the passes only the activation's input is kept, in 8 bits
    (1 + 1/32 bytes per value): the backward pass recomputes the activation
    from it, in the same kernel that takes the gradient through it.  w1 is
    [E, N, H], w2 [E, H, F] with N = F (2F for swiglu); without the expert
    axis for one plain group.

    Like a RoutePlan the network owns the buffers of its results: ``y`` and
    the gradients hold those of the last pass, and the next one overwrites
    them."""

    def __init__(self, rows: ExpertRows, w1, w2, *, b1=None, b2=None, act: str = "swiglu", dtype=torch.bfloat16):
        N, H, _ = rows._weights(w1, torch.bfloat16)
        H2, F, _ = rows._weights(w2, torch.bfloat16)
        if _act(act) == abi.MOE_ACT_NONE:
            raise ValueError("act: an expert network has an activation")
        if H2 != H or N != (2 * F if act == "swiglu" else F):
            raise ValueError(f"w1 {tuple(w1.shape)} and w2 {tuple(w2.shape)} do not fit together for act {act!r}")
        self.rows, self.w1, self.w2, self.b1, self.b2, self.act, self.dtype = rows, w1, w2, b1, b2, act, dtype
        self.saved = rows.new_saved(N)
        self.hidden = rows._new((rows.rows, F))   # act(u): forward, and again in the backward pass
        self.y = rows._new((rows.rows, H))
        self.grads = self._du = None

    def forward(self, x, *, residual=None, out=None):
        """x [rows, H] -> [rows, H] (+ residual), in ``y`` or ``out``."""
        r = self.rows
        r.linear(x, self.w1, bias=self.b1, act=self.act, saved=self.saved, out=self.hidden)
        return r.linear(self.hidden, self.w2, bias=self.b2, residual=residual, out=self.y if out is None else out)

    def backward(self, dy, x) -> FFNGrads:
        """Gradients of the last forward pass; x is its input."""
        r = self.rows
        if self.grads is None:
            self._du = r._new(self.saved.codes.shape)
            like = lambda w: None if w is None else r._new(w.shape, self.dtype)  # noqa: E731
            self.grads = FFNGrads(r._new(self.y.shape), like(self.w1), like(self.w2), like(self.b1), like(self.b2))
        g = self.grads
        du = r.dgrad(dy, self.w2, act=self.act, saved=self.saved, out=self._du, a=self.hidden)
        r.wgrad(dy, self.hidden, dtype=self.dtype, out=g.dw2, out_bias=g.db2)
        r.dgrad(du, self.w1, out=g.dx)
        r.wgrad(du, x, dtype=self.dtype, out=g.dw1, out_bias=g.db1)
        return g
