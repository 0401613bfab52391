"""Fused operators on NVFP4 weights: the projection with bias, activation and
residual in its epilogue, the gated feed-forward block, the product through
the transposed weight, and their gradients (the weight is frozen: gradients go
to the activations, the biases and the residual).

    y = linear(w, X, bias=b, activation="gelu", residual=r)
    h = gated(GatedWeight.from_float(Wg, Wu), X, activation="silu")

Both are differentiable when given the weight's transposed copy
(``transposed=w.transpose()``, made once); ``linear_backward`` and
``gated_backward`` are the same gradients without autograd, for programs that
run their own backward pass and for captured graphs (torch ends the process
where an autograd pass is captured while an eager graph of the same leaves is
alive; these functions have no such graph, and with ``gemm_t`` they refuse
tensors through which a gradient is wanted).  Forward-mode derivatives are
refused everywhere.

Every launch goes to ``stream`` (the current stream by default).  Results and
temporary memory are allocated on it, and tensors of the call are recorded on
it, so that memory freed by the caller is not reused while the launch reads it.
"""
from __future__ import annotations

import ctypes
import functools
import struct
import weakref
from dataclasses import InitVar, dataclass

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import (Nvfp4Error, PackedWeight, _dev, _i32, _i64, _vp, check_devices, lib, packed_codes_bytes,
               packed_scales_bytes)

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


# nvfp4_epilogue: bias, up_bias, residual, preact, ldr, ldp, activation,
# bias_dtype, residual_dtype, out_dtype
_EPILOGUE = struct.Struct("@4P2q4i")

_SIZE = ctypes.c_size_t
_F32 = ctypes.c_float
_SIGNATURES = {
    "nvfp4_linear": (_i32, [_vp, _vp, _F32, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _SIZE, _vp]),
    "nvfp4_linear_workspace_bytes": (_SIZE, [_i32, _i32, _i32]),
    "nvfp4_gated_rows": (_SIZE, [_i32]),
    "nvfp4_fused_geometry": (_i32, [_i32, _i32, _i32] + [ctypes.POINTER(_i32)] * 4),
    "nvfp4_pack_gated": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp]),
    "nvfp4_gated": (_i32, [_vp, _vp, _F32, _F32, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _SIZE, _vp]),
    "nvfp4_gated_workspace_bytes": (_SIZE, [_i32, _i32, _i32]),
    "nvfp4_transposed_codes_bytes": (_SIZE, [_i32, _i32]),
    "nvfp4_transposed_scales_bytes": (_SIZE, [_i32, _i32]),
    "nvfp4_pack_transposed": (_i32, [_vp, _vp, _i32, _i32, _vp, _vp, _vp]),
    "nvfp4_linear_backward": (_i32, [_vp, _vp, _F32, _vp, _i32, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _i32, _i32, _i32,
                                     _i32, _vp, _SIZE, _vp]),
    "nvfp4_linear_backward_workspace_bytes": (_SIZE, [_i32] * 6),
    "nvfp4_gated_backward": (_i32, [_vp, _vp, _F32, _F32, _vp, _i32, _i64, _vp, _i64, _i32, _vp, _i64, _vp, _vp, _i32,
                                    _i32, _i32, _i32, _vp, _SIZE, _vp]),
    "nvfp4_gated_backward_workspace_bytes": (_SIZE, [_i32] * 5),
}


@functools.lru_cache(maxsize=None)
def _call(name: str):
    f = getattr(lib(), name)
    f.restype, f.argtypes = _SIGNATURES[name]
    return f


def _run(name: str, *args) -> None:
    status = _call(name)(*args)
    if status:
        raise Nvfp4Error(status, name)


# ---- checks, streams and memory ---------------------------------------------------

def _act(activation) -> int:
    if activation is None:
        return 0
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(ACTIVATIONS), activation))
    return ACTIVATIONS[activation]


def _typed(t, dtypes, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))


def _mat(t, dtypes, name: str, n, cols) -> torch.Tensor:
    """A device matrix of n rows (None: any) and cols columns, unit stride
    along a row."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes):
        _typed(t, dtypes, name)
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (n is not None and shape[0] != n):
        raise ValueError("%s must be [%s, %d], got %s" % (name, "n" if n is None else n, cols, list(shape)))
    if shape[0] >> 31 or cols >> 31:         # the library's sizes are 32-bit
        raise ValueError("%s must have fewer than 2^31 rows and columns, got %s" % (name, list(shape)))
    if t.stride(1) != 1 and cols > 1 and shape[0] > 0:
        raise ValueError("%s must have unit stride along a row" % name)
    return t


def _ld(t) -> int:
    """Row stride in elements; of no meaning with fewer than two rows."""
    shape = t.shape
    return t.stride(0) if shape[0] > 1 else shape[1]


def _weight(w, cls, name: str = "w"):
    """The classes of weights share field names over layouts of different sizes,
    so one of another class would be read past its end."""
    if not isinstance(w, cls):
        raise TypeError("%s must be a %s, got %s" % (name, cls.__name__, type(w).__name__))


def _vec(t, dtypes, name: str, size: int):
    _typed(t, dtypes, name)
    if t.dim() != 1 or t.shape[0] != size or not t.is_contiguous():
        raise ValueError("%s must be a contiguous [%d]" % (name, size))


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


class _Launch:
    """The stream of a call, after checking that it and every tensor are on
    the current device, and the memory rules of a stream that is not the
    current one.  (With stream None the raw current stream is looked up: a
    torch Stream object costs several times the rest of this.)"""
    __slots__ = ("device", "handle", "stream", "current")

    def __init__(self, stream, *tensors):
        device = self.device = torch.cuda.current_device()
        for t in tensors:
            if t is not None and t.get_device() != device:
                check_devices([t.device], device, torch.device("cuda", device))
        self.stream = None
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(device)
            return
        check_devices((), device, stream.device)
        self.handle = stream.cuda_stream
        self.current = torch.cuda.current_stream()
        if stream != self.current:
            self.stream = stream
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)

    def alloc(self, *shape, dtype):
        """Memory of the launch's stream."""
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device="cuda")
        with torch.cuda.stream(self.stream):
            t = torch.empty(shape, dtype=dtype, device="cuda")
        t.record_stream(self.current)   # a result is read there
        return t

    def workspace(self, given, need: int):
        """(pointer, bytes, tensor) of `need` workspace bytes."""
        if given is None:
            if not need:
                return 0, 0, None
            given = self.alloc(need, dtype=torch.uint8)
        return given.data_ptr(), given.numel(), given


# ---- weights -----------------------------------------------------------------------

@dataclass
class TransposedWeight:
    """The transposed copy of a packed weight, which gradients go through:
    another 9/16 byte a weight, made once where gradients are wanted."""
    codes: torch.Tensor
    scales: torch.Tensor
    gscale: float
    N: int                   # rows of the packed weight
    K: int
    gated: bool = False      # of a GatedWeight
    # The packed codes the copy was made from, held weakly and only to refuse the
    # copy of another weight; a copied or unpickled object has none.
    source: InitVar[torch.Tensor] = None
    _source = None

    def __post_init__(self, source):
        if source is not None:
            self._source = weakref.ref(source)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_source"}


def _check_transposed(wt: TransposedWeight, w) -> None:
    """wt is the transposed copy of w (a PackedWeight or a GatedWeight), as far
    as sizes, kind, tensor scale and the codes it was made from tell."""
    gated = isinstance(w, GatedWeight)
    source = None if wt._source is None else wt._source()
    if ((wt.gated, wt.N, wt.K, wt.gscale) != ((True, gated_rows(w.F), w.K, 1.0) if gated else
                                              (False, w.N, w.K, w.gscale))
            or (source is not None and source.data_ptr() != w.codes.data_ptr())):
        raise ValueError("transposed is not the transposed copy of this weight (w.transpose())")


def _transpose(codes, scales, gscale, N, K, stream, gated=False) -> TransposedWeight:
    at = _Launch(stream, codes, scales)
    ct = at.alloc(int(_call("nvfp4_transposed_codes_bytes")(N, K)), dtype=torch.uint8)
    st = at.alloc(int(_call("nvfp4_transposed_scales_bytes")(N, K)), dtype=torch.uint8)
    _run("nvfp4_pack_transposed", codes.data_ptr(), scales.data_ptr(), N, K, ct.data_ptr(), st.data_ptr(),
         at.handle)
    return TransposedWeight(ct, st, gscale, N, K, gated, codes)


def transpose(w: PackedWeight, stream=None) -> TransposedWeight:
    """The transposed copy of ``w`` (also ``w.transpose()``)."""
    _weight(w, PackedWeight)
    return _transpose(w.codes, w.scales, w.gscale, w.N, w.K, stream)


def gated_rows(F: int) -> int:
    """Rows of the packed weight of a gated block with F outputs."""
    return int(_call("nvfp4_gated_rows")(F))


def fused_geometry(n: int, rows: int, K: int) -> tuple:
    """(weight rows, tokens of a workgroup, K groups in it, K parts) the fused
    operators take for n > 16 tokens (nvfp4_fused_geometry)."""
    v = [_i32() for _ in range(4)]
    _run("nvfp4_fused_geometry", n, rows, K, *(ctypes.byref(x) for x in v))
    return tuple(x.value for x in v)


@dataclass
class GatedWeight:
    """The gate and up weights of a gated block in one packed weight whose
    16-row groups alternate gate, up."""
    codes: torch.Tensor
    scales: torch.Tensor
    gate_gscale: float
    up_gscale: float
    F: int
    K: int

    @classmethod
    def from_packed(cls, gate: PackedWeight, up: PackedWeight, stream=None) -> "GatedWeight":
        _weight(gate, PackedWeight, "gate")
        _weight(up, PackedWeight, "up")
        if (gate.N, gate.K) != (up.N, up.K):
            raise ValueError("the gate and up weights must have one shape")
        at = _Launch(stream, gate.codes, gate.scales, up.codes, up.scales)
        rows = gated_rows(gate.N)
        codes = at.alloc(packed_codes_bytes(rows, gate.K), dtype=torch.uint8)
        scales = at.alloc(packed_scales_bytes(rows, gate.K), dtype=torch.uint8)
        _run("nvfp4_pack_gated", gate.codes.data_ptr(), gate.scales.data_ptr(), up.codes.data_ptr(),
             up.scales.data_ptr(), gate.N, gate.K, codes.data_ptr(), scales.data_ptr(),
             at.handle)
        return cls(codes, scales, gate.gscale, up.gscale, gate.N, gate.K)

    @classmethod
    def from_float(cls, Wg: torch.Tensor, Wu: torch.Tensor, stream=None) -> "GatedWeight":
        """Quantise fp32 or bf16 gate and up weights [F, K], each with its own
        tensor scale."""
        return cls.from_packed(PackedWeight.from_float(Wg, stream), PackedWeight.from_float(Wu, stream), stream)

    def transpose(self, stream=None) -> TransposedWeight:
        """The transposed copy, for gradients (its tensor scales are applied
        to the gradient rows, so its own is 1)."""
        return _transpose(self.codes, self.scales, 1.0, gated_rows(self.F), self.K, stream, gated=True)


# ---- forward -------------------------------------------------------------------------

def _out(at, out, out_dtype, n, cols):
    if out is None:
        if out_dtype not in _DTYPES:
            raise TypeError("out_dtype must be torch.bfloat16 or torch.float32, got %s" % out_dtype)
        return at.alloc(n, cols, dtype=out_dtype)
    if out.dtype != out_dtype:
        raise TypeError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
    return out


def _linear_forward(w, X, bias, act, residual, out, out_dtype, preact, workspace, stream):
    n = X.shape[0]
    at = _Launch(stream, w.codes, w.scales, X, bias, residual, out, preact, workspace)
    Y = _out(at, out, out_dtype, n, w.N)
    ep = _EPILOGUE.pack(_ptr(bias), 0, _ptr(residual), _ptr(preact), 0 if residual is None else _ld(residual),
                        0 if preact is None else _ld(preact), act, 1 if bias is None else _DTYPES[bias.dtype],
                        1 if residual is None else _DTYPES[residual.dtype], _DTYPES[Y.dtype])
    ws, size, keep = at.workspace(workspace, int(_call("nvfp4_linear_workspace_bytes")(n, w.N, w.K)))
    _run("nvfp4_linear", w.codes.data_ptr(), w.scales.data_ptr(), w.gscale, X.data_ptr(), _ld(X),
         Y.data_ptr(), _ld(Y), n, w.N, w.K, ep, ws, size, at.handle)
    return Y


def _gated_forward(w, X, act, gate_bias, up_bias, out, out_dtype, preact, workspace, stream):
    n = X.shape[0]
    at = _Launch(stream, w.codes, w.scales, X, gate_bias, up_bias, out, preact, workspace)
    H = _out(at, out, out_dtype, n, w.F)
    some = gate_bias if gate_bias is not None else up_bias
    ep = _EPILOGUE.pack(_ptr(gate_bias), _ptr(up_bias), 0, _ptr(preact), 0, 0 if preact is None else _ld(preact), act,
                        1 if some is None else _DTYPES[some.dtype], 1, _DTYPES[H.dtype])
    ws, size, keep = at.workspace(workspace, int(_call("nvfp4_gated_workspace_bytes")(n, w.F, w.K)))
    _run("nvfp4_gated", w.codes.data_ptr(), w.scales.data_ptr(), w.gate_gscale, w.up_gscale, X.data_ptr(),
         _ld(X), H.data_ptr(), _ld(H), n, w.F, w.K, ep, ws, size, at.handle)
    return H


_FLOATS = (torch.bfloat16, torch.float32)


def _pad8(cols: int) -> int:
    return (cols + 7) // 8 * 8


def preact_columns(w) -> int:
    """Columns of the fp32 pre-activation buffer of ``w`` (a PackedWeight or a
    GatedWeight): the outputs up to a multiple of 8, or the gated weight's rows."""
    if isinstance(w, GatedWeight):
        return gated_rows(w.F)
    if not isinstance(w, PackedWeight):
        raise TypeError("w must be a PackedWeight or a GatedWeight, got %s" % type(w).__name__)
    return _pad8(w.N)


def _preact_arg(preact, w, n):
    return None if preact is None else _mat(preact, (torch.float32,), "preact", n, preact_columns(w))


def _workspace_arg(workspace):
    return None if workspace is None else _dev(workspace, torch.uint8, "workspace")


def _refuse_tangents(tensors) -> None:
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError("forward-mode derivatives are not available")


def _wants_grad(*tensors) -> bool:
    if forward_ad._current_level >= 0:      # inside a dual_level
        _refuse_tangents(tensors)
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _no_graph(*tensors) -> None:
    """Of a call that makes no graph: a gradient wanted through these would be
    lost without a word."""
    if _wants_grad(*tensors):
        raise ValueError("a gradient through this call is not available (detach the argument, or torch.no_grad())")


def _written(*buffers) -> None:
    """Tell autograd of buffers that a launch overwrites, for the graphs that
    have saved them."""
    for t in buffers:
        if t is not None:
            increment_version(t)


def _check_grad(X, w, transposed, stream, *buffers):
    if any(b is not None for b in buffers):
        raise ValueError("out, preact and workspace go with calls that need no gradient")
    if stream is not None and stream != torch.cuda.current_stream():
        raise ValueError("with gradients the launch stream is the current one (torch.cuda.stream)")
    if X.requires_grad:
        if transposed is None:
            raise ValueError("a gradient of X needs the weight's transposed copy (transposed=w.transpose())")
        _check_transposed(transposed, w)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, bias, residual, w, transposed, act, out_dtype):
        ctx.transposed, ctx.act = transposed, act
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.residual_dtype = None if residual is None else residual.dtype
        preact = None
        if act and (ctx.needs_input_grad[0] or ctx.needs_input_grad[1]):
            preact = torch.empty(X.shape[0], _pad8(w.N), dtype=torch.float32, device=X.device)
        ctx.save_for_backward(preact)
        return _linear_forward(w, X, bias, act, residual, None, out_dtype, preact, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        (preact,) = ctx.saved_tensors
        need_x, need_b, need_r = ctx.needs_input_grad[:3]
        dX = db = None
        if need_x or need_b:
            dX, db = _linear_backward(ctx.transposed if need_x else None, dY, ctx.act, preact,
                                      ctx.bias_dtype if need_b else None, None, None)
        return dX, db, dY.to(ctx.residual_dtype) if need_r else None, None, None, None, None


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, gate_bias, up_bias, w, transposed, act, out_dtype):
        ctx.w, ctx.transposed, ctx.act = w, transposed, act
        ctx.bias_dtype = next((b.dtype for b in (gate_bias, up_bias) if b is not None), None)
        preact = torch.empty(X.shape[0], gated_rows(w.F), dtype=torch.float32, device=X.device)
        ctx.save_for_backward(preact)
        return _gated_forward(w, X, act, gate_bias, up_bias, None, out_dtype, preact, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dH):
        (preact,) = ctx.saved_tensors
        need_x, need_g, need_u = ctx.needs_input_grad[:3]
        grads = _gated_backward(ctx.w, ctx.transposed if need_x else None, dH, ctx.act, preact,
                                ctx.bias_dtype if need_g else None, ctx.bias_dtype if need_u else None, None, None)
        return grads + (None, None, None, None)


def linear(w: PackedWeight, X: torch.Tensor, bias: torch.Tensor = None, activation: str = None,
           residual: torch.Tensor = None, *, transposed: TransposedWeight = None, out: torch.Tensor = None,
           out_dtype=None, preact: torch.Tensor = None, workspace: torch.Tensor = None,
           stream=None) -> torch.Tensor:
    """Y = act(X . dequant(W)^T + bias) + residual for any number of tokens.

    X: bf16 [n, K]; bias: bf16 or fp32 [N]; residual: bf16 or fp32 [n, N] (it
    may be ``out`` itself); Y: bf16, or fp32 with ``out_dtype``.  Rows may be
    strided; X rows are 16-byte aligned.  ``preact`` (fp32 [n,
    preact_columns(w)]) receives the pre-activations ``linear_backward`` needs.
    ``workspace``: uint8, nvfp4_linear_workspace_bytes (allocated otherwise).
    Differentiable in X (given ``transposed``), bias and residual."""
    act = _act(activation)
    _weight(w, PackedWeight)
    if transposed is not None:
        _weight(transposed, TransposedWeight, "transposed")
    _mat(X, (torch.bfloat16,), "X", None, w.K)
    n = X.shape[0]
    if bias is not None:
        _vec(bias, _FLOATS, "bias", w.N)
    if residual is not None:
        _mat(residual, _FLOATS, "residual", n, w.N)
    if out is not None:
        _mat(out, _FLOATS, "out", n, w.N)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if _wants_grad(X, bias, residual):
        _check_grad(X, w, transposed, stream, out, preact, workspace)
        return _Linear.apply(X, bias, residual, w, transposed, act, out_dtype)
    if out is not None or preact is not None:
        _no_graph(out, preact)
        _written(out, preact)
    return _linear_forward(w, X, bias, act, residual, out, out_dtype, _preact_arg(preact, w, n),
                           _workspace_arg(workspace), stream)


def gated(w: GatedWeight, X: torch.Tensor, activation: str = "silu", gate_bias: torch.Tensor = None,
          up_bias: torch.Tensor = None, *, transposed: TransposedWeight = None, out: torch.Tensor = None,
          out_dtype=None, preact: torch.Tensor = None, workspace: torch.Tensor = None,
          stream=None) -> torch.Tensor:
    """H = act(X . dequant(Wg)^T + gate_bias) * (X . dequant(Wu)^T + up_bias),
    both projections, the activation and the product in one launch.  Arguments
    as ``linear``; the biases have one dtype.  Differentiable in X (given
    ``transposed``) and the biases."""
    act = _act(activation)
    _weight(w, GatedWeight)
    if transposed is not None:
        _weight(transposed, TransposedWeight, "transposed")
    _mat(X, (torch.bfloat16,), "X", None, w.K)
    n = X.shape[0]
    for b, name in ((gate_bias, "gate_bias"), (up_bias, "up_bias")):
        if b is not None:
            _vec(b, _FLOATS, name, w.F)
    if gate_bias is not None and up_bias is not None and gate_bias.dtype != up_bias.dtype:
        raise TypeError("gate_bias and up_bias must have one dtype")
    if out is not None:
        _mat(out, _FLOATS, "out", n, w.F)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if _wants_grad(X, gate_bias, up_bias):
        _check_grad(X, w, transposed, stream, out, preact, workspace)
        return _Gated.apply(X, gate_bias, up_bias, w, transposed, act, out_dtype)
    if out is not None or preact is not None:
        _no_graph(out, preact)
        _written(out, preact)
    return _gated_forward(w, X, act, gate_bias, up_bias, out, out_dtype, _preact_arg(preact, w, n),
                          _workspace_arg(workspace), stream)


# ---- backward ------------------------------------------------------------------------

def _incoming(dY, N, name, stream):
    """A gradient as autograd hands it over: any strides.  A copy is made on
    the launch stream, where the caller's ordering holds."""
    if not isinstance(dY, torch.Tensor) or not dY.is_cuda:
        raise TypeError("%s must be a CUDA (HIP) tensor" % name)
    if dY.dim() == 2 and (dY.stride(1) != 1 or dY.stride(0) < dY.shape[1]):
        at = _Launch(stream, dY)
        if at.stream is None:
            dY = dY.contiguous()
        else:
            with torch.cuda.stream(stream):
                dY = dY.contiguous()
    return _mat(dY, _FLOATS, name, None, N)


def _linear_backward(wt, dY, act, preact, bias_dtype, out, stream):
    dY = _incoming(dY, wt.N if wt is not None else dY.shape[-1], "dY", stream)
    n, N = dY.shape
    codes, scales, gscale, K = (wt.codes, wt.scales, wt.gscale, wt.K) if wt is not None else (None, None, 0.0, 0)
    at = _Launch(stream, dY, preact, out, codes, scales)
    dX = (at.alloc(n, K, dtype=torch.bfloat16) if out is None else out) if wt is not None else None
    db = None if bias_dtype is None else at.alloc(N, dtype=bias_dtype)
    ld, dtype, ptr = _ld(dY), _DTYPES[dY.dtype], dY.data_ptr()
    copy = act or dtype == 0 or N % 8 or ptr % 16 or (n > 1 and (ld % 8 or ld > 1 << 22))
    ws, size, keep = at.workspace(None, _call("nvfp4_linear_backward_workspace_bytes")(
        n, N, K, wt is not None, db is not None, 1 if copy else 0))
    _run("nvfp4_linear_backward", _ptr(codes), _ptr(scales), gscale, ptr, dtype, ld, _ptr(preact),
         0 if preact is None else _ld(preact), act, _ptr(dX), K if dX is None else _ld(dX), _ptr(db),
         1 if db is None else _DTYPES[bias_dtype], n, N, K, ws, size, at.handle)
    return dX, db


def _gated_backward(w, wt, dH, act, preact, gate_dtype, up_dtype, out, stream):
    dH = _incoming(dH, w.F, "dH", stream)
    n, F, K = dH.shape[0], w.F, w.K
    codes, scales = (wt.codes, wt.scales) if wt is not None else (None, None)
    at = _Launch(stream, dH, preact, out, codes, scales)
    dX = (at.alloc(n, K, dtype=torch.bfloat16) if out is None else out) if wt is not None else None
    dg = None if gate_dtype is None else at.alloc(F, dtype=gate_dtype)
    du = None if up_dtype is None else at.alloc(F, dtype=up_dtype)
    some = gate_dtype if gate_dtype is not None else up_dtype
    ws, size, keep = at.workspace(None, _call("nvfp4_gated_backward_workspace_bytes")(n, F, K, wt is not None,
                                                                                     some is not None))
    _run("nvfp4_gated_backward", _ptr(codes), _ptr(scales), w.gate_gscale, w.up_gscale, dH.data_ptr(),
         _DTYPES[dH.dtype], _ld(dH), preact.data_ptr(), _ld(preact), act, _ptr(dX), K if dX is None else _ld(dX),
         _ptr(dg), _ptr(du), 1 if some is None else _DTYPES[some], n, F, K, ws, size, at.handle)
    return dX, dg, du


def _grad_args(wt, bias_dtype, out, n):
    if bias_dtype is not None and bias_dtype not in _DTYPES:
        raise TypeError("bias_dtype must be torch.bfloat16 or torch.float32, got %s" % bias_dtype)
    if out is not None:
        if wt is None:
            raise ValueError("out receives dX, which needs the transposed weight")
        _mat(out, (torch.bfloat16,), "out", n, wt.K)


def gemm_t(wt: TransposedWeight, dY: torch.Tensor, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """dX[n, K] = dY[n, N] . dequant(W) (bf16 in and out, fp32 accumulation):
    the gradient of ``gemv``, ``gemm`` or a plain ``linear`` with respect to
    its input.  (The copy of a GatedWeight has no tensor scale: W without its
    two.)  dY rows that are not 16-byte aligned, or an N that is no multiple of
    8, cost a padded copy of dY."""
    _weight(wt, TransposedWeight, "wt")
    _mat(dY, (torch.bfloat16,), "dY", None, wt.N)
    if out is not None:
        _mat(out, (torch.bfloat16,), "out", dY.shape[0], wt.K)
    _no_graph(dY, out)
    _written(out)
    return _linear_backward(wt, dY, 0, None, None, out, stream)[0]


def linear_backward(wt: TransposedWeight, dY: torch.Tensor, activation: str = None, preact: torch.Tensor = None,
                    bias_dtype=None, out: torch.Tensor = None, stream=None):
    """(dX, dbias) of ``linear``: dX bf16 [n, K] (None without ``wt``), dbias in
    ``bias_dtype`` (None without).  ``preact`` as ``linear`` filled it (not
    needed without an activation).  The residual's gradient is dY."""
    if wt is not None:
        _weight(wt, TransposedWeight, "wt")
        if wt.gated:
            raise ValueError("wt is the copy of a gated weight, which gated_backward takes")
    _typed(dY, _FLOATS, "dY")
    act = _act(activation)
    if act:
        if preact is None:
            raise ValueError("the gradient of an activation needs preact")
        _mat(preact, (torch.float32,), "preact", dY.shape[0], _pad8(dY.shape[-1]))
    _grad_args(wt, bias_dtype, out, dY.shape[0])
    _no_graph(dY, preact, out)
    _written(out)
    return _linear_backward(wt, dY, act, preact if act else None, bias_dtype, out, stream)


def gated_backward(w: GatedWeight, wt: TransposedWeight, dH: torch.Tensor, preact: torch.Tensor,
                   activation: str = "silu", bias_dtype=None, out: torch.Tensor = None, stream=None):
    """(dX, dgate_bias, dup_bias) of ``gated``; the bias gradients in
    ``bias_dtype`` (None without)."""
    _weight(w, GatedWeight)
    if wt is not None:
        _weight(wt, TransposedWeight, "wt")
    _typed(dH, _FLOATS, "dH")
    act = _act(activation)
    _mat(preact, (torch.float32,), "preact", dH.shape[0], gated_rows(w.F))
    if wt is not None:
        _check_transposed(wt, w)
    _grad_args(wt, bias_dtype, out, dH.shape[0])
    _no_graph(dH, preact, out)
    _written(out)
    return _gated_backward(w, wt, dH, act, preact, bias_dtype, bias_dtype, out, stream)
