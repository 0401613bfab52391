"""Mixture-of-experts layer on NVFP4 weights: the router from logits to experts
and weights, the whole layer of gated experts, and their gradients (the experts
are frozen: gradients go to the activations, the weights and the logits).

    weights, experts = moe_route(logits, k)              # logits [n, E]
    w = ExpertWeights.from_float(Wg, Wu, Wd)             # [E, F, K], [E, F, K], [E, K, F]
    y = moe(w, X, experts, weights, residual=shared)

``moe_route`` is differentiable in the logits; ``moe`` in X, the weights and the
residual when given the experts' transposed copies (``transposed=w.transpose()``,
made once).  ``moe_route_backward`` and ``moe_backward`` are the same gradients
without autograd.  Streams, memory and refusals as in ``fused.py``.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct
import weakref
from dataclasses import InitVar, dataclass

import torch

from . import Nvfp4Error, PackedWeight, _i32, _i64, _vp, lib, packed_codes_bytes, packed_scales_bytes
from .fused import (_DTYPES, _EPILOGUE, _F32, _FLOATS, _SIZE, GatedWeight, _act, _Launch, _incoming, _ld, _mat, _no_graph, _out,
                    _ptr, _transpose, _typed, _wants_grad, _weight, _workspace_arg,
                    _written)

SCORES = {"softmax": 0, "sigmoid": 1}
MAX_EXPERTS = 1024
MAX_SLOTS = 32

# nvfp4_experts: gate_up codes and scales, down codes and scales, gscale, E, F, K
_EXPERTS = struct.Struct("@5P3i")

_SIGNATURES = {
    "nvfp4_moe_route": (_i32, [_vp, _i32, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _F32, _vp, _vp, _vp]),
    "nvfp4_moe_route_backward": (_i32, [_vp, _i32, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _F32, _vp, _i64, _vp]),
    "nvfp4_moe": (_i32, [_vp, _vp, _i64, _vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _SIZE, _vp]),
    "nvfp4_moe_workspace_bytes": (_SIZE, [_i32] * 6),
    "nvfp4_moe_geometry": (_i32, [_i32] * 5 + [ctypes.POINTER(_i32)] * 2),
    "nvfp4_moe_decode_geometry": (_i32, [_i32, _i32, ctypes.POINTER(_i32)]),
    "nvfp4_moe_backward": (_i32, [_vp, _vp, _i32, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _SIZE, _vp]),
    "nvfp4_moe_backward_workspace_bytes": (_SIZE, [_i32] * 7),
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


# ---- router -------------------------------------------------------------------------

def _scoring(scoring) -> int:
    if scoring not in SCORES:
        raise ValueError("scoring must be one of %s, got %r" % (", ".join(SCORES), scoring))
    return SCORES[scoring]


def _logits(logits):
    _typed(logits, _FLOATS, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [n, E], got %s" % list(logits.shape))
    _mat(logits, _FLOATS, "logits", None, logits.shape[1])
    n, E = logits.shape
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError("logits must be of 1 to %d experts, got %d" % (MAX_EXPERTS, E))
    return n, E


def _slots(k, E=MAX_SLOTS) -> int:
    if not isinstance(k, int) or isinstance(k, bool) or not 1 <= k <= min(E, MAX_SLOTS):
        raise ValueError("k must be an integer from 1 to %d, got %r" % (min(E, MAX_SLOTS), k))
    return k


def _scale(scale) -> float:
    scale = float(scale)
    if not math.isfinite(scale):
        raise ValueError("scale must be finite, got %r" % scale)
    return scale


def _pair_matrix(t, dtype, name, n=None, k=None):
    """A contiguous [n, k] of the pairs of a token and an expert."""
    _typed(t, (dtype,), name)
    if t.dim() != 2 or (n is not None and t.shape[0] != n) or (k is not None and t.shape[1] != k):
        raise ValueError("%s must be [%s, %s], got %s" % (name, "n" if n is None else n, "k" if k is None else k, list(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _route_forward(logits, k, scoring, bias, normalize, scale, stream):
    n, E = logits.shape
    at = _Launch(stream, logits, bias)
    weights = at.alloc(n, k, dtype=torch.float32)
    experts = at.alloc(n, k, dtype=torch.int32)
    _run("nvfp4_moe_route", logits.data_ptr(), _DTYPES[logits.dtype], _ld(logits), _ptr(bias), n, E, k, scoring, normalize,
         scale, weights.data_ptr(), experts.data_ptr(), at.handle)
    return weights, experts


def _route_backward(logits, experts, dweights, scoring, normalize, scale, stream):
    n, E = logits.shape
    at = _Launch(stream, logits, experts, dweights)
    out = at.alloc(n, E, dtype=logits.dtype)
    _run("nvfp4_moe_route_backward", logits.data_ptr(), _DTYPES[logits.dtype], _ld(logits), experts.data_ptr(),
         dweights.data_ptr(), n, E, experts.shape[1], scoring, normalize, scale, out.data_ptr(), E, at.handle)
    return out


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, scoring, bias, normalize, scale):
        weights, experts = _route_forward(logits, k, scoring, bias, normalize, scale, None)
        ctx.save_for_backward(logits, experts)
        ctx.how = scoring, normalize, scale
        ctx.mark_non_differentiable(experts)
        return weights, experts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dweights, _):
        logits, experts = ctx.saved_tensors
        return _route_backward(logits, experts, dweights.contiguous(), *ctx.how, None), None, None, None, None, None


def moe_route(logits: torch.Tensor, k: int, scoring: str = "softmax", bias: torch.Tensor = None, normalize: bool = True,
              scale: float = 1.0, *, stream=None):
    """(weights fp32 [n, k], experts int32 [n, k]): for each token the k experts of
    largest score, largest first, ties to the lowest index.

    logits: fp32 or bf16 [n, E], E <= 1024, k <= 32; -inf masks an expert, and a
    slot for which none is left has expert -1 and weight 0.  Scores are the
    softmax of the row or sigmoids; ``bias`` (fp32 [E]) is added for the choice
    alone.  Weights: scale times the chosen scores, with ``normalize`` over their
    sum.  Differentiable in the logits (the choice has no gradient)."""
    n, E = _logits(logits)
    k, how, scale = _slots(k, E), _scoring(scoring), _scale(scale)
    if bias is not None:
        _typed(bias, (torch.float32,), "bias")
        if bias.shape != (E,) or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous [%d]" % E)
        _no_graph(bias)
    normalize = 1 if normalize else 0
    if _wants_grad(logits):
        if stream is not None and stream != torch.cuda.current_stream():
            raise ValueError("with gradients the launch stream is the current one (torch.cuda.stream)")
        return _Route.apply(logits, k, how, bias, normalize, scale)
    return _route_forward(logits, k, how, bias, normalize, scale, stream)


def moe_route_backward(logits: torch.Tensor, experts: torch.Tensor, dweights: torch.Tensor, scoring: str = "softmax",
                       normalize: bool = True, scale: float = 1.0, *, stream=None) -> torch.Tensor:
    """dlogits [n, E] (in the logits' type) of ``moe_route``, with the experts it chose."""
    n, E = _logits(logits)
    _pair_matrix(experts, torch.int32, "experts", n)
    k = _slots(experts.shape[1], E)
    _pair_matrix(dweights, torch.float32, "dweights", n, k)
    _no_graph(logits, dweights)
    return _route_backward(logits, experts, dweights, _scoring(scoring), 1 if normalize else 0, _scale(scale), stream)


# ---- weights --------------------------------------------------------------------------

@dataclass
class TransposedExperts:
    """The transposed copies of an ExpertWeights, which its gradients go through:
    another 9/16 byte a weight, made once where gradients are wanted."""
    gate_up_codes: torch.Tensor
    gate_up_scales: torch.Tensor
    down_codes: torch.Tensor
    down_scales: torch.Tensor
    gscale: torch.Tensor
    E: int
    F: int
    K: int
    # The gate and up codes the copy was made from, held weakly and only to refuse
    # the copy of other experts; a copied or unpickled object has none.
    source: InitVar[torch.Tensor] = None
    _source = None

    def __post_init__(self, source):
        if source is not None:
            self._source = weakref.ref(source)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_source"}


@dataclass
class ExpertWeights:
    """E gated experts of one shape: for each the gate and up weights in one gated
    weight and the packed down weight, the experts in turn in one buffer each;
    gscale: fp32 [3, E], the tensor scales of gate, up and down."""
    gate_up_codes: torch.Tensor
    gate_up_scales: torch.Tensor
    down_codes: torch.Tensor
    down_scales: torch.Tensor
    gscale: torch.Tensor
    E: int
    F: int
    K: int

    @classmethod
    def from_packed(cls, gate, up, down, stream=None) -> "ExpertWeights":
        """From lists of E packed weights: gate and up F x K, down K x F."""
        gate, up, down = list(gate), list(up), list(down)
        E = len(gate)
        if not 1 <= E <= MAX_EXPERTS or len(up) != E or len(down) != E:
            raise ValueError("gate, up and down must be lists of one length, 1 to %d" % MAX_EXPERTS)
        for ws, name in ((gate, "gate"), (up, "up"), (down, "down")):
            for w in ws:
                _weight(w, PackedWeight, name)
        return cls._build(E, gate[0].N, gate[0].K, lambda e: (gate[e], up[e], down[e]), stream)

    @classmethod
    def from_float(cls, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, stream=None) -> "ExpertWeights":
        """Quantise fp32 or bf16 weights [E, F, K], [E, F, K] and [E, K, F], each
        matrix with its own tensor scale."""
        for W, name in ((Wg, "Wg"), (Wu, "Wu"), (Wd, "Wd")):
            _typed(W, _FLOATS, name)
            if W.dim() != 3:
                raise ValueError("%s must be 3-D, got %s" % (name, list(W.shape)))
        E, F, K = Wg.shape
        if not 1 <= E <= MAX_EXPERTS or Wu.shape != Wg.shape or Wd.shape != (E, K, F):
            raise ValueError("the weights must be [E, F, K], [E, F, K] and [E, K, F] of 1 to %d experts, got %s, %s and %s"
                             % (MAX_EXPERTS, list(Wg.shape), list(Wu.shape), list(Wd.shape)))
        return cls._build(E, F, K, lambda e: tuple(PackedWeight.from_float(W[e], stream) for W in (Wg, Wu, Wd)), stream)

    @classmethod
    def _build(cls, E, F, K, expert, stream):
        """``expert(e)``: the packed gate, up and down weights of expert e."""
        if F % 16 or K % 16 or not 1 <= F <= 1 << 18 or not 1 <= K <= 1 << 18:
            raise ValueError("F and K must be multiples of 16 up to 262144, got %d and %d" % (F, K))
        at = _Launch(stream)
        sizes = [(packed_codes_bytes(2 * F, K), packed_scales_bytes(2 * F, K)), (packed_codes_bytes(K, F), packed_scales_bytes(K, F))]
        gu, gus, d, ds = [at.alloc(E, size, dtype=torch.uint8) for pair in sizes for size in pair]
        scales = []
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            for e in range(E):
                g, u, w = expert(e)
                if (g.N, g.K) != (F, K) or (u.N, u.K) != (F, K) or (w.N, w.K) != (K, F):
                    raise ValueError("expert %d is not of F = %d and K = %d" % (e, F, K))
                _Launch(stream, w.codes, w.scales)
                both = GatedWeight.from_packed(g, u, stream)
                for to, part in ((gu, both.codes), (gus, both.scales), (d, w.codes), (ds, w.scales)):
                    to[e].copy_(part)
                scales.append((g.gscale, u.gscale, w.gscale))
            gscale = torch.tensor(list(zip(*scales)), dtype=torch.float32).cuda()
        if at.stream is not None:
            gscale.record_stream(at.current)
        return cls(gu, gus, d, ds, gscale, E, F, K)

    def transpose(self, stream=None) -> TransposedExperts:
        """The transposed copies, for gradients."""
        at = _Launch(stream, self.gate_up_codes, self.gate_up_scales, self.down_codes, self.down_scales, self.gscale)
        made = []
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            for codes, scales, N, K in ((self.gate_up_codes, self.gate_up_scales, 2 * self.F, self.K),
                                        (self.down_codes, self.down_scales, self.K, self.F)):
                for e in range(self.E):
                    t = _transpose(codes[e], scales[e], 1.0, N, K, stream)
                    if e == 0:
                        made += [at.alloc(self.E, p.numel(), dtype=torch.uint8) for p in (t.codes, t.scales)]
                    made[-2][e].copy_(t.codes)
                    made[-1][e].copy_(t.scales)
        return TransposedExperts(*made, self.gscale, self.E, self.F, self.K, self.gate_up_codes)


def _check_transposed(wt, w):
    """wt is the transposed copy of w, as far as sizes, the codes it was made from and
    the tensor scales tell, which it shares with the weights and so keeps alive."""
    source = None if wt._source is None else wt._source()
    if ((wt.E, wt.F, wt.K) != (w.E, w.F, w.K) or (source is not None and source.data_ptr() != w.gate_up_codes.data_ptr())
            or (wt._source is not None and wt.gscale.data_ptr() != w.gscale.data_ptr())):
        raise ValueError("transposed is not the transposed copy of these experts (w.transpose())")


def _parts(w):
    return w.gate_up_codes, w.gate_up_scales, w.down_codes, w.down_scales, w.gscale


def _struct(w):
    return _EXPERTS.pack(*(t.data_ptr() for t in _parts(w)), w.E, w.F, w.K)


# ---- the layer ---------------------------------------------------------------------------

def _moe_forward(w, X, experts, weights, act, residual, out, out_dtype, preact, workspace, stream):
    n, k = experts.shape
    at = _Launch(stream, *_parts(w), X, experts, weights, residual, out, preact, workspace)
    Y = _out(at, out, out_dtype, n, w.K)
    ep = _EPILOGUE.pack(0, 0, _ptr(residual), _ptr(preact), 0 if residual is None else _ld(residual),
                        0 if preact is None else _ld(preact), act, 1, 1 if residual is None else _DTYPES[residual.dtype],
                        _DTYPES[Y.dtype])
    ws, size, keep = at.workspace(workspace, int(_call("nvfp4_moe_workspace_bytes")(n, k, w.E, w.F, w.K, preact is not None)))
    _run("nvfp4_moe", _struct(w), X.data_ptr(), _ld(X), experts.data_ptr(), weights.data_ptr(), n, k, Y.data_ptr(), _ld(Y), ep,
         ws, size, at.handle)
    return Y


def _moe_backward(wt, dY, experts, weights, preact, act, need_x, need_w, out, stream):
    dY = _incoming(dY, wt.K, "dY", stream)
    n, k = experts.shape
    at = _Launch(stream, *_parts(wt), dY, experts, weights, preact, out)
    dX = (at.alloc(n, wt.K, dtype=torch.bfloat16) if out is None else out) if need_x else None
    dw = at.alloc(n, k, dtype=torch.float32) if need_w else None
    ld, dtype, ptr = _ld(dY), _DTYPES[dY.dtype], dY.data_ptr()
    copy = dtype == 0 or ptr % 16 or (n > 1 and ld % 8)
    ws, size, keep = at.workspace(None, int(_call("nvfp4_moe_backward_workspace_bytes")(n, k, wt.E, wt.F, wt.K, need_x, 1 if copy else 0)))
    _run("nvfp4_moe_backward", _struct(wt), ptr, dtype, ld, experts.data_ptr(), weights.data_ptr(), preact.data_ptr(), _ld(preact),
         act, n, k, _ptr(dX), wt.K if dX is None else _ld(dX), _ptr(dw), ws, size, at.handle)
    return dX, dw


class _Moe(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, weights, residual, w, transposed, experts, act, out_dtype):
        ctx.transposed, ctx.act = transposed, act
        ctx.residual_dtype = None if residual is None else residual.dtype
        preact = None
        if ctx.needs_input_grad[0] or ctx.needs_input_grad[1]:
            preact = torch.empty(experts.numel(), 2 * w.F, dtype=torch.float32, device=X.device)
        ctx.save_for_backward(experts, weights, preact)
        return _moe_forward(w, X, experts, weights, act, residual, None, out_dtype, preact, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        experts, weights, preact = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        dX = dw = None
        if need_x or need_w:
            dX, dw = _moe_backward(ctx.transposed, dY, experts, weights, preact, ctx.act, need_x, need_w, None, None)
        return dX, dw, dY.to(ctx.residual_dtype) if need_r else None, None, None, None, None, None


def moe(w: ExpertWeights, X: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, activation: str = "silu",
        residual: torch.Tensor = None, *, transposed: TransposedExperts = None, out: torch.Tensor = None, out_dtype=None,
        preact: torch.Tensor = None, workspace: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Y[t] = sum_s weights[t, s] FFN(experts[t, s], X[t]) + residual[t], with
    FFN(e, x) = (act(x . Wg_e^T) * (x . Wu_e^T)) . Wd_e^T, for any number of tokens.

    X: bf16 [n, K], rows strided and 16-byte aligned; experts: int32 [n, k] (one
    outside [0, E) is no expert); weights: fp32 [n, k]; residual: bf16 or fp32
    [n, K] (it may be ``out`` itself); Y: bf16, or fp32 with ``out_dtype``.
    ``preact`` (fp32 [n k, 2 F]) receives what ``moe_backward`` needs.

    Between the two products act() * () is held to 16 significant bits up to 16
    tokens; beyond, where K is above 8192 or pre-activations are kept (``preact``,
    gradients), to 11 for a bf16 Y, and to 22, in a second down projection, for an
    fp32 one.

    ``workspace``: uint8, nvfp4_moe_workspace_bytes (allocated otherwise).
    Differentiable in X and weights (given ``transposed``) and the residual."""
    act = _act(activation)
    _weight(w, ExpertWeights)
    if transposed is not None:
        _weight(transposed, TransposedExperts, "transposed")
    _mat(X, (torch.bfloat16,), "X", None, w.K)
    n = X.shape[0]
    _pair_matrix(experts, torch.int32, "experts", n)
    k = _slots(experts.shape[1])
    _pair_matrix(weights, torch.float32, "weights", n, k)
    if residual is not None:
        _mat(residual, _FLOATS, "residual", n, w.K)
    if out is not None:
        _mat(out, _FLOATS, "out", n, w.K)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if preact is not None:
        _mat(preact, (torch.float32,), "preact", n * k, 2 * w.F)
    if _wants_grad(X, weights, residual):
        if out is not None or preact is not None or workspace is not None:
            raise ValueError("out, preact and workspace go with calls that need no gradient")
        if stream is not None and stream != torch.cuda.current_stream():
            raise ValueError("with gradients the launch stream is the current one (torch.cuda.stream)")
        if X.requires_grad or weights.requires_grad:
            if transposed is None:
                raise ValueError("a gradient of X or the weights needs the experts' transposed copies (transposed=w.transpose())")
            _check_transposed(transposed, w)
        return _Moe.apply(X, weights, residual, w, transposed, experts, act, out_dtype)
    if out is not None or preact is not None:
        _no_graph(out, preact)
        _written(out, preact)
    return _moe_forward(w, X, experts, weights, act, residual, out, out_dtype, preact, _workspace_arg(workspace), stream)


def moe_backward(wt: TransposedExperts, dY: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, preact: torch.Tensor,
                 activation: str = "silu", *, out: torch.Tensor = None, stream=None):
    """(dX bf16 [n, K], dweights fp32 [n, k]) of ``moe``, with ``preact`` as it
    filled it.  The residual's gradient is dY.  An fp32 dY has 16 significant bits
    in the products, for which one of them is made twice."""
    act = _act(activation)
    _weight(wt, TransposedExperts, "wt")
    _typed(dY, _FLOATS, "dY")
    if dY.dim() != 2:
        raise ValueError("dY must be [n, %d], got %s" % (wt.K, list(dY.shape)))
    n = dY.shape[0]
    _pair_matrix(experts, torch.int32, "experts", n)
    k = _slots(experts.shape[1])
    _pair_matrix(weights, torch.float32, "weights", n, k)
    _mat(preact, (torch.float32,), "preact", n * k, 2 * wt.F)
    if out is not None:
        _mat(out, (torch.bfloat16,), "out", n, wt.K)
    _no_graph(dY, weights, preact, out)
    _written(out)
    return _moe_backward(wt, dY, experts, weights, preact, act, True, True, out, stream)


def moe_geometry(n: int, k: int, E: int, F: int, K: int) -> tuple:
    """(weight rows, tokens of a workgroup) of the grouped products of ``moe`` for
    more than 16 tokens, or with pre-activations (nvfp4_moe_geometry)."""
    v = [_i32() for _ in range(2)]
    _run("nvfp4_moe_geometry", n, k, E, F, K, *(ctypes.byref(x) for x in v))
    return tuple(x.value for x in v)


def moe_decode_geometry(K: int, compute_units: int) -> int:
    """Outputs of a workgroup in the down projection of ``moe`` for up to 16 tokens on
    a device of so many compute units (nvfp4_moe_decode_geometry)."""
    v = _i32()
    _run("nvfp4_moe_decode_geometry", K, compute_units, ctypes.byref(v))
    return v.value


def moe_workspace_bytes(n: int, k: int, w: ExpertWeights, preact: bool = False) -> int:
    """Workspace bytes ``moe`` needs."""
    _weight(w, ExpertWeights)
    return int(_call("nvfp4_moe_workspace_bytes")(n, k, w.E, w.F, w.K, 1 if preact else 0))
