"""Projection in 8-bit integers, for layers that do not stand four bits: the
weight with a scale for each channel, the activations with one for each token.

    w = Int8Weight.from_float(W)                       # or from_int8(codes, scale)
    y = int8_linear(w, X, bias=b, activation="silu")   # X bf16, quantised in the call
    q, s = int8_quantize(X)                            # once, for several projections
    y = int8_linear(w, q, s)

There are no gradients: rounding to integers has none.  Streams, memory and
refusals as in ``fused.py``.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import Nvfp4Error, _dev, _i32, _i64, _vp, lib
from .fused import (_DTYPES, _EPILOGUE, _FLOATS, _SIZE, _act, _Launch, _ld, _mat, _no_graph, _out, _ptr, _typed, _vec, _weight,
                    _workspace_arg, _written)

_SIGNATURES = {
    "nvfp4_int8_packed_bytes": (_SIZE, [_i32, _i32]),
    "nvfp4_int8_pack": (_i32, [_vp, _i32, _i32, _vp, _vp]),
    "nvfp4_int8_quantize": (_i32, [_vp, _i32, _i64, _i32, _i32, _vp, _i64, _vp, _vp]),
    "nvfp4_int8_linear": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _SIZE, _vp]),
    "nvfp4_int8_linear_workspace_bytes": (_SIZE, [_i32] * 4),
    "nvfp4_int8_geometry": (_i32, [_i32, _i32, _i32] + [ctypes.POINTER(_i32)] * 4),
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


@dataclass
class Int8Weight:
    """An N x K weight in 8-bit integers: packed codes, a scale for each row."""
    codes: torch.Tensor      # int8, nvfp4_int8_packed_bytes(N, K)
    scale: torch.Tensor      # fp32 [N]
    N: int
    K: int

    @classmethod
    def from_int8(cls, codes: torch.Tensor, scale: torch.Tensor, stream=None) -> "Int8Weight":
        """From int8 codes [N, K] and fp32 scales [N]: the weight codes * scale.  Both
        are copied."""
        _dev(codes, torch.int8, "codes")
        if codes.dim() != 2:
            raise ValueError("codes must be [N, K], got %s" % list(codes.shape))
        N, K = codes.shape
        _vec(scale, (torch.float32,), "scale", N)
        _no_graph(scale)
        size = cls._sizes(N, K)
        at = _Launch(stream, codes, scale)
        packed = at.alloc(size, dtype=torch.int8)
        _run("nvfp4_int8_pack", codes.data_ptr(), N, K, packed.data_ptr(), at.handle)
        own = at.alloc(N, dtype=torch.float32)
        with torch.cuda.stream(at.stream):       # (of None: the current one)
            own.copy_(scale.detach())
        return cls(packed, own, N, K)

    @staticmethod
    def _sizes(N, K) -> int:
        """Bytes of the packed codes."""
        size = int(_call("nvfp4_int8_packed_bytes")(N, K)) if N < 1 << 31 and K < 1 << 31 else 0
        if not size:
            raise ValueError("N must be 1 to 2^30 and K a multiple of 16 from 16 to 131056, got %d x %d" % (N, K))
        return size

    @classmethod
    def from_float(cls, W: torch.Tensor, stream=None) -> "Int8Weight":
        """Quantise an fp32 or bf16 weight [N, K], each row as ``int8_quantize`` does."""
        _typed(W, _FLOATS, "W")
        if W.dim() != 2:
            raise ValueError("W must be [N, K], got %s" % list(W.shape))
        cls._sizes(*W.shape)
        q, scale = int8_quantize(W, stream=stream)
        return cls.from_int8(q, scale, stream)


def int8_quantize(X: torch.Tensor, *, stream=None):
    """(q int8 [n, K], scale fp32 [n]) of a bf16 or fp32 matrix: scale = amax / 127,
    q = 127 x / amax to the nearest integer, halves to the even one.  K is a
    multiple of 16, rows may be strided and are 16-byte aligned.  A row of zeros has
    scale 0, one with a NaN or an infinity scale NaN and q 0."""
    _typed(X, _FLOATS, "X")
    if X.dim() != 2:
        raise ValueError("X must be [n, K], got %s" % list(X.shape))
    _mat(X, _FLOATS, "X", None, X.shape[1])
    _no_graph(X)
    n, K = X.shape
    at = _Launch(stream, X)
    q = at.alloc(n, K, dtype=torch.int8)
    scale = at.alloc(n, dtype=torch.float32)
    _run("nvfp4_int8_quantize", X.data_ptr(), _DTYPES[X.dtype], _ld(X), n, K, q.data_ptr(), K, scale.data_ptr(), at.handle)
    return q, scale


def int8_linear(w: Int8Weight, X: torch.Tensor, scale: torch.Tensor = None, bias: torch.Tensor = None, activation: str = None,
                residual: torch.Tensor = None, *, out: torch.Tensor = None, out_dtype=None, workspace: torch.Tensor = None,
                stream=None) -> torch.Tensor:
    """Y = act(X . W^T + bias) + residual for any number of tokens, the product in
    8-bit integers with exact sums.

    X: bf16 [n, K], quantised in the call as by ``int8_quantize``, or int8 [n, K]
    with ``scale`` (fp32 [n]); rows may be strided and are 16-byte aligned.  bias:
    bf16 or fp32 [N]; residual: bf16 or fp32 [n, N] (it may be ``out`` itself); Y:
    bf16, or fp32 with ``out_dtype``.  ``workspace``: uint8,
    nvfp4_int8_linear_workspace_bytes (allocated otherwise)."""
    act = _act(activation)
    _weight(w, Int8Weight)
    _mat(X, (torch.bfloat16,) if scale is None else (torch.int8,), "X", None, w.K)
    n = X.shape[0]
    if scale is not None:
        _vec(scale, (torch.float32,), "scale", n)
    if bias is not None:
        _vec(bias, _FLOATS, "bias", w.N)
    if residual is not None:
        _mat(residual, _FLOATS, "residual", n, w.N)
    if out is not None:
        _mat(out, _FLOATS, "out", n, w.N)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    _no_graph(X, scale, bias, residual, out, w.scale)
    workspace = _workspace_arg(workspace)
    at = _Launch(stream, w.codes, w.scale, X, scale, bias, residual, out, workspace)
    Y = _out(at, out, out_dtype, n, w.N)
    if out is not None:
        _written(out)
    ep = _EPILOGUE.pack(_ptr(bias), 0, _ptr(residual), 0, 0 if residual is None else _ld(residual), 0, act,
                        1 if bias is None else _DTYPES[bias.dtype], 1 if residual is None else _DTYPES[residual.dtype],
                        _DTYPES[Y.dtype])
    ws, size, keep = at.workspace(workspace, int(_call("nvfp4_int8_linear_workspace_bytes")(n, w.N, w.K, scale is None)))
    _run("nvfp4_int8_linear", w.codes.data_ptr(), w.scale.data_ptr(), X.data_ptr(), _ld(X), _ptr(scale), Y.data_ptr(), _ld(Y), n,
         w.N, w.K, ep, ws, size, at.handle)
    return Y


def int8_geometry(n: int, N: int, K: int) -> tuple:
    """(weight rows, tokens of a workgroup, K groups in it, K parts) that
    ``int8_linear`` takes for n > 16 tokens (nvfp4_int8_geometry)."""
    v = [_i32() for _ in range(4)]
    _run("nvfp4_int8_geometry", n, N, K, *(ctypes.byref(x) for x in v))
    return tuple(x.value for x in v)


def int8_linear_workspace_bytes(n: int, N: int, K: int, quantize: bool = True) -> int:
    """Workspace bytes ``int8_linear`` needs; quantize: X is bf16."""
    return int(_call("nvfp4_int8_linear_workspace_bytes")(n, N, K, 1 if quantize else 0))
