"""The fused operators in 64 bits, with bounds on what 32-bit sums and the
roundings to bf16 may differ by.

A sum of m fp32 products in any order is off by at most about m 2^-24 times the
sum of the magnitudes; a rounding to bf16 by 2^-8 of the value, to fp32 by
2^-24 (half a step each).  An error e of a pre-activation moves act(z) by at
most LIP e and act'(z) by at most LIP2 e; the activations themselves are
evaluated in fp32 from an exponential with a relative error of a few 2^-23 and
a reciprocal within one step, which ACT_EPS (1 + |value|) covers.
"""
import numpy as np
from scipy import special

LIP = 1.13       # max |act'|: gelu 1.129, gelu_tanh 1.13, silu 1.1
LIP2 = 1.0       # max |act''|: gelu 0.80, gelu_tanh 0.81, silu 0.5
ACT_EPS = 2.0 ** -20
HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_C = np.sqrt(2 / np.pi)


def act(z, kind):
    if kind == "relu":
        return np.maximum(z, 0)
    if kind == "silu":
        return z * special.expit(z)
    if kind == "gelu":
        return 0.5 * z * special.erfc(-z / np.sqrt(2))
    if kind == "gelu_tanh":
        return z * special.expit(2 * _C * (z + 0.044715 * z ** 3))
    return z


def act_grad(z, kind):
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "silu":
        s = special.expit(z)
        return s * (1 + z * (1 - s))
    if kind == "gelu":
        return 0.5 * special.erfc(-z / np.sqrt(2)) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if kind == "gelu_tanh":
        u = 2 * _C * (z + 0.044715 * z ** 3)
        s = special.expit(u)
        return s + z * s * (1 - s) * 2 * _C * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def half(f32):
    return HALF_F32 if f32 else HALF_BF16


def pre(X, W, bias=None):
    """Pre-activations and their fp32 error bound; W [N, K] with its tensor scale."""
    z = X @ W.T
    mag = np.abs(X) @ np.abs(W).T
    if bias is not None:
        z = z + bias
        mag = mag + np.abs(bias)
    return z, (X.shape[1] + 32) * HALF_F32 * mag


def _activated(z, ez, kind):
    a = act(z, kind)
    lip = 1.0 if kind in ("none", "relu") else LIP
    eps = 0.0 if kind in ("none", "relu") else ACT_EPS * (1 + np.abs(a))
    return a, lip * ez + eps


def linear(X, W, bias=None, kind="none", residual=None, out_f32=False):
    """(Y, bound)"""
    z, ez = pre(X, W, bias)
    y, e = _activated(z, ez, kind)
    if residual is not None:
        y = y + residual
        e = e + HALF_F32 * np.abs(y)
    return y, e + half(out_f32) * (np.abs(y) + e) + 2.0 ** -133


def gated(X, Wg, Wu, bg=None, bu=None, kind="silu", out_f32=False):
    g, eg = pre(X, Wg, bg)
    u, eu = pre(X, Wu, bu)
    a, ea = _activated(g, eg, kind)
    h = a * u
    e = np.abs(a) * eu + np.abs(u) * ea + ea * eu + HALF_F32 * np.abs(h)
    return h, e + half(out_f32) * (np.abs(h) + e) + 2.0 ** -133


def _grad_parts(z, ez, kind):
    """act'(z) and its bound when z is known within ez and stored in fp32."""
    d = act_grad(z, kind)
    e = ez + HALF_F32 * (np.abs(z) + ez)
    if kind == "none":
        return d, np.zeros_like(d)
    if kind == "relu":
        return d, (np.abs(z) <= e).astype(np.float64)
    return d, LIP2 * e + 4 * ACT_EPS * (1 + np.abs(z))


def product_t(dZ, e, W):
    """dZ . W for dZ known within e (before its rounding to bf16): (dX, bound)."""
    dX = dZ @ W
    N = W.shape[0]
    e = e + HALF_BF16 * (np.abs(dZ) + e)
    b = e @ np.abs(W) + (N + 32) * HALF_F32 * ((np.abs(dZ) + e) @ np.abs(W))
    return dX, b + HALF_BF16 * (np.abs(dX) + b) + 2.0 ** -133


def column_sum(d, e, f32):
    s = d.sum(0)
    b = e.sum(0) + (d.shape[0] + 32) * HALF_F32 * (np.abs(d) + e).sum(0)
    return s, b + half(f32) * (np.abs(s) + b) + 2.0 ** -133


def linear_grads(X, W, dY, bias=None, kind="none", bias_f32=False):
    """((dX, bound), (dbias, bound))"""
    z, ez = pre(X, W, bias)
    d, ed = _grad_parts(z, ez, kind)
    dZ, e = dY * d, np.abs(dY) * ed + HALF_F32 * np.abs(dY * d)
    return product_t(dZ, e, W), column_sum(dZ, e, bias_f32)


def gated_grads(X, Wg, Wu, dH, bg=None, bu=None, kind="silu", bias_f32=False):
    """((dX, bound), (dbg, bound), (dbu, bound))"""
    g, eg = pre(X, Wg, bg)
    u, eu = pre(X, Wu, bu)
    d, ed = _grad_parts(g, eg, kind)
    rg = eg + HALF_F32 * (np.abs(g) + eg)      # the stored pre-activations
    ru = eu + HALF_F32 * (np.abs(u) + eu)
    a, ea = _activated(g, rg, kind)
    dG, dU = dH * u * d, dH * a
    eG = np.abs(dH) * (np.abs(u) * ed + ru * np.abs(d) + ru * ed) + 3 * HALF_F32 * np.abs(dG)
    eU = np.abs(dH) * ea + 3 * HALF_F32 * np.abs(dU)
    (x0, b0), (x1, b1) = product_t(dG, eG, Wg), product_t(dU, eU, Wu)
    # one sum and one rounding for both products: the two bounds cover them
    return (x0 + x1, b0 + b1), column_sum(dG, eG, bias_f32), column_sum(dU, eU, bias_f32)
