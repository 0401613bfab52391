"""The router, the expert layer and the 8-bit projection in 64 bits, with bounds
on what 32-bit sums and the roundings to bf16 may differ by (the steps of
fused_reference, whose terms these are)."""
import numpy as np

import fused_reference as R

STEP = R.HALF_F32


def route(logits, k, scoring, bias=None, normalize=True, scale=1.0):
    """(weights, bound, experts) of float64 logits [n, E]; -inf masks.

    A weight is a quotient of exponentials (or sigmoids) and a sum of them.  An
    exponential in fp32 is off by 2 steps of itself and by what its argument is off,
    a difference or a log sigmoid of fp32 numbers, each rounded twice: 4 steps of
    the largest magnitude in the row.  A sum of m terms adds (m / 2 + 8) steps in the wave's
    order (at most 16 in a lane, 6 across), the quotient and the scale 4."""
    n, E = logits.shape
    live = np.isfinite(logits) | np.isposinf(logits)
    l = np.where(live, logits, 0.0)
    if scoring == "softmax":
        top = np.where(live, l, -np.inf).max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        e = np.where(live, np.exp(l - top), 0.0)
        s = e.sum(1, keepdims=True)
        score = e / np.where(s > 0, s, 1.0)
    else:
        score = np.where(live, 1 / (1 + np.exp(-l)), 0.0)
    key = np.where(live, logits if bias is None else score + bias, -np.inf)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ok = np.take_along_axis(live, order, 1)
    w = np.where(ok, np.take_along_axis(score, order, 1), 0.0)
    if normalize:
        s = w.sum(1, keepdims=True)
        w = w / np.where(s > 0, s, 1.0)
    big = np.abs(l).max(1, keepdims=True)
    spread = 2 * big
    return w * scale, scale * w * STEP * (4 * big + 4 * spread + E / 2 + 48) + 2.0 ** -126, np.where(ok, order, -1)


def route_grad(logits, experts, dweights, scoring, normalize, scale):
    """(dlogits, bound): each factor of a gradient within the weights' relative
    bound, on the sum of the magnitudes of its terms."""
    n, E = logits.shape
    live = ~np.isneginf(logits)
    l = np.where(live, logits, 0.0)
    ok = experts >= 0
    idx = np.where(ok, experts, 0)
    dw = np.where(ok, dweights, 0.0)
    lc = np.take_along_axis(l, idx, 1)
    rel = STEP * (4 * 3 * np.abs(l).max(1, keepdims=True) + E / 2 + 48)
    if scoring == "softmax" and not normalize:
        top = np.where(live, l, -np.inf).max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        e = np.where(live, np.exp(l - top), 0.0)
        s = e.sum(1, keepdims=True)
        p = e / np.where(s > 0, s, 1.0)
        full = np.zeros_like(l)
        for j in range(idx.shape[1]):
            np.add.at(full, (np.arange(n), idx[:, j]), dw[:, j])
        dot, mag = (p * full).sum(1, keepdims=True), (p * np.abs(full)).sum(1, keepdims=True)
        return scale * p * (full - dot), 3 * rel * scale * p * (np.abs(full) + mag) + 2.0 ** -126
    sig = 1 / (1 + np.exp(-lc))
    if normalize:
        u = lc if scoring == "softmax" else np.where(lc > 0, 0, lc) - np.log1p(np.exp(-np.abs(lc)))
        u = np.where(ok, u, -np.inf)
        top = u.max(1, keepdims=True)
        e = np.exp(u - np.where(np.isfinite(top), top, 0.0))
        s = e.sum(1, keepdims=True)
        q = e / np.where(s > 0, s, 1.0)
        d, mag = q * (dw - (q * dw).sum(1, keepdims=True)), q * (np.abs(dw) + (q * np.abs(dw)).sum(1, keepdims=True))
    else:
        q = sig
        d, mag = q * dw, q * np.abs(dw)
    if scoring == "sigmoid":
        back = 1 / (1 + np.exp(lc))
        d, mag = d * back, mag * back
    out, bound = np.zeros_like(l), np.zeros_like(l)
    for j in range(idx.shape[1]):
        np.add.at(out, (np.arange(n), idx[:, j]), np.where(ok, d, 0.0)[:, j])
        np.add.at(bound, (np.arange(n), idx[:, j]), np.where(ok, mag, 0.0)[:, j])
    return scale * out, 3 * rel * scale * bound + 2.0 ** -126


def _live(experts, E):
    return (experts >= 0) & (experts < E)


def _kept(v, e):
    """Bound of rows v, known within e, as operands of the next product: fp16 numbers
    with an exponent for each 64 (half of a step of 2^-10: 2^-11 relative), whose
    largest is between 2^14 and 2^15.  A block's numbers are scaled by a power of two
    to the row's exponent, and lost where it is below 2^-24: numbers below 2^15 2^-25,
    against 2^14 at least of the row's largest."""
    a = np.abs(v) + e
    return e + 2.0 ** -11 * a + 2.0 ** -24 * a.max(1, keepdims=True)


def kept_in_bf16_parts(v, e):
    """Two bf16 parts of a value (16 bits): half a step, 2^-8 relative, of what half a
    step of the value left."""
    return e + 2.0 ** -16 * (np.abs(v) + e)


def kept_in_fp16_parts(v, e):
    """_kept, and a second fp16 number of what the first one left, 2^11 times it: 2^-11
    of 2^-11 relative.  (Below fp16's normal numbers half a step is 2^-25, 2^-39 of
    the block's largest, and the second part's 2^-36 2^-14; the row's last term covers
    both, as it covers blocks that are lost.)"""
    a = np.abs(v) + e
    return e + 2.0 ** -22 * a + 2.0 ** -24 * a.max(1, keepdims=True)


def moe(X, Wg, Wu, Wd, experts, weights, kind="silu", residual=None, out_f32=False, kept=_kept):
    """(Y, bound): h kept to 11 bits (_kept) or as `kept` says and its down projection,
    k weighted terms (a weight is multiplied by the tensor scale first: 3 steps), the
    residual, the last rounding."""
    n, k = experts.shape
    F, K = Wg.shape[1:]
    y, b, m = np.zeros((n, K)), np.zeros((n, K)), np.zeros((n, K))
    ok = _live(experts, len(Wg))
    for e in range(len(Wg)):
        t, s = np.nonzero(ok & (experts == e))
        if not len(t):
            continue
        h, eh = R.gated(X[t], Wg[e], Wu[e], kind=kind, out_f32=True)
        eh = kept(h, eh)
        o = h @ Wd[e].T
        eo = eh @ np.abs(Wd[e]).T + (F + 32) * STEP * ((np.abs(h) + eh) @ np.abs(Wd[e]).T)
        w = weights[t, s][:, None]
        np.add.at(y, t, w * o)
        np.add.at(b, t, np.abs(w) * eo)
        np.add.at(m, t, np.abs(w) * (np.abs(o) + eo))
    b = b + (k + 4) * STEP * m
    if residual is not None:
        y = y + residual
        b = b + STEP * np.abs(y)
    return y, b + R.half(out_f32) * (np.abs(y) + b) + 2.0 ** -133


def moe_grads(X, Wg, Wu, Wd, experts, weights, dY, kind="silu", dy_f32=False, dy_step=R.HALF_BF16):
    """((dX, bound), (dweights, bound)); an fp32 dY is an operand within dy_step of its
    value."""
    n, k = experts.shape
    F, K = Wg.shape[1:]
    dx, bx, mx = np.zeros((n, K)), np.zeros((n, K)), np.zeros((n, K))
    dw, bw = np.zeros((n, k)), np.zeros((n, k))
    ok = _live(experts, len(Wg))
    for e in range(len(Wg)):
        t, s = np.nonzero(ok & (experts == e))
        if not len(t):
            continue
        g, eg = R.pre(X[t], Wg[e])
        u, eu = R.pre(X[t], Wu[e])
        rg, ru = eg + STEP * (np.abs(g) + eg), eu + STEP * (np.abs(u) + eu)     # as stored
        a, ea = R._activated(g, rg, kind)
        d, ed = R._grad_parts(g, eg, kind)
        dh = dY[t] @ Wd[e]
        mag = np.abs(dY[t]) @ np.abs(Wd[e])
        eh = (K + 33) * STEP * mag + (dy_step * mag if dy_f32 else 0.0)
        h = a * u
        ehh = np.abs(a) * ru + np.abs(u) * ea + ea * ru + STEP * np.abs(h)
        dw[t, s] = (dh * h).sum(1)
        terms = (np.abs(dh) + eh) * (np.abs(h) + ehh)
        bw[t, s] = (np.abs(dh) * ehh + eh * np.abs(h) + eh * ehh).sum(1) + (F + 32) * STEP * terms.sum(1)
        w = np.abs(weights[t, s])[:, None]
        dG, dU = weights[t, s][:, None] * dh * u * d, weights[t, s][:, None] * dh * a
        eG = w * (eh * np.abs(u * d) + (np.abs(dh) + eh) * (np.abs(u) * ed + ru * np.abs(d) + ru * ed)) + 6 * STEP * np.abs(dG)
        eU = w * (eh * np.abs(a) + (np.abs(dh) + eh) * ea) + 6 * STEP * np.abs(dU)
        kept = _kept(np.hstack((dG, dU)), np.hstack((eG, eU)))
        F = dG.shape[1]
        for v, ev, W in ((dG, kept[:, :F], Wg[e]), (dU, kept[:, F:], Wu[e])):
            p = (np.abs(v) + ev) @ np.abs(W)
            np.add.at(dx, t, v @ W)
            np.add.at(bx, t, ev @ np.abs(W) + (2 * F + 32) * STEP * p)
            np.add.at(mx, t, p)
    bx = bx + (k + 4) * STEP * mx
    return (dx, bx + R.HALF_BF16 * (np.abs(dx) + bx) + 2.0 ** -133), (dw, bw + 2.0 ** -126)


def int8_quantize(X, f32=False):
    """(q, scale) as defined: in exact arithmetic for bf16 values (a half-integer
    quotient is representable, and no other lies within 2^-17 of one), with each
    operation rounded to fp32 otherwise."""
    top = np.abs(X).max(1)
    div = np.where(top > 0, top, 1.0)[:, None]
    if f32:
        with np.errstate(over="ignore"):
            q = np.rint((np.float32(127) * X.astype(np.float32)).astype(np.float32) / div.astype(np.float32))
    else:
        q = np.rint(127 * X / div)
    return q.astype(np.int64), (top.astype(np.float32) / np.float32(127)).astype(np.float64)


def int8_linear(q, scale, wq, wscale, bias=None, kind="none", residual=None, out_f32=False):
    """(Y, bound): the integer sum is exact; its conversion and the two scales are
    three roundings, bias and residual one each."""
    z = (q @ wq.T).astype(np.float64) * scale[:, None] * wscale[None, :]
    e = 3 * STEP * np.abs(z)
    if bias is not None:
        z = z + bias
        e = e + STEP * np.abs(z)
    y, e = R._activated(z, e, kind)
    if residual is not None:
        y = y + residual
        e = e + STEP * np.abs(y)
    return y, e + R.half(out_f32) * (np.abs(y) + e) + 2.0 ** -126
