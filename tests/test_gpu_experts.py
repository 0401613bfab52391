"""GPU parity of the router and the expert layer, with their gradients, against
64-bit arithmetic, through the Python entry points, within the bounds of
experts_reference."""
import copy
import gc

import numpy as np
import pytest
import torch

import experts_reference as X8
import fused_reference as R
import nvfp4_weight_only_02_amd as nv
import oracle as O
from nvfp4_weight_only_02_amd import experts, inputs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    nv.lib()
    yield
    torch.cuda.synchronize()


def say(*a):
    print(*a, flush=True)


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(shape, seed, dtype=BF16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def check(got, want, what):
    ref, bound = want
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all(), what
    assert (err <= bound).all(), "%s: worst err/bound %.3g" % (what, float((err / bound).max()))


def weights(E, F, K, seed=1, std=0.05):
    """(ExpertWeights, [E, F, K], [E, F, K], [E, K, F] in 64 bits)"""
    packed, dense = ([], [], []), ([], [], [])
    for e in range(E):
        for j, (N, C) in enumerate(((F, K), (F, K), (K, F))):
            codes, scales, g = O.quantize(inputs.weights_f32(N, C, seed + 3 * e + j, std))
            packed[j].append(nv.PackedWeight.from_canonical(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(),
                                                            g, N, C))
            dense[j].append(np.asarray(O.dequant(codes, scales, g), dtype=np.float64))
    return (nv.ExpertWeights.from_packed(*packed),) + tuple(np.stack(d) for d in dense)


def choices(n, k, E, seed, empty=0.0):
    rng = np.random.default_rng(seed)
    p = rng.random(E) + 0.2
    ids = np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(n)]) if n else np.zeros((0, k), int)
    ids = np.where(rng.random((n, k)) < empty, -1, ids)
    w = rng.random((n, k)) + 0.1
    return torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(w.astype(np.float32)).cuda()


# ---- router ------------------------------------------------------------------------

def logits_of(n, E, seed, dtype=F32, masked=0.0):
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((n, E)) * 2
    l[rng.random((n, E)) < masked] = -np.inf
    return torch.from_numpy(l.astype(np.float32)).to(dtype).cuda()


@pytest.mark.parametrize("n,E,k", [(1, 1, 1), (1, 64, 8), (5, 3, 3), (16, 65, 6), (33, 128, 1), (7, 130, 32), (300, 256, 8),
                                   (9, 513, 5), (3, 1024, 32), (0, 8, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias,normalize,scale,dtype,masked", [
    (False, True, 1.0, F32, 0.0), (True, True, 2.5, F32, 0.3), (False, False, 1.0, BF16, 0.3), (True, False, 0.5, BF16, 0.0)])
def test_route(n, E, k, scoring, bias, normalize, scale, dtype, masked):
    say("route", n, E, k, scoring, bias, normalize, scale, dtype, masked)
    l = logits_of(n, E, E + n, dtype, masked)
    b = randn((E,), 5, F32, 0.2) if bias else None
    w, e = nv.moe_route(l, k, scoring, b, normalize, scale)
    assert w.dtype == F32 and e.dtype == torch.int32 and w.shape == e.shape == (n, k)
    if n == 0:
        return
    rw, bound, re = X8.route(f64(l), k, scoring, None if b is None else f64(b), normalize, scale)
    assert np.array_equal(e.cpu().numpy(), re)
    check(w, (rw, bound), "weights")
    dw = randn((n, k), 6, F32)
    dl = nv.moe_route_backward(l, e, dw, scoring, normalize, scale)
    assert dl.dtype == dtype
    ref, db = X8.route_grad(f64(l), re, f64(dw), scoring, normalize, scale)
    check(dl, (ref, db + R.half(dtype == F32) * (np.abs(ref) + db)), "dlogits")
    leaf = l.clone().requires_grad_()
    (auto,) = torch.autograd.grad(nv.moe_route(leaf, k, scoring, b, normalize, scale)[0], leaf, dw)
    assert torch.equal(auto, dl)


def test_route_ties_zeros_and_strides():
    say("route ties")
    l = torch.zeros(4, 100, device="cuda")
    l[1, 50:] = -0.0                  # the zeros are alike
    l[2, 7] = l[2, 93] = 1.0
    l[3] = -INF
    l[3, 64] = -500.0
    w, e = nv.moe_route(l, 3)
    assert e.tolist() == [[0, 1, 2], [0, 1, 2], [7, 93, 0], [64, -1, -1]]
    assert w[3].tolist() == [1.0, 0.0, 0.0]
    for scoring in ("softmax", "sigmoid"):
        assert nv.moe_route(l, 3, scoring, bias=torch.zeros(100, device="cuda"))[1][:3].tolist() == e[:3].tolist()
    # bf16 rows are full of ties
    b = logits_of(50, 300, 3, BF16)
    assert np.array_equal(nv.moe_route(b, 8)[1].cpu().numpy(), X8.route(f64(b), 8, "softmax")[2])
    wide = torch.full((9, 200), 77.0, device="cuda")
    wide[:, 20:120] = logits_of(9, 100, 4)
    part = wide[:, 20:120]
    for x, y in zip(nv.moe_route(part, 5), nv.moe_route(part.contiguous(), 5)):
        assert torch.equal(x, y)
    dw = randn((9, 5), 8, F32)
    e = nv.moe_route(part, 5)[1]
    assert torch.equal(nv.moe_route_backward(part, e, dw), nv.moe_route_backward(part.contiguous(), e, dw))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_extremes(scoring, normalize):
    """Empty rows, NaN, infinities and logits whose scores underflow."""
    say("route extremes", scoring, normalize)
    l = logits_of(6, 70, 9)
    l[1] = -INF
    l[2, 33] = NAN
    l[3] = -INF
    l[3, 5], l[3, 69] = -300.0, -301.0
    l[4, 10] = 3e38
    w, e = nv.moe_route(l, 4, scoring, normalize=normalize)
    assert e[1].tolist() == [-1] * 4 and w[1].tolist() == [0.0] * 4
    assert e[2, 0] == 33 and torch.isnan(w[2, 0]) and (normalize or scoring == "sigmoid" or torch.isnan(w[2]).all())
    assert e[3].tolist() == [5, 69, -1, -1]
    if normalize or scoring == "softmax":
        # both exponents are exact: 1 / (1 + 1/e)
        q = 1 / (1 + np.exp(-1.0))
        assert np.allclose(f64(w[3]), [q, 1 - q, 0, 0], rtol=1e-6, atol=0)
    # the sigmoid is 1 there, and so is the softmax; normalized sigmoids share it with the other three
    assert e[4, 0] == 10 and (w[4, 0] == 1.0 or (normalize and scoring == "sigmoid" and 0.25 <= w[4, 0] < 1))
    keep = [0, 5]
    clean = nv.moe_route(l[keep].contiguous(), 4, scoring, normalize=normalize)
    assert torch.equal(w[keep], clean[0]) and torch.equal(e[keep], clean[1])
    dl = nv.moe_route_backward(l, e, torch.ones_like(w), scoring, normalize)
    assert (dl[1] == 0).all() and torch.isfinite(dl[[0, 1, 3, 4, 5]]).all() and torch.isnan(dl[2]).any()
    assert torch.isfinite(dl[3]).all() and (dl[3, 6:69] == 0).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_against_differences(scoring, normalize):
    """Central differences of the 64-bit form with the experts held: off by t^2 / 6
    of the third derivative (below 2 for a sum of two scores' products) and
    2^-50 / t, far below the fp32 bound asked for."""
    say("route differences", scoring, normalize)
    n, E, k = 4, 20, 5
    l = logits_of(n, E, 12)
    w, e = nv.moe_route(l, k, scoring, None, normalize, 1.5)
    dw = randn((n, k), 13, F32)
    dl = f64(nv.moe_route_backward(l, e, dw, scoring, normalize, 1.5))
    ids = e.cpu().numpy()

    def f(x):
        p = np.exp(x - x.max(1, keepdims=True))
        p = p / p.sum(1, keepdims=True) if scoring == "softmax" else 1 / (1 + np.exp(-x))
        q = np.take_along_axis(p, ids, 1)
        return (1.5 * (q / q.sum(1, keepdims=True) if normalize else q) * f64(dw)).sum()
    x, t = f64(l), 1e-5
    for i in range(n):
        for j in range(E):
            d = np.zeros_like(x)
            d[i, j] = t
            assert abs((f(x + d) - f(x - d)) / (2 * t) - dl[i, j]) <= 1e-5


# ---- the layer ------------------------------------------------------------------------

SHAPES = [(1, 16, 16, 1), (5, 48, 144, 2), (13, 400, 656, 3), (70, 144, 272, 8), (4, 272, 2064, 4)]


@pytest.mark.parametrize("E,F,K,k", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 4, 5, 9, 16, 17, 40, 150])
@pytest.mark.parametrize("act,residual,out,empty", [("silu", None, BF16, 0.0), ("gelu", F32, F32, 0.4),
                                                    ("gelu_tanh", BF16, BF16, 0.0), ("relu", F32, BF16, 0.9)])
def test_moe(n, E, F, K, k, act, residual, out, empty):
    say("moe", n, E, F, K, k, act, residual, out, empty)
    w, Wg, Wu, Wd = weights(E, F, K)
    X = randn((n, K), 2)
    e, c = choices(n, k, E, n + E, empty)
    r = None if residual is None else randn((n, K), 4, residual, 2.0)
    Y = nv.moe(w, X, e, c, act, r, out_dtype=out)
    assert Y.dtype == out
    check(Y, X8.moe(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c), act, None if r is None else f64(r), out == F32), "Y")


@pytest.mark.parametrize("n,E,F,K,k,tile", [(60, 6, 80, 144, 2, (128, 32)), (450, 8, 2576, 144, 1, (128, 64)),
                                            (800, 2, 2064, 144, 1, (256, 64))])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_every_tile_of_the_grouped_products(n, E, F, K, k, tile, act):
    say("moe tile", n, E, F, K, k, tile, act)
    assert nv.moe_geometry(n, k, E, F, K) == tile
    w, Wg, Wu, Wd = weights(E, F, K, 60)
    X = randn((n, K), 61).requires_grad_()
    e, c = choices(n, k, E, 62)
    c.requires_grad_()
    dY = randn((n, K), 63, BF16, 0.1)
    Y = nv.moe(w, X, e, c, act, transposed=w.transpose())
    args = (f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c))
    check(Y, X8.moe(*args, act), "Y")
    dX, dc = torch.autograd.grad(Y, [X, c], dY)
    x, d = X8.moe_grads(*args, f64(dY), act)
    check(dX, x, "dX")
    check(dc, d, "dweights")


@pytest.mark.parametrize("n", [9, 40])
def test_values_between_the_products_of_any_size(n):
    """Rows of h from 2^-60 to 2^60, whose columns spread over another 2^32: what is
    kept of a value depends on its own row alone."""
    say("moe sizes", n)
    E, F, K, k = 3, 208, 144, 2
    g = torch.Generator(device="cuda").manual_seed(70)
    spread = 2.0 ** torch.randint(-8, 9, (E, F, 1), generator=g, device="cuda").float()
    packed, dense = ([], [], []), ([], [], [])
    for j, (N, C, m) in enumerate(((F, K, spread), (F, K, spread), (K, F, torch.ones(E, K, 1, device="cuda")))):
        W = torch.randn(E, N, C, generator=g, device="cuda") * 0.1
        for i in range(E):
            codes, scales, t = O.quantize((W[i] * m[i]).cpu().numpy())
            packed[j].append(nv.PackedWeight.from_canonical(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), t, N, C))
            dense[j].append(np.asarray(O.dequant(codes, scales, t), dtype=np.float64))
    w, (Wg, Wu, Wd) = nv.ExpertWeights.from_packed(*packed), (np.stack(d) for d in dense)
    X = (randn((n, K), 71, F32) * 2.0 ** torch.linspace(-30, 30, n, device="cuda").round()[:, None]).to(BF16).requires_grad_()
    e, c = choices(n, k, E, 72)
    c.requires_grad_()
    dY = (randn((n, K), 73, F32) * 2.0 ** torch.linspace(20, -20, n, device="cuda").round()[:, None]).to(BF16)
    args = (f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c))
    with torch.no_grad():
        check(nv.moe(w, X, e, c, "none"), X8.moe(*args, "none"), "Y")
    Y = nv.moe(w, X, e, c, "none", transposed=w.transpose())
    check(Y, X8.moe(*args, "none"), "Y")
    dX, dc = torch.autograd.grad(Y, [X, c], dY)
    x, d = X8.moe_grads(*args, f64(dY), "none")
    check(dX, x, "dX")
    check(dc, d, "dweights")


@pytest.mark.parametrize("E,F,K,k", [(5, 16, 32, 2), (13, 48, 144, 3), (70, 16, 80, 8)])
@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("n", [1, 5, 16, 17, 40, 150, 900])
def test_bits_of_fp32_results(n, E, F, K, k, act):
    """Where the result is fp32, h is held to 16 bits up to 16 tokens and to 22
    beyond (or with pre-activations): sums short enough to show a lost bit."""
    say("moe bits", n, E, F, K, k, act)
    w, Wg, Wu, Wd = weights(E, F, K, 320)
    X = randn((n, K), 321)
    e, c = choices(n, k, E, 322)
    args = f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c), act, None, True
    Y = nv.moe(w, X, e, c, act, out_dtype=F32)
    check(Y, X8.moe(*args, kept=X8.kept_in_bf16_parts if n <= 16 else X8.kept_in_fp16_parts), "Y")
    Y = nv.moe(w, X, e, c, act, out_dtype=F32, preact=torch.empty(n * k, 2 * F, device="cuda"))
    check(Y, X8.moe(*args, kept=X8.kept_in_fp16_parts), "Y with preact")


def test_bits_of_values_of_any_size():
    """Columns of h over 2^40, blocks of zeros, and beside them a token with an infinity:
    the second parts have the first ones' exponents and change nothing there."""
    say("moe bits, sizes")
    E, F, K, k, n = 3, 208, 32, 2, 40
    g = torch.Generator(device="cuda").manual_seed(330)
    spread = 2.0 ** torch.randint(-10, 11, (E, F, 1), generator=g, device="cuda").float()
    spread[:, 64:128] = 0
    packed, dense = ([], [], []), ([], [], [])
    for j, (N, C, m) in enumerate(((F, K, spread), (F, K, spread), (K, F, torch.ones(E, K, 1, device="cuda")))):
        W = torch.randn(E, N, C, generator=g, device="cuda") * 0.1
        for i in range(E):
            codes, scales, t = O.quantize((W[i] * m[i]).cpu().numpy())
            packed[j].append(nv.PackedWeight.from_canonical(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), t, N, C))
            dense[j].append(np.asarray(O.dequant(codes, scales, t), dtype=np.float64))
    w, (Wg, Wu, Wd) = nv.ExpertWeights.from_packed(*packed), (np.stack(d) for d in dense)
    X = (randn((n, K), 331, F32) * 2.0 ** torch.linspace(-20, 20, n, device="cuda").round()[:, None]).to(BF16)
    e, c = choices(n, k, E, 332)
    Y = nv.moe(w, X, e, c, "none", out_dtype=F32)
    check(Y, X8.moe(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c), "none", None, True, kept=X8.kept_in_fp16_parts), "Y")
    X[3] = 2.0 ** 66                       # h is infinite in most columns
    X[5] = 0
    got, low = nv.moe(w, X, e, c, "none", out_dtype=F32), nv.moe(w, X, e, c, "none")
    keep = [t for t in range(n) if t not in (3, 5)]
    assert torch.equal(got[keep], Y[keep]) and (got[5] == 0).all()
    assert torch.equal(torch.isnan(got[3]), torch.isnan(low[3])) and torch.equal(torch.isinf(got[3]), torch.isinf(low[3]))


@pytest.mark.parametrize("n", [3, 50, 300])
def test_bits_of_fp32_dy(n):
    """dweights of an fp32 dY, which enters the product in two bf16 parts."""
    say("moe bits, dY", n)
    E, F, K, k = 5, 48, 32, 2
    w, Wg, Wu, Wd = weights(E, F, K, 340)
    wt = w.transpose()
    X, (e, c) = randn((n, K), 341), choices(n, k, E, 342, 0.2)
    pre = torch.zeros(n * k, 2 * F, device="cuda")
    nv.moe(w, X, e, c, "none", preact=pre)
    dY = randn((n, K + 3), 343, F32)[:, 1:1 + K]
    dX, dc = nv.moe_backward(wt, dY, e, c, pre, "none")
    x, d = X8.moe_grads(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c), f64(dY), "none", True, 2.0 ** -16)
    check(dX, x, "dX")
    check(dc, d, "dweights")
    only = experts._moe_backward(wt, dY, e, c, pre, 0, False, True, None, None)
    assert only[0] is None and torch.equal(only[1], dc)
    big = dY.clone()
    big[1, 2], big[2, 0] = INF, NAN
    got = nv.moe_backward(wt, big, e, c, pre, "none")
    keep = [t for t in range(n) if t not in (1, 2)]
    assert torch.equal(got[0][keep], dX[keep]) and torch.equal(got[1][keep], dc[keep])
    live = (e[1] >= 0).tolist()
    assert not torch.isfinite(got[1][1][live]).any() and torch.isnan(got[1][2][e[2] >= 0]).all()


@pytest.mark.parametrize("K,F,n", [(8192, 32, 16), (8208, 32, 3), (7184, 128, 2), (32, 8208, 5), (1040, 144, 16)])
def test_moe_long_rows(K, F, n):
    """Every wave's share of K up to 8192, the form beyond, long F."""
    say("moe long", K, F, n)
    w, Wg, Wu, Wd = weights(3, F, K, 30, 0.02)
    X = randn((n, K), 31)
    e, c = choices(n, 2, 3, 32)
    check(nv.moe(w, X, e, c), X8.moe(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c)), "Y")


@pytest.mark.parametrize("tiles", range(1, 9))
@pytest.mark.parametrize("n", [2, 7, 13])
def test_every_decode_variant(tiles, n):
    say("decode variant", tiles, n)
    K = tiles * 1024 - 112
    w, Wg, Wu, Wd = weights(3, 32, K, 40 + tiles, 0.02)
    X = randn((n, K), 41)
    e, c = choices(n, 3, 3, 42)
    check(nv.moe(w, X, e, c), X8.moe(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c)), "Y")


@pytest.mark.parametrize("k", [1, 2, 3, 4, 7, 8, 32])
@pytest.mark.parametrize("n", [1, 16])
def test_every_split_of_the_down_projection(k, n):
    say("down split", k, n)
    w, Wg, Wu, Wd = weights(33, 528, 96, 50)
    X = randn((n, 96), 51)
    e, c = choices(n, k, 33, 52)
    check(nv.moe(w, X, e, c), X8.moe(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c)), "Y")


@pytest.mark.parametrize("k", [8, 24, 25, 32])
def test_most_pairs_of_the_down_projection(k):
    """Up to 512 pairs and two windows of rows: the sums take the most LDS there, and
    beyond 384 pairs fewer tiles are fetched ahead."""
    say("moe most pairs", k)
    n, E, F, K = 16, 40, 144, 4112
    w, Wg, Wu, Wd = weights(E, F, K, 85)
    X, (e, c) = randn((n, K), 86), choices(n, k, E, 87)
    check(nv.moe(w, X, e, c, out_dtype=F32), X8.moe(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c), out_f32=True), "Y")


@pytest.mark.parametrize("n", [1, 6, 16, 30, 200])
def test_empty_repeated_and_foreign_experts(n):
    """No expert at all; one expert for all tokens, in every slot; experts that
    are not in [0, E)."""
    say("moe choices", n)
    E, F, K, k = 6, 80, 144, 4
    w, Wg, Wu, Wd = weights(E, F, K, 60)
    X = randn((n, K), 61)
    r = randn((n, K), 62)
    c = choices(n, k, E, 63)[1]
    none = torch.full((n, k), -1, dtype=torch.int32, device="cuda")
    assert (nv.moe(w, X, none, c) == 0).all()
    assert torch.equal(nv.moe(w, X, none, c, residual=r), r)
    nan = torch.full_like(c, NAN)
    assert torch.equal(nv.moe(w, X, none, nan, residual=r), r)      # no expert: its weight is not used
    same = torch.full((n, k), 3, dtype=torch.int32, device="cuda")
    check(nv.moe(w, X, same, c), X8.moe(f64(X), Wg, Wu, Wd, same.cpu().numpy(), f64(c)), "one expert")
    rng = np.random.default_rng(64)
    mix = torch.from_numpy(rng.choice([-2 ** 31, -7, -1, 0, 2, 5, 6, 1000, 2 ** 31 - 1], (n, k)).astype(np.int32)).cuda()
    check(nv.moe(w, X, mix, c), X8.moe(f64(X), Wg, Wu, Wd, mix.cpu().numpy(), f64(c)), "foreign")


def test_many_experts():
    say("1024 experts")
    E, F, K = 1024, 16, 32
    Wg, Wu, Wd = (randn((E,) + s, 70 + i, F32, 0.2) for i, s in enumerate(((F, K), (F, K), (K, F))))
    w = nv.ExpertWeights.from_float(Wg, Wu, Wd)
    deq = []
    for W in (Wg, Wu, Wd):
        q = [O.quantize(W[e].cpu().numpy()) for e in range(E)]
        deq.append(np.stack([np.asarray(O.dequant(*a), dtype=np.float64) for a in q]))
    for n in (16, 300):
        X = randn((n, K), 75)
        e, c = choices(n, 32, E, 76)
        check(nv.moe(w, X, e, c), X8.moe(f64(X), *deq, e.cpu().numpy(), f64(c)), "Y")


@pytest.mark.parametrize("n", [7, 60])
def test_nonfinite_stays_in_its_token(n):
    """A NaN or an infinity in a token's activations, and a NaN scale in an expert
    that only one token takes, reach that token alone."""
    say("moe nonfinite", n)
    E, F, K, k = 5, 80, 272, 2
    w, _, _, _ = weights(E, F, K, 80)
    X = randn((n, K), 81)
    e, c = choices(n, k, E - 1, 82)
    clean = nv.moe(w, X, e, c)
    dirty = X.clone()
    dirty[3, 100], dirty[5, 0] = NAN, INF
    got = nv.moe(w, dirty, e, c)
    keep = [t for t in range(n) if t not in (3, 5)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[5]).any()
    # the last expert, of token 2 alone, has NaN scales
    w.gate_up_scales[E - 1] = 0x7F
    w.down_scales[E - 1] = 0x7F
    e2 = e.clone()
    e2[2, 1] = E - 1
    got = nv.moe(w, X, e2, c)
    keep = [t for t in range(n) if t != 2]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[2]).all()
    c2 = c.clone()
    c2[4, 0] = NAN
    got = nv.moe(w, X, e, c2)
    keep = [t for t in range(n) if t != 4]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[4]).all()


def test_decode_does_not_depend_on_the_batch_and_results_repeat():
    say("moe batch identity")
    E, F, K, k = 11, 272, 1040, 3
    w, _, _, _ = weights(E, F, K, 90)
    X = randn((16, K), 91)
    e, c = choices(16, k, E, 92, 0.2)
    whole = nv.moe(w, X, e, c)
    for a, b in ((0, 1), (3, 8), (5, 14), (15, 16)):
        assert torch.equal(nv.moe(w, X[a:b], e[a:b].contiguous(), c[a:b].contiguous()), whole[a:b])
    for n in (16, 40, 300):
        X = randn((n, K), 93)
        e, c = choices(n, k, E, 94)
        first = nv.moe(w, X, e, c)
        for _ in range(3):
            assert torch.equal(nv.moe(w, X, e, c), first)


@pytest.mark.parametrize("n", [5, 30])
def test_strides_guards_workspaces_and_in_place_residual(n):
    say("moe strides", n)
    E, F, K, k = 5, 48, 144, 2
    w, _, _, _ = weights(E, F, K, 100)
    buf = randn((n, 3 * K + 8), 101)
    X = buf[:, 8:8 + K]
    e, c = choices(n, k, E, 102, 0.2)
    want = nv.moe(w, X.contiguous(), e, c)
    assert torch.equal(nv.moe(w, X, e, c), want)
    for col in (0, 3, 4):                       # the last two: element and vector alignment
        out = torch.full((n + 2, K + 9), 7.0, device="cuda", dtype=BF16)
        assert torch.equal(nv.moe(w, X, e, c, out=out[1:n + 1, col:col + K]), want)
        out[1:n + 1, col:col + K] = 7.0
        assert (out == 7.0).all()
    r = randn((n, K + 3), 103, F32)
    want = nv.moe(w, X, e, c, residual=r[:, 1:1 + K], out_dtype=F32)
    got = r.clone()
    nv.moe(w, X, e, c, residual=got[:, 1:1 + K], out=got[:, 1:1 + K])
    assert torch.equal(got[:, 1:1 + K], want) and torch.equal(got[:, 0], r[:, 0]) and torch.equal(got[:, 1 + K:], r[:, 1 + K:])
    need = nv.moe_workspace_bytes(n, k, w)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")      # NaN where it is read unwritten
    assert torch.equal(nv.moe(w, X, e, c, residual=r[:, 1:1 + K], out_dtype=F32, workspace=ws[:need]), want)
    assert (ws[need:] == 255).all()


@pytest.mark.parametrize("n", [12, 90])
def test_columns_that_do_not_exist_read_as_zero(n):
    """After a call full of NaN (left behind in LDS and in the workspace), sizes
    that end inside a tile still give finite results."""
    say("moe stale", n)
    big, _, _, _ = weights(4, 256, 512, 110)
    w, _, _, _ = weights(4, 144, 336, 111)
    X = randn((n, 336), 112)
    e, c = choices(n, 2, 4, 113)
    want = nv.moe(w, X, e, c)
    ws = torch.empty(max(nv.moe_workspace_bytes(n, 2, big), nv.moe_workspace_bytes(n, 2, w)), dtype=torch.uint8, device="cuda")
    nv.moe(big, torch.full((n, 512), NAN, device="cuda", dtype=BF16), e, c, workspace=ws)
    assert torch.equal(nv.moe(w, X, e, c, workspace=ws), want)


@pytest.mark.parametrize("n,E,F,K,k", [(1, 3, 16, 16, 1), (9, 5, 48, 144, 2), (33, 5, 144, 272, 3), (150, 3, 272, 528, 2),
                                       (700, 4, 64, 96, 2)])
@pytest.mark.parametrize("act,dtype,empty", [("silu", BF16, 0.0), ("gelu", F32, 0.3), ("gelu_tanh", BF16, 0.9), ("none", BF16, 0.0)])
def test_moe_gradients(n, E, F, K, k, act, dtype, empty):
    say("moe grad", n, E, F, K, k, act, dtype, empty)
    w, Wg, Wu, Wd = weights(E, F, K, 120)
    wt = w.transpose()
    X = randn((n, K), 121).requires_grad_()
    e, c = choices(n, k, E, 122, empty)
    c.requires_grad_()
    r = randn((n, K), 123).requires_grad_()
    dY = randn((n, K), 124, dtype, 0.1)
    Y = nv.moe(w, X, e, c, act, r, transposed=wt, out_dtype=dtype)
    args = (f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c))
    check(Y, X8.moe(*args, act, f64(r), dtype == F32), "Y")
    dX, dc, dr = torch.autograd.grad(Y, [X, c, r], dY)
    x, d = X8.moe_grads(*args, f64(dY), act, dtype == F32)
    check(dX, x, "dX")
    check(dc, d, "dweights")
    assert torch.equal(dr, dY.to(BF16))
    pre = torch.full((n * k, 2 * F), NAN, device="cuda")
    with torch.no_grad():
        assert torch.equal(nv.moe(w, X, e, c, act, r, out_dtype=dtype, preact=pre), Y)
    for a, b in zip(nv.moe_backward(wt, dY, e, c.detach(), pre, act), (dX, dc)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("F", [4096, 4112, 4400, 8208])
@pytest.mark.parametrize("n", [2, 40])
def test_gradients_of_rows_longer_than_the_registers_hold(F, n):
    """From F = 4096 on, the rest of a row's gradients is computed again once the row's
    largest is known; in some rows that lies in the rest."""
    say("moe grad, long F", F, n)
    E, K, k = 2, 48, 1
    w, Wg, Wu, Wd = weights(E, F, K, 360)
    wt = w.transpose()
    X, (e, c) = randn((n, K), 361), choices(n, k, E, 362)
    dY = randn((n, K), 363, BF16, 0.1)
    pre = torch.zeros(n * k, 2 * F, device="cuda")
    nv.moe(w, X, e, c, preact=pre)
    args = f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c)
    dX, dc = nv.moe_backward(wt, dY, e, c, pre)
    x, d = X8.moe_grads(*args, f64(dY))
    check(dX, x, "dX")
    check(dc, d, "dweights")


def test_gradients_of_repeated_experts_and_expanded_dy():
    say("moe grad repeated")
    E, F, K, k, n = 4, 64, 96, 3, 21
    w, Wg, Wu, Wd = weights(E, F, K, 130)
    wt = w.transpose()
    X = randn((n, K), 131).requires_grad_()
    e = torch.full((n, k), 2, dtype=torch.int32, device="cuda")
    e[:, 1] = -1
    c = choices(n, k, E, 132)[1].requires_grad_()
    Y = nv.moe(w, X, e, c, transposed=wt)
    dX, dc = torch.autograd.grad(Y.sum(), [X, c])
    x, d = X8.moe_grads(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c), np.ones((n, K)))
    check(dX, x, "dX")
    check(dc, d, "dweights")
    assert (dc[:, 1] == 0).all()
    buf = randn((n, K + 5), 133, BF16)          # rows that are not 16-byte aligned
    pre = torch.empty(n * k, 2 * F, device="cuda")
    nv.moe(w, X.detach(), e, c.detach(), preact=pre)
    for a, b in zip(nv.moe_backward(wt, buf[:, 3:3 + K], e, c.detach(), pre),
                    nv.moe_backward(wt, buf[:, 3:3 + K].contiguous(), e, c.detach(), pre)):
        assert torch.equal(a, b)


def test_reference_gradients_against_differences():
    """The formulas that the kernels are held to, against central differences in 64 bits."""
    rng = np.random.default_rng(140)
    E, F, K, k, n = 3, 8, 6, 2, 4
    Wg, Wu, Wd = rng.standard_normal((E, F, K)), rng.standard_normal((E, F, K)), rng.standard_normal((E, K, F))
    X, c, dY = rng.standard_normal((n, K)), rng.standard_normal((n, k)), rng.standard_normal((n, K))
    e = rng.integers(-1, E, (n, k))
    for kind in ("silu", "gelu", "gelu_tanh"):
        (dx, _), (dc, _) = X8.moe_grads(X, Wg, Wu, Wd, e, c, dY, kind)

        def f(x, w):
            return (X8.moe(x, Wg, Wu, Wd, e, w, kind)[0] * dY).sum()
        t = 1e-5
        for i in range(n):
            for j in range(K):
                v = np.zeros_like(X)
                v[i, j] = t
                assert abs((f(X + v, c) - f(X - v, c)) / (2 * t) - dx[i, j]) < 1e-6 * (1 + abs(dx[i, j]))
            for j in range(k):
                v = np.zeros_like(c)
                v[i, j] = t
                assert abs((f(X, c + v) - f(X, c - v)) / (2 * t) - dc[i, j]) < 1e-6 * (1 + abs(dc[i, j]))


def test_transposed_copies_of_experts_that_are_gone():
    say("moe transposed")
    E, F, K, k, n = 2, 32, 48, 1, 5
    X, (e, c) = randn((n, K), 351).requires_grad_(), choices(n, k, E, 352)
    w = weights(E, F, K, 350)[0]
    wt = w.transpose()
    nv.moe(w, X, e, c, transposed=wt).sum().backward()
    w = weights(E, F, K, 353)[0]          # the first ones are freed
    gc.collect()
    assert wt._source() is None
    with pytest.raises(ValueError):
        nv.moe(w, X, e, c, transposed=wt)
    nv.moe(w, X, e, c, transposed=w.transpose()).sum().backward()
    whole = copy.deepcopy((w, w.transpose()))      # both copied: nothing tells them apart
    nv.moe(whole[0], X, e, c, transposed=whole[1]).sum().backward()


def test_no_tokens():
    say("moe no tokens")
    w, _, _, _ = weights(2, 32, 48, 150)
    X = torch.empty(0, 48, device="cuda", dtype=BF16, requires_grad=True)
    e, c = choices(0, 2, 2, 151)
    c = c.reshape(0, 2).requires_grad_()
    Y = nv.moe(w, X, e.reshape(0, 2), c, transposed=w.transpose())
    dX, dc = torch.autograd.grad(Y, [X, c], torch.empty(0, 48, device="cuda", dtype=BF16))
    assert Y.shape == (0, 48) and dX.shape == (0, 48) and dc.shape == (0, 2)


def test_several_chunks():
    """More than 2^16 pairs are handled in parts: the same results as of the parts."""
    say("moe chunks")
    E, F, K, k, n = 7, 32, 48, 32, 5000          # chunks of 2048 tokens
    w, _, _, _ = weights(E, F, K, 160)
    wt = w.transpose()
    X, dY = randn((n, K), 161), randn((n, K), 162)
    rng = np.random.default_rng(163)
    e = torch.from_numpy(rng.integers(-1, E, (n, k)).astype(np.int32)).cuda()
    c = torch.from_numpy(rng.random((n, k)).astype(np.float32)).cuda()
    pre = torch.zeros(n * k, 2 * F, device="cuda")
    Y = nv.moe(w, X, e, c, preact=pre)
    dX, dc = nv.moe_backward(wt, dY, e, c, pre)
    for a in range(0, n, 2048):
        b = min(n, a + 2048)
        part = torch.zeros((b - a) * k, 2 * F, device="cuda")
        assert torch.equal(nv.moe(w, X[a:b], e[a:b], c[a:b], preact=part), Y[a:b])
        assert torch.equal(part, pre[a * k:b * k])
        x, d = nv.moe_backward(wt, dY[a:b], e[a:b], c[a:b], part)
        assert torch.equal(x, dX[a:b]) and torch.equal(d, dc[a:b])


@pytest.mark.parametrize("wide", ["X", "dY", "both"])
def test_chunks_do_not_depend_on_the_strides(wide):
    """Rows so far apart that fewer of them than a chunk's fit 32-bit offsets, in
    one direction or both: the bits of the same rows next to each other.  The
    pre-activations are in the experts' order within a chunk, so that both
    directions have to cut the tokens alike."""
    say("moe chunk strides", wide)
    E, F, K, k, n, ld = 4, 32, 48, 1, 5000, 1 << 18       # 4094 rows of this stride
    w, Wg, Wu, Wd = weights(E, F, K, 300)
    wt = w.transpose()
    X, dY, (e, c) = randn((n, K), 301), randn((n, K), 302), choices(n, k, E, 303)

    def apart(t):
        rows = torch.empty(n, ld, device="cuda", dtype=BF16)[:, 64:64 + K]
        rows.copy_(t)
        return rows
    Xs, dYs = apart(X) if wide != "dY" else X, apart(dY) if wide != "X" else dY
    pre, pres = (torch.zeros(n * k, 2 * F, device="cuda") for _ in range(2))
    Y, Ys = nv.moe(w, X, e, c, preact=pre), nv.moe(w, Xs, e, c, preact=pres)
    assert torch.equal(Ys, Y) and torch.equal(pres, pre)
    for need_x in (True, False):
        got, want = (experts._moe_backward(wt, g, e, c, p, 2, need_x, True, None, None) for g, p in ((dYs, pres), (dY, pre)))
        assert torch.equal(got[1], want[1]) and (not need_x or torch.equal(got[0], want[0]))
    dX, dc = nv.moe_backward(wt, dYs, e, c, pres)
    x, d = X8.moe_grads(f64(X), Wg, Wu, Wd, e.cpu().numpy(), f64(c), f64(dY))
    check(dX, x, "dX")
    check(dc, d, "dweights")


# ---- together, streams, graphs -------------------------------------------------------------

def test_layer_as_it_is_used():
    """Router logits from a projection, the router, the experts, a shared block in
    8 bits added by the layer: forward against 64 bits, gradients through the
    router and the experts against differences of the 64-bit layer."""
    say("layer")
    n, E, F, K, k = 24, 8, 96, 160, 2
    w, Wg, Wu, Wd = weights(E, F, K, 170)
    wt = w.transpose()
    rw, Wr = nv.PackedWeight.from_float(randn((E, K), 171, F32, 0.1)), None
    codes, scales, g = O.quantize(randn((E, K), 171, F32, 0.1).cpu().numpy())
    Wr = np.asarray(O.dequant(codes, scales, g), dtype=np.float64)
    shared = nv.Int8Weight.from_float(randn((K, K), 172, F32, 0.05))
    X = randn((n, K), 173).requires_grad_()
    logits = nv.linear(rw, X, out_dtype=F32, transposed=rw.transpose())
    weights_, experts = nv.moe_route(logits, k)
    side = nv.int8_linear(shared, X.detach())
    Y = nv.moe(w, X, experts, weights_, residual=side, transposed=wt)
    ids = experts.cpu().numpy()

    def f(x):
        l = x @ Wr.T
        a = np.take_along_axis(l, ids, 1)
        q = np.exp(a - a.max(1, keepdims=True))
        return X8.moe(x, Wg, Wu, Wd, ids, q / q.sum(1, keepdims=True))
    ref, bound = f(f64(X))
    # the weights are off by what the logits are: sums of K products
    el = (K + 32) * R.HALF_F32 * (np.abs(f64(X)) @ np.abs(Wr).T).max()
    assert np.array_equal(ids, np.argsort(-(f64(X) @ Wr.T), 1, kind="stable")[:, :k])
    ref, y = ref + f64(side), f64(Y)
    assert (np.abs(y - ref) <= bound + 4 * el * np.abs(ref - f64(side)).max() + R.HALF_BF16 * np.abs(ref)).all()
    (dX,) = torch.autograd.grad(Y.sum(), X)
    rng = np.random.default_rng(174)
    for _ in range(6):
        v = rng.standard_normal((n, K))
        t = 1e-4
        diff = (f(f64(X) + t * v)[0].sum() - f(f64(X) - t * v)[0].sum()) / (2 * t)
        got = float((f64(dX) * v).sum())
        # roundings to bf16 of h's gradient, of dX, of dlogits for their product and of the two summed parts
        assert abs(got - diff) <= 8 * R.HALF_BF16 * float((np.abs(f64(dX)) * np.abs(v)).sum()) + 1e-3


def step(w, wt, X, dY, logits):
    weights_, experts = nv.moe_route(logits, 2, "sigmoid")
    pre = torch.empty(X.shape[0] * 2, 2 * w.F, device="cuda")
    Y = nv.moe(w, X, experts, weights_, preact=pre)
    dX, dc = nv.moe_backward(wt, dY, experts, weights_, pre)
    return Y, nv.moe(w, X, experts, weights_), dX, nv.moe_route_backward(logits, experts, dc, "sigmoid")


def test_graph_replays_match_eager():
    say("moe graphs")
    E, F, K = 5, 80, 144
    w, _, _, _ = weights(E, F, K, 180)
    wt = w.transpose()
    graphs = []
    for n in (6, 90):
        X, dY, l = randn((n, K), 181), randn((n, K), 182), logits_of(n, E, 183)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(w, wt, X, dY, l)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(w, wt, X, dY, l)
        graphs.append((n, X, dY, l, graph, out))
    for trip in range(4):
        for n, X, dY, l, graph, out in graphs:
            X.copy_(randn((n, K), 190 + trip))
            dY.copy_(randn((n, K), 200 + trip))
            l.copy_(logits_of(n, E, 210 + trip, masked=0.3))
            graph.replay()
            torch.cuda.synchronize()
            for o, x in zip(out, step(w, wt, X, dY, l)):
                assert torch.equal(o, x), (trip, n)


def test_side_stream():
    say("moe stream")
    E, F, K, k = 4, 48, 144, 2
    for n in (5, 60):
        w, _, _, _ = weights(E, F, K, 220)
        X, dY, l = randn((n, K), 221), randn((n, K), 222), logits_of(n, E, 223)
        e, c = nv.moe_route(l, k)[::-1]
        pre = torch.zeros(n * k, 2 * F, device="cuda")
        want = (nv.moe(w, X, e, c, preact=pre),) + nv.moe_backward(w.transpose(), dY, e, c, pre)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        e2, c2 = nv.moe_route(l, k, stream=s)[::-1]
        pre2 = torch.zeros(n * k, 2 * F, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        Y = nv.moe(w, X, e2, c2, preact=pre2, stream=s)
        wt = w.transpose(stream=s)
        got = (Y,) + nv.moe_backward(wt, dY, e2, c2, pre2, stream=s)
        s.synchronize()
        for a, b in zip(got + (e2, c2, pre2), want + (e, c, pre)):
            assert torch.equal(a, b)
    assert torch.equal(nv.ExpertWeights.from_float(*(randn(sh, 224, F32) for sh in ((2, 32, 48), (2, 32, 48), (2, 48, 32))), stream=s).gscale,
                       nv.ExpertWeights.from_float(*(randn(sh, 224, F32) for sh in ((2, 32, 48), (2, 32, 48), (2, 48, 32)))).gscale)


def test_refusals():
    say("moe refusals")
    E, F, K, k, n = 3, 32, 48, 2, 4
    w, _, _, _ = weights(E, F, K, 230)
    other, _, _, _ = weights(E, F, K, 250)
    wt = w.transpose()
    X, (e, c) = randn((n, K), 231), choices(n, k, E, 232)
    l = logits_of(n, E, 233)
    pre = torch.empty(n * k, 2 * F, device="cuda")
    bad = [
        (TypeError, lambda: nv.moe(wt, X, e, c)), (TypeError, lambda: nv.moe(w, X.float(), e, c)),
        (TypeError, lambda: nv.moe(w, X, e.long(), c)), (TypeError, lambda: nv.moe(w, X, e, c.to(BF16))),
        (ValueError, lambda: nv.moe(w, X[:, :32], e, c)), (ValueError, lambda: nv.moe(w, X[:3], e, c)),
        (ValueError, lambda: nv.moe(w, X, e[:, :1], c)), (ValueError, lambda: nv.moe(w, X, e, c.t().contiguous().t())),
        (ValueError, lambda: nv.moe(w, X, e, c, "swish")), (ValueError, lambda: nv.moe(w, X, e.expand(n, k)[:, :0], c[:, :0])),
        (ValueError, lambda: nv.moe(w, X, e, c, preact=pre[:3])), (ValueError, lambda: nv.moe(w, X, e, c, residual=X[:2])),
        (TypeError, lambda: nv.moe(w, X, e, c, out_dtype=torch.float16)), (TypeError, lambda: nv.moe(w, X.cpu(), e, c)),
        (nv.Nvfp4Error, lambda: nv.moe(w, X, e, c, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (nv.Nvfp4Error, lambda: nv.moe(w, X, e, c, out=X)),
        (ValueError, lambda: nv.moe(w, X.clone().requires_grad_(), e, c)),
        (ValueError, lambda: nv.moe(w, X.clone().requires_grad_(), e, c, transposed=other.transpose())),
        (ValueError, lambda: nv.moe(w, X.clone().requires_grad_(), e, c, transposed=wt, out=torch.empty_like(X))),
        (ValueError, lambda: nv.moe_backward(wt, X.clone().requires_grad_(), e, c, pre)),
        (TypeError, lambda: nv.moe_backward(w, X, e, c, pre)), (ValueError, lambda: nv.moe_backward(wt, X, e, c, pre[:, :60])),
        (TypeError, lambda: nv.ExpertWeights.from_packed([w], [w], [w])),
        (ValueError, lambda: nv.ExpertWeights.from_float(*[randn((2, 32, 40), 1, F32)] * 2, randn((2, 40, 32), 1, F32))),
        (ValueError, lambda: nv.moe_route(l, 4)), (ValueError, lambda: nv.moe_route(l, 0)), (ValueError, lambda: nv.moe_route(l, 2.0)),
        (ValueError, lambda: nv.moe_route(l, 2, "max")), (ValueError, lambda: nv.moe_route(l, 2, scale=NAN)),
        (TypeError, lambda: nv.moe_route(l.double(), 2)), (ValueError, lambda: nv.moe_route(l, 2, bias=torch.zeros(2, device="cuda"))),
        (ValueError, lambda: nv.moe_route(l, 2, bias=torch.zeros(E, device="cuda", requires_grad=True))),
        (ValueError, lambda: nv.moe_route(torch.zeros(2, 1025, device="cuda"), 2)), (ValueError, lambda: nv.moe_route(l.t(), 2)),
        (ValueError, lambda: nv.moe_route_backward(l, e, c.clone().requires_grad_())),
        (ValueError, lambda: nv.moe_route_backward(l, e[:2], c)),
    ]
    for i, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            say("not refused:", i)
    Y = nv.moe(w, X, e, c)
    with pytest.raises(RuntimeError):            # a buffer that a graph has saved, overwritten
        leaf = c.clone().requires_grad_()
        z = nv.moe(w, X, e, leaf, transposed=wt)
        e.fill_(0)
        z.sum().backward()
    assert torch.isfinite(Y).all()
