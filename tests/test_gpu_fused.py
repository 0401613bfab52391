"""GPU parity of the fused operators (projection with epilogue, gated block,
product through the transposed weight, gradients) against 64-bit arithmetic,
through the Python entry points, within the bounds of fused_reference."""
import numpy as np
import pytest
import torch

import fused_reference as R
import nvfp4_weight_only_02_amd as nv
import oracle as O
from nvfp4_weight_only_02_amd import fused, inputs

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


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


def weight(N, K, seed, std=0.05):
    """(PackedWeight, its 64-bit values)"""
    codes, scales, g = O.quantize(inputs.weights_f32(N, K, seed, std))
    pw = nv.PackedWeight.from_canonical(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), g, N, K)
    return pw, np.asarray(O.dequant(codes, scales, g), dtype=np.float64)


def randn(shape, seed, dtype=BF16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def check(got, want, what):
    ref, bound = want
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all(), what
    assert (err <= bound).all(), "%s: worst err/bound %.3g" % (what, float((err / bound).max()))


SHAPES = [(1, 16), (37, 144), (200, 656), (64, 8208), (330, 2064)]
LINEAR = [  # activation, bias, residual, out
    ("none", None, None, BF16), ("silu", BF16, BF16, BF16), ("gelu", F32, F32, F32),
    ("gelu_tanh", BF16, F32, BF16), ("relu", F32, BF16, F32)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("n", [1, 4, 13, 16, 17, 40, 70, 150])
@pytest.mark.parametrize("act,bias,residual,out", LINEAR)
def test_linear(n, N, K, act, bias, residual, out):
    say("linear", n, N, K, act, bias, residual, out)
    w, W = weight(N, K, 1 + N)
    X = randn((n, K), 2)
    b = None if bias is None else randn((N,), 3, bias)
    r = None if residual is None else randn((n, N), 4, residual, 3.0)
    Y = nv.linear(w, X, bias=b, activation=act, residual=r, out_dtype=out)
    assert Y.dtype == out
    check(Y, R.linear(f64(X), W, None if b is None else f64(b), act, None if r is None else f64(r), out == F32), "Y")


@pytest.mark.parametrize("F,K", [(1, 16), (17, 144), (40, 656), (64, 8208), (129, 2064)])
@pytest.mark.parametrize("n", [1, 4, 13, 16, 17, 40, 150])
@pytest.mark.parametrize("act,bias,out", [("silu", None, BF16), ("gelu", F32, F32), ("gelu_tanh", BF16, BF16),
                                          ("relu", None, F32), ("none", BF16, BF16)])
def test_gated(n, F, K, act, bias, out):
    say("gated", n, F, K, act, bias, out)
    (g, Wg), (u, Wu) = weight(F, K, 5, 0.05), weight(F, K, 6, 0.02)
    X = randn((n, K), 7)
    bg = None if bias is None else randn((F,), 8, bias)
    bu = None if bias is None else randn((F,), 9, bias)
    H = nv.gated(nv.GatedWeight.from_packed(g, u), X, activation=act, gate_bias=bg, up_bias=bu, out_dtype=out)
    check(H, R.gated(f64(X), Wg, Wu, None if bg is None else f64(bg), None if bu is None else f64(bu), act,
                     out == F32), "H")


@pytest.mark.parametrize("N,K", SHAPES + [(129, 48)])
@pytest.mark.parametrize("n", [1, 15, 33, 70, 150])
def test_gemm_t(n, N, K):
    say("gemm_t", n, N, K)
    w, W = weight(N, K, 10 + K)
    dY = randn((n, N), 11)
    dX = nv.gemm_t(w.transpose(), dY)
    D = f64(dY)
    ref = D @ W
    b = (N + 32) * R.HALF_F32 * (np.abs(D) @ np.abs(W))
    check(dX, (ref, b + R.HALF_BF16 * (np.abs(ref) + b) + 2.0 ** -133), "dX")


def test_gemm_t_one_hot_is_exact_dequant():
    say("gemm_t one-hot")
    rng = np.random.default_rng(22)
    N, K = 80, 272
    codes = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    scales = rng.integers(0, 0x7F, size=(N, K // 16), dtype=np.uint8)
    w = nv.PackedWeight.from_canonical(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 1.0, N, K)
    dX = nv.gemm_t(w.transpose(), torch.eye(N, device="cuda", dtype=BF16))
    assert np.array_equal(f64(dX), O.dequant(codes, scales, 1.0))


@pytest.mark.parametrize("n,N,K", [(3, 200, 656), (16, 37, 144), (21, 330, 272), (150, 129, 656)])
@pytest.mark.parametrize("act,bias", [("none", F32), ("silu", BF16), ("gelu", BF16), ("gelu_tanh", F32),
                                      ("relu", None)])
def test_linear_gradients(n, N, K, act, bias):
    say("linear grad", n, N, K, act, bias)
    w, W = weight(N, K, 12)
    X = randn((n, K), 13).requires_grad_()
    b = None if bias is None else randn((N,), 14, bias).requires_grad_()
    r = randn((n, N), 15).requires_grad_()
    dY = randn((n, N), 16, std=0.1)
    Y = nv.linear(w, X, bias=b, activation=act, residual=r, transposed=w.transpose())
    check(Y, R.linear(f64(X), W, None if b is None else f64(b), act, f64(r)), "Y")
    grads = torch.autograd.grad(Y, [X, r] + ([b] if b is not None else []), dY)
    dX, db = R.linear_grads(f64(X), W, f64(dY), None if b is None else f64(b), act, bias == F32)
    check(grads[0], dX, "dX")
    assert torch.equal(grads[1], dY)
    if b is not None:
        assert grads[2].dtype == bias
        check(grads[2], db, "db")


@pytest.mark.parametrize("n,F,K", [(3, 200, 656), (16, 17, 144), (21, 330, 272), (150, 129, 656)])
@pytest.mark.parametrize("act,bias", [("silu", None), ("gelu", BF16), ("gelu_tanh", F32), ("none", F32)])
def test_gated_gradients(n, F, K, act, bias):
    say("gated grad", n, F, K, act, bias)
    (g, Wg), (u, Wu) = weight(F, K, 17), weight(F, K, 18, 0.02)
    w = nv.GatedWeight.from_packed(g, u)
    X = randn((n, K), 19).requires_grad_()
    bg = None if bias is None else randn((F,), 20, bias).requires_grad_()
    bu = None if bias is None else randn((F,), 21, bias).requires_grad_()
    dH = randn((n, F), 22, std=0.1)
    H = nv.gated(w, X, activation=act, gate_bias=bg, up_bias=bu, transposed=w.transpose())
    grads = torch.autograd.grad(H, [X] + ([bg, bu] if bias is not None else []), dH)
    none = bias is None
    dX, dbg, dbu = R.gated_grads(f64(X), Wg, Wu, f64(dH), None if none else f64(bg), None if none else f64(bu), act,
                                 bias == F32)
    check(grads[0], dX, "dX")
    if not none:
        check(grads[1], dbg, "dbg")
        check(grads[2], dbu, "dbu")


@pytest.mark.parametrize("act", R.ACTS)
def test_elementwise_gradient_tight(act):
    """Column sums of act'(z) over a wide range of z."""
    say("dZ", act)
    n, N, K = 40, 333, 16
    w, _ = weight(N, K, 23)
    z = torch.zeros(n, 336, device="cuda")
    z[:, :N] = randn((n, N), 24, F32, 4.0)
    z[:, N:] = float("nan")              # columns that do not exist
    dY = torch.ones(n, N, device="cuda", dtype=BF16)
    _, db = nv.linear_backward(None, dY, activation=act, preact=z, bias_dtype=F32)
    d = R.act_grad(f64(z)[:, :N], act)
    s, b = R.column_sum(d, 4 * R.ACT_EPS * (1 + np.abs(f64(z)[:, :N])), True)
    check(db, (s, b), "column sums")


@pytest.mark.parametrize("act", R.ACTS)
def test_gradient_of_huge_preactivations(act):
    """act'(z) up to the end of fp32's range, where squares and cubes of z
    overflow: 0 or 1 by then, so the bound is the one at |z| = 16."""
    z = [s * v for v in (0.0, 1.0, 15.0, 17.0, 90.0, 1e4, 1e13, 1e19, 2e19, 3e38) for s in (1, -1)]
    say("huge z", act)
    z = torch.tensor([z], device="cuda", dtype=F32)
    p = torch.zeros(1, 24, device="cuda")
    p[:, :20] = z
    _, db = nv.linear_backward(None, torch.ones(1, 20, device="cuda"), activation=act, preact=p, bias_dtype=F32)
    check(db[None], (R.act_grad(f64(z), act), 4 * R.ACT_EPS * (1 + np.minimum(np.abs(f64(z)), 16))), "act'")


def test_strides_guards_and_in_place_residual():
    """Strided X with NaN between its rows, an unaligned strided output whose
    surroundings stay as they were, the residual in place."""
    for n in (5, 16, 40):
        say("strides", n)
        N, K = 93, 208
        w, W = weight(N, K, 25)
        big = torch.full((n, K + 24), float("nan"), device="cuda", dtype=BF16)
        big[:, :K] = randn((n, K), 26)
        X = big[:, :K]
        for dtype in (BF16, F32):
            buf = torch.full((n + 2, 131), 7.0, device="cuda", dtype=dtype)
            out = buf[1:n + 1, 3:3 + N]
            r = randn((n, N), 27, dtype)
            out.copy_(r)
            Y = nv.linear(w, X, residual=out, out=out)
            assert Y.data_ptr() == out.data_ptr()
            check(out, R.linear(f64(X), W, None, "none", f64(r), dtype == F32), "in place")
            buf[1:n + 1, 3:3 + N] = 7.0
            assert (buf == 7.0).all()
        g, _ = weight(N, K, 28)
        gw = nv.GatedWeight.from_packed(w, g)
        buf = torch.full((n + 2, 140), 7.0, device="cuda", dtype=BF16)
        H = nv.gated(gw, X, out=buf[1:n + 1, 5:5 + N])
        assert torch.equal(H, nv.gated(gw, X.contiguous()))
        buf[1:n + 1, 5:5 + N] = 7.0
        assert (buf == 7.0).all()


def test_results_repeat_and_decode_does_not_depend_on_the_batch():
    say("repeat, batch identity")
    N, K = 200, 656
    w, _ = weight(N, K, 29)
    gw = nv.GatedWeight.from_packed(w, w)
    wt = w.transpose()
    X, dY = randn((300, K), 30), randn((300, N), 31)
    for n in (17, 64, 300):
        first = nv.linear(w, X[:n], activation="silu"), nv.gated(gw, X[:n]), nv.gemm_t(wt, dY[:n])
        again = nv.linear(w, X[:n], activation="silu"), nv.gated(gw, X[:n]), nv.gemm_t(wt, dY[:n])
        for p, q in zip(first, again):
            assert torch.equal(p, q), n
    one = nv.linear(w, X[:16]), nv.gated(gw, X[:16])
    for a, b in ((0, 1), (3, 9), (15, 16)):
        assert torch.equal(nv.linear(w, X[a:b]), one[0][a:b])
        assert torch.equal(nv.gated(gw, X[a:b]), one[1][a:b])


@pytest.mark.parametrize("n", [9, 33, 90, 300])
def test_columns_that_do_not_exist_read_as_zero(n):
    """After a call whose activations are NaN everywhere (its slices stay behind
    in LDS), a K and an N that end inside a tile still give finite results."""
    say("stale LDS", n)
    big, _ = weight(2048, 1024, 70)
    w, W = weight(328, 336, 71)
    gw, wt = nv.GatedWeight.from_packed(w, w), w.transpose()
    bt = big.transpose()
    X, dY = randn((n, 336), 72), randn((n, 328), 73)
    want = nv.linear(w, X), nv.gated(gw, X), nv.gemm_t(wt, dY)
    for f, v in ((lambda: nv.linear(w, X), want[0]), (lambda: nv.gated(gw, X), want[1]),
                 (lambda: nv.gemm_t(wt, dY), want[2])):
        nan = torch.full((n, 2048), float("nan"), device="cuda", dtype=BF16)
        nv.linear(big, nan[:, :1024])
        nv.gemm_t(bt, nan)
        got = f()
        assert torch.isfinite(got).all()
        assert torch.equal(got, v)


def test_linear_without_epilogue_is_gemv():
    say("linear == gemv")
    w, _ = weight(200, 656, 32)
    X = randn((9, 656), 33)
    assert torch.equal(nv.linear(w, X), nv.gemv(w, X))


def test_nonfinite_stays_in_its_token():
    for n in (9, 50):
        say("nonfinite", n)
        w, _ = weight(70, 272, 34)
        gw = nv.GatedWeight.from_packed(w, w)
        wt = w.transpose()
        X, dY = randn((n, 272), 35), randn((n, 70), 36)
        clean = nv.linear(w, X, activation="gelu"), nv.gated(gw, X), nv.gemm_t(wt, dY)
        X[4, 100], dY[4, 69] = float("nan"), float("inf")
        dirty = nv.linear(w, X, activation="gelu"), nv.gated(gw, X), nv.gemm_t(wt, dY)
        keep = [t for t in range(n) if t != 4]
        for c, d in zip(clean, dirty):
            assert torch.equal(c[keep], d[keep])
            assert not torch.isfinite(d[4]).any()


def test_no_tokens():
    say("no tokens")
    w, _ = weight(70, 272, 37)
    gw = nv.GatedWeight.from_packed(w, w)
    X = torch.empty(0, 272, device="cuda", dtype=BF16, requires_grad=True)
    b = randn((70,), 38).requires_grad_()
    Y = nv.linear(w, X, bias=b, activation="silu", transposed=w.transpose())
    dX, db = torch.autograd.grad(Y, [X, b], torch.empty(0, 70, device="cuda", dtype=BF16))
    assert Y.shape == (0, 70) and dX.shape == (0, 272) and (db == 0).all()
    H = nv.gated(gw, X, gate_bias=b, transposed=gw.transpose())
    dX, db = torch.autograd.grad(H, [X, b], torch.empty(0, 70, device="cuda", dtype=BF16))
    assert H.shape == (0, 70) and dX.shape == (0, 272) and (db == 0).all()
    assert nv.gemm_t(w.transpose(), torch.empty(0, 70, device="cuda", dtype=BF16)).shape == (0, 272)


def block(g, u, d, gt, dt, X, bg, bd):
    """A feed-forward block: gated, then the down projection onto the residual stream."""
    h = nv.gated(g, X, gate_bias=bg, transposed=gt)
    return nv.linear(d, h, bias=bd, residual=X, transposed=dt)


@pytest.mark.parametrize("n", [1, 16, 64])
def test_block_forward_and_backward(n):
    """The operators as a program runs them together, with an expanded
    incoming gradient, against central differences of the 64-bit block."""
    say("block", n)
    K, F = 160, 96
    (g, Wg), (u, Wu), (d, Wd) = weight(F, K, 40), weight(F, K, 41), weight(K, F, 42)
    gw = nv.GatedWeight.from_packed(g, u)
    X = randn((n, K), 43).requires_grad_()
    bg = randn((F,), 44, F32).requires_grad_()
    bd = randn((K,), 45, F32).requires_grad_()
    Y = block(gw, u, d, gw.transpose(), d.transpose(), X, bg, bd)

    def f(x, b):
        return x + f64(bd) + R.gated(x, Wg, Wu, b, None, "silu")[0] @ Wd.T
    x, b = f64(X), f64(bg)
    ref = f(x, b)
    scale = np.abs(ref).max()
    # h and Y are rounded to bf16: 2^-8 of each term of the down projection, and of Y
    assert np.abs(f64(Y) - ref).max() <= R.HALF_BF16 * (scale + (np.abs(R.gated(x, Wg, Wu, b)[0]) @ np.abs(Wd).T).max())
    dX, dbg, dbd = torch.autograd.grad(Y.sum(), [X, bg, bd])
    assert np.array_equal(f64(dbd), np.full(K, float(n)))
    rng = np.random.default_rng(46)
    for leaf, grad, which in ((x, dX, 0), (b, dbg, 1)):
        for _ in range(8):
            v = rng.standard_normal(leaf.shape)
            t = 1e-4
            args = lambda s: (x + s * v, b) if which == 0 else (x, b + s * v)   # noqa: E731
            diff = (f(*args(t)).sum() - f(*args(-t)).sum()) / (2 * t)
            got = float((f64(grad) * v).sum())
            # at most three roundings to bf16 (h's gradient, dZ, dX) and that of
            # h itself, on every term
            assert abs(got - diff) <= 8 * R.HALF_BF16 * float((np.abs(f64(grad)) * np.abs(v)).sum()) + 1e-3, which


def test_graph_replays_match_eager():
    """Forward and backward captured, two graphs with their own memory, replayed
    with changing inputs between eager calls."""
    say("graphs")
    K, F = 272, 144
    (g, _), (u, _), (d, _) = weight(F, K, 50), weight(F, K, 51), weight(K, F, 52)
    gw = nv.GatedWeight.from_packed(g, u)
    gt, dt = gw.transpose(), d.transpose()

    def step(X, dY, b):
        n = X.shape[0]
        pre = torch.empty(n, nv.preact_columns(gw), device="cuda")
        H = nv.gated(gw, X, gate_bias=b, preact=pre)
        Y = nv.linear(d, H, residual=X)
        dH, _ = nv.linear_backward(dt, dY)
        dX, db, _ = nv.gated_backward(gw, gt, dH, pre, bias_dtype=F32)
        return Y, dX, db

    graphs = []
    for n in (6, 200):
        X, dY, b = randn((n, K), 53), randn((n, K), 54), randn((F,), 55, F32)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(X, dY, b)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(X, dY, b)
        graphs.append((n, X, dY, b, graph, out))
    for trip in range(4):
        for n, X, dY, b, graph, out in graphs:
            X.copy_(randn((n, K), 60 + trip))
            dY.copy_(randn((n, K), 70 + trip))
            graph.replay()
            torch.cuda.synchronize()
            for o, e in zip(out, step(X, dY, b)):
                assert torch.equal(o, e), (trip, n)


def test_side_stream_and_given_buffers():
    say("streams")
    w, _ = weight(64, 8208, 56)
    gw = nv.GatedWeight.from_packed(w, w)
    X = randn((7, 8208), 57)
    want = nv.linear(w, X, activation="silu"), nv.gated(gw, X), nv.gemm_t(w.transpose(), randn((7, 64), 58))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    a = nv.linear(w, X, activation="silu", stream=s)
    b = nv.gated(gw, X, workspace=ws, stream=s)
    c = nv.gemm_t(w.transpose(stream=s), randn((7, 64), 58), stream=s)
    s.synchronize()
    for p, q in zip((a, b, c), want):
        assert torch.equal(p, q)


def test_unaligned_and_expanded_gradients():
    say("unaligned dY")
    w, W = weight(40, 272, 59)
    wt = w.transpose()
    buf = randn((30, 101), 61)
    dY = buf[:, 1:41]                       # rows not 16-byte aligned
    assert torch.equal(nv.gemm_t(wt, dY), nv.gemm_t(wt, dY.contiguous()))
    X = randn((30, 272), 62).requires_grad_()
    Y = nv.linear(w, X, transposed=wt)
    (a,) = torch.autograd.grad(Y.sum(), X)
    assert torch.equal(a, nv.gemm_t(wt, torch.ones(30, 40, device="cuda", dtype=BF16)))


def test_gradient_copies_are_made_on_the_launch_stream():
    # the current stream is kept busy (tens of ms): what a call on another
    # stream computes may not wait for it, nor read what it has yet to write
    w, W = weight(64, 144, 71)
    wt = w.transpose()
    gw = nv.GatedWeight.from_packed(w, w)
    gt = gw.transpose()
    big = randn((64, 21), 72, F32)
    X = randn((21, 144), 73)
    z = torch.empty(21, nv.preact_columns(gw), dtype=F32, device="cuda")
    nv.gated(gw, X, preact=z)
    s = torch.cuda.Stream()

    def both(d, stream=None):
        return (nv.linear_backward(wt, d, bias_dtype=F32, stream=stream) +
                nv.gated_backward(gw, gt, d, z, bias_dtype=F32, stream=stream))

    for stream in (None, s):        # memory that is used again holds another gradient's values
        both(-big.t(), stream)
        both((-big).t(), stream)
    torch.cuda.synchronize()
    say("gradients on another stream")
    torch.cuda._sleep(50_000_000)
    got = both(big.t(), s)
    with torch.cuda.stream(s):
        got = [t.cpu() for t in got]
    for a, b in zip(got, both(big.t().contiguous())):
        assert torch.equal(a, b.cpu())


def test_gradient_refusals():
    w, _ = weight(40, 272, 63)
    gw = nv.GatedWeight.from_packed(w, w)
    wt, gt = w.transpose(), gw.transpose()
    dY = randn((5, 40), 64)
    z = torch.zeros(5, nv.preact_columns(gw), device="cuda")
    out = torch.empty(5, 272, device="cuda", dtype=BF16)
    for call in (lambda **k: nv.linear_backward(k.pop("wt"), dY, **k),
                 lambda **k: nv.gated_backward(gw, gt if k.pop("wt") is wt else None, dY, z, **k)):
        with pytest.raises(TypeError):
            call(wt=wt, bias_dtype=torch.float16)
        with pytest.raises(ValueError):
            call(wt=None, bias_dtype=F32, out=out)       # no dX to receive
        with pytest.raises(ValueError):
            call(wt=wt, out=out[:4])
        with pytest.raises(TypeError):
            call(wt=wt, out=out.float())
        assert call(wt=wt, out=out)[0] is out


def test_refusals():
    say("refusals")
    w, _ = weight(40, 272, 63)
    gw = nv.GatedWeight.from_packed(w, w)
    X = randn((5, 272), 64)
    with pytest.raises(ValueError):
        nv.linear(w, X, activation="tanh")
    with pytest.raises(ValueError):
        nv.linear(w, X.t().contiguous().t())
    with pytest.raises(ValueError):
        nv.linear(w, X[:, :256])
    with pytest.raises(TypeError):
        nv.linear(w, X.float())
    with pytest.raises(ValueError):
        nv.linear(w, X, bias=randn((41,), 65))
    with pytest.raises(ValueError):
        nv.linear(w, X.clone().requires_grad_())                     # no transposed copy
    with pytest.raises(ValueError):
        nv.linear(w, X.clone().requires_grad_(), transposed=gw.transpose())
    with pytest.raises(TypeError):
        nv.gated(gw, X, gate_bias=randn((40,), 66), up_bias=randn((40,), 67, F32))
    with pytest.raises(ValueError):
        nv.GatedWeight.from_packed(w, weight(41, 272, 68)[0])
    odd = torch.empty(5 * 273 + 8, device="cuda", dtype=BF16)
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.linear(w, odd[:5 * 273].view(5, 273)[:, :272])
    assert e.value.status == 3
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.linear(w, X, out=X.view(-1)[:200].view(5, 40))
    assert e.value.status == 10


# ---- every tile of the many-token product -------------------------------------------

def device_weight(N, K, seed):
    """(PackedWeight, its 64-bit values on the device), quantised there."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes, scales, ts = nv.quantize(torch.randn(N, K, generator=g, device="cuda") * 0.05)
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    nib = torch.stack((codes & 15, codes >> 4), dim=2).view(N, K)
    v = torch.where(nib >= 8, -lut[(nib & 7).long()], lut[(nib & 7).long()])
    s = scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=1)
    gscale = float(ts[0].item())
    return nv.PackedWeight.from_canonical(codes, scales, gscale, N, K), v * s * gscale


def device_check(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    assert (err <= bound).all(), "%s: worst err/bound %.3g" % (what, float((err / bound).max()))


# (n, rows, K) of each tile (rows, tokens, K groups), in one part and in several,
# with n, rows and K that end inside a tile
TILES = [((32, 32, 4), 1, (45, 176, 272)), ((32, 32, 4), 2, (17, 80, 6160)),
         ((32, 32, 8), 1, (17, 4112, 3088)), ((32, 32, 8), 2, (33, 80, 12304)),
         ((64, 32, 4), 1, (33, 4624, 144)), ((64, 32, 4), 2, (33, 1040, 6160)),
         ((64, 64, 4), 1, (100, 5136, 784)), ((64, 64, 4), 2, (193, 1328, 9232)),
         ((128, 64, 2), 1, (201, 5136, 272)), ((128, 64, 2), 2, (33, 2576, 16400)),
         ((256, 128, 2), 1, (701, 8208, 1552)), ((256, 128, 2), 2, (401, 5136, 6160)),
         ((256, 128, 1), 1, (257, 16400, 272)), ((256, 128, 1), 2, (1001, 5136, 6160))]


@pytest.mark.parametrize("tile,parts,shape", TILES)
def test_every_tile(tile, parts, shape):
    n, rows, K = shape
    say("tile", tile, parts, shape)
    w, W = device_weight(rows, K, 80)
    X = randn((n, K), 81)
    F = rows // 32 * 16 - 3
    for geo in (nv.fused_geometry(n, rows, K), nv.fused_geometry(n, nv.gated_rows(F), K)):
        assert geo[:3] == tile and min(geo[3], 2) == parts, geo
    mag = X.double().abs() @ W.abs().t()
    ref = X.double() @ W.t()
    sums = (K + 32) * R.HALF_F32 * mag
    device_check(nv.linear(w, X, out_dtype=F32), ref, sums + R.HALF_F32 * ref.abs(), "linear")
    # the gated weight of the same number of packed rows
    (g, Wg), (u, Wu) = device_weight(F, K, 82), device_weight(F, K, 83)
    gw = nv.GatedWeight.from_packed(g, u)
    G, U = X.double() @ Wg.t(), X.double() @ Wu.t()
    eg = (K + 32) * R.HALF_F32 * (X.double().abs() @ Wg.abs().t())
    eu = (K + 32) * R.HALF_F32 * (X.double().abs() @ Wu.abs().t())
    device_check(nv.gated(gw, X, activation="none", out_dtype=F32), G * U,
                 G.abs() * eu + U.abs() * eg + eg * eu + 2 * R.HALF_F32 * (G * U).abs(), "gated")
    # the other way: a weight of K rows and `rows` columns
    t, Wt = device_weight(K - 5, rows, 84)
    dY = randn((n, K - 5), 85)
    ref = dY.double() @ Wt
    b = (K + 32) * R.HALF_F32 * (dY.double().abs() @ Wt.abs())
    device_check(nv.gemm_t(t.transpose(), dY), ref, b + R.HALF_BF16 * (ref.abs() + b) + 2.0 ** -133, "gemm_t")


def test_offsets_beyond_32_bits():
    """Rows of the output, the residual and the pre-activations that lie more
    than 2^31 elements into their buffers."""
    say("far rows")
    n, N, K, ld = 1100, 72, 144, 1 << 21
    w, W = device_weight(N, K, 86)
    X = randn((n, K), 87)
    r = randn((n, N), 88)
    far = torch.empty_strided((n, N), (ld, 1), dtype=BF16, device="cuda")
    out = torch.empty_strided((n, N), (ld, 1), dtype=BF16, device="cuda")
    pre = torch.empty_strided((n, N), (ld, 1), dtype=F32, device="cuda")
    far.copy_(r)
    assert torch.equal(nv.linear(w, X, activation="silu", residual=far, out=out, preact=pre),
                       nv.linear(w, X, activation="silu", residual=r))
    dY = randn((n, N), 89)
    far.copy_(dY)
    near = torch.empty(n, N, device="cuda")
    near.copy_(pre)
    wt = w.transpose()
    for a, b in zip(nv.linear_backward(wt, far, "silu", pre, F32), nv.linear_backward(wt, dY, "silu", near, F32)):
        assert torch.equal(a, b)
    Xf = torch.empty_strided((n, K), (ld, 1), dtype=BF16, device="cuda")
    Xf.copy_(X)
    assert torch.equal(nv.linear(w, Xf), nv.linear(w, X))
    assert torch.equal(nv.linear(w, Xf[1090:]), nv.linear(w, X[1090:]))


# ---- every specialisation of the decode product -----------------------------------------

@pytest.mark.parametrize("n", [1, 6, 11, 16])
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("tiles", range(1, 9))
def test_every_decode_variant(tiles, exact, n):
    """The linear form without an epilogue gives the plain projection's bits, the
    gated form without an activation the product of two fp32 projections."""
    K, N = 1024 * tiles - (0 if exact else 112), 83
    say("decode", tiles, exact, n)
    assert nv.gemv_variant(n, N, K)[:3] == (tiles, (n + 3) // 4, int(exact))
    (g, _), (u, _) = device_weight(N, K, 90), device_weight(N, K, 91)
    X = randn((n, K), 92)
    assert torch.equal(nv.linear(g, X), nv.gemv(g, X))
    want = nv.linear(g, X, out_dtype=F32) * nv.linear(u, X, out_dtype=F32)
    assert torch.equal(nv.gated(nv.GatedWeight.from_packed(g, u), X, activation="none", out_dtype=F32), want)


# (128-column tiles a wave, N, K) of calls in K parts
PARTS = [(1, 83, 8208), (1, 83, 30000), (2, 20000, 20480), (3, 1000, 9216), (4, 1003, 13312), (5, 1000, 17408),
         (6, 1000, 24576), (7, 877, 59072), (8, 1000, 30000)]


@pytest.mark.parametrize("n", [1, 6, 11, 16])
@pytest.mark.parametrize("tiles,N,K", PARTS)
def test_every_decode_part_variant(tiles, N, K, n):
    say("decode parts", tiles, N, K, n)
    assert nv.gemv_variant(n, N, K, 0)[0] == tiles and nv.gemv_kparts(N, K) > 1
    (g, _), (u, _) = device_weight(N, K, 93), device_weight(N, K, 94)
    X = randn((n, K), 95)
    assert torch.equal(nv.linear(g, X), nv.gemv_ws(g, X))
    H = nv.gated(nv.GatedWeight.from_packed(g, u), X, activation="none", out_dtype=F32)
    G, U = nv.linear(g, X, out_dtype=F32), nv.linear(u, X, out_dtype=F32)
    # the gated weight has more rows, so maybe another number of parts: the order of the sums
    e = 64 * R.HALF_F32 * (G.abs().max() * U.abs().max())
    assert (H - G * U).abs().max() <= e * (K / 64)


@pytest.mark.parametrize("n", [3, 16])
def test_decode_with_many_row_groups(n):
    """More row groups a workgroup than LDS has places for: several batches."""
    say("many rows", n)
    N, K = 70003, 144
    (g, _), (u, _) = device_weight(N, K, 96), device_weight(N, K, 97)
    X = randn((n, K), 98)
    r = randn((n, N), 99)
    assert torch.equal(nv.linear(g, X), nv.gemv(g, X))
    G, U = nv.linear(g, X, out_dtype=F32), nv.linear(u, X, out_dtype=F32)
    assert torch.equal(nv.linear(g, X, residual=r), (G + r.float()).to(BF16))
    assert torch.equal(nv.gated(nv.GatedWeight.from_packed(g, u), X, activation="none", out_dtype=F32), G * U)


# ---- transposed copies that belong to another weight ----------------------------------

def test_transposed_copy_of_another_weight():
    say("foreign transposed copies")
    w, _ = weight(96, 144, 100)
    other, _ = weight(96, 144, 101)
    gw, go = nv.GatedWeight.from_packed(w, other), nv.GatedWeight.from_packed(other, w)
    plain = nv.PackedWeight(gw.codes, gw.scales, 1.0, nv.gated_rows(96), 144)    # the gated rows as one weight
    X = randn((5, 144), 102).requires_grad_()
    for f, a, foreign in ((nv.linear, w, (other.transpose(),)), (nv.linear, plain, (gw.transpose(),)),
                          (nv.gated, gw, (go.transpose(), plain.transpose()))):
        for t in foreign:
            with pytest.raises(ValueError, match="transposed copy"):
                f(a, X, transposed=t)
        assert torch.isfinite(torch.autograd.grad(f(a, X, transposed=a.transpose()).sum(), X)[0]).all()
    z = torch.zeros(5, nv.preact_columns(gw), device="cuda")
    dH = randn((5, 96), 103)
    for t in (go.transpose(), plain.transpose()):
        with pytest.raises(ValueError, match="transposed copy"):
            nv.gated_backward(gw, t, dH, z)
    with pytest.raises(ValueError, match="gated weight"):
        nv.linear_backward(gw.transpose(), randn((5, nv.gated_rows(96)), 104))


# ---- derivatives that would be lost -----------------------------------------------------

def test_derivatives_are_not_dropped():
    """Calls without a graph refuse what asks for one, and forward-mode tangents."""
    say("dropped derivatives")
    from torch.autograd import forward_ad as fwd
    w, _ = weight(40, 272, 105)
    gw = nv.GatedWeight.from_packed(w, w)
    wt, gt = w.transpose(), gw.transpose()
    X, dY, r, b = randn((5, 272), 106), randn((5, 40), 107), randn((5, 40), 108), randn((40,), 109)
    z = torch.zeros(5, nv.preact_columns(gw), device="cuda")
    out = torch.empty(5, 40, device="cuda", dtype=BF16)
    zl = torch.zeros(5, nv.preact_columns(w), device="cuda")
    calls = {  # by the argument that carries the derivative
        "gemm_t dY": (dY, lambda t: nv.gemm_t(wt, t)),
        "linear_backward dY": (dY, lambda t: nv.linear_backward(wt, t, bias_dtype=F32)),
        "linear_backward preact": (zl, lambda t: nv.linear_backward(wt, dY, "silu", t)),
        "gated_backward dH": (dY, lambda t: nv.gated_backward(gw, gt, t, z)),
        "gated_backward preact": (z, lambda t: nv.gated_backward(gw, gt, dY, t)),
        "linear out": (out, lambda t: nv.linear(w, X, out=t)),
        "gated out": (out, lambda t: nv.gated(gw, X, out=t)),
        "linear preact": (zl, lambda t: nv.linear(w, X, preact=t)),
    }
    for name, (t, f) in calls.items():
        leaf = t.clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            f(leaf)
        with torch.no_grad():
            f(leaf)                                   # nothing is asked for
        f(leaf.detach())
    tangents = dict(calls, **{
        "linear X": (X, lambda t: nv.linear(w, t)),
        "linear bias": (b, lambda t: nv.linear(w, X, bias=t)),
        "linear residual": (r, lambda t: nv.linear(w, X, residual=t)),
        "gated X": (X, lambda t: nv.gated(gw, t)),
        "gated bias": (b, lambda t: nv.gated(gw, X, up_bias=t)),
    })
    for name, (t, f) in tangents.items():
        want = f(t.clone())
        with fwd.dual_level():
            with pytest.raises(ValueError, match="forward-mode"):
                f(fwd.make_dual(t.clone(), torch.ones_like(t)))
            got = f(t.clone())                        # no tangent, nothing lost
        for p, q in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
            assert p is None or torch.equal(p, q), name


def test_written_buffers_are_modified_in_place():
    """A buffer that a graph saved and a call then overwrote is an error of that
    graph's backward pass, not another gradient."""
    say("versions")
    w, _ = weight(40, 272, 110)
    gw = nv.GatedWeight.from_packed(w, w)
    wt, gt = w.transpose(), gw.transpose()
    X, dY = randn((5, 272), 111), randn((5, 40), 112)
    z = torch.zeros(5, nv.preact_columns(gw), device="cuda")
    calls = {
        "linear out": ((5, 40), BF16, lambda t: nv.linear(w, X, out=t)),
        "linear preact": ((5, nv.preact_columns(w)), F32, lambda t: nv.linear(w, X, preact=t)),
        "gated out": ((5, 40), BF16, lambda t: nv.gated(gw, X, out=t)),
        "gated preact": ((5, nv.preact_columns(gw)), F32, lambda t: nv.gated(gw, X, preact=t)),
        "gemm_t out": ((5, 272), BF16, lambda t: nv.gemm_t(wt, dY, out=t)),
        "linear_backward out": ((5, 272), BF16, lambda t: nv.linear_backward(wt, dY, out=t)),
        "gated_backward out": ((5, 272), BF16, lambda t: nv.gated_backward(gw, gt, dY, z, out=t)),
    }
    for name, (shape, dtype, f) in calls.items():
        buf = torch.zeros(shape, device="cuda", dtype=dtype)
        f(buf)
        leaf = torch.ones_like(buf).requires_grad_()
        y = (leaf * buf).sum()
        f(buf)
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
        f(buf)
        (leaf * buf).sum().backward()
        assert torch.equal(leaf.grad, buf), name
        with torch.inference_mode():
            f(torch.zeros(shape, device="cuda", dtype=dtype))


# ---- the left tail of gelu ----------------------------------------------------------------

# Phi(z) in units of 2^-24 of its value: t = 1 / (1 + 0.4 x) is off by 4 (x, the
# sum, the reciprocal), the polynomial by 6, the two exponentials by 2 each, five
# products by 1 each, the fit by 1.5: 20.5.  2^-126 is where they are flushed.
PHI_EPS = 2.0 ** -19


@pytest.mark.parametrize("n", [1, 20])
def test_gelu_keeps_its_relative_precision(n):
    say("gelu tail", n)
    N, K = 4003, 16
    w, _ = weight(N, K, 113)
    z = torch.linspace(-14, 9, N, device="cuda")
    Y = nv.linear(w, torch.zeros(n, K, device="cuda", dtype=BF16), bias=z, activation="gelu", out_dtype=F32)
    z64 = f64(z)
    ref = R.act(z64, "gelu")
    bound = PHI_EPS * np.abs(ref) + np.abs(z64) * 2.0 ** -126
    check(Y, (np.tile(ref, (n, 1)), np.tile(bound, (n, 1))), "gelu")


def test_gelu_gradient_keeps_its_relative_precision():
    """Phi(z) + z phi(z), against the sum of both terms' magnitudes."""
    say("gelu gradient tail")
    N = 4000
    z = torch.linspace(-14, 9, N, device="cuda")[None]
    _, db = nv.linear_backward(None, torch.ones(1, N, device="cuda"), "gelu", z, F32)
    z64 = f64(z)[0]
    phi = np.exp(-z64 * z64 / 2) / np.sqrt(2 * np.pi)
    terms = 0.5 * R.special.erfc(-z64 / np.sqrt(2)) + np.abs(z64) * phi
    check(db, (R.act_grad(z64, "gelu"), PHI_EPS * terms + np.abs(z64) * 2.0 ** -125), "gelu'")


# ---- column slices of one buffer ----------------------------------------------------------

@pytest.mark.parametrize("n,N,K", [(5, 40, 272), (16, 93, 144), (40, 93, 272), (33, 72, 8208)])
def test_neighbouring_columns_of_one_buffer(n, N, K):
    """X, the residual and the output side by side in one buffer, the gradient's
    dY and dX in another: what contiguous calls give, and nothing else moves."""
    say("columns", n, N, K)
    w, _ = weight(N, K, 114)
    wt = w.transpose()
    X, r, dY = randn((n, K), 115), randn((n, N), 116), randn((n, N), 117)
    want = nv.linear(w, X, activation="silu", residual=r)
    pad = 4 + (-(K + 2 * N + 4)) % 8
    buf = torch.full((n, K + 2 * N + pad), 7.0, device="cuda", dtype=BF16)
    x, res, out = buf[:, :K], buf[:, K:K + N], buf[:, K + N + 1:K + 2 * N + 1]
    x.copy_(X)
    res.copy_(r)
    nv.linear(w, x, activation="silu", residual=res, out=out)
    assert torch.equal(out, want) and torch.equal(x, X) and torch.equal(res, r)
    assert (buf[:, K + N] == 7).all() and (buf[:, K + 2 * N + 1:] == 7).all()
    dX, db = nv.linear_backward(wt, dY, bias_dtype=F32)
    buf = torch.full((n, K + N + 8), 7.0, device="cuda", dtype=BF16)
    dy, dx = buf[:, 1:1 + N], buf[:, 3 + N:3 + N + K]
    dy.copy_(dY)
    got = nv.linear_backward(wt, dy, bias_dtype=F32, out=dx)
    assert torch.equal(dx, dX) and torch.equal(got[1], db) and torch.equal(dy, dY)
    assert (buf[:, 0] == 7).all() and (buf[:, 1 + N:3 + N] == 7).all() and (buf[:, 3 + N + K:] == 7).all()
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.linear_backward(wt, dy, out=buf[:, N:N + K])
    assert e.value.status == 10


def test_sizes_beyond_32_bits_are_refused():
    """A row or column count that the library's int would cut to a small one."""
    say("sizes beyond 32 bits")
    big = torch.zeros((1 << 32) + 64, device="cuda", dtype=BF16)
    for dY in (big[:, None], big[None]):
        with pytest.raises(ValueError, match="2\\^31"):
            nv.linear_backward(None, dY, bias_dtype=F32)
    w, _ = weight(1, 16, 118)
    with pytest.raises(ValueError, match="2\\^31"):
        nv.gemm_t(w.transpose(), big[:, None])
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.gemm_t(w.transpose(), big[:(1 << 20) + 1, None])
    assert e.value.status == 2


def test_quantising_on_another_stream_reads_its_own_tensor_scale():
    """The launch stream is behind (tens of ms) when the tensor scale is read."""
    say("from_float on a stream")
    W, V = randn((64, 256), 119, F32, 0.05), randn((64, 256), 120, F32, 0.02)
    want, gated = nv.PackedWeight.from_float(W), nv.GatedWeight.from_float(W, V)
    old = [torch.full((2,), 123.0, device="cuda") for _ in range(64)]
    del old                               # what new small tensors find in their memory
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):            # the same for memory of that stream
        old = [torch.full((2,), 123.0, device="cuda") for _ in range(64)]
        del old
    torch.cuda.synchronize()

    def behind():
        with torch.cuda.stream(s):
            torch.cuda._sleep(50_000_000)
    behind()
    w = nv.PackedWeight.from_float(W, stream=s)
    assert w.gscale == want.gscale
    behind()
    g = nv.GatedWeight.from_float(W, V, stream=s)
    assert (g.gate_gscale, g.up_gscale) == (gated.gate_gscale, gated.up_gscale)
    s.synchronize()
    assert torch.equal(w.codes, want.codes) and torch.equal(w.scales, want.scales)
    assert torch.equal(g.codes, gated.codes) and torch.equal(g.scales, gated.scales)


# ---- gradients in K parts, of many row blocks, of fp32 gradients; every tile's epilogue ---

def linear_step(w, W, n, seed, act, out=BF16, bias=F32, what=""):
    """A training step in two ways, with and without autograd, against 64 bits:
    output, pre-activations, dX and the bias gradient."""
    N, K = W.shape
    wt = w.transpose()
    X, b, r = randn((n, K), seed), randn((N,), seed + 1, bias), randn((n, N), seed + 2, out, 2.0)
    dY = randn((n, N), seed + 3, out, 0.1)
    z = torch.full((n, nv.preact_columns(w)), float("nan"), device="cuda")
    Y = nv.linear(w, X, bias=b, activation=act, residual=r, out_dtype=out, preact=z)
    x, bb = f64(X), f64(b)
    check(Y, R.linear(x, W, bb, act, f64(r), out == F32), what + " Y")
    p, ep = R.pre(x, W, bb)
    check(z[:, :N], (p, ep + R.HALF_F32 * (np.abs(p) + ep)), what + " preact")
    dX, db = nv.linear_backward(wt, dY, act, z, bias)
    want_x, want_b = R.linear_grads(x, W, f64(dY), bb, act, bias == F32)
    check(dX, want_x, what + " dX")
    check(db, want_b, what + " db")
    Xg, bg = X.clone().requires_grad_(), b.clone().requires_grad_()
    Yg = nv.linear(w, Xg, bias=bg, activation=act, residual=r, out_dtype=out, transposed=wt)
    for a, q in zip((Yg,) + torch.autograd.grad(Yg, [Xg, bg], dY), (Y, dX, db)):
        assert torch.equal(a, q), what


def gated_step(g, Wg, u, Wu, n, seed, act, out=BF16, bias=F32, what=""):
    F, K = Wg.shape
    w = nv.GatedWeight.from_packed(g, u)
    wt = w.transpose()
    X, bg, bu = randn((n, K), seed), randn((F,), seed + 1, bias), randn((F,), seed + 2, bias)
    dH = randn((n, F), seed + 3, out, 0.1)
    z = torch.full((n, nv.preact_columns(w)), float("nan"), device="cuda")
    H = nv.gated(w, X, activation=act, gate_bias=bg, up_bias=bu, out_dtype=out, preact=z)
    x, gb, ub = f64(X), f64(bg), f64(bu)
    check(H, R.gated(x, Wg, Wu, gb, ub, act, out == F32), what + " H")
    rows = torch.arange(F, device="cuda")
    rows = rows // 16 * 32 + rows % 16
    for W, b, at in ((Wg, gb, rows), (Wu, ub, rows + 16)):
        p, ep = R.pre(x, W, b)
        check(z[:, at], (p, ep + R.HALF_F32 * (np.abs(p) + ep)), what + " preact")
    got = nv.gated_backward(w, wt, dH, z, act, bias)
    for a, want, name in zip(got, R.gated_grads(x, Wg, Wu, f64(dH), gb, ub, act, bias == F32), ("dX", "dbg", "dbu")):
        check(a, want, what + " " + name)
    leaves = [t.clone().requires_grad_() for t in (X, bg, bu)]
    Hg = nv.gated(w, leaves[0], activation=act, gate_bias=leaves[1], up_bias=leaves[2], out_dtype=out, transposed=wt)
    for a, q in zip((Hg,) + torch.autograd.grad(Hg, leaves, dH), (H,) + got):
        assert torch.equal(a, q), what


@pytest.mark.parametrize("n", [1, 7, 16])
@pytest.mark.parametrize("act,out,bias", [("silu", BF16, F32), ("gelu", F32, BF16)])
def test_training_step_with_a_decode_product_in_parts(n, act, out, bias):
    """K > 8192 at few tokens: the second launch stores the pre-activations."""
    say("step, decode parts", n, act)
    N, K = 83, 8208
    assert nv.gemv_kparts(N, K) > 1 and nv.gemv_kparts(nv.gated_rows(N), K) > 1
    (g, Wg), (u, Wu) = weight(N, K, 121), weight(N, K, 122, 0.02)
    linear_step(g, Wg, n, 123, act, out, bias, "linear")
    gated_step(g, Wg, u, Wu, n, 127, act, out, bias, "gated")


@pytest.mark.parametrize("n,N,K", [(33, 5140, 8208), (100, 5140, 4112)])
def test_training_step_in_parts_both_ways(n, N, K):
    """Forward and backward products in K parts, with bias gradients of several
    row blocks: the workspace holds dZ, column sums and partial sums."""
    say("step, parts", n, N, K)
    F = N // 2
    for rows, k in ((N, K), (nv.gated_rows(F), K), (K, N + (-N) % 8), (K, nv.gated_rows(F))):
        assert nv.fused_geometry(n, rows, k)[3] > 1
    w, W = device_weight(N, K, 131)
    linear_step(w, f64(W), n, 132, "gelu_tanh", what="linear")
    (g, Wg), (u, Wu) = device_weight(F, K, 136), device_weight(F, K, 137)
    gated_step(g, f64(Wg), u, f64(Wu), n, 138, "silu", what="gated")


@pytest.mark.parametrize("n,N", [(450, 16400), (1001, 8210), (40000, 40)])
def test_column_sums_of_many_rows_a_block(n, N):
    """More token rows a block of the gradient kernel than its eight at a time
    (2048 blocks in all, 256 columns each), and the same bits again."""
    say("rows a block", n, N)
    K = 48
    assert n > 8 * -(-2048 // -(-N // 256))
    (g, Wg), (u, Wu) = weight(N, K, 142), weight(N, K, 143, 0.02)
    linear_step(g, Wg, n, 144, "silu", what="linear")
    gated_step(g, Wg, u, Wu, n, 148, "gelu", what="gated")
    wt, dY, z = g.transpose(), randn((n, N), 152), randn((n, nv.preact_columns(g)), 153, F32)
    first = nv.linear_backward(wt, dY, "gelu", z, F32)
    for _ in range(3):
        for a, b in zip(first, nv.linear_backward(wt, dY, "gelu", z, F32)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n,N,K", [(1, 93, 144), (16, 200, 656), (33, 93, 144), (150, 330, 272), (33, 5140, 4112)])
def test_fp32_gradients(n, N, K):
    """dY and dH in fp32, rows unaligned, without an activation and with one."""
    say("fp32 dY", n, N, K)
    (w, W), (u, U) = device_weight(N, K, 154), device_weight(N, K, 155)
    W, U = f64(W), f64(U)
    X = randn((n, K), 156)
    buf = randn((n, N + 3), 157, F32, 0.1)
    dY = buf[:, 1:N + 1]
    z = torch.empty(n, nv.preact_columns(w), device="cuda")
    for act in ("none", "gelu"):
        nv.linear(w, X, activation=act, preact=z)
        dX, db = nv.linear_backward(w.transpose(), dY, act, z, BF16)
        want_x, want_b = R.linear_grads(f64(X), W, f64(dY), None, act, False)
        check(dX, want_x, "dX " + act)
        check(db, want_b, "db " + act)
    gw = nv.GatedWeight.from_packed(w, u)
    z = torch.empty(n, nv.preact_columns(gw), device="cuda")
    nv.gated(gw, X, preact=z)
    for a, want in zip(nv.gated_backward(gw, gw.transpose(), dY, z, "silu", F32),
                       R.gated_grads(f64(X), W, U, f64(dY), None, None, "silu", True)):
        check(a, want, "gated")


@pytest.mark.parametrize("tile,parts,shape", TILES)
def test_every_tile_with_an_epilogue(tile, parts, shape):
    """Bias, activation, residual and pre-activations in each tile, in one part
    and in several; the bounds of fused_reference.linear and gated."""
    n, rows, K = shape
    say("tile epilogue", tile, parts, shape)
    F = rows // 32 * 16 - 3
    for geo in (nv.fused_geometry(n, rows, K), nv.fused_geometry(n, nv.gated_rows(F), K)):
        assert geo[:3] == tile and min(geo[3], 2) == parts, geo
    X = randn((n, K), 158)
    x = X.double()

    def pre(W, b):
        p = x @ W.t() + b.double()
        return p, (K + 32) * R.HALF_F32 * (x.abs() @ W.abs().t() + b.double().abs())

    def silu(p, e):
        a = p * torch.sigmoid(p)
        return a, R.LIP * e + R.ACT_EPS * (1 + a.abs())

    w, W = device_weight(rows, K, 159)
    b, r = randn((rows,), 160), randn((n, rows), 161, F32, 2.0)
    z = torch.full((n, nv.preact_columns(w)), float("nan"), device="cuda")
    Y = nv.linear(w, X, bias=b, activation="silu", residual=r, preact=z)
    p, e = pre(W, b)
    device_check(z[:, :rows], p, e + R.HALF_F32 * (p.abs() + e), "preact")
    y, e = silu(p, e)
    y = y + r.double()
    e = e + R.HALF_F32 * y.abs()
    device_check(Y, y, e + R.HALF_BF16 * (y.abs() + e) + 2.0 ** -133, "linear")
    del W, y, p, e
    (g, Wg), (u, Wu) = device_weight(F, K, 162), device_weight(F, K, 163)
    gw = nv.GatedWeight.from_packed(g, u)
    bg, bu = randn((F,), 164, F32), randn((F,), 165, F32)
    z = torch.full((n, nv.preact_columns(gw)), float("nan"), device="cuda")
    H = nv.gated(gw, X, gate_bias=bg, up_bias=bu, preact=z)
    at = torch.arange(F, device="cuda")
    at = at // 16 * 32 + at % 16
    (pg, eg), (pu, eu) = pre(Wg, bg), pre(Wu, bu)
    device_check(z[:, at], pg, eg + R.HALF_F32 * (pg.abs() + eg), "gate preact")
    device_check(z[:, at + 16], pu, eu + R.HALF_F32 * (pu.abs() + eu), "up preact")
    a, ea = silu(pg, eg)
    h = a * pu
    e = a.abs() * eu + pu.abs() * ea + ea * eu + R.HALF_F32 * h.abs()
    device_check(H, h, e + R.HALF_BF16 * (h.abs() + e) + 2.0 ** -133, "gated")


def test_graphs_of_steps_in_parts():
    """Captured training steps whose products run in K parts, each with workspaces
    of its graph, replayed in turn between eager calls."""
    say("graphs, parts")
    N, K = 83, 8208
    (g, _), (u, _) = weight(N, K, 166), weight(N, K, 167, 0.02)
    gw = nv.GatedWeight.from_packed(g, u)
    wt, gt = g.transpose(), gw.transpose()
    assert nv.fused_geometry(70, N, K)[3] > 1 and nv.fused_geometry(70, nv.gated_rows(N), K)[3] > 1

    def step(X, dY, b):
        z = torch.empty(X.shape[0], nv.preact_columns(g), device="cuda")
        zg = torch.empty(X.shape[0], nv.preact_columns(gw), device="cuda")
        Y = nv.linear(g, X, bias=b, activation="silu", preact=z)
        H = nv.gated(gw, X, gate_bias=b, preact=zg)
        return (Y, H) + nv.linear_backward(wt, dY, "silu", z, F32) + nv.gated_backward(gw, gt, dY, zg, "silu", F32)

    graphs = []
    for n in (5, 70):
        args = randn((n, K), 168), randn((n, N), 169), randn((N,), 170, F32)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            step(*args)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*args)
        graphs.append((args, graph, out))
    for trip in range(4):
        for args, graph, out in graphs:
            args[0].copy_(randn(args[0].shape, 171 + trip))
            args[1].copy_(randn(args[1].shape, 175 + trip))
            graph.replay()
            torch.cuda.synchronize()
            for o, e in zip(out, step(*args)):
                assert torch.equal(o, e), trip


@pytest.mark.parametrize("n,N,ldp,col", [(3, 92, 192, 100), (20, 93, 192, 96), (9, 1, 8, 4), (300, 332, 440, 108)])
def test_preactivations_in_the_last_columns_of_a_buffer(n, N, ldp, col):
    """Through the C entry points: nothing behind column N of the last row is
    theirs to read."""
    say("last columns", n, N, ldp, col)
    K = 144
    w, W = weight(N, K, 180)
    wt = w.transpose()
    X, dY = randn((n, K), 181), randn((n, N), 182)
    whole = torch.full((n * ldp,), float("nan"), device="cuda")
    whole = whole[:(n - 1) * ldp + col + N]
    stream = torch.cuda.current_stream().cuda_stream
    Y, dX, db = (torch.empty(s, device="cuda", dtype=t) for s, t in (((n, N), BF16), ((n, K), BF16), ((N,), F32)))
    ep = fused._EPILOGUE.pack(0, 0, 0, whole.data_ptr() + 4 * col, 0, ldp, 2, 1, 1, 1)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    fused._run("nvfp4_linear", w.codes.data_ptr(), w.scales.data_ptr(), w.gscale, X.data_ptr(), K, Y.data_ptr(), N, n,
               N, K, ep, ws.data_ptr(), ws.numel(), stream)
    fused._run("nvfp4_linear_backward", wt.codes.data_ptr(), wt.scales.data_ptr(), wt.gscale, dY.data_ptr(), 1, N,
               whole.data_ptr() + 4 * col, ldp, 2, dX.data_ptr(), K, db.data_ptr(), 0, n, N, K, ws.data_ptr(),
               ws.numel(), stream)
    check(Y, R.linear(f64(X), W, None, "silu"), "Y")
    want_x, want_b = R.linear_grads(f64(X), W, f64(dY), None, "silu", True)
    check(dX, want_x, "dX")
    check(db, want_b, "db")
    assert torch.isnan(whole[:col]).all()
