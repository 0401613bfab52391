"""GPU parity of the 8-bit projection: quantisation bit for bit, products against
exact integers within the bounds of experts_reference."""
import numpy as np
import pytest
import torch

import experts_reference as X8
import nvfp4_weight_only_02_amd as nv
from nvfp4_weight_only_02_amd import int8

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


def codes(shape, seed, low=-127):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, 128, shape, generator=g, dtype=torch.int32).to(torch.int8).cuda()


def check(got, want, what):
    ref, bound = want
    err = np.abs(f64(got) - ref)
    assert np.isfinite(f64(got)).all(), what
    assert (err <= bound).all(), "%s: worst err/bound %.3g" % (what, float((err / bound).max()))


def weight(N, K, seed, low=-127):
    q = codes((N, K), seed, low)
    s = randn((N,), seed + 1, F32).abs() * 0.01 + 1e-4
    return nv.Int8Weight.from_int8(q, s), q.cpu().numpy().astype(np.int64), f64(s)


# ---- quantisation -----------------------------------------------------------------------

@pytest.mark.parametrize("n,K", [(1, 16), (7, 48), (33, 2064), (3, 8192), (2, 8208), (5, 20000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize(n, K, dtype):
    say("quantize", n, K, dtype)
    X = randn((n, K), K, dtype) * torch.rand(n, 1, device="cuda").to(dtype) * 3
    q, s = nv.int8_quantize(X)
    rq, rs = X8.int8_quantize(f64(X), dtype == F32)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(f64(s), rs)
    assert q.dtype == torch.int8 and (q.abs().amax(1) == 127).all()


def test_quantize_halves_and_every_pair_of_mantissas():
    """All quotients of a bf16 mantissa and a maximum's, at the exponents where
    the result is not zero: the halves among them go to the even integer."""
    say("quantize mantissas")
    tops = (torch.arange(128, 256, dtype=F32) / 128).cuda()
    vals = torch.cat([(torch.arange(128, 256, dtype=F32) / 128) * 2.0 ** -e for e in range(0, 10)]).cuda()
    X = vals.repeat(128, 1)
    X = torch.where(X <= tops[:, None], X, torch.zeros_like(X)) * torch.tensor([1.0, -1.0], device="cuda").repeat(640)
    X = torch.cat([tops[:, None], torch.zeros(128, 15, device="cuda"), X], 1).to(BF16)
    q, s = nv.int8_quantize(X)
    rq, rs = X8.int8_quantize(f64(X))
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(f64(s), rs)


@pytest.mark.parametrize("n,K", [(3, 32784), (2, 131056), (1, 200000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_rows_longer_than_the_registers_hold(n, K, dtype):
    """The rest of a row is read again for the division; in one row the largest value
    lies there, in another before."""
    say("quantize again", n, K, dtype)
    X = randn((n, K), K, dtype)
    X[0, K - 5] = 9.0
    X[n - 1, 11] = -8.5 if n > 1 else 1.0
    q, s = nv.int8_quantize(X)
    rq, rs = X8.int8_quantize(f64(X), dtype == F32)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(f64(s), rs)


@pytest.mark.parametrize("dtype,K", [(F32, (1 << 29) + 16), (BF16, (1 << 30) + 16)])
def test_quantize_rows_of_more_than_2_31_bytes(dtype, K):
    say("quantize long", dtype, K)
    X = torch.zeros(1, K, device="cuda", dtype=dtype)
    X[0, 5], X[0, K // 2 + 3], X[0, K - 9], X[0, K - 1] = 1.0, -0.5, -2.0, 0.25
    q, s = nv.int8_quantize(X)
    assert f64(s)[0] == np.float32(2) / np.float32(127)
    # 63.5, 31.75, 127 and 15.875 steps: halves go to the even integer
    assert [int(q[0, c]) for c in (5, K // 2 + 3, K - 9, K - 1)] == [64, -32, -127, 16]
    assert int(torch.count_nonzero(q)) == 4


def test_from_float_refuses_a_row_too_long_before_reading_it():
    say("int8 from_float long")
    for K in (131072, 131064, 8):
        with pytest.raises(ValueError):
            nv.Int8Weight.from_float(torch.ones(1, 1, device="cuda").expand(2, K))
    with pytest.raises(ValueError):
        nv.Int8Weight.from_float(torch.ones(64, device="cuda"))


def test_the_weight_keeps_its_own_scales():
    """The caller's buffers may be used again, for the next weight say."""
    say("int8 own scales")
    q, s, X = codes((40, 64), 50), randn((40,), 51, F32).abs(), randn((5, 64), 52)
    w = nv.Int8Weight.from_int8(q, s)
    want = nv.int8_linear(w, X)
    q.zero_()
    s.fill_(7.0)
    assert torch.equal(nv.int8_linear(w, X), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s = codes((40, 64), 50), randn((40,), 51, F32).abs()
    side.wait_stream(torch.cuda.current_stream())
    w = nv.Int8Weight.from_int8(q, s, stream=side)
    side.synchronize()
    s.fill_(7.0)
    assert torch.equal(nv.int8_linear(w, X), want)
    with pytest.raises(ValueError):
        nv.Int8Weight.from_int8(q, s.requires_grad_())


def test_quantize_extremes():
    say("quantize extremes")
    X = randn((8, 64), 3)
    X[1] = 0
    X[2, 5] = NAN
    X[3, 6] = -INF
    X[4] = 0
    X[4, 7], X[4, 8] = 2.0 ** -133, -(2.0 ** -133)      # the least bf16
    X[5] = 3.3895313892515355e38                         # the largest
    X[5, 1] = -X[5, 0]
    X[6, 9] = 2.0 ** 120
    q, s = nv.int8_quantize(X)
    assert (q[1] == 0).all() and s[1] == 0
    assert (q[2] == 0).all() and (q[3] == 0).all() and torch.isnan(s[2:4]).all()
    assert q[4, 7] == 127 and q[4, 8] == -127 and (q[4, :7] == 0).all()
    assert (q[5, 2:] == 127).all() and q[5, 1] == -127 and torch.isfinite(s[5])
    assert q[6, 9] == 127 and q[6].abs().sum() == 127
    keep = [0, 7]
    rq, rs = X8.int8_quantize(f64(X[keep]))
    assert np.array_equal(q[keep].cpu().numpy(), rq) and np.array_equal(f64(s[keep]), rs)


# ---- product ------------------------------------------------------------------------------

SHAPES = [(1, 16), (37, 144), (200, 656), (64, 8208), (330, 2064), (1040, 272)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 64, 100, 300, 520])
@pytest.mark.parametrize("quantized,act,bias,residual,out", [
    (False, "none", None, None, BF16), (True, "silu", BF16, BF16, BF16), (True, "gelu", F32, F32, F32),
    (False, "gelu_tanh", F32, None, F32), (True, "relu", None, F32, BF16), (True, "none", None, None, F32)])
def test_linear(n, N, K, quantized, act, bias, residual, out):
    say("int8 linear", n, N, K, quantized, act, bias, residual, out)
    w, wq, ws = weight(N, K, N, -128)
    b = None if bias is None else randn((N,), 3, bias)
    r = None if residual is None else randn((n, N), 4, residual, 3.0)
    if quantized:
        q, s = codes((n, K), 5, -128), randn((n,), 6, F32).abs() * 0.01
        Y = nv.int8_linear(w, q, s, b, act, r, out_dtype=out)
        rq, rs = q.cpu().numpy().astype(np.int64), f64(s)
    else:
        X = randn((n, K), 7)
        Y = nv.int8_linear(w, X, None, b, act, r, out_dtype=out)
        rq, rs = X8.int8_quantize(f64(X))
        q, s = nv.int8_quantize(X)
        assert torch.equal(nv.int8_linear(w, q, s, b, act, r, out_dtype=out), Y)
    assert Y.dtype == out
    check(Y, X8.int8_linear(rq, rs, wq, ws, None if b is None else f64(b), act, None if r is None else f64(r), out == F32), "Y")


@pytest.mark.parametrize("n,N,K,geometry", [
    (60, 330, 2064, (64, 32, 4, 1)), (40, 40, 8208, (64, 32, 4, 8)), (70, 9000, 144, (128, 64, 1, 1)),
    (75, 2000, 8208, (128, 64, 1, 8)), (520, 1040, 1040, (128, 64, 2, 1)), (40, 9000, 8208, (128, 64, 2, 3)),
    (520, 4090, 144, (128, 128, 1, 1)), (150, 4096, 8208, (128, 128, 1, 4)), (2000, 4090, 272, (256, 128, 1, 1)),
    (2050, 5120, 400, (256, 256, 1, 1)), (520, 4090, 8208, (256, 128, 1, 3))])
def test_every_tile(n, N, K, geometry):
    """Every tile of the many-token product, with K parts where it takes them, the
    sizes no multiple of the tile's."""
    say("int8 tile", n, N, K, geometry)
    assert nv.int8_geometry(n, N, K) == geometry
    w, wq, ws = weight(N, K, 40, -128)
    q, s = codes((n, K), 41, -128), randn((n,), 42, F32).abs() * 0.01
    b, r = randn((N,), 43, F32), randn((n, N), 44, BF16, 3.0)
    # (sums below 2^31: exact in 64-bit floats too)
    args = f64(q), f64(s), wq.astype(np.float64), ws, f64(b)
    check(nv.int8_linear(w, q, s, b, "silu", r), X8.int8_linear(*args, "silu", f64(r)), "Y")
    check(nv.int8_linear(w, q, s, b, "none", out_dtype=F32), X8.int8_linear(*args, "none", None, True), "Y")


@pytest.mark.parametrize("n,K", [(8, 6144), (5, 4112), (7, 7008), (3, 16384), (2, 24576), (1, 49152), (1, 33040)])
def test_rows_that_a_decode_launch_quantises_longer_than_its_registers_hold(n, K):
    say("int8 decode, long rows", n, K)
    assert nv.int8_linear_workspace_bytes(n, 70, K) == 0       # quantised in the launch
    w, wq, ws = weight(70, K, 60)
    X = randn((n, K), 61)
    X[0, K - 3] = 12.0
    q, s = X8.int8_quantize(f64(X))
    Y = nv.int8_linear(w, X, out_dtype=F32)
    check(Y, X8.int8_linear(q, s, wq, ws, out_f32=True), "Y")
    assert torch.equal(nv.int8_linear(w, *nv.int8_quantize(X), out_dtype=F32), Y)


@pytest.mark.parametrize("N,n", [(16384, 3), (9000, 16), (2000, 1), (16001, 5), (5120, 700)])
def test_many_rows(N, n):
    say("int8 rows", N, n)
    w, wq, ws = weight(N, 400, 9)
    X = randn((n, 400), 10)
    check(nv.int8_linear(w, X, out_dtype=F32), X8.int8_linear(*X8.int8_quantize(f64(X)), wq, ws, out_f32=True), "Y")


@pytest.mark.parametrize("n", [1, 16, 20, 70, 600])
def test_largest_sums_are_exact(n):
    """-128 everywhere at the longest rows: 128 * 128 * 131056 is just below 2^31."""
    say("int8 largest", n)
    N, K = 48, 131056
    w = nv.Int8Weight.from_int8(torch.full((N, K), -128, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda"))
    q = torch.full((n, K), -128, dtype=torch.int8, device="cuda")
    Y = nv.int8_linear(w, q, torch.ones(n, device="cuda"), out_dtype=F32)
    assert (Y == float(np.float32(128 * 128 * K))).all()
    q[0] = 127
    Y = nv.int8_linear(w, q, torch.ones(n, device="cuda"), out_dtype=F32)
    assert (Y[0] == float(np.float32(-127 * 128 * K))).all()


def test_from_float_is_the_row_quantisation():
    say("int8 from_float")
    for dtype in (F32, BF16):
        W = randn((70, 272), 11, dtype, 0.02)
        w = nv.Int8Weight.from_float(W)
        q, s = nv.int8_quantize(W)
        v = nv.Int8Weight.from_int8(q, s)
        assert torch.equal(w.codes, v.codes) and torch.equal(w.scale, s)


@pytest.mark.parametrize("n", [3, 40, 530])
def test_strides_guards_workspaces_and_in_place_residual(n):
    say("int8 strides", n)
    N, K = 69, 272
    w, _, _ = weight(N, K, 12)
    X = randn((n, 2 * K + 16), 13)[:, 16:16 + K]
    want = nv.int8_linear(w, X.contiguous())
    assert torch.equal(nv.int8_linear(w, X), want)
    q = codes((n, K + 48), 14)[:, 32:32 + K]
    s = randn((n,), 15, F32).abs()
    assert torch.equal(nv.int8_linear(w, q, s), nv.int8_linear(w, q.contiguous(), s))
    for col in (0, 3, 4):
        out = torch.full((n + 2, N + 9), 7.0, device="cuda", dtype=BF16)
        assert torch.equal(nv.int8_linear(w, X, out=out[1:n + 1, col:col + N]), want)
        out[1:n + 1, col:col + N] = 7.0
        assert (out == 7.0).all()
    r = randn((n, N + 3), 16, F32)
    want = nv.int8_linear(w, X, residual=r[:, 1:1 + N], out_dtype=F32)
    got = r.clone()
    nv.int8_linear(w, X, residual=got[:, 1:1 + N], out=got[:, 1:1 + N])
    assert torch.equal(got[:, 1:1 + N], want) and torch.equal(got[:, 0], r[:, 0])
    need = nv.int8_linear_workspace_bytes(n, N, K)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(nv.int8_linear(w, X, residual=r[:, 1:1 + N], out_dtype=F32, workspace=ws[:need]), want)
    assert (ws[need:] == 255).all()


@pytest.mark.parametrize("n", [9, 100])
def test_results_repeat_and_do_not_depend_on_the_batch(n):
    """Integer sums have no order: a token's result is the same in any batch."""
    say("int8 batch", n)
    w, _, _ = weight(200, 2064, 17)
    X = randn((600, 2064), 18)
    for bias in (None, randn((200,), 30, F32)):
        whole = nv.int8_linear(w, X, bias=bias, activation="silu", out_dtype=F32)
        for a in (0, 31, 600 - n):
            assert torch.equal(nv.int8_linear(w, X[a:a + n], bias=bias, activation="silu", out_dtype=F32), whole[a:a + n])


@pytest.mark.parametrize("n", [6, 80, 530])
def test_nonfinite_stays_in_its_token(n):
    say("int8 nonfinite", n)
    w, _, _ = weight(70, 272, 19)
    X = randn((n, 272), 20)
    clean = nv.int8_linear(w, X)
    X[4, 100] = NAN
    X[2, 3] = INF
    got = nv.int8_linear(w, X)
    keep = [t for t in range(n) if t not in (2, 4)]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[[2, 4]]).all()


def test_no_tokens():
    say("int8 none")
    w, _, _ = weight(70, 272, 21)
    assert nv.int8_linear(w, torch.empty(0, 272, device="cuda", dtype=BF16)).shape == (0, 70)
    q, s = nv.int8_quantize(torch.empty(0, 272, device="cuda", dtype=BF16))
    assert q.shape == (0, 272) and s.shape == (0,)


def test_graph_replays_and_streams():
    say("int8 graphs")
    w, _, _ = weight(300, 4112, 22)
    graphs = []
    for n in (1, 7, 40, 600):
        X = randn((n, 4112), 23)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            nv.int8_linear(w, X)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = nv.int8_linear(w, X)
        graphs.append((X, graph, out))
    for trip in range(4):
        for X, graph, out in graphs:
            X.copy_(randn(tuple(X.shape), 24 + trip))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, nv.int8_linear(w, X))
    s = torch.cuda.Stream()
    X = graphs[2][0]
    s.wait_stream(torch.cuda.current_stream())
    Y = nv.int8_linear(w, X, stream=s)
    q, sc = nv.int8_quantize(X, stream=s)
    Z = nv.int8_linear(nv.Int8Weight.from_float(randn((32, 4112), 25, F32), stream=s), q, sc, stream=s)
    s.synchronize()
    assert torch.equal(Y, nv.int8_linear(w, X))
    assert torch.equal(Z, nv.int8_linear(nv.Int8Weight.from_float(randn((32, 4112), 25, F32)), X))


def test_refusals():
    say("int8 refusals")
    w, _, _ = weight(40, 64, 26)
    pw = nv.PackedWeight.from_float(randn((40, 64), 27, F32))
    X, q, s = randn((5, 64), 28), codes((5, 64), 29), torch.ones(5, device="cuda")
    bad = [
        (TypeError, lambda: nv.int8_linear(pw, X)), (TypeError, lambda: nv.linear(w, X)), (TypeError, lambda: nv.int8_linear(w, X, s)),
        (TypeError, lambda: nv.int8_linear(w, q)), (ValueError, lambda: nv.int8_linear(w, q, s[:4])), (TypeError, lambda: nv.int8_linear(w, X.float())),
        (ValueError, lambda: nv.int8_linear(w, X[:, :48])), (ValueError, lambda: nv.int8_linear(w, X, activation="tanh")),
        (ValueError, lambda: nv.int8_linear(w, X.clone().requires_grad_())),
        (ValueError, lambda: nv.int8_linear(w, X, bias=torch.zeros(40, device="cuda", requires_grad=True))),
        (ValueError, lambda: nv.int8_quantize(X.clone().requires_grad_())), (TypeError, lambda: nv.int8_quantize(q)),
        (nv.Nvfp4Error, lambda: nv.int8_quantize(X[:, :40])), (nv.Nvfp4Error, lambda: nv.int8_quantize(X[:, 4:20])),
        (nv.Nvfp4Error, lambda: nv.int8_linear(w, randn((20, 64), 1), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (ValueError, lambda: nv.Int8Weight.from_int8(codes((4, 40), 1), torch.ones(4, device="cuda"))),
        (ValueError, lambda: nv.Int8Weight.from_int8(codes((1, 131072), 1), torch.ones(1, device="cuda"))),
        (ValueError, lambda: nv.Int8Weight.from_int8(codes((4, 64), 1), torch.ones(3, device="cuda"))),
        (TypeError, lambda: nv.int8_linear(w, X.cpu())), (ValueError, lambda: nv.int8_linear(w, X, residual=X[:, :40][:4])),
    ]
    for i, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            say("not refused:", i)
    assert int8._call("nvfp4_int8_packed_bytes")(40, 64) == 3 * 2048
