"""Argument checks and host functions of the router, the expert layer and the
8-bit projection, no GPU: every refusal comes before any HIP call."""
import pytest
from hypothesis import given, settings, strategies as st

import nvfp4_weight_only_02_amd as nv
from nvfp4_weight_only_02_amd import experts, int8
from test_fused_host import ALIGN, DEVICE, NULL, OK, OVERLAP, RANGE, SHAPE, WORKSPACE, at, epilogue

BIG = 1 << 30


def args(base, kw):
    assert set(kw) <= set(base), set(kw) - set(base)
    return {**base, **kw}


def route(**kw):
    a = args(dict(l=at(0), dt=0, ldl=64, b=at(1), n=5, E=64, k=4, how=0, norm=1, w=at(2), e=at(3)), kw)
    return experts._call("nvfp4_moe_route")(a["l"], a["dt"], a["ldl"], a["b"], a["n"], a["E"], a["k"], a["how"], a["norm"], 1.0,
                                            a["w"], a["e"], None)


def route_backward(**kw):
    a = args(dict(l=at(0), dt=0, ldl=64, e=at(1), dw=at(2), n=5, E=64, k=4, how=0, dl=at(3), ldd=64), kw)
    return experts._call("nvfp4_moe_route_backward")(a["l"], a["dt"], a["ldl"], a["e"], a["dw"], a["n"], a["E"], a["k"],
                                                     a["how"], 1, 1.0, a["dl"], a["ldd"], None)


SHARED = [(dict(l=None), NULL), (dict(n=-1), RANGE), (dict(E=0), RANGE), (dict(E=1025, ldl=1025), RANGE), (dict(k=0), RANGE),
          (dict(k=33), RANGE), (dict(E=3), RANGE), (dict(how=2), RANGE), (dict(dt=2), RANGE), (dict(ldl=63), RANGE),
          (dict(l=at(0) + 2), ALIGN)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(w=None), NULL), (dict(e=None), NULL), (dict(b=at(1) + 2), ALIGN), (dict(w=at(2) + 2), ALIGN), (dict(e=at(3) + 1), ALIGN),
    (dict(w=at(0)), OVERLAP), (dict(w=at(0) + 4 * (4 * 64 + 60)), OVERLAP), (dict(e=at(2)), OVERLAP), (dict(e=at(1) + 252), OVERLAP)])
def test_route_refuses(kw, status):
    assert route(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(e=None), NULL), (dict(dw=None), NULL), (dict(dl=None), NULL), (dict(ldd=63), RANGE), (dict(dl=at(3) + 2), ALIGN),
    (dict(dl=at(0)), OVERLAP), (dict(dl=at(2) - 4), OVERLAP), (dict(dl=at(1)), OVERLAP)])
def test_route_backward_refuses(kw, status):
    assert route_backward(**kw) == status


def layer(a):
    return experts._EXPERTS.pack(a["gc"], a["gs"], a["dc"], a["ds"], a["g"], a["E"], a["F"], a["K"])


LAYER = dict(gc=at(10), gs=at(11), dc=at(12), ds=at(13), g=at(14), E=6, F=48, K=64, x=at(0), ldx=64, e=at(1), w=at(2), n=5, k=3)


def moe(**kw):
    a = args(dict(LAYER, y=at(3), ldy=64, ep=epilogue(), ws=at(4), size=BIG, null=False), kw)
    return experts._call("nvfp4_moe")(None if a["null"] else layer(a), a["x"], a["ldx"], a["e"], a["w"], a["n"], a["k"], a["y"],
                                      a["ldy"], a["ep"], a["ws"], a["size"], None)


def moe_backward(**kw):
    a = args(dict(LAYER, dt=1, z=at(3), ldp=96, act=2, dx=at(4), lddx=64, dw=at(5), ws=at(6), size=BIG), kw)
    return experts._call("nvfp4_moe_backward")(layer(a), a["x"], a["dt"], a["ldx"], a["e"], a["w"], a["z"], a["ldp"], a["act"],
                                               a["n"], a["k"], a["dx"], a["lddx"], a["dw"], a["ws"], a["size"], None)


SIZES = [(dict(n=-1), RANGE), (dict(n=(1 << 20) + 1), RANGE), (dict(k=0), RANGE), (dict(k=33), RANGE), (dict(E=0), RANGE),
         (dict(E=1025), RANGE), (dict(F=0), RANGE), (dict(K=0), RANGE), (dict(F=40), SHAPE), (dict(K=56), SHAPE),
         (dict(F=(1 << 18) + 16), SHAPE), (dict(gc=0), NULL), (dict(ds=0), NULL), (dict(g=0), NULL), (dict(gs=at(11) + 8), ALIGN),
         (dict(dc=at(12) + 4), ALIGN), (dict(g=at(14) + 2), ALIGN), (dict(x=None), NULL), (dict(e=None), NULL), (dict(w=None), NULL),
         (dict(ldx=56), RANGE), (dict(ldx=(1 << 18) + 8), SHAPE), (dict(e=at(1) + 2), ALIGN), (dict(w=at(2) + 1), ALIGN),
         (dict(ws=None), WORKSPACE), (dict(size=64), WORKSPACE)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(null=True), NULL), (dict(ep=None), NULL), (dict(y=None), NULL), (dict(ldx=68), ALIGN), (dict(x=at(0) + 8), ALIGN),
    (dict(ldy=63), RANGE), (dict(ep=epilogue(bias=at(5))), RANGE), (dict(ep=epilogue(up_bias=at(5))), RANGE),
    (dict(ep=epilogue(activation=5)), RANGE), (dict(ep=epilogue(out_dtype=3)), RANGE), (dict(ep=epilogue(residual=at(5), ldr=63)), RANGE),
    (dict(ep=epilogue(preact=at(5), ldp=95)), RANGE), (dict(ep=epilogue(preact=at(5), ldp=100)), ALIGN),
    (dict(ep=epilogue(preact=at(5) + 8, ldp=96)), ALIGN), (dict(ws=at(4) + 8), ALIGN), (dict(y=at(0)), OVERLAP), (dict(y=at(2)), OVERLAP),
    (dict(y=at(10) + 64), OVERLAP), (dict(y=at(13) - 16), OVERLAP), (dict(y=at(14)), OVERLAP), (dict(ws=at(3)), OVERLAP),
    (dict(ws=at(1)), OVERLAP), (dict(ep=epilogue(residual=at(4), ldr=64)), OVERLAP), (dict(ep=epilogue(residual=at(3) + 2, ldr=64)), OVERLAP),
    (dict(ep=epilogue(preact=at(3), ldp=96)), OVERLAP), (dict(ep=epilogue(preact=at(0), ldp=96)), OVERLAP),
    (dict(y=at(3) + 1), ALIGN)])
def test_moe_refuses(kw, status):
    assert moe(**kw) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(z=None), NULL), (dict(act=5), RANGE), (dict(dt=4), RANGE), (dict(ldp=95), RANGE), (dict(ldp=98), ALIGN), (dict(lddx=63), RANGE),
    (dict(dx=at(4) + 1), ALIGN), (dict(dw=at(5) + 2), ALIGN), (dict(dx=at(0)), OVERLAP), (dict(dx=at(3)), OVERLAP), (dict(dw=at(2)), OVERLAP),
    (dict(dw=at(4)), OVERLAP), (dict(ws=at(4) - 64), OVERLAP), (dict(dx=at(12)), OVERLAP), (dict(ws=at(0)), OVERLAP)])
def test_moe_backward_refuses(kw, status):
    assert moe_backward(**kw) == status


def test_workspaces():
    need = experts._call("nvfp4_moe_workspace_bytes")
    assert need(5, 3, 6, 48, 64, 0) == 5 * 3 * 128 * 4                 # the rows of h in two parts, whole tiles
    assert need(0, 3, 6, 48, 64, 0) == need(5, 33, 6, 48, 64, 0) == need(5, 3, 6, 40, 64, 0) == 0
    assert moe(size=5 * 3 * 512 - 1) == WORKSPACE
    for n, pre in ((17, 0), (5, 1)):
        size = need(n, 3, 6, 48, 64, pre)
        assert size >= n * 3 * (48 * 2 + 64 * 4)
        ep = epilogue(preact=at(5), ldp=96) if pre else epilogue()
        assert moe(n=n, ep=ep, size=size - 1) == WORKSPACE
    # it does not grow beyond 2^16 pairs, and never shrinks with more tokens
    for E, k in ((6, 3), (1023, 8), (1000, 32), (1024, 1)):
        sizes = [need(n, k, E, 16, 16, 1) for n in list(range(1, 200)) + list(range(60000 // k, 70000 // k)) + [1 << 20]]
        assert sizes == sorted(sizes) and sizes[-1] == need(-(-70000 // k), k, E, 16, 16, 1)
    back = experts._call("nvfp4_moe_backward_workspace_bytes")
    assert back(5, 3, 6, 48, 64, 0, 0) < back(5, 3, 6, 48, 64, 0, 1) < back(5, 3, 6, 48, 64, 1, 1)
    assert moe_backward(size=back(5, 3, 6, 48, 64, 1, 0) - 1) == WORKSPACE
    assert moe_backward(ldx=65, size=back(5, 3, 6, 48, 64, 1, 1) - 1) == WORKSPACE


def int8_linear(**kw):
    a = args(dict(wq=at(0), ws=at(1), x=at(2), ldx=None, xs=None, y=at(3), ldy=None, n=4, N=40, K=64, ep=epilogue(), work=at(4), size=BIG), kw)
    ldx, ldy = a["K"] if a["ldx"] is None else a["ldx"], a["N"] if a["ldy"] is None else a["ldy"]
    return int8._call("nvfp4_int8_linear")(a["wq"], a["ws"], a["x"], ldx, a["xs"], a["y"], ldy, a["n"], a["N"], a["K"], a["ep"],
                                           a["work"], a["size"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(wq=None), NULL), (dict(ws=None), NULL), (dict(x=None), NULL), (dict(y=None), NULL), (dict(ep=None), NULL),
    (dict(n=-1), RANGE), (dict(n=(1 << 20) + 1), RANGE), (dict(N=0), RANGE), (dict(N=(1 << 30) + 1), RANGE), (dict(K=0), RANGE),
    (dict(K=72), SHAPE), (dict(K=131072), SHAPE), (dict(ldx=56), RANGE), (dict(ldy=39), RANGE), (dict(ldx=(1 << 22) + 16), SHAPE),
    (dict(ldx=68), ALIGN), (dict(xs=at(5), ldx=72), ALIGN), (dict(x=at(2) + 8), ALIGN), (dict(wq=at(0) + 8), ALIGN),
    (dict(ws=at(1) + 2), ALIGN), (dict(xs=at(5) + 2), ALIGN), (dict(y=at(3) + 1), ALIGN), (dict(n=20, work=None), WORKSPACE),
    (dict(n=20, size=255), WORKSPACE), (dict(n=20, work=at(4) + 8), ALIGN), (dict(ep=epilogue(up_bias=at(5))), RANGE),
    (dict(ep=epilogue(preact=at(5), ldp=64)), RANGE), (dict(ep=epilogue(activation=7)), RANGE), (dict(ep=epilogue(out_dtype=2)), RANGE),
    (dict(ep=epilogue(residual=at(5), ldr=39)), RANGE), (dict(ep=epilogue(bias=at(5) + 1)), ALIGN), (dict(y=at(2)), OVERLAP),
    (dict(y=at(0)), OVERLAP), (dict(y=at(1) + 156), OVERLAP), (dict(xs=at(3)), OVERLAP), (dict(ep=epilogue(bias=at(3))), OVERLAP),
    (dict(n=20, work=at(3)), OVERLAP), (dict(n=20, work=at(2)), OVERLAP), (dict(n=20, ep=epilogue(residual=at(4), ldr=40)), OVERLAP),
    (dict(ep=epilogue(residual=at(3) + 2, ldr=40)), OVERLAP)])
def test_int8_linear_refuses(kw, status):
    assert int8_linear(**kw) == status


def quantize(**kw):
    a = args(dict(x=at(0), dt=1, ldx=64, n=4, K=64, q=at(1), ldq=64, s=at(2)), kw)
    return int8._call("nvfp4_int8_quantize")(a["x"], a["dt"], a["ldx"], a["n"], a["K"], a["q"], a["ldq"], a["s"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(s=None), NULL), (dict(n=-1), RANGE), (dict(K=0), RANGE), (dict(dt=3), RANGE),
    (dict(ldx=56), RANGE), (dict(ldq=48), RANGE), (dict(K=56, ldx=64), SHAPE), (dict(ldx=68), ALIGN), (dict(ldq=72), ALIGN),
    (dict(x=at(0) + 8), ALIGN), (dict(q=at(1) + 8), ALIGN), (dict(s=at(2) + 2), ALIGN), (dict(q=at(0)), OVERLAP), (dict(s=at(1)), OVERLAP),
    (dict(s=at(0) + 4), OVERLAP)])
def test_int8_quantize_refuses(kw, status):
    assert quantize(**kw) == status


def test_int8_sizes_and_pack_refusals():
    size = int8._call("nvfp4_int8_packed_bytes")
    assert size(1, 16) == 2048 and size(17, 144) == 2 * 2 * 2048 and size(16384, 5120) == 16384 * 5120
    assert size(0, 16) == size(1, 8) == size(1, 131072) == size((1 << 30) + 1, 16) == 0
    pack = int8._call("nvfp4_int8_pack")
    assert pack(None, 4, 64, at(1), None) == pack(at(0), 4, 64, None, None) == NULL
    assert pack(at(0), 4, 72, at(1), None) == SHAPE and pack(at(0), 0, 64, at(1), None) == RANGE
    assert pack(at(0), 4, 64, at(1) + 8, None) == ALIGN and pack(at(0), 4, 64, at(0) + 16, None) == OVERLAP
    need = nv.int8_linear_workspace_bytes
    assert need(20, 40, 64) == 20 * 64 + 256 and need(20, 40, 64, False) == 0 and need(0, 40, 64) == 0 and need(20, 40, 72) == 0
    # a decode launch quantises few activations itself
    assert need(4, 40, 64) == need(8, 40, 6144) == 0 and need(8, 40, 6160) == 8 * 6160 + 128 + 256 and need(9, 40, 64) == 9 * 64 + 192 + 256
    assert need(17, 40, 8192, False) > 0           # K parts: one row tile alone


def test_valid_calls_reach_the_device_check():
    if nv.torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    assert route() == route(b=None, dt=1) == route_backward() == DEVICE
    for kw in (dict(), dict(n=40), dict(ep=epilogue(residual=at(3), ldr=64)), dict(n=1, ldx=65), dict(ep=epilogue(preact=at(5), ldp=96))):
        assert moe(**kw) == DEVICE
    for kw in (dict(), dict(dx=None), dict(dw=None), dict(dt=0, ldx=65)):
        assert moe_backward(**kw) == DEVICE
    for kw in (dict(), dict(n=40), dict(n=600), dict(xs=at(5), ldx=80), dict(n=1, ldx=65), dict(ep=epilogue(residual=at(3), ldr=40))):
        assert int8_linear(**kw) == DEVICE
    assert quantize() == DEVICE and quantize(n=1, ldx=65, ldq=67) == DEVICE
    # nothing to do: no device is asked for
    assert route(n=0, l=None, w=None, e=None) == route_backward(n=0, l=None) == quantize(n=0, x=None) == OK
    assert moe(n=0, x=None, y=None, e=None, w=None, ws=None) == moe_backward(n=0, x=None, e=None, w=None, z=None) == OK
    assert moe_backward(dx=None, dw=None, ws=None) == int8_linear(n=0, x=None, y=None, work=None) == OK


def test_geometry():
    assert nv.moe_geometry(1, 1, 1, 16, 16) == (128, 32) and nv.moe_geometry(1 << 20, 32, 1024, 16, 16) == (128, 64)
    for a, status in (((0, 1, 1, 16, 16), RANGE), ((1, 33, 40, 16, 16), RANGE), ((1, 1, 0, 16, 16), RANGE), ((1, 1, 1, 8, 16), SHAPE)):
        with pytest.raises(nv.Nvfp4Error) as e:
            nv.moe_geometry(*a)
        assert e.value.status == status
    for a, status in (((16, 64, 64), RANGE), ((17, 0, 64), RANGE), ((17, 64, 72), SHAPE), ((17, 64, 131072), SHAPE)):
        with pytest.raises(nv.Nvfp4Error) as e:
            nv.int8_geometry(*a)
        assert e.value.status == status
    assert int8._call("nvfp4_int8_geometry")(17, 64, 64, None, None, None, None) == NULL
    assert experts._call("nvfp4_moe_geometry")(17, 1, 1, 64, 64, None, None) == NULL


def test_decode_geometry():
    """Any number of compute units serves every K of the decode form: a device may be
    partitioned into 2, 4 or 8."""
    assert [nv.moe_decode_geometry(5120, c) for c in (256, 128, 64)] == [20, 32, 32]
    assert nv.moe_decode_geometry(8192, 256) == 32 and nv.moe_decode_geometry(16, 256) == 4
    for units in list(range(1, 40)) + [64, 80, 128, 160, 256, 304, (1 << 31) - 1]:
        for K in range(16, 8193, 16):
            r = nv.moe_decode_geometry(K, units)
            assert 4 <= r <= 32 and r % 4 == 0 and (r == 32 or -(-K // r) <= units)
    for a, status in (((0, 256), RANGE), ((64, 0), RANGE), ((72, 256), SHAPE), ((8208, 256), SHAPE)):
        with pytest.raises(nv.Nvfp4Error) as e:
            nv.moe_decode_geometry(*a)
        assert e.value.status == status
    assert experts._call("nvfp4_moe_decode_geometry")(64, 256, None) == NULL


@settings(max_examples=300, deadline=None)
@given(n=st.integers(17, 1 << 20), N=st.integers(1, 1 << 17), T=st.integers(1, 1023), tail=st.sampled_from([0, 16, 112]))
def test_int8_geometry_rule(n, N, T, tail):
    K = T * 128 - tail
    r, t, kg, ks = nv.int8_geometry(n, N, K)
    assert (r, t, kg) in {(64, 32, 4), (128, 64, 2), (128, 64, 1), (128, 128, 1), (256, 128, 1), (256, 256, 1)}
    tp = -(-2 * T // ks)
    assert 1 <= ks <= 8 and (ks - 1) * tp < 2 * T        # no part is empty
    assert (nv.int8_linear_workspace_bytes(n, N, K, False) > 0) == (ks > 1)
