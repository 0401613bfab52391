"""Argument checks and host functions of the fused operators, no GPU: every
refusal comes before any HIP call."""
import numpy as np
import pytest
from hypothesis import given, settings
from hypothesis import strategies as st

import fused_reference as R
import nvfp4_weight_only_02_amd as nv
from nvfp4_weight_only_02_amd import fused

OK, NULL, RANGE, ALIGN, SHAPE, DEVICE, WORKSPACE, OVERLAP = 0, 1, 2, 3, 4, 7, 8, 10


def at(i):
    """Fake device addresses, far apart."""
    return (i + 1) * (1 << 40)


def epilogue(**kw):
    base = dict(bias=0, up_bias=0, residual=0, preact=0, ldr=0, ldp=0, activation=0, bias_dtype=1, residual_dtype=1,
                out_dtype=1)
    base.update(kw)
    return fused._EPILOGUE.pack(*base.values())


def linear(wq=at(0), ws=at(1), x=at(2), ldx=None, y=at(3), ldy=None, n=4, N=64, K=256, ep=None, work=None, size=0):
    ep = ep if ep is not None else epilogue()
    return fused._call("nvfp4_linear")(wq, ws, 1.0, x, K if ldx is None else ldx, y, N if ldy is None else ldy, n, N,
                                       K, ep if ep != 0 else None, work, size, None)


def gated(x=at(2), ldx=None, h=at(3), ldh=None, n=4, F=64, K=256, ep=None, work=None, size=0):
    ep = ep if ep is not None else epilogue()
    return fused._call("nvfp4_gated")(at(0), at(1), 1.0, 1.0, x, K if ldx is None else ldx, h,
                                      F if ldh is None else ldh, n, F, K, ep, work, size, None)


@pytest.mark.parametrize("kw,status", [
    (dict(wq=None), NULL), (dict(x=None), NULL), (dict(y=None), NULL), (dict(ep=0), NULL),
    (dict(n=-1), RANGE), (dict(n=(1 << 20) + 1), RANGE), (dict(N=0), RANGE), (dict(K=0), RANGE),
    (dict(K=250), SHAPE), (dict(K=(1 << 18) + 16), SHAPE), (dict(ldx=240), RANGE), (dict(ldy=63), RANGE),
    (dict(ldx=260), ALIGN), (dict(x=at(2) + 8), ALIGN), (dict(wq=at(0) + 4), ALIGN), (dict(y=at(3) + 1), ALIGN),
    (dict(ldx=(1 << 22) + 8), SHAPE),
    (dict(ep=epilogue(activation=5)), RANGE), (dict(ep=epilogue(activation=-1)), RANGE),
    (dict(ep=epilogue(out_dtype=2)), RANGE), (dict(ep=epilogue(up_bias=at(5))), RANGE),
    (dict(ep=epilogue(bias=at(5), bias_dtype=7)), RANGE), (dict(ep=epilogue(bias=at(5) + 1)), ALIGN),
    (dict(ep=epilogue(residual=at(5), ldr=63)), RANGE), (dict(ep=epilogue(residual=at(5) + 2, ldr=64, residual_dtype=0)), ALIGN),
    (dict(ep=epilogue(preact=at(5), ldp=60)), RANGE), (dict(ep=epilogue(preact=at(5), ldp=68)), ALIGN),
    (dict(ep=epilogue(preact=at(5) + 8, ldp=64)), ALIGN),
    (dict(y=at(2)), OVERLAP), (dict(y=at(2) + 3 * 512 + 510), OVERLAP), (dict(y=at(0)), OVERLAP),
    (dict(ep=epilogue(residual=at(3) + 2, ldr=64)), OVERLAP), (dict(ep=epilogue(residual=at(3), ldr=72)), OVERLAP),
    (dict(ep=epilogue(residual=at(3), ldr=64, residual_dtype=0)), OVERLAP),
    (dict(ep=epilogue(preact=at(3), ldp=64)), OVERLAP), (dict(ep=epilogue(bias=at(3))), OVERLAP),
    (dict(ep=epilogue(preact=at(2), ldp=64)), OVERLAP),
])
def test_linear_refuses(kw, status):
    assert linear(**kw) == status


def test_valid_calls_reach_the_device_check():
    # valid arguments: the first thing that can fail is the missing GPU (with
    # one, these addresses would be launched on)
    if nv.torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    for kw in (dict(), dict(n=40), dict(ep=epilogue(residual=at(3), ldr=64)), dict(n=1, ldx=257)):
        assert linear(**kw) == DEVICE
    assert linear(n=0) == OK and linear(n=0, x=None, y=None) == OK and gated(n=0) == OK


def test_long_rows_need_a_workspace():
    need = fused._call("nvfp4_linear_workspace_bytes")(4, 64, 8208)
    assert need == nv.gemv_kparts(64, 8208) * 4 * 64 * 4
    assert linear(K=8208) == WORKSPACE
    assert linear(K=8208, work=at(7), size=need - 1) == WORKSPACE
    assert linear(K=8208, work=at(7) + 4, size=need) == ALIGN
    for other in (2, 3):                             # X, Y
        assert linear(K=8208, work=at(other) - 16, size=need) == OVERLAP
    assert linear(K=8208, work=at(7), size=need, ep=epilogue(residual=at(7), ldr=64)) == OVERLAP
    codes, scales = 4 * 65 * 1024, 4 * 65 * 128     # bytes of the weight
    for q, size in ((at(0), codes), (at(1), scales)):
        assert linear(K=8208, work=q - 16, size=need) == linear(K=8208, work=q + size - 16, size=need) == OVERLAP
    for n in (4, 17):
        big = fused._call("nvfp4_linear_workspace_bytes")(n, 64, 8208)
        assert linear(n=n, K=8208, work=at(0), size=big) == OVERLAP
        assert linear(n=n, K=8208, work=at(7), size=big, ep=epilogue(bias=at(7) + 64)) == OVERLAP
    assert linear(n=17, K=8208) == WORKSPACE        # many columns for one row tile: K parts here too
    assert fused._call("nvfp4_linear_workspace_bytes")(4, 64, 8192) == 0
    rows = nv.gated_rows(50)
    assert rows == 128
    assert fused._call("nvfp4_gated_workspace_bytes")(4, 50, 8208) == nv.gemv_kparts(rows, 8208) * 4 * rows * 4
    assert gated(F=50, K=8208) == WORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(F=0), RANGE), (dict(ep=epilogue(residual=at(5), ldr=64)), RANGE),
    (dict(ep=epilogue(preact=at(5), ldp=64)), RANGE), (dict(ep=epilogue(up_bias=at(3))), OVERLAP),
    (dict(K=264), SHAPE), (dict(ldh=60), RANGE), (dict(x=None), NULL)])
def test_gated_refuses(kw, status):
    assert gated(**kw) == status


def linear_backward(**kw):
    a = dict(c=at(0), s=at(1), dy=at(2), dt=1, ldy=93, z=at(3), ldp=96, act=2, dx=at(4), ldx=None, db=at(5), bt=0, n=4,
             N=93, K=48, ws=at(6), size=1 << 30)
    a.update(kw)
    if a["ldx"] is None:
        a["ldx"] = a["K"]
    return fused._call("nvfp4_linear_backward")(a["c"], a["s"], 1.0, a["dy"], a["dt"], a["ldy"], a["z"], a["ldp"],
                                                a["act"], a["dx"], a["ldx"], a["db"], a["bt"], a["n"], a["N"], a["K"],
                                                a["ws"], a["size"], None)


BACKWARD = [
    (dict(dy=None), NULL), (dict(z=None), NULL), (dict(c=None), NULL), (dict(n=-1), RANGE), (dict(act=9), RANGE),
    (dict(dt=3), RANGE), (dict(bt=2), RANGE), (dict(N=0), RANGE), (dict(K=0), RANGE), (dict(K=40), SHAPE),
    (dict(ldy=90), RANGE), (dict(ldp=88), RANGE), (dict(ldx=40), RANGE), (dict(ldp=95), ALIGN), (dict(dx=at(4) + 1), ALIGN),
    (dict(dy=at(2) + 1), ALIGN), (dict(db=at(5) + 2), ALIGN), (dict(ws=at(6) + 8), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(size=4 * 96 * 2 - 1), WORKSPACE), (dict(dx=at(2)), OVERLAP), (dict(dx=at(0)), OVERLAP), (dict(db=at(4)), OVERLAP),
    (dict(db=at(3)), OVERLAP), (dict(ws=at(4) - 256), OVERLAP), (dict(ws=at(2) - 256), OVERLAP),
    (dict(ldy=(1 << 31)), SHAPE), (dict(n=4000, N=2000, ldy=2000, ldp=2000, act=0, dx=None, size=15), WORKSPACE)]


@pytest.mark.parametrize("kw,status", BACKWARD)
def test_linear_backward_refuses(kw, status):
    assert linear_backward(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), NULL), (dict(F=0), RANGE), (dict(ldp=64), RANGE), (dict(dg=at(4)), OVERLAP), (dict(du=at(5)), OVERLAP),
    (dict(ws=None), WORKSPACE), (dict(K=40), SHAPE), (dict(s=None), NULL), (dict(act=-1), RANGE)])
def test_gated_backward_refuses(kw, status):
    a = dict(c=at(0), s=at(1), dy=at(2), z=at(3), ldp=96, act=2, dx=at(4), dg=at(5), du=at(7), n=4, F=33, K=48, ws=at(6))
    a.update(kw)
    f = a["F"]
    assert fused._call("nvfp4_gated_backward")(a["c"], a["s"], 1.0, 1.0, a["dy"], 1, f, a["z"], a["ldp"], a["act"],
                                               a["dx"], a["K"], a["dg"], a["du"], 0, a["n"], f, a["K"], a["ws"],
                                               1 << 20, None) == status


def test_backward_workspace():
    f = fused._call("nvfp4_linear_backward_workspace_bytes")
    assert f(4, 96, 48, 1, 0, 0) == 0                # dY as it is, one part, no sums
    assert f(4, 93, 48, 1, 0, 1) == 768              # dZ: 4 x 96 bf16
    assert f(4, 93, 48, 0, 0, 1) == 0 and f(0, 93, 48, 1, 1, 1) == 0
    assert f(4000, 2000, 48, 0, 1, 1) > 0            # column sums of row blocks
    assert fused._call("nvfp4_gated_backward_workspace_bytes")(4, 33, 48, 1, 0) == 4 * 96 * 2
    # no GPU, no tokens: refused only where memory would be touched
    assert linear_backward(n=0, db=None, dx=None) in (OK, DEVICE)


def test_pack_refuses():
    f = fused._call("nvfp4_pack_gated")
    assert f(at(0), at(1), at(2), at(3), 0, 256, at(4), at(5), None) == RANGE
    assert f(at(0), at(1), at(2), at(3), 16, 250, at(4), at(5), None) == SHAPE
    assert f(at(0), at(1), at(2), None, 16, 256, at(4), at(5), None) == NULL
    assert f(at(0), at(1), at(2), at(3), 16, 256, at(0), at(5), None) == OVERLAP
    assert f(at(0) + 8, at(1), at(2), at(3), 16, 256, at(4), at(5), None) == ALIGN
    t = fused._call("nvfp4_pack_transposed")
    assert t(at(0), at(1), 0, 256, at(4), at(5), None) == RANGE
    assert t(at(0), at(1), 16, 256, at(1), at(5), None) == OVERLAP
    assert t(at(0), at(1), 16, 256, at(4), at(5) + 1, None) == ALIGN


def test_transposed_sizes():
    c, s = fused._call("nvfp4_transposed_codes_bytes"), fused._call("nvfp4_transposed_scales_bytes")
    assert c(256, 64) == 256 * 64 // 2 and s(256, 64) == 256 * 64 // 16
    assert c(129, 16) == 256 * 16 // 2 and s(129, 16) == 256
    assert c(0, 16) == 0 and s(16, 24) == 0
    assert c(1 << 20, 1 << 18) == (1 << 37)


@pytest.mark.parametrize("kind", R.ACTS)
def test_reference_gradients_are_differences(kind):
    z = np.linspace(-9, 9, 4001) + 1e-3
    t = 1e-5
    diff = (R.act(z + t, kind) - R.act(z - t, kind)) / (2 * t)
    assert np.abs(diff - R.act_grad(z, kind)).max() < 1e-8
    assert np.abs(R.act_grad(z, kind)).max() <= R.LIP


@settings(max_examples=300, deadline=None)
@given(n=st.integers(17, 1 << 20), rows=st.integers(1, 1 << 17), T=st.integers(1, 2048), tail=st.sampled_from([0, 8, 16, 112]))
def test_fused_geometry_rule(n, rows, T, tail):
    K = T * 128 - tail if T * 128 > tail else 8
    r, t, kg, ks = nv.fused_geometry(n, rows, K)
    assert (r, t, kg) in {(32, 32, 4), (32, 32, 8), (64, 32, 4), (64, 64, 4), (128, 64, 2), (256, 128, 2), (256, 128, 1)}
    tiles = -(-K // 128)
    tp = -(-tiles // ks)
    assert 1 <= ks <= 12 and (ks - 1) * tp < tiles        # no part is empty
    if K % 16 == 0 and K <= 1 << 18:
        need = fused._call("nvfp4_linear_workspace_bytes")(n, rows, K)
        assert need == (ks * n * -(-rows // 16) * 16 * 4 if ks > 1 else 0)


def test_fused_geometry_refuses():
    for args, status in (((16, 64, 256), RANGE), ((17, 0, 256), RANGE), ((17, 64, 0), RANGE), ((17, 64, 260), SHAPE)):
        with pytest.raises(nv.Nvfp4Error) as e:
            nv.fused_geometry(*args)
        assert e.value.status == status


# ---- weights of the wrong kind -------------------------------------------------------

def weights(N=64, K=256):
    """A weight of each class over host memory: refused for its class before any
    of it is looked at."""
    b = nv.torch.empty(16, dtype=nv.torch.uint8)
    return {"PackedWeight": nv.PackedWeight(b, b, 1.0, N, K), "GatedWeight": nv.GatedWeight(b, b, 1.0, 1.0, N, K),
            "TransposedWeight": nv.TransposedWeight(b, b, 1.0, N, K)}


CALLS = [  # what the call takes, the call on a weight and a matrix
    ("PackedWeight", lambda w, x: nv.linear(w, x)),
    ("PackedWeight", lambda w, x: nv.transpose(w)),
    ("PackedWeight", lambda w, x: nv.GatedWeight.from_packed(w, weights()["PackedWeight"])),
    ("PackedWeight", lambda w, x: nv.GatedWeight.from_packed(weights()["PackedWeight"], w)),
    ("GatedWeight", lambda w, x: nv.gated(w, x)),
    ("GatedWeight", lambda w, x: nv.gated_backward(w, None, x, x)),
    ("TransposedWeight", lambda w, x: nv.gemm_t(w, x)),
    ("TransposedWeight", lambda w, x: nv.linear_backward(w, x)),
    ("TransposedWeight", lambda w, x: nv.gated_backward(weights()["GatedWeight"], w, x, x)),
    ("PackedWeight", lambda w, x: nv.gemv(w, x)),
    ("PackedWeight", lambda w, x: nv.gemv_ws(w, x)),
    ("PackedWeight", lambda w, x: nv.gemv_ws_static(w, x)),
    ("PackedWeight", lambda w, x: nv.gemv_sched(w, x, [1])),
    ("PackedWeight", lambda w, x: nv.gemm(w, x)),
    ("PackedWeight", lambda w, x: nv.gemv_qkv(w, x, (32, 16, 16), (0, 32, 48), 64)),
]


@pytest.mark.parametrize("call", range(len(CALLS)))
@pytest.mark.parametrize("kind", ["PackedWeight", "GatedWeight", "TransposedWeight", "other"])
def test_weight_of_another_class_is_refused(call, kind):
    """A transposed copy has the fields of a packed weight and other sizes: read
    as one, its tiles would be read past their end."""
    want, f = CALLS[call]
    if kind == want or (kind == "other" and call >= 9):    # the projections look at no other class
        return
    w = object() if kind == "other" else weights()[kind]
    x = nv.torch.empty(4, 256, dtype=nv.torch.bfloat16)
    with pytest.raises(TypeError, match=want):
        f(w, x)


def test_transposed_argument_is_a_transposed_weight():
    x = nv.torch.empty(4, 256, dtype=nv.torch.bfloat16)
    for f, kind in ((nv.linear, "PackedWeight"), (nv.gated, "GatedWeight")):
        for other in ("PackedWeight", "GatedWeight"):
            with pytest.raises(TypeError, match="TransposedWeight"):
                f(weights()[kind], x, transposed=weights()[other])
    with pytest.raises(TypeError, match="PackedWeight or a GatedWeight"):
        nv.preact_columns(weights()["TransposedWeight"])


def test_transposed_copy_of_another_weight_is_refused():
    """What autograd and gated_backward can tell apart: the kind of weight, its
    sizes, its tensor scale and the codes the copy was made from."""
    import copy
    import pickle
    t = lambda: nv.torch.empty(16, dtype=nv.torch.uint8)     # noqa: E731
    w = nv.PackedWeight(t(), t(), 0.5, 96, 64)
    gw = nv.GatedWeight(t(), t(), 0.5, 0.25, 48, 64)
    wt = nv.TransposedWeight(t(), t(), 0.5, 96, 64, source=w.codes)
    gt = nv.TransposedWeight(t(), t(), 1.0, 96, 64, gated=True, source=gw.codes)
    check = fused._check_transposed
    check(wt, w)
    check(gt, gw)
    # the same memory in another object, and copies that go without a source
    check(wt, nv.PackedWeight(w.codes[:], w.scales, 0.5, 96, 64))
    for again in (copy.deepcopy(wt), pickle.loads(pickle.dumps(wt)), nv.TransposedWeight(t(), t(), 0.5, 96, 64)):
        assert again.gscale == 0.5 and not again.gated
        check(again, w)
    for other, weight in ((gt, w), (wt, gw),                                           # the other kind
                          (wt, nv.PackedWeight(t(), t(), 0.5, 96, 64)),                # other codes
                          (gt, nv.GatedWeight(t(), t(), 0.5, 0.25, 48, 64)),
                          (wt, nv.PackedWeight(w.codes, w.scales, 0.75, 96, 64)),      # another tensor scale
                          (wt, nv.PackedWeight(w.codes, w.scales, 0.5, 80, 64)),       # other sizes
                          (wt, nv.PackedWeight(w.codes, w.scales, 0.5, 96, 80))):
        with pytest.raises(ValueError, match="transposed copy"):
            check(other, weight)
    # the copy does not keep the packed weight's memory, and outlives it
    import gc
    import weakref
    alive = weakref.ref(w.codes)
    del w, weight
    gc.collect()
    assert alive() is None
    check(wt, nv.PackedWeight(t(), t(), 0.5, 96, 64))
    x = nv.torch.empty(4, 96, dtype=nv.torch.bfloat16)
    with pytest.raises(ValueError, match="gated weight"):
        nv.linear_backward(gt, x)


# ---- column slices of one buffer -----------------------------------------------------------

def test_disjoint_columns_do_not_overlap():
    """Matrices whose rows take turns in memory: neighbouring columns of one
    row-major buffer."""
    if nv.torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    base, ld = at(2), 512                                  # bf16 rows of 1 KiB
    col = lambda c, size=2: base + c * size                # noqa: E731
    # X in columns 0 .. 255, Y in 256 .. 319, residual in 320 .. 383
    ep = epilogue(residual=col(320), ldr=ld)
    assert linear(x=col(0), ldx=ld, y=col(256), ldy=ld, ep=ep) == DEVICE
    assert linear(x=col(256), ldx=ld, y=col(0), ldy=ld, ep=epilogue(residual=col(64), ldr=ld)) == DEVICE
    # Y reaches one column into X, into the residual, and around a row's end into X
    assert linear(x=col(0), ldx=ld, y=col(255), ldy=ld) == OVERLAP
    assert linear(x=col(0), ldx=ld, y=col(257), ldy=ld, ep=ep) == OVERLAP
    assert linear(x=col(0), ldx=ld, y=col(449), ldy=ld) == OVERLAP
    assert linear(x=col(0), ldx=ld, y=col(448), ldy=ld) == DEVICE
    # a row further on the columns are the same ones; one row alone lies between rows
    assert linear(x=col(0), ldx=ld, y=col(256 + 2 * ld), ldy=ld) == DEVICE
    assert linear(x=col(0), ldx=ld, y=col(2 * ld), ldy=ld) == OVERLAP
    assert linear(n=1, x=col(0), y=col(256), ep=epilogue(residual=col(320), ldr=64)) == DEVICE
    # another stride in bytes: by their spans
    assert linear(x=col(0), ldx=ld, y=col(256), ldy=ld, ep=epilogue(out_dtype=0)) == OVERLAP
    assert linear(x=col(0), ldx=ld, y=col(256), ldy=ld // 2, ep=epilogue(out_dtype=0)) == DEVICE
    # a bias between two rows of Y, a pre-activation buffer beside the output
    assert linear(y=col(0), ldy=ld, x=at(4), ep=epilogue(bias=col(64))) == DEVICE
    assert linear(y=col(0), ldy=ld, x=at(4), ep=epilogue(bias=col(449))) == OVERLAP
    assert linear(y=col(0), ldy=ld, x=at(4), ep=epilogue(preact=col(256), ldp=ld // 2)) == DEVICE
    assert linear(y=col(0), ldy=ld, x=at(4), ep=epilogue(preact=col(448), ldp=ld // 2)) == OVERLAP
    # gradients: dX beside dY; dX over its columns
    assert linear_backward(dy=col(48), ldy=ld, dx=col(0), ldx=ld) == DEVICE
    assert linear_backward(dy=col(47), ldy=ld, dx=col(0), ldx=ld) == OVERLAP


def test_rows_beyond_the_limit():
    """2^30 rows, as the packing steps and the geometry take: beyond, a row count
    rounded up to a tile would leave 32 bits."""
    f, g = fused._call("nvfp4_linear_workspace_bytes"), fused._call("nvfp4_gated_workspace_bytes")
    for N in ((1 << 30) + 1, (1 << 31) - 16, (1 << 31) - 1):
        for n in (4, 40):
            assert linear(n=n, N=N, K=16, y=at(60)) == RANGE
            assert f(n, N, 16384) == 0
    assert f(4, 1 << 30, 16384) == nv.gemv_kparts(1 << 30, 16384) * 4 * (1 << 30) * 4
    assert gated(F=(1 << 29) + 1, h=at(60)) == RANGE and g(4, (1 << 29) + 1, 16384) == 0
