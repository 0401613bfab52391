"""Cases of the fused NVFP4 operators: the projection with bias, activation and
residual in its epilogue (``linear``), the gated feed-forward block (``gated``)
and the product through the transposed weight (``gemm_t``), each with the
gradients it has.

``own`` false computes them with elementary torch operations in 32 bits on the
canonical NVFP4 weight; ``own`` true makes the package's calls on the weight as
a program keeps it (packed once at load time).
"""
import math

import numpy as np
import torch

own = False

ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---- cases ---------------------------------------------------------------------

def _linear(name, n, N, K, act="none", bias="none", residual="none", out="bf16", train=False):
    return {"name": name, "op": "linear", "n": n, "N": N, "K": K, "act": act, "bias": bias,
            "residual": residual, "out": out, "train": train}


def _gated(name, n, N, K, act="silu", bias="none", train=False):
    return {"name": name, "op": "gated", "n": n, "N": N, "K": K, "act": act, "bias": bias, "train": train}


def _gemm_t(name, n, N, K):
    return {"name": name, "op": "gemm_t", "n": n, "N": N, "K": K, "train": False}


def listed():
    return [
        # One sequence decoding: the output projection added to the residual stream.
        _linear("linear_decode_1", 1, 5120, 6144, residual="bf16"),
        # Sixteen sequences decoding: a wide fused projection with a bias.
        _linear("linear_decode_16", 16, 16384, 5120, bias="bf16"),
        # Twelve sequences: a down projection (long rows) into an fp32 residual stream.
        _linear("linear_down_12", 12, 5120, 17408, residual="f32", out="f32"),
        # A small layer with sizes that fit no tile, a short prompt.
        _linear("linear_ragged_47", 47, 1237, 2064, act="gelu", bias="f32", residual="bf16"),
        # A prompt through the output projection and the residual.
        _linear("linear_prompt_1000", 1000, 5120, 6144, residual="bf16"),
        # A training step's two-layer MLP first half: bias, activation, gradients.
        _linear("linear_train_1536", 1536, 16384, 5120, act="gelu_tanh", bias="bf16", train=True),
        # One sequence decoding through the gated block.
        _gated("gated_decode_1", 1, 17408, 5120),
        # A small gated block with biases and sizes that fit no tile.
        _gated("gated_ragged_33", 33, 1111, 1040, act="gelu", bias="bf16"),
        # A long prompt through the gated block: the largest forward.
        _gated("gated_prompt_2048", 2048, 17408, 5120),
        # A training step of the gated block: forward and gradients.
        _gated("gated_train_1024", 1024, 17408, 5120, train=True),
        # Input gradients of a few tokens (a learned prompt) and of a batch.
        _gemm_t("gemm_t_24", 24, 5120, 6144),
        _gemm_t("gemm_t_777", 777, 16384, 5120),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(("linear", "linear", "gated", "gated", "gemm_t"))
        n = _log_int(rng, 1, 2048)
        N = _log_int(rng, 64, 20000)
        if rng.random() < 0.5:
            N = (N + 127) // 128 * 128
        K = 16 * _log_int(rng, 4, 1088)
        if rng.random() < 0.5:
            K = (K + 127) // 128 * 128
        train = rng.random() < 0.4
        # relu's derivative jumps at zero, where a rounding decides it: forward only
        act = rng.choice([a for a in ACTIVATIONS if not (train and a == "relu")])
        if op == "linear":
            # fp32 bias gradients go with the identity: their values are then sums of the
            # incoming gradient alone
            bias = rng.choice(("none", "bf16", "f32"))
            if train and bias == "f32":
                act = "none"
            out = rng.choice(("bf16", "bf16", "f32"))
            residual = rng.choice(("none", out))
            case = _linear("", n, N, K, act, bias, residual, out, train)
        elif op == "gated":
            case = _gated("", n, min(N, 17408), K, act, rng.choice(("none", "bf16")), train)
        else:
            case = _gemm_t("", n, N, K)
        del case["name"]
        if work(case)["flops"] <= most:
            return case


def work(case):
    n, N, K = case["n"], case["N"], case["K"]
    halves = 2 if case["op"] == "gated" else 1
    weight = halves * (N * K // 2 + N * K // 16)
    flops = 2 * n * N * K * halves
    size = {"none": 0, "bf16": 2, "f32": 4}
    nbytes = weight + 2 * n * K + size[case.get("out", "bf16")] * n * N
    nbytes += halves * N * size[case.get("bias", "none")] + n * N * size[case.get("residual", "none")]
    if case["train"]:
        # the incoming gradient, the input gradient, the bias gradients; the
        # product of the gradient with the weight
        nbytes += size[case.get("out", "bf16")] * n * N + 2 * n * K + halves * N * size[case.get("bias", "none")]
        flops *= 2
    return {"bytes": nbytes, "flops": flops}


# ---- inputs ----------------------------------------------------------------------

def _quantize(W):
    """fp32 [N, K] -> NVFP4 codes [N, K/2], E4M3 scale bytes [N, K/16], tensor scale."""
    N, K = W.shape
    gscale = float(np.float32(float(W.abs().max()) / 2688.0))
    blocks = W.view(N, K // 16, 16)
    s8 = (blocks.abs().amax(2) / (6.0 * gscale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = (s8.float() * gscale).unsqueeze(2)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=W.device)
    mag = torch.bucketize(torch.where(step > 0, blocks.abs() / step, torch.zeros_like(blocks)), edges)
    code = (mag.to(torch.uint8) + 8 * (blocks < 0).to(torch.uint8)).view(N, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), s8.view(torch.uint8), gscale


def _weight(N, K, gen):
    W = torch.randn(N, K, generator=gen, device="cuda") * 0.02
    codes, scales, gscale = _quantize(W)
    return {"codes": codes.contiguous(), "scales": scales.contiguous(), "gscale": gscale, "N": N, "K": K}


def prepare(case, seed):
    return _inputs(case, seed, keep=True)


def _inputs(case, seed, keep):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, N, K = case["n"], case["N"], case["K"]
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    st = {"case": case}

    def rand(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    st["w"] = [_weight(N, K, gen) for _ in range(2 if case["op"] == "gated" else 1)]
    if case["op"] == "gemm_t":
        st["dY"] = rand(n, N, std=0.01)
    else:
        # normalised activations, rows of somewhat different size
        row = torch.rand(n, 1, generator=gen, device="cuda") * 1.5 + 0.5
        st["X"] = (torch.randn(n, K, generator=gen, device="cuda") * row).to(torch.bfloat16)
        st["bias"] = [None if case["bias"] == "none" else rand(N, std=0.5, dtype=dt[case["bias"]]) for _ in st["w"]]
        if case.get("residual", "none") != "none":
            st["residual"] = rand(n, N, std=4.0, dtype=dt[case["residual"]])
        if case["train"]:
            st["dY"] = rand(n, N, std=0.01, dtype=dt[case.get("out", "bf16")])
            if keep and own:
                st["X"].requires_grad_(True)
                for b in st["bias"]:
                    if b is not None:
                        b.requires_grad_(True)
    if keep and own:
        import nvfp4_weight_only_02_amd as nv
        packed = [nv.PackedWeight.from_canonical(w["codes"], w["scales"], w["gscale"], N, K) for w in st["w"]]
        st["packed"] = nv.GatedWeight.from_packed(*packed) if case["op"] == "gated" else packed[0]
        st["transposed"] = st["packed"].transpose() if case["train"] or case["op"] == "gemm_t" else None
    return st


# ---- one pass ----------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import nvfp4_weight_only_02_amd as nv
    c = st["case"]
    if c["op"] == "gemm_t":
        return nv.gemm_t(st["transposed"], st["dY"])
    if c["op"] == "linear":
        y = nv.linear(st["packed"], st["X"], bias=st["bias"][0], activation=c["act"],
                      residual=st.get("residual"), transposed=st["transposed"],
                      out_dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16)
    else:
        y = nv.gated(st["packed"], st["X"], activation=c["act"], gate_bias=st["bias"][0], up_bias=st["bias"][1],
                     transposed=st["transposed"])
    if not c["train"]:
        return y
    leaves = [st["X"]] + [b for b in st["bias"] if b is not None]
    return (y.detach(),) + torch.autograd.grad(y, leaves, st["dY"])


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _dequant(w):
    """fp32 [N, K] of the weight without its tensor scale (exact)."""
    lut = torch.tensor(_E2M1, device=w["codes"].device)
    low = lut[(w["codes"] & 15).long()]
    high = lut[(w["codes"] >> 4).long()]
    vals = torch.stack((low, high), dim=2).view(w["N"], w["K"] // 16, 16)
    return (vals * w["scales"].view(torch.float8_e4m3fn).float().unsqueeze(2)).view(w["N"], w["K"])


def _act(z, kind):
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if kind == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if kind == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _run_plain(st):
    c = st["case"]
    bf16 = torch.bfloat16
    if c["op"] == "gemm_t":
        w = st["w"][0]
        return ((st["dY"].float() @ _dequant(w)) * w["gscale"]).to(bf16)
    x = st["X"].float()
    dense = [_dequant(w) for w in st["w"]]
    z = [(x @ d.t()) * w["gscale"] for d, w in zip(dense, st["w"])]
    z = [a if b is None else a + b.float() for a, b in zip(z, st["bias"])]
    if c["op"] == "linear":
        y = _act(z[0], c["act"])
        if "residual" in st:
            y = y + st["residual"].float()
        y = y.to(torch.float32 if c["out"] == "f32" else bf16)
    else:
        y = (_act(z[0], c["act"]) * z[1]).to(bf16)
    if not c["train"]:
        return y
    dy = st["dY"].float()
    if c["op"] == "linear":
        dz = [dy * _act_grad(z[0], c["act"])]
    else:
        dz = [dy * z[1] * _act_grad(z[0], c["act"]), dy * _act(z[0], c["act"])]
    dx = sum((g @ d) * w["gscale"] for g, d, w in zip(dz, dense, st["w"])).to(bf16)
    return (y, dx) + tuple(g.sum(0).to(b.dtype) for g, b in zip(dz, st["bias"]) if b is not None)


# ---- the definition in 64 bits -------------------------------------------------------

def exact(case, seed):
    st = _inputs(case, seed, keep=False)
    f64 = torch.float64
    bf16 = torch.bfloat16

    def weight64(w):
        # sign, exponent and mantissa fields of both formats, evaluated
        c = torch.empty(w["N"], w["K"], dtype=torch.uint8, device="cuda")
        c[:, 0::2] = w["codes"] & 15
        c[:, 1::2] = w["codes"] >> 4
        e, m = (c >> 1) & 3, (c & 1).to(f64)
        mag = torch.where(e == 0, 0.5 * m, torch.exp2(e.to(f64) - 1) * (1 + 0.5 * m))
        val = torch.where(c >= 8, -mag, mag)
        s = w["scales"]
        se, sm = (s >> 3) & 15, (s & 7).to(f64) / 8
        scale = torch.where(se == 0, sm * 2.0 ** -6, torch.exp2(se.to(f64) - 7) * (1 + sm))
        return val * scale.repeat_interleave(16, dim=1) * float(np.float32(w["gscale"]))

    root2 = math.sqrt(2.0)

    def act64(z, kind):
        """(value, derivative)"""
        if kind == "relu":
            return z.clamp(min=0), (z > 0).to(f64)
        if kind == "silu":
            s = torch.sigmoid(z)
            return z * s, s + z * s * torch.sigmoid(-z)
        if kind == "gelu":
            cdf = 0.5 * torch.special.erfc(-z / root2)
            return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if kind == "gelu_tanh":
            k = math.sqrt(2 / math.pi)
            t = torch.tanh(k * (z + 0.044715 * z ** 3))
            s = torch.sigmoid(2 * k * (z + 0.044715 * z ** 3))
            return z * s, s + 0.5 * z * (1 - t * t) * k * (1 + 0.134145 * z ** 2)
        return z, torch.ones_like(z)

    if case["op"] == "gemm_t":
        return torch.mm(st["dY"].to(f64), weight64(st["w"][0]))
    x = st["X"].to(f64)
    pre = []
    for w, b in zip(st["w"], st["bias"]):
        p = torch.mm(x, weight64(w).t())
        pre.append(p if b is None else p + b.to(f64))
    a, da = act64(pre[0], case["act"])
    if case["op"] == "linear":
        y = a + st["residual"].to(f64) if "residual" in st else a
    else:
        y = a * pre[1]
    if not case["train"]:
        return y
    dy = st["dY"].to(f64)
    grads = [dy * da] if case["op"] == "linear" else [dy * pre[1] * da, dy * a]
    dx = torch.zeros_like(x)
    for g, w in zip(grads, st["w"]):
        dx += torch.mm(g, weight64(w))
    return (y, dx) + tuple(g.sum(0) for g, b in zip(grads, st["bias"]) if b is not None)
