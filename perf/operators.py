"""The 4-bit and orthogonalising operators, as they are measured: MXFP4 quantisation and its
inverse, the product of two MXFP4 matrices, the product of binary16 activations with an MXFP4
weight, and the Newton-Schulz orthogonalisation of an update.

``run`` computes an operator in elementary float32 torch operations, or, where ``own`` is true,
through the package's entry points. An MXFP4 matrix (R x K) is a pair (codes, scales): codes
uint8 (R, 16 KB), KB = ceil(K / 32), two E2M1 codes a byte, the even k in the low half, zero
codes past K; scales uint8 (R, KB), byte s standing for 2^(s - 127), in rows padded to 16 bytes.
"""
import math

import torch

own = False

BLOCK = 32
NS_A, NS_B, NS_C, NS_EPS = 3.4445, -4.7750, 2.0315, 1e-7
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One token's activations brought to the grid of four bits and back: latency.
        {"name": "roundtrip_token", "op": "roundtrip", "R": 1, "K": 4096, "dims": "rows"},
        # Ragged activations: 3000 is no multiple of the block of 32.
        {"name": "roundtrip_ragged", "op": "roundtrip", "R": 4095, "K": 3000, "dims": "rows"},
        # A training batch along both of its axes, as the two products of a backward pass read it.
        {"name": "roundtrip_both", "op": "roundtrip", "R": 16384, "K": 4096, "dims": "both"},
        # A row shard of a linear layer, both operands in four bits.
        {"name": "mxfp4_shard", "op": "mxfp4", "M": 512, "N": 4096, "K": 4096, "relu": True},
        # The largest product of two 4-bit matrices.
        {"name": "mxfp4_8192", "op": "mxfp4", "M": 8192, "N": 8192, "K": 8192, "relu": False},
        # One training step of a linear layer on a ragged batch: output and both gradients.
        {"name": "mxfp4_train", "op": "train", "M": 4095, "N": 4096, "K": 4096},
        # Serving one token: bound by reading the weight.
        {"name": "weight_token", "op": "weight", "M": 1, "N": 8192, "K": 4096, "relu": False},
        # A few sequences decoded together, an output width that is no multiple of a tile.
        {"name": "weight_batch", "op": "weight", "M": 37, "N": 3000, "K": 4096, "relu": True},
        # A prompt.
        {"name": "weight_prompt", "op": "weight", "M": 4096, "N": 4096, "K": 4096, "relu": False},
        # A frozen 4-bit layer inside a fine-tuned model: output and the input's gradient.
        {"name": "weight_tune", "op": "tune", "M": 2048, "N": 4096, "K": 1024},
        # The momenta of a stack of small layers, kept in float32.
        {"name": "orth_stack", "op": "orth", "batch": 16, "R": 512, "C": 2048, "dtype": "float32", "steps": 5},
        # One large square layer's update.
        {"name": "orth_4096", "op": "orth", "batch": 1, "R": 4096, "C": 4096, "dtype": "float16", "steps": 5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """Sizes over the logarithm of their range; half of them rounded to whole multiples of 64."""
    def size(lo, hi):
        v = _log_int(rng, lo, hi)
        return v if rng.random() < 0.5 or v < 64 else v // 64 * 64

    op = rng.choice(["roundtrip", "mxfp4", "train", "weight", "weight", "tune", "orth"])
    if op == "roundtrip":
        return {"op": op, "R": size(1, 16384), "K": size(33, 4096), "dims": rng.choice(["rows", "cols", "both"])}
    if op in ("mxfp4", "weight"):
        return {"op": op, "M": size(1, 4096), "N": size(64, 8192), "K": size(64, 8192), "relu": rng.random() < 0.5}
    if op in ("train", "tune"):
        return {"op": op, "M": size(16, 4096), "N": size(64, 4096), "K": size(64, 4096)}
    return {"op": op, "batch": rng.choice([1, 1, 2, 5, 12]), "R": size(64, 2048), "C": size(64, 2048),
            "dtype": rng.choice(["float16", "float32"]), "steps": rng.choice([4, 5, 6])}


def _blocks(k):
    return -(-k // BLOCK)


# ---------------------------------------------------------------- plain forms
def _code_magnitudes(a):
    """E2M1 code (0..7) of a >= 0: to nearest, ties to the even code, saturated at 6."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _quant(x):
    """(codes, scales) of a 2-D x along its last axis: scale 2^(floor(log2 amax) - 2) for each
    block of 32 (1 for a block of zeros)."""
    rows, k = x.shape
    kb = _blocks(k)
    v = torch.zeros((rows, kb * BLOCK), dtype=torch.float32, device=x.device)
    v[:, :k] = x.float()
    v = v.view(rows, kb, BLOCK)
    amax = v.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1].to(torch.int32) - 3, torch.zeros((), dtype=torch.int32, device=x.device))
    code = _code_magnitudes(torch.ldexp(v.abs(), -e[..., None]))
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).view(rows, kb * BLOCK // 2, 2)
    pad = torch.zeros((rows, -(-kb // 16) * 16), dtype=torch.uint8, device=x.device)
    pad[:, :kb] = (e + 127).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), pad[:, :kb]


def _values(codes, scales):
    """The float32 values (R, 32 KB) of an MXFP4 matrix."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    rows, kb = scales.shape
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).view(rows, kb, BLOCK)
    return torch.ldexp(v, scales.to(torch.int32)[..., None] - 127).view(rows, kb * BLOCK)


def _rounded(x):
    """The values of x (R x K) after quantisation along its last axis."""
    return _values(*_quant(x))[:, : x.shape[1]]


def _orthogonalised(g, steps):
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt() + NS_EPS).float()
    for _ in range(steps):
        a = x @ x.transpose(1, 2)
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x.transpose(1, 2).contiguous() if tall else x


# ---------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, m, k):
    """Normal activations, a few channels much larger than the rest, as trained models have them."""
    gain = torch.where(torch.rand(k, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
    return (_normal(gen, m, k) * gain).half()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = dict(case)
    if op == "roundtrip":
        state["x"] = _activations(gen, case["R"], case["K"])
    elif op == "mxfp4":
        state["a"], state["sa"] = _quant(_activations(gen, case["M"], case["K"]))
        state["b"], state["sb"] = _quant((_normal(gen, case["N"], case["K"]) / math.sqrt(case["K"])).half())
    elif op == "train":
        state["x"] = _activations(gen, case["M"], case["K"]).requires_grad_()
        state["w"] = (_normal(gen, case["N"], case["K"]) / math.sqrt(case["K"])).half().requires_grad_()
        state["dy"] = (_normal(gen, case["M"], case["N"]) * 0.01).half()
    elif op in ("weight", "tune"):
        state["x"] = _activations(gen, case["M"], case["K"]).requires_grad_(op == "tune")
        state["q"], state["s"] = _quant((_normal(gen, case["N"], case["K"]) / math.sqrt(case["K"])).half())
        if op == "tune":
            state["dy"] = (_normal(gen, case["M"], case["N"]) * 0.01).half()
    else:
        b, r, c = case["batch"], case["R"], case["C"]
        # a gradient: a few strong directions over a floor of noise
        g = _normal(gen, b, r, 8) @ _normal(gen, b, 8, c) * 1e-3 + _normal(gen, b, r, c) * 3e-3
        state["g"] = g.to(getattr(torch, case["dtype"]))
    return state


# ---------------------------------------------------------------- one pass
def _run_own(s):
    import tiled_dense_gemm_04_amd as tg

    op = s["op"]
    if op == "roundtrip":
        r, k = s["R"], s["K"]
        q = tg.mxfp4_quant(s["x"], s["dims"])
        if s["dims"] == "rows":
            return tg.mxfp4_dequant(q[0], q[1], k)
        if s["dims"] == "cols":
            return tg.mxfp4_dequant(q[0], q[1], r)
        return tg.mxfp4_dequant(q[0], q[1], k), tg.mxfp4_dequant(q[2], q[3], r)
    if op == "mxfp4":
        return tg.mxfp4_gemm(s["a"], s["sa"], s["b"], s["sb"], relu=s["relu"])
    if op == "train":
        y = tg.Mxfp4LinearFunction.apply(s["x"], s["w"])
        return (y.detach(), *torch.autograd.grad(y, (s["x"], s["w"]), s["dy"]))
    if op == "weight":
        return tg.mxfp4_gemm_f16(s["x"], s["q"], s["s"], relu=s["relu"])
    if op == "tune":
        y = tg.Mxfp4WeightFunction.apply(s["x"], s["q"], s["s"])
        return (y.detach(), *torch.autograd.grad(y, (s["x"],), s["dy"]))
    return tg.orthogonalize(s["g"], steps=s["steps"])


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    with torch.no_grad():
        if op == "roundtrip":
            x = s["x"]
            if s["dims"] == "rows":
                return _rounded(x).half()
            if s["dims"] == "cols":
                return _rounded(x.t()).half()
            return _rounded(x).half(), _rounded(x.t()).half()
        if op == "mxfp4":
            y = _values(s["a"], s["sa"]) @ _values(s["b"], s["sb"]).t()
            return (y.clamp_min(0) if s["relu"] else y).half()
        if op == "train":
            x, w, dy = s["x"], s["w"], s["dy"]
            y = _rounded(x) @ _rounded(w).t()
            dx = _rounded(dy) @ _rounded(w.t()).t()
            dw = _rounded(dy.t()) @ _rounded(x.t()).t()
            return y.half(), dx.half(), dw.half()
        if op in ("weight", "tune"):
            w = _values(s["q"], s["s"])[:, : s["K"]].half().float()  # the weight in the activations' type
            y = s["x"].float() @ w.t()
            if op == "weight":
                return (y.clamp_min(0) if s["relu"] else y).half()
            return y.half(), (s["dy"].float() @ w).half()
        return _orthogonalised(s["g"], s["steps"]).half()


def work(case):
    op = case["op"]

    def packed(r, k):  # bytes of an MXFP4 matrix
        return r * _blocks(k) * 17

    if op == "roundtrip":
        r, k = case["R"], case["K"]
        ways = 2 if case["dims"] == "both" else 1
        return {"bytes": 2 * r * k * (1 + ways), "flops": 4 * r * k * ways}
    if op == "orth":
        b, m, n = case["batch"], min(case["R"], case["C"]), max(case["R"], case["C"])
        size = 2 if case["dtype"] == "float16" else 4
        # the two symmetric products need half of their entries each
        return {"bytes": b * m * n * (size + 2), "flops": case["steps"] * b * (m * m * n + m * m * m + 2 * m * m * n)}
    m, n, k = case["M"], case["N"], case["K"]
    if op == "mxfp4":
        return {"bytes": packed(m, k) + packed(n, k) + 2 * m * n, "flops": 2 * m * n * k}
    if op == "train":
        return {"bytes": 2 * (2 * m * k + 2 * n * k + 2 * m * n), "flops": 6 * m * n * k}
    if op == "weight":
        return {"bytes": 2 * m * k + packed(n, k) + 2 * m * n, "flops": 2 * m * n * k}
    return {"bytes": 4 * m * k + packed(n, k) + 4 * m * n, "flops": 4 * m * n * k}


# ---------------------------------------------------------------- 64-bit definitions
def _grid64(x):
    """Quantised values of a 2-D x along its last axis, in float64: the multiple of the local
    step of E2M1 that is nearest, ties to even."""
    rows, k = x.shape
    v = torch.nn.functional.pad(x.detach().double(), (0, -k % BLOCK)).reshape(rows, -1, BLOCK)
    top = v.abs().max(-1, keepdim=True).values
    scale = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 4.0))) - 2)
    u = v / scale
    step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(1.0))) - 1)
    u = (torch.round(u / step) * step).clamp(-6.0, 6.0)
    return (u * scale).reshape(rows, -1)[:, :k]


def _decoded64(codes, scales):
    """float64 values of packed codes, from the fields of E2M1: sign, two exponent bits, one fraction bit."""
    c = torch.stack((codes % 16, codes // 16), -1).reshape(codes.shape[0], -1).double()
    sign = torch.where(c >= 8, -1.0, 1.0)
    c = c % 8
    e, f = torch.floor(c / 2), c % 2
    mag = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * torch.exp2(e - 1))
    return sign * mag * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op == "roundtrip":
            x = s["x"]
            if s["dims"] == "rows":
                return _grid64(x)
            if s["dims"] == "cols":
                return _grid64(x.t())
            return _grid64(x), _grid64(x.t())
        if op == "mxfp4":
            y = _decoded64(s["a"], s["sa"]) @ _decoded64(s["b"], s["sb"]).t()
            return torch.relu(y) if s["relu"] else y
        if op == "train":
            x, w, dy = s["x"], s["w"], s["dy"]
            return (_grid64(x) @ _grid64(w).t(), _grid64(dy) @ _grid64(w.t()).t(),
                    _grid64(dy.t()) @ _grid64(x.t()).t())
        if op in ("weight", "tune"):
            w = _decoded64(s["q"], s["s"])[:, : s["K"]].half().double()  # binary16 weights by definition
            y = s["x"].double() @ w.t()
            if op == "weight":
                return torch.relu(y) if s["relu"] else y
            return y, s["dy"].double() @ w
        x = s["g"].double()
        x = x / (torch.linalg.matrix_norm(x)[:, None, None] + NS_EPS)
        for _ in range(s["steps"]):
            if x.shape[1] <= x.shape[2]:
                a = torch.bmm(x, x.mT.contiguous())
                x = NS_A * x + torch.bmm(NS_B * a + NS_C * torch.bmm(a, a), x)
            else:
                a = torch.bmm(x.mT.contiguous(), x)
                x = NS_A * x + torch.bmm(x, NS_B * a + NS_C * torch.bmm(a, a))
        return x
