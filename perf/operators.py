"""Dense-layer and gradient operators: their cases, plain forms and exact values.

Three operators, each in three element types (float32, bfloat16, float16):

* ``fwd``   y = act(x W^T + b + r), with z = x W^T + b + r kept for the backward pass where asked for;
* ``grad``  its backward pass: dx, dW, db and, for the residual, dr;
* ``clip``  the global L2 norm of a list of gradients, and the gradients scaled down to a largest norm.

``own`` chooses between the plain form (elementary torch operations in 32 bits, rounded once at the end) and the
library's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "silu")


def listed():
    return [
        # one input (one token) through a wide layer: only the weights' bytes count
        {"name": "fwd one token", "op": "fwd", "dtype": "bf16", "M": 1, "N": 4096, "K": 1024, "act": "gelu",
         "res": False, "z": False, "pad": 0},
        # a layer of the 8-32-32-4 network on its 64 centres: nothing but latency
        {"name": "fwd tiny mlp", "op": "fwd", "dtype": "f32", "M": 64, "N": 32, "K": 8, "act": "relu",
         "res": False, "z": False, "pad": 0},
        # a small batch of tokens through a projection with its residual
        {"name": "fwd 16 tokens", "op": "fwd", "dtype": "bf16", "M": 16, "N": 2048, "K": 8192, "act": "none",
         "res": True, "z": False, "pad": 0},
        # the first layer of the 784-256x3-10 network on its 1024 centres
        {"name": "fwd mlp 784-256", "op": "fwd", "dtype": "f32", "M": 1024, "N": 256, "K": 784, "act": "relu",
         "res": False, "z": False, "pad": 0},
        # a 1024-wide layer on 4096 centres, closing a residual block
        {"name": "fwd wide residual", "op": "fwd", "dtype": "f32", "M": 4096, "N": 1024, "K": 1024, "act": "relu",
         "res": True, "z": False, "pad": 0},
        # odd sizes, rows of a wider buffer, everything in the epilogue
        {"name": "fwd odd strided", "op": "fwd", "dtype": "f16", "M": 777, "N": 1001, "K": 515, "act": "silu",
         "res": True, "z": True, "pad": 5},
        # a training layer of a large model: the largest forward product
        {"name": "fwd large", "op": "fwd", "dtype": "bf16", "M": 8192, "N": 4096, "K": 4096, "act": "gelu",
         "res": False, "z": True, "pad": 0},
        # training the 784-256x3-10 network
        {"name": "grad mlp 784-256", "op": "grad", "dtype": "f32", "M": 1024, "N": 256, "K": 784, "act": "relu",
         "res": False, "z": True, "pad": 0},
        # odd sizes and strides with the residual's gradient
        {"name": "grad odd strided", "op": "grad", "dtype": "f16", "M": 333, "N": 517, "K": 1001, "act": "silu",
         "res": True, "z": True, "pad": 3},
        # the largest backward pass
        {"name": "grad large", "op": "grad", "dtype": "bf16", "M": 8192, "N": 4096, "K": 4096, "act": "gelu",
         "res": False, "z": True, "pad": 0},
        # the weight and bias gradients of the 784-256x3-10 network: 8 tensors, latency
        {"name": "clip mlp", "op": "clip", "dtype": "f32", "count": 8, "total": 335114, "over": 4.0, "scale": 1.0},
        # the gradients of a model of 280 million weights, larger than the L2 cache
        {"name": "clip large", "op": "clip", "dtype": "bf16", "count": 48, "total": 280_000_001, "over": 2.6,
         "scale": 0.125},
    ]


def _spread(rng, lo, hi):
    """A size spread over the logarithm of its range."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "grad", "grad", "clip"))
    dtype = rng.choice(("f32", "bf16", "f16"))
    if op == "clip":
        return {"op": op, "dtype": dtype, "count": _spread(rng, 1, 60), "total": _spread(rng, 1000, 140_000_000),
                "over": rng.choice((0.5, 3.0)), "scale": rng.choice((1.0, 1.0 / 64))}
    case = {"op": op, "dtype": dtype, "M": _spread(rng, 1, 8192), "N": _spread(rng, 4, 4096),
            "K": _spread(rng, 4, 4096), "act": rng.choice(ACTS), "res": rng.random() < 0.5,
            "z": op == "grad" or rng.random() < 0.5, "pad": rng.choice((0, 0, 1, 8))}
    if rng.random() < 0.5:  # widths as models have them
        case["N"], case["K"] = -(-case["N"] // 64) * 64, -(-case["K"] // 64) * 64
    return case


def _sizes(case):
    """The lengths of a list of gradients: weights and short vectors in turn, `total` values in all."""
    rng = random.Random(case["count"] * 1_000_003 + case["total"])
    parts = [rng.random() ** 2 * (1.0 if i % 2 == 0 else 0.01) + 1e-4 for i in range(case["count"])]
    sizes = [int(case["total"] * p / sum(parts)) for p in parts]
    sizes[0] += case["total"] - sum(sizes)
    return sizes


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(rows, cols, std, pad=0):
        t = torch.randn(rows, cols + pad, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)
        return t[:, :cols]

    if case["op"] == "clip":
        sizes = _sizes(case)
        flat = torch.randn(case["total"], generator=gen, device="cuda", dtype=torch.float32).mul_(0.02).to(dtype)
        # each gradient is an allocation of its own, as a training program has them
        grads = [g.clone() for g in torch.split(flat, sizes)]
        norm = 0.02 * case["scale"] * math.sqrt(case["total"])
        return {"case": case, "grads": grads, "out": [torch.empty_like(g) for g in grads],
                "max_norm": norm / case["over"]}
    M, N, K, pad = case["M"], case["N"], case["K"], case["pad"]
    s = {"case": case, "W": normal(N, K, math.sqrt(2.0 / K)), "b": normal(1, N, 0.1)[0]}
    # inputs as a ReLU layer before leaves them for half of the seeds, signed for the others
    s["x"] = normal(M, K, 1.0, pad)
    if seed % 2:
        s["x"] = s["x"].clamp_(min=0)
    if case["op"] == "fwd":
        s["r"] = normal(M, N, 1.0, pad) if case["res"] else None
    else:
        s["dy"] = normal(M, N, 0.01, pad)
        s["z"] = normal(M, N, 1.4, pad)
    return s


# --------------------------------------------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * (0.5 * torch.erfc(z * -math.sqrt(0.5)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _plain(s):
    case, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    if case["op"] == "clip":
        norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
        norm = norm * case["scale"]
        clip = torch.isfinite(norm) & (norm > s["max_norm"])
        f = torch.where(clip, s["max_norm"] / norm, torch.ones_like(norm)) * case["scale"]
        f = f.float()
        return {"norm": norm.float(), "out": [(g.float() * f).to(dtype) for g in s["grads"]]}
    x, W = s["x"].float(), s["W"].float()
    if case["op"] == "fwd":
        z = x @ W.t() + s["b"].float()
        if case["res"]:
            z = z + s["r"].float()
        return {"y": _act(z, case["act"]).to(dtype), "z": z.to(dtype) if case["z"] else None}
    g = s["dy"].float() * _act_grad(s["z"].float(), case["act"])
    return {"dx": (g @ W).to(dtype), "dW": (g.t() @ x).to(dtype), "db": g.sum(0).to(dtype),
            "dr": g.to(dtype) if case["res"] else None}


def run(state):
    if not own:
        return _plain(state)
    from linear_bound_propagation_b200 import vf

    case = state["case"]
    if case["op"] == "clip":
        norm, out = vf.clip_grad_norm(state["grads"], state["max_norm"], scale=case["scale"], out=state["out"])
        return {"norm": norm, "out": out}
    if case["op"] == "fwd":
        out = vf.linear(state["x"], state["W"], state["b"], residual=state["r"], act=case["act"], want_z=case["z"])
        return {"y": out["y"], "z": out["z"]}
    need = ("dx", "dW", "db", "dr") if case["res"] else ("dx", "dW", "db")
    out = vf.linear_grad(state["dy"], state["x"], state["W"], act=case["act"], z=state["z"], need=need)
    return {k: out[k] for k in ("dx", "dW", "db", "dr")}


def work(case):
    """Each input read once and each output written once; the products' operations."""
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "clip":
        return {"bytes": 2 * e * case["total"] + 4, "flops": 3 * case["total"]}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "fwd":
        outs = 1 + (1 if case["z"] else 0) + (1 if case["res"] else 0)
        return {"bytes": e * (M * K + N * K + N + outs * M * N), "flops": 2 * M * N * K}
    outs = 1 + (1 if case["act"] != "none" else 0) + (1 if case["res"] else 0)
    return {"bytes": e * (2 * M * K + 2 * N * K + N + outs * M * N), "flops": 4 * M * N * K}


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "clip":
        squares = sum(float((g.double() ** 2).sum()) for g in s["grads"])
        norm = case["scale"] * math.sqrt(squares)
        f = case["scale"] * (s["max_norm"] / norm if norm > s["max_norm"] else 1.0)
        return {"norm": torch.tensor(norm, dtype=torch.float64), "out": [g.double() * f for g in s["grads"]]}
    x, W, root = s["x"].double(), s["W"].double(), math.sqrt(2.0)
    if case["op"] == "fwd":
        z = torch.addmm(s["b"].double(), x, W.t())
        if s["r"] is not None:
            z += s["r"].double()
        y = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, torch.zeros_like(z)),
             "gelu": lambda: z * (1.0 + torch.erf(z / root)) / 2.0, "silu": lambda: z / (1.0 + torch.exp(-z))}[case["act"]]()
        return {"y": y, "z": z if case["z"] else None}
    z, g = s["z"].double(), s["dy"].double()
    if case["act"] == "relu":
        g = torch.where(z > 0, g, torch.zeros_like(g))
    elif case["act"] == "gelu":
        density = torch.exp(-(z ** 2) / 2.0) / math.sqrt(2.0 * math.pi)
        g = g * ((1.0 + torch.erf(z / root)) / 2.0 + z * density)
    elif case["act"] == "silu":
        e = 1.0 + torch.exp(-z)
        g = g * (1.0 / e + z * (e - 1.0) / (e * e))
    return {"dx": torch.mm(g, W), "dW": torch.mm(g.t(), x), "db": torch.sum(g, 0), "dr": g if case["res"] else None}
