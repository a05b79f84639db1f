"""The dense-layer and gradient operators (vf.linear, vf.linear_grad, vf.clip_grad_norm) on a B200, against plain
formulas in 64 bits.

Tolerances are worst-case sums of the roundings each output passes (u = 2^-24):
* a product of T terms held in fp32 or fp32 accumulators: (1.1 T + 16) 2^-23 of sum |a||b|. This covers a chain of
  fused multiply-adds (T u), matrix instructions that add 16 products and the accumulator with one truncation of 2^-23
  for each of the 17, and an fp32 operand taken as three 8-bit pieces with the products below 2^-24 left out (2^-23);
* the activation, evaluated in fp32: slope at most 1.13 times the error of z, plus (10 + z^2) u |y| (a few ulp, and
  erfc's argument rounded to u, which erfc's logarithmic slope of about z turns into z^2 u);
* its slope: 2^-20 absolute;
* g rounded to a 16-bit type before it enters a product: half a step of |g|, and half a subnormal step for float16;
* the output's own rounding: half a step, eps / 2 relative, plus half a subnormal step for float16.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from linear_bound_propagation_b200 import synth

vf = pytest.importorskip("linear_bound_propagation_b200.vf")
pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
U = 2.0 ** -24


def acc_tol(T):
    return (1.1 * T + 16) * 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sub_step(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def act64(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    return torch.ones_like(z)


def randn(gen, rows, cols, dtype, std=1.0, pad=0, off=0):
    """[rows, cols] view of a buffer with `pad` extra columns, starting `off` elements in."""
    t = torch.randn(rows * (cols + pad) + off, generator=gen, device="cuda").mul_(std).to(dtype)
    return t[off:].view(rows, cols + pad)[:, :cols]


def worst(got, want, tol):
    """Largest |got - want| / tol; shapes equal and everything finite."""
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    if not got.numel():
        return 0.0
    return float(((got.double() - want).abs() / (tol + 1e-300)).max())


def check_forward(dtype, M, N, K, act, bias, res, pad, off, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, W = randn(gen, M, K, dtype, 1.0, pad, off), randn(gen, N, K, dtype, K ** -0.5 if K else 1.0, pad, off)
    b = randn(gen, 1, N, dtype)[0] if bias else None
    r = randn(gen, M, N, dtype, 1.0, pad, off) if res else None
    got = vf.linear(x, W, b, residual=r, act=act, want_z=True)
    vf.ops_check()
    z, S = x.double() @ W.double().t(), x.double().abs() @ W.double().abs().t()
    for t in (b, r):
        if t is not None:
            z, S = z + t.double(), S + t.double().abs()
    ez = acc_tol(K) * S
    y = act64(z, act)
    ey = 1.13 * ez + (10 + z * z) * U * y.abs()
    hs, ss = half_step(dtype), sub_step(dtype)
    assert worst(got["z"], z, ez + hs * (z.abs() + ez) + ss) <= 1.0
    assert worst(got["y"], y, ey + hs * (y.abs() + ey) + ss) <= 1.0


def check_grad(dtype, M, N, K, act, pad, off, seed, need=("dx", "dW", "db", "dr")):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, W = randn(gen, M, K, dtype, 1.0, pad, off), randn(gen, N, K, dtype, 0.1, pad, off)
    dy, z = randn(gen, M, N, dtype, 1.0, pad, off), randn(gen, M, N, dtype, 1.5, pad, off)
    got = vf.linear_grad(dy, x, W, act=act, z=None if act == "none" else z, need=need)
    vf.ops_check()
    assert all((got[k] is not None) == (k in need) for k in ("dx", "dW", "db", "dr"))
    hs, ss = half_step(dtype), sub_step(dtype)
    g = dy.double() * slope64(z.double(), act)
    eg = 2.0 ** -20 * dy.double().abs() if act in ("gelu", "silu") else torch.zeros_like(g)
    ein = eg + (hs * g.abs() + ss if act in ("gelu", "silu") and dtype != torch.float32 else 0)
    want = {"dx": g @ W.double(), "dW": g.t() @ x.double(), "db": g.sum(0), "dr": g}
    tol = {"dx": acc_tol(N) * (g.abs() @ W.double().abs()) + ein @ W.double().abs(),
           "dW": acc_tol(M) * (g.abs().t() @ x.double().abs()) + ein.t() @ x.double().abs(),
           "db": acc_tol(M) * g.abs().sum(0) + eg.sum(0), "dr": eg}
    for k in need:
        t = tol[k] + hs * (want[k].abs() + tol[k]) + ss
        assert worst(got[k], want[k], t) <= 1.0, k


SHAPES = [(1, 1, 1), (1, 1000, 70), (2, 3, 515), (3, 5, 0), (7, 130, 33), (8, 4096, 1024), (16, 512, 4096),
          (33, 64, 200), (64, 32, 8), (100, 1, 300), (128, 256, 64), (129, 257, 65), (200, 100, 784), (300, 520, 1001),
          (1000, 384, 320), (1025, 1025, 129)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_matches_formula(dtype, shape):
    for i, (act, bias, res, pad, off) in enumerate([("none", False, False, 0, 0), ("relu", True, True, 0, 0),
                                                    ("gelu", True, False, 8, 8), ("silu", True, True, 3, 1)]):
        check_forward(dtype, *shape, act, bias, res, pad, off, 100 + i)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_grad_matches_formula(dtype, shape):
    for i, (act, pad, off) in enumerate([("none", 0, 0), ("relu", 0, 0), ("gelu", 8, 8), ("silu", 3, 1)]):
        check_grad(dtype, *shape, act, pad, off, 200 + i)


@pytest.mark.parametrize("need", [("dx",), ("dW",), ("db",), ("dr",), ("dx", "db"), ()])
def test_linear_grad_of_some_outputs(need):
    for dtype in DTYPES:
        check_grad(dtype, 150, 200, 130, "silu", 0, 0, 5, need)
        check_grad(dtype, 3, 20, 10, "relu", 1, 0, 6, need)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (5, 40, 333), (16, 128, 1024), (130, 70, 100), (257, 513, 448),
                                   (384, 640, 512), (2000, 300, 64)])
def test_small_whole_numbers_are_exact(dtype, M, N, K):
    """Products of whole numbers in -2..2 stay below 2^24, so every sum is exact and only the output rounds."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    x, W, r, dy = (torch.randint(-2, 3, s, generator=gen, device="cuda").to(dtype) for s in ((M, K), (N, K), (M, N), (M, N)))
    z = (x.double() @ W.double().t() + r.double()).to(dtype)
    assert torch.equal(vf.linear(x, W, residual=r)["y"], z)
    assert torch.equal(vf.linear(x, W, residual=r, act="relu")["y"], z.clamp(min=0))
    g = dy.double() * (r.double() > 0)
    got = vf.linear_grad(dy, x, W, act="relu", z=r, need=("dx", "dW", "db", "dr"))
    assert torch.equal(got["dx"], (g @ W.double()).to(dtype))
    assert torch.equal(got["dW"], (g.t() @ x.double()).to(dtype))
    assert torch.equal(got["db"], g.sum(0).to(dtype))
    assert torch.equal(got["dr"], g.to(dtype))
    vf.ops_check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(4090, 1016, 72), (4096, 1020, 200), (2050, 2048, 2040), (8200, 520, 264)])
def test_many_large_tiles(dtype, M, N, K):
    """Sizes whose tiles are 256 x 256 and shared by a pair of CTAs, several per pair, ragged in every direction."""
    check_forward(dtype, M, N, K, "relu", True, True, 0, 0, 1)
    check_forward(dtype, M, N, K, "gelu", True, False, 3, 1, 2)
    check_grad(dtype, M, N, K, "silu", 0, 0, 3)
    check_grad(dtype, M, N, K, "relu", 8, 8, 4, ("dx", "dW"))
    gen = torch.Generator(device="cuda").manual_seed(M)
    x, W, r = (torch.randint(-2, 3, s, generator=gen, device="cuda").to(dtype) for s in ((M, K), (N, K), (M, N)))
    assert torch.equal(vf.linear(x, W, residual=r)["y"], (x.double() @ W.double().t() + r.double()).to(dtype))
    got = vf.linear_grad(r, x, W)
    assert torch.equal(got["dx"], (r.double() @ W.double()).to(dtype))
    assert torch.equal(got["dW"], (r.double().t() @ x.double()).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(5557, 64, 64), (8000, 10, 200), (3000, 300, 40), (64, 5000, 24), (24, 40, 6000),
                                   (6, 3000, 520), (8, 33, 1027)])
def test_unequal_products_of_the_backward_pass(dtype, M, N, K):
    """Long reductions behind few tiles, few rows, and one product much larger than the other: exact on whole numbers
    (every sum stays below 2^24), and within the roundings with an activation."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    x, W, r, dy = (torch.randint(-2, 3, s, generator=gen, device="cuda").to(dtype) for s in ((M, K), (N, K), (M, N), (M, N)))
    g = dy.double() * (r.double() > 0)
    want = {"dx": g @ W.double(), "dW": g.t() @ x.double(), "db": g.sum(0), "dr": g}
    for need in (("dx", "dW", "db", "dr"), ("dx",), ("dW",), ("dW", "db"), ("dx", "dr")):
        got = vf.linear_grad(dy, x, W, act="relu", z=r, need=need)
        for k in need:
            assert torch.equal(got[k], want[k].to(dtype)), (need, k)
    check_grad(dtype, M, N, K, "gelu", 0, 0, 7)
    check_grad(dtype, M, N, K, "silu", 3, 1, 8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(4096, 1016, 256), (2050, 264, 72), (700, 1030, 64), (16, 640, 2048)])
def test_in_place_over_the_residual(dtype, M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, W, r = randn(gen, M, K, dtype), randn(gen, N, K, dtype, K ** -0.5), randn(gen, M, N, dtype)
    want = vf.linear(x, W, residual=r, act="gelu")["y"]
    for _ in range(2):
        buf = r.clone()
        assert vf.linear(x, W, residual=buf, act="gelu", out=buf)["y"] is buf
        assert torch.equal(buf, want)


def test_offsets_beyond_32_bits():
    """Rows of x, y and z whose elements lie more than 2^31 apart, forward and backward, against sampled rows."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    M, N, K = 33000, 24, 66000
    x = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
    for i in range(0, M, 3000):
        x[i:i + 3000] = torch.randn(3000, K, generator=gen, device="cuda")[:x[i:i + 3000].shape[0]].bfloat16()
    W = randn(gen, N, K, torch.bfloat16, K ** -0.5)
    rows = torch.tensor([0, 1, 2048, 32766, M - 1], device="cuda")
    y = vf.linear(x, W)["y"]
    z, S = x[rows].double() @ W.double().t(), x[rows].double().abs() @ W.double().abs().t()
    ez = acc_tol(K) * S
    assert worst(y[rows], z, ez + 2.0 ** -8 * (z.abs() + ez)) <= 1.0
    dy = randn(gen, M, N, torch.bfloat16)
    g = vf.linear_grad(dy, x, W, need=("dx", "dW"))
    dx, S = dy[rows].double() @ W.double(), dy[rows].double().abs() @ W.double().abs()
    ex = acc_tol(N) * S
    assert worst(g["dx"][rows], dx, ex + 2.0 ** -8 * (dx.abs() + ex)) <= 1.0
    cols = torch.tensor([0, 40000, K - 1], device="cuda")
    dW, S = dy.double().t() @ x[:, cols].double(), dy.double().abs().t() @ x[:, cols].double().abs()
    ew = acc_tol(M) * S
    assert worst(g["dW"][:, cols], dW, ew + 2.0 ** -8 * (dW.abs() + ew)) <= 1.0
    vf.ops_check()
    del dx, dW, S, z, g, y, dy
    flat = x.view(-1)[:2 ** 31 + 4099]
    flat[2 ** 31 + 7] = 3000.0
    want = math.sqrt(sum(float((c.double() ** 2).sum()) for c in torch.split(flat, 1 << 27)))
    norm, _ = vf.clip_grad_norm([flat], float("inf"))
    assert abs(float(norm) - want) <= 18 * U * want
    vf.clip_grad_norm([flat], want / 2)
    assert abs(float(flat[2 ** 31 + 7]) - 1500.0) <= 1500.0 * 2.0 ** -8


def test_workspace_is_checked_before_anything_runs():
    x, W = torch.ones(300, 200, device="cuda"), torch.ones(400, 200, device="cuda")
    y = torch.full((300, 400), 7.0, device="cuda")
    L = vf.lib()
    args = (0, 0, x.data_ptr(), 200, W.data_ptr(), 200, None, None, 0)
    buf = torch.empty(1 << 20, device="cuda", dtype=torch.uint8)
    dW, dy = torch.full((4000, 200), 7.0, device="cuda"), torch.ones(3000, 4000, device="cuda")
    xl = torch.ones(3000, 200, device="cuda")
    for work, nbytes, code in ((None, 0, vf.VF_ERR_WORKSPACE), (buf.data_ptr(), 1 << 20, vf.VF_ERR_WORKSPACE),
                               (buf.data_ptr() + 8, 1 << 19, vf.VF_ERR_ARG)):
        assert L.vf_linear_grad(0, 0, dy.data_ptr(), 4000, None, 0, xl.data_ptr(), 200, None, 0, 3000, 4000, 200, None, 0,
                                dW.data_ptr(), 200, None, None, 0, work, nbytes, None) == code
    assert L.vf_linear(*args, 300, 400, 200, y.data_ptr(), 400, None, 0, None, 0, None) in (vf.VF_OK, vf.VF_ERR_WORKSPACE)
    torch.cuda.synchronize()
    assert (dW == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [2, 4, 5, 8, 9, 13, 16, 17])
@pytest.mark.parametrize("N,K,pad", [(1, 129, 0), (517, 36, 4), (4099, 264, 8), (2050, 515, 1)])
def test_backward_of_a_few_rows_is_exact_on_whole_numbers(dtype, M, N, K, pad):
    """Every sum is a whole number below 2^24, so fp32 holds it and one rounding remains. Nothing is written behind a row."""
    gen = torch.Generator(device="cuda").manual_seed(M * 7 + N)

    def whole(rows, cols):
        return torch.randint(-3, 4, (rows, cols + pad), generator=gen, device="cuda").to(dtype)[:, :cols]

    dy, z, x, W = whole(M, N), whole(M, N), whole(M, K), whole(N, K)
    g = dy.double() * (z > 0)
    got = vf.linear_grad(dy, x, W, act="relu", z=z, need=("dx", "dW", "db", "dr"))
    for name, want in (("dx", g @ W.double()), ("dW", g.t() @ x.double()), ("db", g.sum(0)), ("dr", g)):
        assert torch.equal(got[name], want.to(dtype)), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9])
@pytest.mark.parametrize("N,K,pad", [(1, 1, 0), (6, 33, 0), (1183, 264, 8), (1190, 2056, 0), (130, 1030, 1), (4097, 8, 8)])
def test_forward_of_a_few_rows_is_exact_on_whole_numbers(dtype, M, N, K, pad):
    """As above, with bias and z, the output in the residual's place; what lies beside and behind it stays."""
    gen = torch.Generator(device="cuda").manual_seed(M * 5 + N)

    def whole(rows, cols):
        return torch.randint(-3, 4, (rows, cols + pad), generator=gen, device="cuda").to(dtype)[:, :cols]

    x, W, b = whole(M, K), whole(N, K), whole(1, N + 8)[0, :N].contiguous()
    buf = torch.randint(-3, 4, (M + 1, N + 3), generator=gen, device="cuda").to(dtype)
    before, r = buf.clone(), buf[:M, :N]
    want = x.double() @ W.double().t() + b.double() + r.double()
    got = vf.linear(x, W, b, residual=r, act="relu", want_z=True, out=r)
    assert torch.equal(got["z"], want.to(dtype))
    assert torch.equal(r, want.clamp(min=0).to(dtype))
    assert torch.equal(buf[M], before[M]) and torch.equal(buf[:, N:], before[:, N:])


@pytest.mark.parametrize("pad_x,pad_w", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_alignment_changes_the_kernel_not_the_result(pad_x, pad_w):
    """One wave of tiles in fp32: rows of 16-byte alignment need no workspace, others may go through a laid-out copy.
    Whole numbers: every sum is exact."""
    M, N, K = 500, 1000, 900
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randint(-3, 4, (M, K + pad_x), generator=gen, device="cuda").float()[:, :K]
    W = torch.randint(-3, 4, (N, K + pad_w), generator=gen, device="cuda").float()[:, :K]
    assert vf._linear_work(0, M, N, K, vf.VF_FORWARD_ALIGNED) == 0 < vf._linear_work(0, M, N, K, 0)
    assert (vf.linear(x, W)["y"].double() == x.double() @ W.double().t()).all()


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    """Host-set hook: the first CTA never makes its first copies, so its bounded waits expire; the call returns, the
    check reports it once, and later calls are right. One CTA per tile, and a pair of CTAs."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    for M, N, K in ((64, 128, 256), (4096, 1024, 256)):
        x, W = randn(gen, M, K, torch.bfloat16), randn(gen, N, K, torch.bfloat16)
        want = vf.linear(x, W)["y"].clone()
        vf.ops_check()
        monkeypatch.setenv("VF_TEST_OPS_STALL", "1")
        vf.linear(x, W)
        monkeypatch.delenv("VF_TEST_OPS_STALL")
        with pytest.raises(vf.VfError) as e:
            vf.ops_check()
        assert e.value.code == vf.VF_ERR_TIMEOUT
        vf.ops_check()
        assert torch.equal(vf.linear(x, W)["y"], want)


def test_the_first_calls_of_a_process_can_be_captured():
    code = """
import torch
from linear_bound_propagation_b200 import vf
x, W = torch.ones(512, 256, device="cuda"), torch.ones(384, 256, device="cuda")
xb, Wb = x.bfloat16(), W.bfloat16()
few = torch.ones(3, 256, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = [vf.linear(x, W)["y"], vf.linear(xb, Wb, act="relu")["y"], vf.linear(x[:, 1:], W[:, 1:])["y"]]
    d = vf.linear_grad(torch.ones_like(outs[0]), x, W)
    f = vf.linear_grad(torch.ones(3, 384, device="cuda"), few, W)
    norm, c = vf.clip_grad_norm([d["dW"]], 1.0, out=[torch.empty_like(d["dW"])])
g.replay()
torch.cuda.synchronize()
assert (outs[0] == 256).all() and (outs[1] == 256).all() and (outs[2] == 255).all()
assert (d["dx"] == 384).all() and (d["dW"] == 512).all() and (f["dx"] == 384).all() and (f["dW"] == 3).all()
assert abs(float(norm) - 512 * (384 * 256) ** 0.5) < 1
vf.ops_check()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(9, 200, 300), (130, 140, 520), (300, 3712, 1472)])
def test_one_operand_off_its_alignment(dtype, M, N, K):
    """x or W alone starts, or has rows, off a 16-byte boundary: exact on whole numbers."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    x, W = (torch.randint(-2, 3, s, generator=gen, device="cuda").to(dtype) for s in ((M, K), (N, K)))
    want = (x.double() @ W.double().t()).to(dtype)
    px = torch.zeros(M, K + 1, device="cuda", dtype=dtype)[:, :K].copy_(x)
    pw = torch.zeros(N * K + 1, device="cuda", dtype=dtype)[1:].view(N, K).copy_(W)
    assert torch.equal(vf.linear(px, W)["y"], want)
    assert torch.equal(vf.linear(x, pw)["y"], want)
    assert torch.equal(vf.linear(px, pw)["y"], want)
    dy = torch.randint(-2, 3, (M, N), generator=gen, device="cuda").to(dtype)
    for a, b in ((px, W), (x, pw)):
        got = vf.linear_grad(dy, a, b)
        assert torch.equal(got["dx"], (dy.double() @ W.double()).to(dtype))
        assert torch.equal(got["dW"], (dy.double().t() @ x.double()).to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_empty_sizes(dtype):
    e = lambda *s: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
    assert vf.linear(e(0, 4), e(3, 4), e(3))["y"].shape == (0, 3)
    assert vf.linear(e(4, 5), e(0, 5))["y"].shape == (4, 0)
    b = torch.tensor([1.0, -2.0], device="cuda", dtype=dtype)
    assert torch.equal(vf.linear(e(3, 0), e(2, 0), b, act="relu")["y"], b.clamp(min=0).expand(3, 2))
    g = vf.linear_grad(e(0, 3), e(0, 4), e(3, 4))
    assert g["dx"].shape == (0, 4) and not g["dW"].any() and not g["db"].any()
    g = vf.linear_grad(e(5, 0), e(5, 4), e(0, 4))
    assert not g["dx"].any() and g["dx"].shape == (5, 4) and g["dW"].shape == (0, 4)
    g = vf.linear_grad(torch.ones(5, 3, device="cuda", dtype=dtype), e(5, 0), e(3, 0), need=("dx", "dW", "db", "dr"))
    assert g["dx"].shape == (5, 0) and torch.equal(g["db"], torch.full((3,), 5.0, device="cuda", dtype=dtype))
    vf.ops_check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(1, 65, 64), (40, 70, 50), (300, 264, 256)])
def test_strided_output_leaves_its_surroundings(dtype, M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, W = randn(gen, M, K, dtype), randn(gen, N, K, dtype)
    buf = torch.full((M + 2, N + 7), 9.0, device="cuda", dtype=dtype)
    vf.linear(x, W, out=buf[1:M + 1, 3:N + 3])
    assert torch.equal(buf[1:M + 1, 3:N + 3], vf.linear(x, W)["y"])
    buf[1:M + 1, 3:N + 3] = 9.0
    assert (buf == 9.0).all()
    r = randn(gen, M, N, dtype)
    want = vf.linear(x, W, residual=r, act="relu")["y"]
    vf.linear(x, W, residual=r, act="relu", out=r)  # in place over the residual
    assert torch.equal(r, want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [2, 200])
def test_non_finite_rows_stay_in_their_rows(dtype, M):
    """An infinity or NaN in row 0 of x makes row 0 non-finite and leaves every other row's bits; an infinite dy behind
    a closed ReLU contributes nothing."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    N, K = 160, 192
    x, W = randn(gen, M, K, dtype), randn(gen, N, K, dtype)
    clean = vf.linear(x, W, act="none")["y"]
    for bad in (float("inf"), float("nan")):
        xb = x.clone()
        xb[0, 5] = bad
        y = vf.linear(xb, W)["y"]
        assert not torch.isfinite(y[0]).any()
        assert torch.equal(y[1:], clean[1:])
    z = randn(gen, M, N, dtype)
    dy = randn(gen, M, N, dtype)
    want = vf.linear_grad(torch.where(z > 0, dy, torch.zeros_like(dy)), x, W, act="relu", z=z)
    got = vf.linear_grad(torch.where(z > 0, dy, torch.full_like(dy, float("inf"))), x, W, act="relu", z=z)
    for k in ("dx", "dW", "db"):
        assert torch.equal(got[k], want[k])


def test_activation_limits():
    """Far arguments: gelu and silu reach 0 and z, their slopes 0 and 1, without inf * 0."""
    z = torch.tensor([[-3e38, -1e4, -100.0, -0.0, 0.0, 100.0, 1e4, 3e38]], device="cuda")
    one = torch.ones(1, 1, device="cuda")
    W = torch.zeros(8, 1, device="cuda")
    for act in ("gelu", "silu", "relu"):
        y = vf.linear(one, W, residual=z, act=act)["y"]
        assert torch.equal(y, z.clamp(min=0))
        dr = vf.linear_grad(torch.ones_like(z), one, W, act=act, z=z, need=("dr",))["dr"]
        want = [0.0, 0.0, 0.0, 0.5, 0.5, 1.0, 1.0, 1.0] if act != "relu" else [0.0] * 5 + [1.0] * 3
        assert dr[0].tolist() == want


def test_largest_and_smallest_fp32_values():
    """fp32 layers keep fp32's range: values near its largest and smallest normals."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    for M in (4, 160):
        x, W = randn(gen, M, 64, torch.float32), randn(gen, 200, 64, torch.float32)
        for s, t in ((2.0 ** 100, 2.0 ** 20), (2.0 ** -60, 2.0 ** -50), (2.0 ** 60, 2.0 ** -100)):
            y = vf.linear(x * s, W * t)["y"]
            z, S = (x * s).double() @ (W * t).double().t(), (x * s).double().abs() @ (W * t).double().abs().t()
            assert worst(y, z, acc_tol(64) * S + U * z.abs()) <= 1.0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M", [3, 300])
def test_repeats_streams_and_graphs_give_the_same_bits(dtype, M):
    gen = torch.Generator(device="cuda").manual_seed(8)
    N, K = 250, 328
    x, W, b, dy = randn(gen, M, K, dtype), randn(gen, N, K, dtype), randn(gen, 1, N, dtype)[0], randn(gen, M, N, dtype)

    def step(stream=None):
        f = vf.linear(x, W, b, act="gelu", want_z=True, stream=stream)
        g = vf.linear_grad(dy, x, W, act="gelu", z=f["z"], stream=stream)
        norm, out = vf.clip_grad_norm([g["dW"], g["db"]], 0.5, stream=stream)
        return [f["y"], f["z"], g["dx"], norm, *out]

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):  # calls in flight at once, each with a workspace of its own
        for s in streams:
            got.append(step(s))
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, c) for a, c in zip(o, want))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        o1 = step()
    with torch.cuda.graph(g2):
        o2 = step()
    for t in o1 + o2:
        t.fill_(7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):  # two captured steps replayed at once
        g1.replay()
        with torch.cuda.stream(side):
            g2.replay()
    torch.cuda.synchronize()
    for o in (o1, o2):
        assert all(torch.equal(a, c) for a, c in zip(o, want))
    x.copy_(randn(gen, M, K, dtype))  # a replay reads its inputs anew
    g1.replay()
    fresh = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(o1, fresh))
    vf.ops_check()


def test_gradient_against_differences():
    """d/dt of sum(dy * act(layer at p + t d)) at t = 0, by a central difference in 64 bits, for every input."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    M, N, K = 37, 45, 51
    for act in ("none", "relu", "gelu", "silu"):
        p = {"x": randn(gen, M, K, torch.float32), "W": randn(gen, N, K, torch.float32, 0.2),
             "b": randn(gen, 1, N, torch.float32)[0], "r": randn(gen, M, N, torch.float32)}
        dy = randn(gen, M, N, torch.float32)
        z = vf.linear(p["x"], p["W"], p["b"], residual=p["r"], act=act, want_z=True)["z"]
        if act == "relu":  # keep clear of the kink: a step of h |d| moves z by less than this
            dy = torch.where(z.abs() > 1e-3, dy, torch.zeros_like(dy))
        g = vf.linear_grad(dy, p["x"], p["W"], act=act, z=z, need=("dx", "dW", "db", "dr"))
        h = 1e-6

        def loss(q):
            zz = q["x"] @ q["W"].t() + q["b"] + q["r"]
            return float((dy.double() * act64(zz, act)).sum())

        for k, name in (("x", "dx"), ("W", "dW"), ("b", "db"), ("r", "dr")):
            d = torch.randn(p[k].shape, generator=gen, device="cuda", dtype=torch.float64)
            up, dn = ({j: v.double() + (s * h * d if j == k else 0) for j, v in p.items()} for s in (1, -1))
            num = (loss(up) - loss(dn)) / (2 * h)
            ana = float((g[name].double() * d).sum())
            # differences: h^2 times a third derivative of order one, and 2^-52 of a loss of order 1e3 over h;
            # the gradient: fp32 sums of at most 51 terms
            size = float((g[name].double().abs() * d.abs()).sum())
            assert abs(num - ana) <= 1e-6 * size + 1e-5, (act, name)


# ------------------------------------------------------------------------------------------------------ clipping
def clip_check(grads, max_norm, scale, out, in_place=False):
    want = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads)) * scale
    f = scale * (max_norm / want if want > max_norm else 1.0)
    copies = [g.clone() for g in grads]
    norm, got = vf.clip_grad_norm(grads, max_norm, scale=scale, out=None if in_place else out)
    # fp32 sums of at most 32 squares: 33 u relative of the square, half of it of the norm; then the norm's rounding
    assert abs(float(norm) - want) <= (17 + 1) * U * want
    for o, g in zip(got, copies):
        w = g.double() * f
        # the factor is off by 17 u and its own rounding, the product rounds twice
        tol = 20 * U * w.abs() + half_step(g.dtype) * w.abs() * (1 + 20 * U) + sub_step(g.dtype)
        tol = tol + (2.0 ** -134 if g.dtype == torch.bfloat16 else 2.0 ** -150)  # half a subnormal step
        assert worst(o, w, tol) <= 1.0
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(grads, copies))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [[1], [0], [5, 0, 3], [4096], [4095, 8193, 1, 16384, 12345], [3] * 230, [1_000_003, 77]])
def test_clip_matches_formula(dtype, sizes):
    gen = torch.Generator(device="cuda").manual_seed(len(sizes))
    for max_norm, scale in ((0.3, 1.0), (1e6, 1.0), (0.3, 0.125), (float("inf"), 0.5), (0.0, 1.0)):
        for off in (0, 1, 5):  # views that start off a 16-byte boundary
            grads = [randn(gen, 1, n + off, dtype)[0][off:] for n in sizes]
            out = [torch.empty(n + 3, device="cuda", dtype=dtype)[3 if off == 1 else off if off else 0:][:n] for n in sizes]
            out = [o if o.numel() == g.numel() else torch.empty_like(g) for o, g in zip(out, grads)]
            clip_check(grads, max_norm, scale, out)
        clip_check([randn(gen, 1, n, dtype)[0] for n in sizes], max_norm, scale, None, in_place=True)


def test_clip_of_many_large_gradients():
    """More gradients than one launch takes, each launch with a full grid: the partial sums are added apart."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    flat = torch.randn(250 * 60000, generator=gen, device="cuda")
    grads = list(torch.split(flat, 60000))
    clip_check(grads, 10.0, 1.0, [torch.empty_like(g) for g in grads])


def test_clip_of_mixed_types_and_shapes():
    gen = torch.Generator(device="cuda").manual_seed(2)
    grads = [torch.randn(s, generator=gen, device="cuda").to(t)
             for s, t in (((300, 70), torch.float32), ((70,), torch.bfloat16), ((3, 5, 7), torch.float16), ((), torch.float32))]
    clip_check(grads, 1.0, 1.0, [torch.empty_like(g) for g in grads])
    norm, out = vf.clip_grad_norm([], 1.0)
    assert float(norm) == 0.0 and out == []


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -90, 2.0 ** -130])
def test_clip_has_no_overflow_or_underflow(dtype, size):
    gen = torch.Generator(device="cuda").manual_seed(2)
    g = (torch.randn(20000, generator=gen, device="cuda") * size).to(dtype)
    g[7:300] = 0
    clip_check([g], 0.5 * size * math.sqrt(20000.0), 1.0, [torch.empty_like(g)])


def test_clip_reports_a_norm_that_is_not_finite_and_clips_nothing():
    for bad in (float("inf"), float("nan")):
        g = [torch.ones(5000, device="cuda"), torch.full((100,), 2.0, device="cuda")]
        g[0][4321] = bad
        norm, out = vf.clip_grad_norm(g, 0.1, scale=0.5, out=[torch.empty_like(t) for t in g])
        assert not math.isfinite(float(norm))
        assert torch.equal(out[1], torch.full((100,), 1.0, device="cuda"))
        assert torch.equal(out[0].nan_to_num(9, 9), (g[0] * 0.5).nan_to_num(9, 9))


def test_clip_of_the_slope_gradients():
    """The intended neighbour: vf_alpha_grad's gradient, one block per ReLU, limited in place."""
    w = synth.workload(2, B=4)
    net = vf.Net(w.net)
    centres, C = torch.from_numpy(w.centres).cuda(), torch.from_numpy(w.C).cuda()
    B, R = 4, C.shape[1]
    alpha = torch.full((net.alpha_size(B, R),), 0.5, device="cuda")
    _, grad = net.alpha_grad(centres, w.eps, C, alpha)
    blocks = list(torch.split(grad, [B * R * net.sizes[v] for v in net.relu_ids]))
    want = float(grad.double().norm())
    assert want > 0
    keep = grad.clone()
    norm, _ = vf.clip_grad_norm(blocks, want / 3)
    assert abs(float(norm) - want) <= 18 * U * want
    ok = (grad.double() - keep.double() / 3).abs() <= 21 * U * keep.double().abs() / 3 + 2.0 ** -150
    assert ok.all()


def test_training_steps_then_bounds():
    """The operators as they are used together: a two-block residual network takes gradient steps with clipping, every
    gradient of the last step agrees with differences of the loss in 64 bits, and the trained network's bounds (vf.Net)
    enclose the values that vf.linear gives at the centres."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    B, D, H, O = 96, 24, 40, 4
    dims = [(H, D), (H, H), (O, H)]
    P = [(randn(gen, n, k, torch.float32, k ** -0.5), randn(gen, 1, n, torch.float32, 0.1)[0]) for n, k in dims]
    x, target = randn(gen, B, D, torch.float32), randn(gen, B, O, torch.float32)

    def forward(P):
        h1 = vf.linear(x, *P[0], act="relu", want_z=True)
        h2 = vf.linear(h1["y"], *P[1], residual=h1["y"], act="relu", want_z=True)  # relu(W h + b + h)
        return h1, h2, vf.linear(h2["y"], *P[2])

    def loss64(P):
        Q = [(W.double(), b.double()) for W, b in P]
        h1 = torch.clamp(x.double() @ Q[0][0].t() + Q[0][1], min=0)
        h2 = torch.clamp(h1 @ Q[1][0].t() + Q[1][1] + h1, min=0)
        e = h2 @ Q[2][0].t() + Q[2][1] - target.double()
        return float(0.5 * (e * e).sum())

    for step in range(4):
        h1, h2, y = forward(P)
        g3 = vf.linear_grad(y["y"] - target, h2["y"], P[2][0])
        g2 = vf.linear_grad(g3["dx"], h1["y"], P[1][0], act="relu", z=h2["z"], need=("dx", "dW", "db", "dr"))
        g1 = vf.linear_grad(g2["dx"] + g2["dr"], x, P[0][0], act="relu", z=h1["z"], need=("dW", "db"))
        raw = [g1["dW"], g1["db"], g2["dW"], g2["db"], g3["dW"], g3["db"]]
        norm, clipped = vf.clip_grad_norm(raw, 1.0, out=[torch.empty_like(t) for t in raw])
        if step == 3:
            assert float(norm) > 1.0
            total = math.sqrt(sum(float((c.double() ** 2).sum()) for c in clipped))
            assert abs(total - 1.0) <= 1e-5
            for i in range(3):
                for j, t in enumerate(P[i]):
                    d = torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)
                    h = 1e-7
                    up = [tuple(v.double() + (h * d if (a, c) == (i, j) else 0) for c, v in enumerate(p)) for a, p in enumerate(P)]
                    dn = [tuple(v.double() - (h * d if (a, c) == (i, j) else 0) for c, v in enumerate(p)) for a, p in enumerate(P)]
                    num = (loss64(up) - loss64(dn)) / (2 * h)
                    g = raw[2 * i + j].double()
                    # fp32 gradients through three layers, and ReLUs within h of their kink (each moves the
                    # difference by at most h of its own term)
                    assert abs(num - float((g * d).sum())) <= 1e-4 * float((g.abs() * d.abs()).sum()) + 1e-3
        P = [(W - 0.05 * clipped[2 * i], b - 0.05 * clipped[2 * i + 1]) for i, (W, b) in enumerate(P)]
    nd = synth.Node
    c = [(W.cpu().numpy(), b.cpu().numpy()) for W, b in P]
    nodes = [nd("input", shape=(D,)), nd("dense", src=0, W=c[0][0], b=c[0][1]), nd("relu", src=1),
             nd("dense", src=2, W=c[1][0], b=c[1][1]), nd("add", src=3, src2=2), nd("relu", src=4),
             nd("dense", src=5, W=c[2][0], b=c[2][1])]
    net = vf.Net(nodes)
    C = torch.eye(O, device="cuda").reshape(1, O, O).contiguous()
    out = net.verify(x, 0.01, C, both_sides=True)
    y = forward(P)[2]["y"]
    slack = 1e-4 * (y.abs() + 1)  # the parity tolerance of the bounds
    assert (out["lb"] <= y + slack).all() and (out["ub"] >= y - slack).all()
    assert np.isfinite(out["lb"].cpu().numpy()).all()
    vf.ops_check()
