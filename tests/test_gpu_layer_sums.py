"""Long reductions of the 16-bit layer products (vf.linear, vf.linear_grad) on a B200: the error's mean over many outputs,
which a rounding of the output leaves near zero and a sum that truncates does not.

A matrix instruction adds 16 products to its fp32 accumulator. It cuts each product two bits below the accumulator's last place, at
2^-25 of its leading power of two, and the new sum at 2^-23: less than 2^-21 + 2^-23 of the sum. (Measured, about a third of it: 64
instructions lower a sum of positive terms by 5.8e-6, which is half of 64 cuts of 1.8e-7.) Terms of one sign grow the sum
evenly, so the partial sums are half of the last on average. The accumulators are added to fp32 sums, rounding to nearest, every
2048 steps (128 instructions) at the latest:
  mean error <= 64 (2^-21 + 2^-23) (of each run, so of their sum) + T / 2048 additions of 2^-24 each, halved.
Without that, 2^18 rows gave 1.7e-3, seven half steps of float16.
The outputs' roundings are independent and even over (-half step, half step): six standard deviations of their mean."""
import math

import pytest
import torch

vf = pytest.importorskip("linear_bound_propagation_b200.vf")
pytestmark = pytest.mark.gpu


def mean_error(got, want):
    return float(((got.double() - want) / want).mean())


def mean_tol(T, dtype, outputs):
    return 64 * (2.0 ** -21 + 2.0 ** -23) + T / 2048 * 2.0 ** -25 + 6 * torch.finfo(dtype).eps / 2 / math.sqrt(3 * outputs)


def positive(gen, rows, cols, dtype, pad=0):
    """Values in (0, 1/4), every column with a scale of its own, so that the outputs lie anywhere between two steps."""
    t = torch.rand(rows, cols + pad, generator=gen, device="cuda") * (0.125 + 0.125 * torch.rand(cols + pad, generator=gen, device="cuda"))
    return t.to(dtype)[:, :cols]


def test_weight_gradients_over_many_rows():
    """2^18 rows: eight runs of the accumulators at least for each part of the reduction."""
    gen = torch.Generator(device="cuda").manual_seed(31)
    T, N, K = 1 << 18, 2048, 2048
    for dtype in (torch.float16, torch.bfloat16):
        dy, x = positive(gen, T, N, dtype), positive(gen, T, K, dtype)
        got = vf.linear_grad(dy, x, torch.empty(N, K, device="cuda", dtype=dtype), need=("dW",))["dW"]
        vf.ops_check()
        want = dy[:, :1024].double().t() @ x[:, :1024].double()
        assert abs(mean_error(got[:1024, :1024], want)) <= mean_tol(T, dtype, want.numel())


@pytest.mark.parametrize("M,N,pad", [(64, 2048, 0), (300, 1000, 0), (16, 2000, 0), (50, 300, 1), (16, 200, 3)])
def test_forward_over_many_columns(M, N, pad):
    """Aligned rows (fed by TMA, over a cluster or not) and rows that the kernel lays out itself."""
    gen = torch.Generator(device="cuda").manual_seed(32 + M)
    T = 60000
    x, W = positive(gen, T, M, torch.float16).t().contiguous(), positive(gen, T, N, torch.float16).t().contiguous()
    if pad:
        x, W = (torch.cat([t, t[:, :pad]], 1)[:, :T] for t in (x, W))
    got = vf.linear(x, W)["y"]
    vf.ops_check()
    want = x.double() @ W.double().t()
    assert abs(mean_error(got, want)) <= mean_tol(T, torch.float16, want.numel())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1024, 2047, 2048, 2049, 3000, 4097, 70000])
@pytest.mark.parametrize("pad", [0, 1])
def test_every_step_of_a_long_reduction_counts_once(dtype, T, pad):
    """Row n of W has a single 1, spread over the whole reduction: the output is x's element there, exactly, and in the backward
    pass the gradient of that element."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    for M, N in ((40, 3000), (700, 1100)):
        at = torch.randperm(T, generator=gen, device="cuda")[:N]
        if at.numel() < N:
            at = at.repeat(-(-N // T))[:N]
        x = torch.randn(M, T + pad, generator=gen, device="cuda").to(dtype)[:, :T]
        W = torch.zeros(N, T + pad, device="cuda", dtype=dtype)[:, :T]
        W[torch.arange(N, device="cuda"), at] = 1
        got = vf.linear(x, W, want_z=True)
        assert torch.equal(got["z"], x[:, at]) and torch.equal(got["y"], x[:, at])
        # the same product as dx of a layer with T outputs
        if T <= 4097:
            Wt = torch.zeros(T, N + pad, device="cuda", dtype=dtype)[:, :N].copy_(W.t())
            got = vf.linear_grad(x, torch.zeros(M, N, device="cuda", dtype=dtype), Wt, need=("dx",))
            assert torch.equal(got["dx"], x[:, at])
        # and as dW of one with T rows
        xt = torch.zeros(T, M + pad, device="cuda", dtype=dtype)[:, :M].copy_(x.t())
        dy = torch.zeros(T, N, device="cuda", dtype=dtype)
        dy[at, torch.arange(N, device="cuda")] = 1
        got = vf.linear_grad(dy, xt, torch.empty(N, M, device="cuda", dtype=dtype), need=("dW",))
        assert torch.equal(got["dW"], x[:, at].t())
    vf.ops_check()
