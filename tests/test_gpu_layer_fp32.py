"""fp32 layers (vf.linear, vf.linear_grad) on a B200: the three bf16 pieces of an operand, their six products and the long
sums, against 64 bits. u = 2^-24.

A value's pieces are rounded to nearest: h holds 8 significand bits, m is at most 2^-8 and l at most 2^-17 of the
leading power of two. Together they hold all 24 bits. The products left out (m l, l m, l l) are at most 2^-24 (1 + 2^-10) of
the product of the leading powers.

* One product per output: left out u, and one rounding when the h h product and the small ones are added, u; the
  accumulator of the small products is below 2^-7 and truncates by 2^-23 of that for each of five instructions.
* Sums: an accumulator of h h products takes 16 instructions (256 steps), each of which truncates by at most 2^-23 of the
  sum, and is then added to the others, rounding to nearest; terms of one sign grow the sums evenly, so half of either counts:
  8 2^-23 + ceil(T / 256) 2^-25. The small products' accumulator takes up to 640 instructions at 2^-7 of the sum: 640 2^-31. Left
  out: u. The output and the final addition: 2 u. In the 2-norm, relative."""
import pytest
import torch

vf = pytest.importorskip("linear_bound_propagation_b200.vf")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def full(gen, rows, cols, pad=0):
    """Values of both signs whose 24 significand bits are all in use, over 16 powers of two."""
    s = torch.randint(2 ** 23, 2 ** 24, (rows, cols + pad), generator=gen, device="cuda").double()
    s = (s * 2 - 2 ** 24 + 1).abs() + 2 ** 22  # odd and even alike, leading powers 2^22 to 2^24
    s = torch.where(s >= 2 ** 24, s / 2, s).floor()
    sign = torch.randint(0, 2, s.shape, generator=gen, device="cuda") * 2 - 1
    e = torch.randint(-8, 8, s.shape, generator=gen, device="cuda").double()
    return (s * sign * torch.exp2(e - 23)).float()[:, :cols]


def one_hot(gen, rows, cols, pad=0):
    """Rows with a single power of two, spread over the columns; returns the matrix, the places and the values."""
    at = torch.randperm(cols, generator=gen, device="cuda")
    at = at.repeat(-(-rows // cols))[:rows]
    v = torch.exp2(torch.randint(-6, 7, (rows,), generator=gen, device="cuda").float())
    m = torch.zeros(rows, cols + pad, device="cuda")[:, :cols]
    m[torch.arange(rows, device="cuda"), at] = v
    return m, at, v


SIZES = [(40, 300, 1024), (9, 200, 300), (300, 520, 2049), (700, 1100, 4100), (2100, 2200, 515), (16, 512, 8200), (130, 70, 30000)]


@pytest.mark.parametrize("M,N,T", SIZES)
@pytest.mark.parametrize("pad", [0, 1])
def test_all_pieces_of_every_step_arrive_once(M, N, T, pad):
    """One operand holds all its 24 bits, the other one power of two per output: the output is the shifted value, exactly. So for
    each operand, forward, dx and dW."""
    gen = torch.Generator(device="cuda").manual_seed(M + T)
    x = full(gen, M, T, pad)
    W, at, v = one_hot(gen, N, T, pad)
    want = x[:, at] * v
    assert torch.equal(vf.linear(x, W)["y"], want)
    assert torch.equal(vf.linear(W, x)["y"], want.t())
    if T <= 8200:
        Wt = torch.zeros(T, N + pad, device="cuda")[:, :N].copy_(W.t())
        assert torch.equal(vf.linear_grad(x, torch.zeros(M, N, device="cuda"), Wt, need=("dx",))["dx"], want)
        xt = torch.zeros(T, M + pad, device="cuda")[:, :M].copy_(x.t())
        assert torch.equal(vf.linear_grad(W, torch.zeros(N, M, device="cuda"), xt, need=("dx",))["dx"], want.t())
        e = torch.empty(N, M, device="cuda")
        assert torch.equal(vf.linear_grad(Wt, xt, e, need=("dW",))["dW"], want.t())
        assert torch.equal(vf.linear_grad(xt, Wt, e.t().contiguous(), need=("dW",))["dW"], want)
    vf.ops_check()


@pytest.mark.parametrize("M,N,T", [(40, 300, 1024), (700, 1100, 520), (130, 70, 3000)])
@pytest.mark.parametrize("pad", [0, 1])
def test_one_product_is_as_exact_as_fp32(M, N, T, pad):
    """One product of two values with all 24 bits per output. The worst operands of pieces cut by truncation are among them: for
    x = W = 1 + 2^-7 - 2^-23 those leave out 4.7e-7 of the product."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, (W, at, _) = full(gen, M, T, pad), one_hot(gen, N, T, pad)
    x[: M // 2] = 1 + 2.0 ** -7 - 2.0 ** -23
    w = full(gen, 1, N)[0]
    w[: N // 2] = 1 + 2.0 ** -7 - 2.0 ** -23
    W[torch.arange(N, device="cuda"), at] = w
    want = x[:, at].double() * w.double()
    tol = 2 * U * (1 + 2.0 ** -9) + 5 * 2.0 ** -30

    def off(got, want):
        return float(((got.double() - want) / want).abs().max())

    assert off(vf.linear(x, W)["y"], want) <= tol
    Wt = torch.zeros(T, N + pad, device="cuda")[:, :N].copy_(W.t())
    xt = torch.zeros(T, M + pad, device="cuda")[:, :M].copy_(x.t())
    assert off(vf.linear_grad(x, torch.zeros(M, N, device="cuda"), Wt, need=("dx",))["dx"], want) <= tol
    assert off(vf.linear_grad(Wt, xt, torch.empty(N, M, device="cuda"), need=("dW",))["dW"], want.t()) <= tol
    vf.ops_check()


def norm_tol(T):
    return 8 * 2.0 ** -23 + -(-T // 256) * 2.0 ** -25 + 640 * 2.0 ** -31 + 3 * U


def norm_error(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("signed", [True, False])
@pytest.mark.parametrize("T", [1024, 2049, 4096, 8200])
@pytest.mark.parametrize("M,N,pad", [(16, 512, 0), (16, 512, 1), (300, 520, 0), (300, 520, 1), (2100, 1100, 0)])
def test_error_of_long_sums(M, N, T, pad, signed):
    gen = torch.Generator(device="cuda").manual_seed(T + N)

    def mat(rows, cols):
        t = torch.randn(rows, cols + pad, generator=gen, device="cuda")
        return (t if signed else t.abs())[:, :cols]

    x, W = mat(M, T), mat(N, T)
    want = x.double() @ W.double().t()
    assert norm_error(vf.linear(x, W)["y"], want) <= norm_tol(T)
    Wt, xt = mat(T, N), mat(T, M)
    assert norm_error(vf.linear_grad(x, torch.zeros(M, N, device="cuda"), Wt, need=("dx",))["dx"], x.double() @ Wt.double()) <= norm_tol(T)
    assert norm_error(vf.linear_grad(xt, Wt, torch.empty(M, N, device="cuda"), need=("dW",))["dW"], xt.double().t() @ Wt.double()) <= norm_tol(T)
    vf.ops_check()


def test_error_does_not_jump_where_the_kernel_changes():
    """Rows from one to 33 through the few-row kernels and the tensor cores, forward and backward, at one bound."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    T, N = 1024, 512
    W = torch.randn(N, T, generator=gen, device="cuda")
    Wb = torch.randn(T, N, generator=gen, device="cuda")
    for M in (1, 2, 7, 8, 9, 15, 16, 17, 33):
        x = torch.randn(M, T, generator=gen, device="cuda")
        assert norm_error(vf.linear(x, W)["y"], x.double() @ W.double().t()) <= norm_tol(T)
        dx = vf.linear_grad(x, torch.zeros(M, N, device="cuda"), Wb, need=("dx",))["dx"]
        assert norm_error(dx, x.double() @ Wb.double()) <= norm_tol(T)
    vf.ops_check()


@pytest.mark.parametrize("M", [4, 40, 300])
@pytest.mark.parametrize("pad", [0, 1])
def test_values_next_to_the_largest(M, pad):
    """Values that bf16 would round to infinity are cut instead: their products with ordinary and small values are finite and exact
    to a rounding."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    N, T = 264, 200
    big = torch.tensor([0x7f7f7fff, 0x7f7f8000, 0x7f7fffff, 0x7f7fff80, 0x7f000001], device="cuda", dtype=torch.int32).view(torch.float32)
    x = torch.zeros(M, T + pad, device="cuda")[:, :T]
    i = torch.arange(M, device="cuda")
    x[i, i % T] = big[i % 5] * (1 - 2 * (i % 2)).float()
    W = full(gen, N, T, pad) * 2.0 ** -40
    want = x.double() @ W.double().t()
    got = vf.linear(x, W)["y"]
    assert torch.isfinite(got).all()
    assert float(((got.double() - want) / want).abs().max()) <= 2 * U * (1 + 2.0 ** -6) + 5 * 2.0 ** -30
    y = vf.linear(W, x)["y"]
    assert float(((y.double() - want.t()) / want.t()).abs().max()) <= 2 * U * (1 + 2.0 ** -6) + 5 * 2.0 ** -30
    vf.ops_check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [4, 8, 9, 40, 300])
@pytest.mark.parametrize("pad", [0, 1])
def test_infinities_are_those_of_fp32(M, pad, dtype):
    """An infinity against finite values that are not zero gives the infinity that fp32 arithmetic gives, whatever the number of rows:
    so a relu of minus infinity is 0. NaN stays NaN."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    N, T = 264, 200
    x, W = (torch.zeros(n, T + pad, device="cuda", dtype=dtype)[:, :T].copy_(full(gen, n, T)) for n in (M, N))
    clean = vf.linear(x, W)["y"]
    for r, (k, bad) in enumerate([(3, float("inf")), (5, float("-inf")), (T - 1, float("nan"))]):
        x[r, k] = bad
    want = x.double() @ W.double().t()  # rows 0 to 2: +-inf by the sign of W, NaN
    got = vf.linear(x, W, act="relu", want_z=True)
    assert torch.equal(got["z"][:2], want[:2].to(dtype)) and got["z"][2].isnan().all()
    assert torch.equal(got["y"][:2], want[:2].to(dtype).clamp(min=0)) and got["y"][2].isnan().all()
    assert torch.equal(got["z"][3:], clean[3:])
    got = vf.linear(W, x)["y"]
    assert torch.equal(got[:, :2], want[:2].to(dtype).t()) and got[:, 2].isnan().all()
    Wt = torch.zeros(T, N + pad, device="cuda", dtype=dtype)[:, :N].copy_(W.t())
    dx = vf.linear_grad(x, torch.zeros(M, N, device="cuda", dtype=dtype), Wt, need=("dx",))["dx"]
    assert torch.equal(dx[:2], want[:2].to(dtype)) and dx[2].isnan().all()
    vf.ops_check()


@pytest.mark.parametrize("M", [4, 40, 700])
@pytest.mark.parametrize("pad", [0, 1])
def test_small_values_keep_their_bits_down_to_2_to_the_minus_110(M, pad):
    """The lowest of 24 bits of a value of 2^-110 is 2^-133, the lowest that bf16 holds; below that what lies under 2^-133 is cut off or
    rounded there, and the few-row kernels keep all."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    N, T = 264, 520
    for e in (-80, -110, -118, -126):
        x = torch.randint(2 ** 23, 2 ** 24, (M, T + pad), generator=gen, device="cuda").float()[:, :T] * 2.0 ** (e - 23)
        W, at, v = one_hot(gen, N, T, pad)
        W, v = W * 2.0 ** 60, v * 2.0 ** 60
        y, want = vf.linear(x, W)["y"], x[:, at].double() * v.double()
        if e >= -110 or M == 4:
            assert torch.equal(y.double(), want)
        else:
            assert float(((y.double() - want).abs() / v.double()).max()) <= 2.0 ** -134 + 2.0 ** (e - 24)
    vf.ops_check()
