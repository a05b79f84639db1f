"""float16 gradients of any size through gelu and silu (vf.linear_grad) on a B200, against the formulas in 64 bits.

g = dy act'(z) enters the products in 16 bits: half a step of |g|, and, since it is multiplied by the power of two that brings
the largest |dy| to 2^13 or more before it is rounded, half a subnormal step of float16 (2^-25) at 2^13: 2^-38 of the largest |dy|.
Everything else as in test_gpu_operators.py."""
import pytest
import torch

from tests.test_gpu_operators import acc_tol, half_step, randn, slope64, sub_step, worst

vf = pytest.importorskip("linear_bound_propagation_b200.vf")
pytestmark = pytest.mark.gpu
F16 = torch.float16


def check(M, N, K, act, size, std_x, std_w, pad=0, need=("dx", "dW", "db", "dr"), z_at=0.0, off=0):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    x, W = randn(gen, M, K, F16, std_x, pad, off), randn(gen, N, K, F16, std_w, pad, off)
    dy, z = (randn(gen, M, N, F16, 1.0, pad, off) * size).clamp(-65504, 65504), randn(gen, M, N, F16, 1.5, pad, off) + z_at
    if pad:
        dy, z = (torch.cat([t, t[:, :pad]], 1)[:, :N] for t in (dy, z))
    got = vf.linear_grad(dy, x, W, act=act, z=z, need=need)
    vf.ops_check()
    hs, ss = half_step(F16), sub_step(F16)
    g = dy.double() * slope64(z.double(), act)
    eg = 2.0 ** -20 * dy.double().abs()
    ein = eg + hs * g.abs() + 2.0 ** -38 * dy.double().abs().max()
    want = {"dx": g @ W.double(), "dW": g.t() @ x.double(), "db": g.sum(0), "dr": g}
    tol = {"dx": acc_tol(N) * (g.abs() @ W.double().abs()) + ein @ W.double().abs(),
           "dW": acc_tol(M) * (g.abs().t() @ x.double().abs()) + ein.t() @ x.double().abs(),
           "db": acc_tol(M) * g.abs().sum(0) + eg.sum(0), "dr": eg}
    for k in need:
        finite = want[k].abs() < 65000  # what lies beyond float16's largest may round to infinity
        t = tol[k] + hs * (want[k].abs() + tol[k]) + ss
        assert worst(got[k][finite], want[k][finite], t[finite]) <= 1.0, k
        assert finite.float().mean() > 0.5 or k in ("db", "dr")


SHAPES = [(9, 130, 72), (40, 4096, 64), (200, 256, 192), (333, 517, 101), (5557, 64, 64), (1025, 1025, 129), (4096, 1016, 256)]


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_small_gradients_keep_their_bits(act, M, N, K):
    """dy of 1e-6 and 1e-5 beside inputs and weights of 300: g lies among float16's subnormals, the outputs do not."""
    check(M, N, K, act, 1e-6, 300.0, 300.0)
    check(M, N, K, act, 1e-5, 300.0, 300.0, pad=3, off=1)
    check(M, N, K, act, 1e-6, 300.0, 300.0, need=("dx",))
    check(M, N, K, act, 1e-6, 300.0, 300.0, need=("dW", "dr"))


@pytest.mark.parametrize("act,z_at", [("gelu", 1.4), ("silu", 2.4)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gradients_near_the_largest_stay_finite(act, z_at, M, N, K):
    """Slopes above one carry g beyond 65504; its products with small weights and inputs are ordinary."""
    check(M, N, K, act, 50000.0, 1e-3, 1e-3, z_at=z_at, need=("dx", "dW"))


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_all_slopes_small(act):
    """Every z far below zero: slopes of 1e-4 and less."""
    check(150, 264, 136, act, 1.0, 300.0, 300.0, z_at=-9.0 if act == "silu" else -4.5)


def test_the_largest_of_every_magnitude_gives_the_same_bits():
    """A power of two in dy is one in dx: no rounding depends on it as long as outputs stay normal."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, W, z = randn(gen, 300, 200, F16), randn(gen, 264, 200, F16, 8.0), randn(gen, 300, 264, F16, 1.5)
    dy = (torch.randint(1, 2048, (300, 264), generator=gen, device="cuda") * 2.0 ** -11).to(F16)  # 11 bits: exact at every scale
    want = vf.linear_grad(dy, x, W, act="gelu", z=z)
    for p in (-8, -3, 3, 5):
        got = vf.linear_grad(dy * 2.0 ** p, x, W, act="gelu", z=z)
        for k in ("dx", "dW"):
            normal = (want[k].abs() > 2.0 ** -5) & (want[k].abs() < 1000)
            assert normal.any() and torch.equal(got[k][normal], (want[k] * 2.0 ** p)[normal])


def test_zeros_and_what_is_not_finite():
    """An all-zero dy gives zeros; an infinite or NaN dy makes its own row of dx non-finite and leaves the other rows' bits."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, W, z, dy = randn(gen, 100, 72, F16), randn(gen, 136, 72, F16), randn(gen, 100, 136, F16), randn(gen, 100, 136, F16)
    got = vf.linear_grad(torch.zeros_like(dy), x, W, act="silu", z=z)
    assert not any(got[k].any() for k in ("dx", "dW", "db"))
    clean = vf.linear_grad(torch.cat([torch.zeros_like(dy[:1]), dy[1:]]), x, W, act="silu", z=z)["dx"]
    for bad in (float("inf"), float("-inf"), float("nan")):
        d = dy.clone()
        d[0] = 0
        d[0, 5] = bad
        dx = vf.linear_grad(d, x, W, act="silu", z=z)["dx"]
        assert not torch.isfinite(dx[0]).any() and torch.equal(dx[1:], clean[1:])
    vf.ops_check()


def test_captured_passes_keep_their_own_scale():
    """Two captured passes with gradients of very different size, replayed in turn and at once."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, W, z = randn(gen, 100, 72, F16, 100.0), randn(gen, 136, 72, F16, 100.0), randn(gen, 100, 136, F16)
    dys = [randn(gen, 100, 136, F16, s) for s in (1e-5, 1.0)]
    want = [vf.linear_grad(d, x, W, act="gelu", z=z) for d in dys]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in dys], []
    for g, d in zip(graphs, dys):
        with torch.cuda.graph(g):
            outs.append(vf.linear_grad(d, x, W, act="gelu", z=z))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(o[k], w[k]) for k in ("dx", "dW", "db"))
    vf.ops_check()
