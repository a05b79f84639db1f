"""vf.clip_grad_norm on a B200 at the ends of fp32's range, and long lists of every type, against 64 bits."""
import math

import pytest
import torch

from tests.test_gpu_operators import U, clip_check, half_step, randn, worst

vf = pytest.importorskip("linear_bound_propagation_b200.vf")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("in_place", [False, True])
def test_a_norm_beyond_fp32_clips_nothing(dtype, in_place):
    """100 finite values of 1e38: their norm, 1e39, is reported as infinity, and what is reported is not finite clips nothing."""
    g = torch.full((100,), 1e38, device="cuda", dtype=dtype)
    keep = g.clone()
    for scale in (1.0, 0.5):
        g.copy_(keep)
        norm, (o,) = vf.clip_grad_norm([g], 1.0, scale=scale, out=None if in_place else [torch.empty_like(g)])
        if scale == 1.0:
            assert float(norm) == float("inf") and torch.equal(o, keep)
        else:
            assert float(norm) == float("inf") and torch.equal(o, keep * 0.5)
    # the same gradients under a scale that brings the norm back into range are clipped
    g.copy_(keep)
    norm, (o,) = vf.clip_grad_norm([g], 1.0, scale=2.0 ** -10, out=None if in_place else [torch.empty_like(g)])
    want = float(keep[0].double()) * 10 * 2.0 ** -10
    assert abs(float(norm) - want) <= 18 * U * want
    w = torch.full((100,), 0.1, device="cuda", dtype=torch.float64)
    assert worst(o, w, 21 * U * w + half_step(dtype) * w * (1 + 21 * U)) <= 1.0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [5, 3000, 300_001])
def test_a_factor_below_the_normal_numbers_keeps_its_bits(dtype, n):
    """Values of 1e35 and a largest norm of 1, 1e-4 and 1e-6: the factor is a subnormal number or less, the outputs are not."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    g = (torch.randn(n, generator=gen, device="cuda") * 1e35).to(dtype)
    g[0] = 3e38
    want = float(g.double().norm())
    for max_norm in (1.0, 1e-4, 1e-6):
        out = torch.empty_like(g)
        norm, _ = vf.clip_grad_norm([g], max_norm, out=[out])
        assert abs(float(norm) - want) <= 18 * U * want
        w = g.double() * (max_norm / want)
        # the factor and the product as elsewhere, another rounding by the second factor where that is subnormal
        tol = 21 * U * w.abs() + half_step(dtype) * w.abs() * (1 + 21 * U) + (2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149)
        assert worst(out, w, tol) <= 1.0
    out = torch.empty_like(g)
    assert not vf.clip_grad_norm([g], 0.0, out=[out])[1][0].any()


def test_a_scale_below_the_normal_numbers():
    g = torch.randn(1000, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * 1e30
    scale = float(torch.tensor(1e-40))
    norm, (o,) = vf.clip_grad_norm([g], float("inf"), scale=scale, out=[torch.empty_like(g)])
    w = g.double() * scale
    assert worst(o, w, 3 * U * w.abs() + 2.0 ** -149) <= 1.0
    want = float(g.double().norm()) * scale
    assert abs(float(norm) - want) <= 18 * U * want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("in_place", [False, True])
def test_long_lists_of_every_type(dtype, in_place):
    """More than 64 MiB and more than 100 tensors: odd lengths, starts on and off 16-byte boundaries, short ones among them."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    total = (80 << 20) // torch.finfo(dtype).bits * 8
    sizes = [(7 * i * i + 13 * i) % 5000 + 1 for i in range(120)]
    sizes[5], sizes[60] = total // 2, total // 2 + 12345
    grads = [randn(gen, 1, n + i % 3, dtype, 0.02)[0][i % 3:] for i, n in enumerate(sizes)]
    out = [torch.empty(n + i % 2, device="cuda", dtype=dtype)[i % 2:] for i, n in enumerate(sizes)]
    for max_norm in (0.7, 1e6):
        clip_check([g.clone() for g in grads] if in_place else grads, max_norm, 0.5, None if in_place else out, in_place)


def test_long_list_of_mixed_types():
    gen = torch.Generator(device="cuda").manual_seed(4)
    types = [torch.float32, torch.bfloat16, torch.float16]
    grads = [randn(gen, 1, 150_001 + i, types[i % 3], 0.02)[0] for i in range(230)]
    assert sum(g.numel() * g.element_size() for g in grads) > 64 << 20
    clip_check(grads, 1.0, 1.0, [torch.empty_like(g) for g in grads])
