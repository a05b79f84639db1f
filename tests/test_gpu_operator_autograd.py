"""What vf.linear and vf.clip_grad_norm write in place, as autograd sees it, on a B200."""
import pytest
import torch

vf = pytest.importorskip("linear_bound_propagation_b200.vf")
pytestmark = pytest.mark.gpu


def test_writes_in_place_count_as_such():
    """A graph that saved a tensor refuses its backward pass after the tensor was overwritten."""
    x, W = torch.ones(4, 8, device="cuda"), torch.ones(6, 8, device="cuda")
    w = torch.ones(4, 6, device="cuda", requires_grad=True)
    r, g = torch.ones(4, 6, device="cuda"), torch.ones(4, 6, device="cuda")
    for t, write in ((r, lambda: vf.linear(x, W, residual=r, out=r)), (g, lambda: vf.clip_grad_norm([g], 1.0)),
                     (g, lambda: vf.clip_grad_norm([g, r], 1.0, stream=torch.cuda.Stream())),
                     (r, lambda: vf.clip_grad_norm([g], 1.0, out=[r]))):
        loss = (w * t).sum()
        before = t._version
        write()
        assert t._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        torch.cuda.synchronize()


def test_what_is_only_read_counts_as_unchanged():
    x, W, r = torch.ones(4, 8, device="cuda"), torch.ones(6, 8, device="cuda"), torch.ones(4, 6, device="cuda")
    f = vf.linear(x, W, residual=r, want_z=True)
    vf.linear_grad(f["y"], x, W)
    vf.clip_grad_norm([r], 1.0, out=[torch.empty_like(r)])
    assert x._version == W._version == r._version == f["y"]._version == 0


def test_inference_tensors_are_taken():
    with torch.inference_mode():
        x, W, r = torch.ones(4, 8, device="cuda"), torch.ones(6, 8, device="cuda"), torch.ones(4, 6, device="cuda")
        assert (vf.linear(x, W, residual=r, out=r)["y"] == 9).all()
        assert float(vf.clip_grad_norm([r], 1.0)[0]) > 1


def test_a_function_around_both_passes():
    """linear and linear_grad as a torch.autograd.Function: gradients of a two-layer network against those of torch's own operations in 64 bits."""

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, W, b):
            f = vf.linear(x, W, b, act="gelu", want_z=True)
            ctx.save_for_backward(x, W, f["z"])
            return f["y"]

        @staticmethod
        def backward(ctx, dy):
            x, W, z = ctx.saved_tensors
            g = vf.linear_grad(dy.contiguous(), x, W, act="gelu", z=z)
            return g["dx"], g["dW"], g["db"]

    gen = torch.Generator(device="cuda").manual_seed(1)
    p = [torch.randn(s, generator=gen, device="cuda").mul_(0.3).requires_grad_() for s in ((30, 20), (40, 20), (40,), (10, 40), (10,))]
    Layer.apply(Layer.apply(*p[:3]), *p[3:]).square().sum().backward()
    q = [t.detach().double().requires_grad_() for t in p]
    gelu = lambda z: z * 0.5 * torch.erfc(z * -0.5 ** 0.5)  # noqa: E731
    gelu(gelu(q[0] @ q[1].t() + q[2]) @ q[3].t() + q[4]).square().sum().backward()
    for a, c in zip(p, q):
        # sums of at most 40 fp32 terms per layer, two layers forward and back
        assert float((a.grad.double() - c.grad).norm() / c.grad.norm()) <= 4 * 40 * 2.0 ** -24
    vf.ops_check()
