"""Calls on a stream that is given: memory of temporaries, on a B200."""
import pytest
import torch

from linear_bound_propagation_b200 import synth

vf = pytest.importorskip("linear_bound_propagation_b200.vf")
pytestmark = pytest.mark.gpu


def busy_stream():
    """A stream that has waited for the current one and is held up for a while."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    return s


def overwrite(like, count=4):
    """What the allocator hands out next for this size, overwritten."""
    return [torch.full_like(t, float("nan")) for t in like for _ in range(count)]


@pytest.mark.parametrize("M", [4, 900])
def test_temporaries_outlive_the_call_on_another_stream(M):
    """Arguments dropped right after a call on a stream that has not begun: their memory is not handed out before it has."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    N, K = 520, 264
    x, W, b, r, dy, z = (torch.randn(s, generator=gen, device="cuda") for s in ((M, K), (N, K), (N,), (M, N), (M, N), (M, N)))
    want = vf.linear(x * 2, W * 2, b * 2, residual=r * 2, act="gelu")["y"]
    wg = vf.linear_grad(dy * 2, x * 2, W * 2, act="gelu", z=z * 2)
    wn, wc = vf.clip_grad_norm([x * 2, W * 2], 1.0)
    for call in ("linear", "grad", "clip"):
        s = busy_stream()
        t = [v * 2 for v in (x, W, b, r, dy, z)]
        s.wait_stream(torch.cuda.current_stream())
        if call == "linear":
            got = vf.linear(t[0], t[1], t[2], residual=t[3], act="gelu", stream=s)["y"]
        elif call == "grad":
            got = vf.linear_grad(t[4], t[0], t[1], act="gelu", z=t[5], stream=s)
        else:
            norm, _ = vf.clip_grad_norm(t[:2], 1.0, out=[torch.empty_like(v) for v in t[:2]], stream=s)
        assert not s.query()
        del t
        junk = overwrite((x, W, b, r, dy, z))
        torch.cuda.synchronize()
        if call == "linear":
            assert torch.equal(got, want)
        elif call == "grad":
            assert all(torch.equal(got[k], wg[k]) for k in ("dx", "dW", "db"))
        else:
            assert torch.equal(norm, wn)
        del junk


def test_temporaries_of_the_bounds_calls_outlive_them():
    """The same for calls of a network's handle and for concretisation."""
    w = synth.workload(2, B=8)
    net = vf.Net(w.net)
    centres, C = torch.from_numpy(w.centres).cuda(), torch.from_numpy(w.C).cuda()
    alpha = torch.full((net.alpha_size(8, C.shape[1]),), 0.5, device="cuda")
    lb_all, ub_all = net.ibp(centres, w.eps)
    last = len(net.sizes) - 1
    lam = C.expand(8, -1, -1).contiguous()
    li, cst = net.crown_backward(last, lam, lb_all, ub_all, 8)
    lc = vf.concretize(li, cst, centres, w.eps)
    vw, vc, vg = net.verify(centres, w.eps, C, no_host_sync=True), net.alpha_crown(centres, w.eps, C, iters=2), net.alpha_grad(centres, w.eps, C, alpha)
    torch.cuda.synchronize()
    for call in ("ibp", "backward", "concretize", "verify", "alpha", "grad"):
        s = busy_stream()
        c, c2, a, lo, hi, l2, i2, k2 = (v * 1 for v in (centres, C, alpha, lb_all, ub_all, lam, li, cst))
        s.wait_stream(torch.cuda.current_stream())
        if call == "ibp":
            got, want = net.ibp(c, w.eps, stream=s), (lb_all, ub_all)
        elif call == "backward":
            got, want = net.crown_backward(last, l2, lo, hi, 8, stream=s), (li, cst)
        elif call == "concretize":
            got, want = (vf.concretize(i2, k2, c, w.eps, stream=s),), (lc,)
        elif call == "verify":
            o = net.verify(c, w.eps, c2, no_host_sync=True, stream=s)
            got, want = (o["lb"], o["lb_ibp"]), (vw["lb"], vw["lb_ibp"])
        elif call == "alpha":
            got, want = (net.alpha_crown(c, w.eps, c2, iters=2, stream=s)["lb"],), (vc["lb"],)
        else:
            got, want = net.alpha_grad(c, w.eps, c2, a, stream=s), vg
        del c, c2, a, lo, hi, l2, i2, k2
        junk = overwrite((centres, C, alpha, lb_all, lam, li, cst))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), call
        del junk
