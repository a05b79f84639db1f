"""Argument checks of the dense-layer and gradient operators: refused on the host, before any device work, with an error
code and a message. Pointers are made-up addresses that nothing may read, so these run without a GPU."""
import ctypes

import pytest
import torch

from linear_bound_propagation_b200 import vf

P = 1 << 20  # an aligned address


def linear(**kw):
    a = dict(dtype=0, act=0, x=P, ldx=8, W=2 * P, ldw=8, b=None, r=None, ldr=0, M=4, N=6, K=8, y=3 * P, ldy=6, z=None,
             ldz=0, work=None, work_bytes=0)
    a.update(kw)
    return vf.lib().vf_linear(*a.values(), None)


def grad(**kw):
    a = dict(dtype=0, act=1, dy=P, lddy=6, z=2 * P, ldz=6, x=3 * P, ldx=8, W=4 * P, ldw=8, M=4, N=6, K=8, dx=5 * P,
             lddx=8, dW=6 * P, lddw=8, db=None, dr=None, lddr=0, work=None, work_bytes=0)
    a.update(kw)
    return vf.lib().vf_linear_grad(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(dtype=-1), dict(act=4), dict(act=-1), dict(M=-1), dict(N=-1),
                                 dict(K=-1), dict(x=None), dict(W=None), dict(y=None), dict(ldx=7), dict(ldw=7),
                                 dict(ldy=5), dict(r=P, ldr=5), dict(z=P, ldz=5), dict(x=P + 2), dict(W=P + 1),
                                 dict(y=P + 2), dict(b=P + 2), dict(ldx=1 << 41)])
def test_linear_refuses(bad):
    assert linear(**bad) == vf.VF_ERR_ARG
    assert vf.lib().vf_last_error()


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(act=9), dict(M=-1), dict(dy=None), dict(z=None), dict(x=None),
                                 dict(W=None), dict(lddy=5), dict(ldz=5), dict(ldx=7), dict(ldw=7), dict(lddx=7),
                                 dict(lddw=7), dict(dr=P, lddr=5), dict(db=P + 1), dict(dx=P + 2)])
def test_linear_grad_refuses(bad):
    assert grad(**bad) == vf.VF_ERR_ARG
    assert vf.lib().vf_last_error()


def test_sizes_beyond_32_bit_tiles_are_refused():
    assert linear(M=1 << 31) == vf.VF_ERR_UNSUPPORTED
    assert grad(M=1 << 40) == vf.VF_ERR_UNSUPPORTED
    n = ctypes.c_size_t()
    assert vf.lib().vf_linear_workspace(0, 1 << 31, 8, 8, 0, ctypes.byref(n)) == vf.VF_ERR_UNSUPPORTED
    assert vf.lib().vf_linear_workspace(7, 8, 8, 8, 0, ctypes.byref(n)) == vf.VF_ERR_ARG
    assert vf.lib().vf_linear_workspace(0, 8, 8, 8, 0, None) == vf.VF_ERR_ARG
    assert vf.lib().vf_linear_workspace(0, 8, 8, 8, 3, ctypes.byref(n)) == vf.VF_ERR_ARG


def test_empty_outputs_are_no_ops_without_a_device():
    assert linear(M=0) == vf.VF_OK
    assert linear(N=0, W=None, y=None) == vf.VF_OK


def clip(grads, outs, sizes, dtypes=None, scale=1.0, max_norm=1.0, norm=P, n=None):
    k = len(grads)
    arr = lambda t, v: (t * k)(*v)  # noqa: E731
    return vf.lib().vf_clip_grad_norm(k if n is None else n, arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, outs),
                                      arr(ctypes.c_longlong, sizes), arr(ctypes.c_int, dtypes or [0] * k), scale,
                                      max_norm, norm, None, 0, None)


def test_clip_refuses():
    ok = dict(grads=[P], outs=[P], sizes=[8])
    for bad in (dict(n=-1), dict(norm=None), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(dtypes=[5]),
                dict(sizes=[-1]), dict(grads=[None]), dict(outs=[None]), dict(grads=[P + 2], outs=[P + 2])):
        assert clip(**{**ok, **bad}) == vf.VF_ERR_ARG, bad
    for scale in (float("inf"), float("nan"), -1.0):
        assert clip(**ok, scale=scale) == vf.VF_ERR_NONFINITE
    assert clip([P], [P], [1 << 42], dtypes=[0]) != vf.VF_OK


def test_clip_refuses_overlaps():
    # the same gradient twice in place, outputs that overlap, and an output over another gradient
    assert clip([P, P], [P, P], [8, 8]) == vf.VF_ERR_ARG
    assert clip([P, 2 * P], [3 * P, 3 * P + 16], [8, 8]) == vf.VF_ERR_ARG
    assert clip([P, 2 * P], [3 * P, P + 28], [8, 8]) == vf.VF_ERR_ARG
    assert clip([P, 2 * P], [P + 4, 4 * P], [8, 8]) == vf.VF_ERR_ARG  # shifted onto itself
    assert b"overlap" in vf.lib().vf_last_error()
    # in place, apart, and one gradient read twice: past the overlap check (it is the device query or the missing
    # workspace that ends these calls)
    for g, o in (([P, 2 * P], [P, 2 * P]), ([P, P + 32], [2 * P, 2 * P + 32]), ([P, P], [2 * P, 3 * P])):
        assert clip(g, o, [8, 8]) in (vf.VF_ERR_CUDA, vf.VF_ERR_WORKSPACE)
        assert b"overlap" not in vf.lib().vf_last_error()


def test_binding_refuses_what_is_not_on_a_gpu():
    x, W = torch.zeros(2, 3), torch.zeros(4, 3)
    with pytest.raises(ValueError):
        vf.linear(x, W)
    with pytest.raises(ValueError):
        vf.linear(x.double(), W.double())
    with pytest.raises(ValueError):
        vf.linear(x, W, act="tanh")
    with pytest.raises(ValueError):
        vf.linear_grad(torch.zeros(2, 4), x, W, act="relu")
    with pytest.raises(ValueError):
        vf.clip_grad_norm([x], 1.0)
    with pytest.raises(ValueError):
        vf.clip_grad_norm([x], 1.0, out=[])
