"""vf_linear and vf_linear_grad called through the C ABI on a B200: matrices of one row, and workspaces that are too small."""
import ctypes

import pytest
import torch

vf = pytest.importorskip("linear_bound_propagation_b200.vf")
pytestmark = pytest.mark.gpu
CODE = vf.VF_DTYPES


def p(t):
    return None if t is None else t.data_ptr()


def work_for(dtype, M, N, K, grad):
    n = ctypes.c_size_t()
    assert vf.lib().vf_linear_workspace(CODE[dtype], M, N, K, grad, ctypes.byref(n)) == vf.VF_OK
    return torch.empty(n.value, device="cuda", dtype=torch.uint8), n.value


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ld", [0, -7, 3, 1 << 38])
def test_the_stride_of_a_single_row_is_not_used(dtype, ld):
    """Whole numbers, so every kernel's result is exact; one row of x, y, r and z, or one of W and dW."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def whole(*s):
        return torch.randint(-2, 3, s, generator=gen, device="cuda").to(dtype)

    L, s = vf.lib(), torch.cuda.current_stream().cuda_stream
    for M, N, K in ((1, 8192, 4096), (1, 40, 30), (64, 1, 1024), (700, 1, 1021), (9, 1, 4000), (17, 1, 30)):
        x, W, r, dy = whole(M, K), whole(N, K), whole(M, N), whole(M, N)
        one = lambda rows, cols: ld if rows == 1 else cols  # noqa: E731
        y, z = torch.full((M, N), 7.0, device="cuda", dtype=dtype), torch.full((M, N), 7.0, device="cuda", dtype=dtype)
        work, n = work_for(dtype, M, N, K, 0)
        assert L.vf_linear(CODE[dtype], 0, p(x), one(M, K), p(W), one(N, K), None, p(r), one(M, N), M, N, K, p(y), one(M, N),
                           p(z), one(M, N), p(work), n, s) == vf.VF_OK, L.vf_last_error()
        want = x.double() @ W.double().t() + r.double()
        assert torch.equal(y, want.to(dtype)) and torch.equal(z, y)
        dx, dW, db, dr = (torch.full(t, 7.0, device="cuda", dtype=dtype) for t in ((M, K), (N, K), (N,), (M, N)))
        work, n = work_for(dtype, M, N, K, 1)
        assert L.vf_linear_grad(CODE[dtype], 1, p(dy), one(M, N), p(r), one(M, N), p(x), one(M, K), p(W), one(N, K), M, N, K,
                                p(dx), one(M, K), p(dW), one(N, K), p(db), p(dr), one(M, N), p(work), n, s) == vf.VF_OK, L.vf_last_error()
        g = dy.double() * (r.double() > 0)
        for got, w in ((dx, g @ W.double()), (dW, g.t() @ x.double()), (db, g.sum(0)), (dr, g)):
            assert torch.equal(got, w.to(dtype))
    vf.ops_check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_a_forward_call_without_its_workspace_writes_nothing(dtype):
    M, N, K = 2000, 1500, 333
    x, W = torch.ones(M, K + 1, device="cuda", dtype=dtype)[:, :K], torch.ones(N, K + 1, device="cuda", dtype=dtype)[:, :K]
    y = torch.full((M, N), 7.0, device="cuda", dtype=dtype)
    work, n = work_for(dtype, M, N, K, 0)
    assert n > 0
    L, s = vf.lib(), torch.cuda.current_stream().cuda_stream
    for w, size, code in ((None, n, vf.VF_ERR_WORKSPACE), (p(work), 0, vf.VF_ERR_WORKSPACE), (p(work), 1024, vf.VF_ERR_WORKSPACE),
                          (p(work) + 16, n, vf.VF_ERR_ARG)):
        assert L.vf_linear(CODE[dtype], 0, p(x), K + 1, p(W), K + 1, None, None, 0, M, N, K, p(y), N, None, 0, w, size, s) == code
    torch.cuda.synchronize()
    assert (y == 7.0).all()
    assert L.vf_linear(CODE[dtype], 0, p(x), K + 1, p(W), K + 1, None, None, 0, M, N, K, p(y), N, None, 0, p(work), n, s) == vf.VF_OK
    assert (y == K).all()
    vf.ops_check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(1, 20000, 1024), (9, 1, 200000), (40000, 1, 64)])
def test_the_workspace_of_aligned_rows_is_enough_for_any_stride_of_a_single_row(dtype, M, N, K):
    """16-byte rows of x and W, the size of VF_FORWARD_ALIGNED; the one row's stride is a multiple of 16 bytes beyond any tensor map's."""
    x, W = torch.ones(M, K, device="cuda", dtype=dtype), torch.ones(N, K, device="cuda", dtype=dtype)
    y = torch.full((M, N), 7.0, device="cuda", dtype=dtype)
    work, n = work_for(dtype, M, N, K, vf.VF_FORWARD_ALIGNED)
    assert vf.lib().vf_linear(CODE[dtype], 0, p(x), 1 << 38 if M == 1 else K, p(W), 1 << 38 if N == 1 else K, None, None, 0, M, N, K,
                              p(y), N, None, 0, p(work), n, torch.cuda.current_stream().cuda_stream) == vf.VF_OK, vf.lib().vf_last_error()
    assert (y == torch.tensor(float(K), device="cuda").to(dtype)).all()
    vf.ops_check()
