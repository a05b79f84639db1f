// C entry points of the dense-layer and gradient operators: argument checks, workspace sizes and the choice of kernel.
// Handle-less like vf_concretize: everything a call needs is in its arguments, and the caller owns the workspace.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <vector>

#include "vf.h"
#include "vf_internal.cuh"
#include "vf_ops.cuh"

using namespace vf;

namespace {

int ops_fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_last_error(code, buf);
}

#define OPS_TRY(call)                \
    do {                             \
        const int rc_ = (call);      \
        if (rc_ != VF_OK) return rc_; \
    } while (0)

int elem_bytes(int dtype) { return dtype == VF_F32 ? 4 : 2; }

int check_kind(int dtype, int act) {
    if (dtype != VF_F32 && dtype != VF_BF16 && dtype != VF_F16) return ops_fail(VF_ERR_ARG, "unknown dtype %d", dtype);
    if (act < VF_ACT_NONE || act > VF_ACT_SILU) return ops_fail(VF_ERR_ARG, "unknown activation %d", act);
    return VF_OK;
}

int check_sizes(long long M, int N, int K) {
    if (M < 0 || N < 0 || K < 0) return ops_fail(VF_ERR_ARG, "negative size: M %lld, N %d, K %d", M, N, K);
    // tile coordinates are 32-bit, with room for one tile past the end
    if (M > 0x7fffff00LL || N > 0x7fffff00 || K > 0x7fffff00)
        return ops_fail(VF_ERR_UNSUPPORTED, "M %lld, N %d and K %d must stay below 2^31 - 256", M, N, K);
    return VF_OK;
}

// A row-major matrix argument: present, aligned to its element, rows at least `cols` apart.
int check_matrix(const char* name, const void* p, long long rows, long long cols, long long ld, int dtype) {
    if (rows == 0 || cols == 0) return VF_OK;
    if (p == nullptr) return ops_fail(VF_ERR_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % elem_bytes(dtype) != 0)
        return ops_fail(VF_ERR_ARG, "%s is not aligned to its element", name);
    if (ld < cols && rows > 1)
        return ops_fail(VF_ERR_ARG, "%s: row stride %lld is below its %lld columns", name, ld, cols);
    if (ld > (1LL << 40)) return ops_fail(VF_ERR_ARG, "%s: row stride %lld is not one", name, ld);
    return VF_OK;
}

// The stride of a single row is not used; where rows have to be 16 bytes apart it must not decide either.
long long stride(long long rows, long long cols, long long ld) { return rows > 1 ? ld : (cols + 7) / 8 * 8; }

int check_vector(const char* name, const void* p, int dtype) {
    if (reinterpret_cast<uintptr_t>(p) % elem_bytes(dtype) != 0)
        return ops_fail(VF_ERR_ARG, "%s is not aligned to its element", name);
    return VF_OK;
}

int check_aligned(const void* work) {
    if (reinterpret_cast<uintptr_t>(work) % 256 != 0) return ops_fail(VF_ERR_ARG, "workspace is not 256-byte aligned");
    return VF_OK;
}

int check_work(size_t have, size_t need) {
    if (have < need) return ops_fail(VF_ERR_WORKSPACE, "workspace of %zu bytes, this call needs %zu", have, need);
    return VF_OK;
}

int launched(cudaError_t e) {
    if (e == cudaSuccess) return VF_OK;
    cudaGetLastError();  // reported here, not by the caller's next check
    return ops_fail(VF_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
}

// Runs an entry point's body; what the C++ library throws (it can run out of host memory) does not cross the ABI.
template <typename F>
int guarded(F body) {
    try {
        try {
            return body();
        } catch (const std::exception& e) {
            return ops_fail(VF_ERR_CUDA, "host: %s", e.what());
        }
    } catch (...) {  // nor does the message's own memory
        return VF_ERR_CUDA;
    }
}

int sm_count(int* sms) {
    const cudaError_t e = device_sms(sms);
    if (e == cudaSuccess) return VF_OK;
    cudaGetLastError();
    return ops_fail(VF_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
}

struct Range {
    uintptr_t lo, hi;
    int t;
};

// Every output range is disjoint from every other output and from every input but, exactly, its own.
int check_overlaps(const ClipList& l) {
    std::vector<Range> outs;
    outs.reserve(l.n);
    for (int t = 0; t < l.n; ++t) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(l.out[t]);
        if (l.size[t] > 0) outs.push_back(Range{lo, lo + (uintptr_t)l.size[t] * elem_bytes(l.dtype[t]), t});
    }
    std::sort(outs.begin(), outs.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    for (size_t i = 1; i < outs.size(); ++i)
        if (outs[i].lo < outs[i - 1].hi)
            return ops_fail(VF_ERR_ARG, "outputs %d and %d overlap", outs[i - 1].t, outs[i].t);
    for (int t = 0; t < l.n; ++t) {
        if (l.size[t] == 0) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(l.in[t]);
        const uintptr_t hi = lo + (uintptr_t)l.size[t] * elem_bytes(l.dtype[t]);
        // the outputs are disjoint and sorted: the first that ends after lo is the only one to begin looking at
        auto it = std::upper_bound(outs.begin(), outs.end(), lo, [](uintptr_t v, const Range& r) { return v < r.hi; });
        for (; it != outs.end() && it->lo < hi; ++it)
            if (it->t != t || it->lo != lo)
                return ops_fail(VF_ERR_ARG, "gradient %d overlaps output %d", t, it->t);
    }
    return VF_OK;
}

// Small products, and empty ones, run on the FFMA kernels, whose time goes with the reduction's length. M x N x K in us, FFMA
// and tensor cores: fp32 forward 64x32x8 3.7 and 5.1, 64x32x16 3.4 and 5.1, 16x32x64 4.4 and 4.3, 16x16x256 11.1 and 5.5, backward
// 20x32x32 4.9 and 6.2, 16x32x64 4.2 and 6.0, 64x32x32 8.1 and 7.0; bf16 forward 64x32x16 4.8 and 4.3, 16x16x256 17.3 and 4.4,
// backward 16x64x128 5.6 and 6.1, 128x64x32 11.3 and 6.7. The rule goes by the volume alone and so takes the slower side for few
// outputs of a long reduction below it: fp32 forward 32x1x1000 38 and 7.5, 9x1x3640 129 and 13, backward 64x16x16 8.2 and 6.5,
// 2000x4x4 194 and 16, 8191x1x3 505 and 20.
bool use_tc(long long M, int N, int K) { return linear_tc_supported(M, N, K) && (double)M * N * K >= 32768.0; }

}  // namespace

extern "C" {

int vf_linear_workspace(int dtype, long long M, int N, int K, int grad, size_t* bytes) {
    return guarded([&]() -> int {
        if (bytes == nullptr) return ops_fail(VF_ERR_ARG, "NULL pointer");
        OPS_TRY(check_kind(dtype, VF_ACT_NONE));
        OPS_TRY(check_sizes(M, N, K));
        const bool aligned = grad == VF_FORWARD_ALIGNED;
        if (grad < 0 || grad > VF_FORWARD_ALIGNED) return ops_fail(VF_ERR_ARG, "grad = %d", grad);
        if (grad == 1 && linear_few_supported(dtype, M, N, K))
            *bytes = linear_few_workspace(dtype, M, N, K);
        else if (!use_tc(M, N, K) || (grad != 1 && linear_few_forward(dtype, M, N, K)) ||
                 (aligned && (dtype != VF_F32 || linear_direct_fits(dtype, M, N, K, true, true))) ||
                 (grad == 0 && linear_direct_fits(dtype, M, N, K, false, false)))
            *bytes = 0;
        else
            *bytes = linear_tc_workspace(dtype, M, N, K, grad == 1);
        return VF_OK;
    });
}

int vf_linear(int dtype, int act, const void* x, long long ldx, const void* W, long long ldw, const void* b,
              const void* r, long long ldr, long long M, int N, int K, void* y, long long ldy, void* z, long long ldz,
              void* work, size_t work_bytes, void* stream) {
    return guarded([&]() -> int {
        OPS_TRY(check_kind(dtype, act));
        OPS_TRY(check_sizes(M, N, K));
        if (M == 0 || N == 0) return VF_OK;
        OPS_TRY(check_matrix("x", x, M, K, ldx, dtype));
        OPS_TRY(check_matrix("W", W, N, K, ldw, dtype));
        OPS_TRY(check_vector("b", b, dtype));
        if (r != nullptr) OPS_TRY(check_matrix("r", r, M, N, ldr, dtype));
        OPS_TRY(check_matrix("y", y, M, N, ldy, dtype));
        if (z != nullptr) OPS_TRY(check_matrix("z", z, M, N, ldz, dtype));
        ldx = stride(M, K, ldx), ldw = stride(N, K, ldw), ldr = stride(M, N, ldr), ldy = stride(M, N, ldy), ldz = stride(M, N, ldz);
        const LinearFwd p{dtype, act, x, ldx, W, ldw, b, r, ldr, M, N, K, y, ldy, z, ldz};
        if (linear_few_forward(dtype, M, N, K)) return launched(launch_linear_few(p, (cudaStream_t)stream));
        if (!use_tc(M, N, K)) return launched(launch_linear_ffma(p, (cudaStream_t)stream));
        if (!linear_tc_in_place(p) && linear_direct_fits(dtype, M, N, K, aligned16(x, ldx, elem_bytes(dtype)), aligned16(W, ldw, elem_bytes(dtype))))
            return launched(launch_linear_direct(p, (cudaStream_t)stream));
        OPS_TRY(check_aligned(work));
        size_t need = 0;
        const size_t have = work == nullptr ? 0 : work_bytes;
        OPS_TRY(launched(launch_linear_tc(p, work, have, &need, (cudaStream_t)stream)));
        return check_work(have, need);
    });
}

int vf_linear_grad(int dtype, int act, const void* dy, long long lddy, const void* z, long long ldz, const void* x,
                   long long ldx, const void* W, long long ldw, long long M, int N, int K, void* dx, long long lddx,
                   void* dW, long long lddw, void* db, void* dr, long long lddr, void* work, size_t work_bytes,
                   void* stream) {
    return guarded([&]() -> int {
        OPS_TRY(check_kind(dtype, act));
        OPS_TRY(check_sizes(M, N, K));
        OPS_TRY(check_matrix("dy", dy, M, N, lddy, dtype));
        if (act != VF_ACT_NONE) OPS_TRY(check_matrix("z", z, M, N, ldz, dtype));
        if (dx != nullptr) {
            OPS_TRY(check_matrix("W", W, N, K, ldw, dtype));
            OPS_TRY(check_matrix("dx", dx, M, K, lddx, dtype));
        }
        if (dW != nullptr) {
            OPS_TRY(check_matrix("x", x, M, K, ldx, dtype));
            OPS_TRY(check_matrix("dW", dW, N, K, lddw, dtype));
        }
        OPS_TRY(check_vector("db", db, dtype));
        if (dr != nullptr) OPS_TRY(check_matrix("dr", dr, M, N, lddr, dtype));
        lddy = stride(M, N, lddy), ldz = stride(M, N, ldz), ldx = stride(M, K, ldx), ldw = stride(N, K, ldw);
        lddx = stride(M, K, lddx), lddw = stride(N, K, lddw), lddr = stride(M, N, lddr);
        const LinearGrad p{dtype, act, dy, lddy, z, ldz, x, ldx, W, ldw, M, N, K, dx, lddx, dW, lddw, db, dr, lddr};
        const bool few = linear_few_supported(dtype, M, N, K);
        if (!few && !use_tc(M, N, K)) return launched(launch_linear_grad_ffma(p, (cudaStream_t)stream));
        OPS_TRY(check_aligned(work));
        size_t need = 0;
        const size_t have = work == nullptr ? 0 : work_bytes;
        OPS_TRY(launched(few ? launch_linear_few_grad(p, work, have, &need, (cudaStream_t)stream)
                             : launch_linear_grad_tc(p, work, have, &need, (cudaStream_t)stream)));
        return check_work(have, need);
    });
}

int vf_ops_check(void) {
    return guarded([]() -> int {
        int timeout = 0;
        cudaError_t e = cudaDeviceSynchronize();
        if (e == cudaSuccess) e = ops_take_timeout(&timeout);
        if (e != cudaSuccess) return ops_fail(VF_ERR_CUDA, "asynchronous CUDA error: %s", cudaGetErrorString(e));
        if (timeout) return ops_fail(VF_ERR_TIMEOUT, "a kernel gave up a bounded wait; its outputs are not valid");
        return VF_OK;
    });
}

int vf_clip_workspace(int n, size_t* bytes) {
    return guarded([&]() -> int {
        if (bytes == nullptr) return ops_fail(VF_ERR_ARG, "NULL pointer");
        if (n < 0) return ops_fail(VF_ERR_ARG, "negative number of gradients");
        int sms = 0;
        OPS_TRY(sm_count(&sms));
        *bytes = (size_t)clip_work_doubles(n, sms) * sizeof(double);
        return VF_OK;
    });
}

int vf_clip_grad_norm(int n, const void* const* grads, void* const* outs, const long long* sizes, const int* dtypes,
                      float scale, float max_norm, float* norm, void* work, size_t work_bytes, void* stream) {
    return guarded([&]() -> int {
        if (n < 0) return ops_fail(VF_ERR_ARG, "negative number of gradients");
        if (norm == nullptr || (n > 0 && (!grads || !outs || !sizes || !dtypes))) return ops_fail(VF_ERR_ARG, "NULL pointer");
        if (!std::isfinite(scale) || scale < 0.f) return ops_fail(VF_ERR_NONFINITE, "scale must be finite and >= 0");
        if (std::isnan(max_norm) || max_norm < 0.f) return ops_fail(VF_ERR_ARG, "max_norm must be >= 0");
        const ClipList l{n, grads, outs, sizes, dtypes};
        long long bytes = 0;
        for (int t = 0; t < n; ++t) {
            OPS_TRY(check_kind(dtypes[t], VF_ACT_NONE));
            if (sizes[t] < 0 || sizes[t] > (1LL << 42)) return ops_fail(VF_ERR_ARG, "gradient %d has %lld elements", t, sizes[t]);
            OPS_TRY(check_matrix("gradient", grads[t], 1, sizes[t], sizes[t], dtypes[t]));
            OPS_TRY(check_matrix("output", outs[t], 1, sizes[t], sizes[t], dtypes[t]));
            bytes += sizes[t] * elem_bytes(dtypes[t]);
            if (bytes > (1LL << 44)) return ops_fail(VF_ERR_UNSUPPORTED, "gradients of over 16 TiB");
        }
        OPS_TRY(check_overlaps(l));
        size_t need = 0;
        OPS_TRY(vf_clip_workspace(n, &need));
        OPS_TRY(check_aligned(work));
        OPS_TRY(check_work(work == nullptr ? 0 : work_bytes, need));
        return launched(launch_clip(l, scale, max_norm, norm, (double*)work, (cudaStream_t)stream));
    });
}

}  // extern "C"
