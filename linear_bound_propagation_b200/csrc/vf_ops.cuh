// Shared by the dense-layer and gradient operators (k_linear.cu, k_linear_tc.cu, k_clip.cu, vf_ops.cu): element
// types, activations and the launch interfaces. Nothing here is part of the public ABI (include/vf.h).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "vf.h"

namespace vf {

// ------------------------------------------------------------------------------------------ element types
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}

// Eight values that lie together, as the words they are loaded and stored in (elements held one by one would take
// a register each in the 16-bit types).
template <typename T>
struct alignas(16) Pack8 {
    uint32_t w[2 * sizeof(T)];
};
__device__ __forceinline__ void unpack8(const Pack8<float>& p, float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = __uint_as_float(p.w[u]);
}
__device__ __forceinline__ void unpack8(const Pack8<__nv_bfloat16>& p, float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        v[2 * u] = __uint_as_float(p.w[u] << 16);
        v[2 * u + 1] = __uint_as_float(p.w[u] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack8(const Pack8<__half>& p, float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p.w[u]));
        v[2 * u] = f.x;
        v[2 * u + 1] = f.y;
    }
}
__device__ __forceinline__ void pack8(Pack8<float>& p, const float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) p.w[u] = __float_as_uint(v[u]);
}
__device__ __forceinline__ void pack8(Pack8<__nv_bfloat16>& p, const float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * u], v[2 * u + 1]);
        p.w[u] = *reinterpret_cast<const uint32_t*>(&h);
    }
}
__device__ __forceinline__ void pack8(Pack8<__half>& p, const float (&v)[8]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const __half2 h = __floats2half2_rn(v[2 * u], v[2 * u + 1]);
        p.w[u] = *reinterpret_cast<const uint32_t*>(&h);
    }
}
// One element's bits; or_elem on a pack that holds zeros there.
template <typename T>
__device__ __forceinline__ void or_elem(Pack8<T>& p, int u, T x) {
    if (sizeof(T) == 4)
        p.w[u] = *reinterpret_cast<const uint32_t*>(&x);
    else
        p.w[u >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(&x) << (16 * (u & 1));
}
template <typename T>
__device__ __forceinline__ T get_elem(const Pack8<T>& p, int u) {
    T x;
    if (sizeof(T) == 4)
        *reinterpret_cast<uint32_t*>(&x) = p.w[u];
    else
        *reinterpret_cast<uint16_t*>(&x) = (uint16_t)(p.w[u >> 1] >> (16 * (u & 1)));
    return x;
}
template <typename T>
__device__ __forceinline__ void zero8(Pack8<T>& p) {
#pragma unroll
    for (int u = 0; u < (int)(2 * sizeof(T)); ++u) p.w[u] = 0;
}
// The first n (8 at most) of eight values, zeros behind them. vec: p is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load_raw8(const T* p, int n, bool vec, Pack8<T>& v) {
    if (vec && n >= 8) {
        v = *reinterpret_cast<const Pack8<T>*>(p);
    } else {
        zero8(v);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (u < n) or_elem(v, u, p[u]);
    }
}
template <typename T>
__device__ __forceinline__ void store_raw8(T* p, int n, bool vec, const Pack8<T>& v) {
    if (vec && n >= 8) {
        *reinterpret_cast<Pack8<T>*>(p) = v;
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (u < n) p[u] = get_elem(v, u);
    }
}

// -------------------------------------------------------------------------------------------- activations
__device__ __forceinline__ float exp2f_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Clamps that keep NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Evaluated in fp32. FAST serves the 16-bit types, whose rounding (2^-9, 2^-12) lies far above its error; float32 takes
// CUDA's erfcf and expf.
//
// Phi(z), the normal distribution, and e = exp(-z^2 / 2). Accurate form: erfc(-z / sqrt 2) / 2, which keeps its relative
// accuracy for negative z where 1 + erf(z / sqrt 2) cancels. Fast form: Phi(-a) = exp(-a^2 / 2) Q(a) for a = |z|, with
// Q(a) = erfcx(a / sqrt 2) / 2 as a polynomial in t = 1 / (1 + 0.3 a) (the form of Abramowitz & Stegun 7.1.26; the
// coefficients are a weighted least-squares fit of Q over 0 <= a <= 14.5, relative error 1.6e-7). In fp32 it is within
// (15 + z^2) 2^-24 of Phi(z), relative (simulated on 3 million points), and one exponential serves Phi and e.
template <bool FAST>
__device__ __forceinline__ float phi(float z, float& e) {
    if (!FAST) {
        e = expf(-0.5f * z * z);
        return 0.5f * erfcf(z * -0.70710678118654752f);
    }
    const float a = fabsf(z);
    e = exp2f_approx(z * z * -0.72134752044448170f);
    const float t = rcp_approx(fmaf(0.3f, a, 1.f));
    float q = 0.035423859484090325f;
    q = fmaf(q, t, -0.15615893604759168f);
    q = fmaf(q, t, 0.204557570019329f);
    q = fmaf(q, t, -0.052034684620186886f);
    q = fmaf(q, t, 0.12769209473926563f);
    q = fmaf(q, t, 0.1001758593708425f);
    q = fmaf(q, t, 0.12071214884669218f);
    q = fmaf(q, t, 0.11963200649944138f);
    const float tail = q * t * e;
    return z > 0.f ? 1.f - tail : tail;
}
// 1 / (1 + exp(-z)) and e = exp(-z).
template <bool FAST>
__device__ __forceinline__ float sigmoid(float z, float& e) {
    e = FAST ? exp2f_approx(z * -1.4426950408889634f) : expf(-z);
    return FAST ? rcp_approx(1.f + e) : 1.f / (1.f + e);
}

// relu passes NaN on (z < 0 is false for it); gelu and silu take their limit 0 at -inf.
template <bool FAST>
__device__ __forceinline__ float act_value(float z, int act) {
    float e;
    switch (act) {
        case VF_ACT_RELU: return z < 0.f ? 0.f : z;
        case VF_ACT_GELU: {
            const float f = phi<FAST>(z, e);
            return f == 0.f ? 0.f : z * f;
        }
        case VF_ACT_SILU: {
            const float f = sigmoid<FAST>(z, e);
            return f == 0.f ? 0.f : z * f;
        }
        default: return z;
    }
}
// dy act'(z); relu'(0) = 0, and relu selects instead of multiplying, so an infinite dy behind a closed ReLU stays 0.
// silu' = s (1 + z (1 - s)) with 1 - s formed as e s (e = exp(-z)), so it does not cancel for large z; where e
// overflows (z < -88) the slope is below 1e-36 and taken as 0. Beyond |z| = 80 gelu's slope, and above 80 silu's, are
// their limits in fp32; the clamps keep 0 * inf away there.
template <bool FAST>
__device__ __forceinline__ float act_grad(float dy, float z, int act) {
    float e;
    if (act == VF_ACT_NONE) return dy;
    if (act == VF_ACT_RELU) return z <= 0.f ? 0.f : dy;
    z = min_nan(z, 80.f);
    if (act == VF_ACT_GELU) {
        z = max_nan(z, -80.f);
        const float f = phi<FAST>(z, e);
        return dy * fmaf(z * 0.39894228040143268f, e, f);
    }
    const float s = sigmoid<FAST>(z, e);
    return s == 0.f ? 0.f : dy * (s * fmaf(z, e * s, 1.f));
}

// ------------------------------------------------------------------------------------------ launch interfaces
// Rows of 16-byte alignment (ld in elements of e bytes) that TMA can address too: its strides end at 2^40 bytes.
inline bool aligned16(const void* p, long long ld, int e) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * e) % 16 == 0 && ld < (1LL << 37);
}

// One dense layer, forward: y = act(z), z = x W^T + b + r. Row strides in elements.
struct LinearFwd {
    int dtype, act;
    const void* x;
    long long ldx;
    const void* W;
    long long ldw;
    const void* b;  // or nullptr
    const void* r;  // or nullptr
    long long ldr;
    long long M;
    int N, K;
    void* y;
    long long ldy;
    void* z;  // or nullptr
    long long ldz;
};

// Its backward pass: g = dy act'(z); dx = g W, dW = g^T x, db = sum_m g, dr = g (any output may be nullptr).
struct LinearGrad {
    int dtype, act;
    const void* dy;
    long long lddy;
    const void* z;  // nullptr only for VF_ACT_NONE
    long long ldz;
    const void* x;
    long long ldx;
    const void* W;
    long long ldw;
    long long M;
    int N, K;
    void* dx;
    long long lddx;
    void* dW;
    long long lddw;
    void* db;
    void* dr;
    long long lddr;
};

// FFMA kernels (k_linear.cu): any strides and alignment, no workspace.
cudaError_t launch_linear_ffma(const LinearFwd& p, cudaStream_t s);
cudaError_t launch_linear_grad_ffma(const LinearGrad& p, cudaStream_t s);

// A few rows, forward (k_linear_few.cu): any strides and alignment, no workspace.
bool linear_few_forward(int dtype, long long M, int N, int K);
cudaError_t launch_linear_few(const LinearFwd& p, cudaStream_t s);

// Backward pass of a few rows (k_linear_few.cu); workspace as for the tensor-core launches below.
bool linear_few_supported(int dtype, long long M, int N, int K);
size_t linear_few_workspace(int dtype, long long M, int N, int K);
cudaError_t launch_linear_few_grad(const LinearGrad& p, void* work, size_t have, size_t* need, cudaStream_t s);

// Tensor-core kernels (k_linear_tc.cu). linear_tc_workspace: the most any strides and alignment take. The launches write
// to *need what this call takes of `work` (256-byte aligned) and launch nothing if that is more than `have`.
bool linear_tc_supported(long long M, int N, int K);
// Whether TMA can read x and W in place.
bool linear_tc_in_place(const LinearFwd& p);
size_t linear_tc_workspace(int dtype, long long M, int N, int K, bool grad);
cudaError_t launch_linear_tc(const LinearFwd& p, void* work, size_t have, size_t* need, cudaStream_t s);
cudaError_t launch_linear_grad_tc(const LinearGrad& p, void* work, size_t have, size_t* need, cudaStream_t s);
cudaError_t ops_take_timeout(int* flag);
cudaError_t device_sms(int* sms);  // SMs of the current device

// Forward product that lays its operands out itself (k_linear_direct.cu): any strides and alignment, no workspace, for the
// sizes that `fits` accepts.
bool linear_direct_fits(int dtype, long long M, int N, int K, bool x_aligned, bool w_aligned);
cudaError_t launch_linear_direct(const LinearFwd& p, cudaStream_t s);
cudaError_t direct_take_timeout(int* flag);

// Gradient norm and clipping (k_clip.cu); ranges as in vf_clip_grad_norm. `work` holds clip_work_doubles(n, SMs) doubles.
struct ClipList {
    int n;
    const void* const* in;
    void* const* out;
    const long long* size;
    const int* dtype;
};
long long clip_work_doubles(int n, int sms);
cudaError_t launch_clip(const ClipList& l, float scale, float max_norm, float* norm, double* work, cudaStream_t s);

}  // namespace vf
