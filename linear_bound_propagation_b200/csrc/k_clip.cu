// Global L2 norm of a list of gradients, and the gradients scaled down to a largest norm.
//
//   norm = scale * sqrt(sum_t sum_i g_ti^2),  out_ti = g_ti * f,  f = scale * (max_norm / norm if norm > max_norm else 1)
//
// Two passes over the list: no element may be written before the norm over all of them is known. Each pass is one
// launch per MAX_TENSORS tensors; the table of pointers travels in the kernel's parameters, so nothing is copied to the
// device and a captured launch keeps its own table. Pass 1 leaves one partial sum per block, pass 2 adds them in a
// fixed order in every block: no atomics, the same bits on every run.
//
// Squares are added in fp32 over one thread's 32 bytes (at most 16 terms) and in fp64 beyond that. Where such a
// partial sum leaves the range in which fp32 squares are exact enough (overflow above 1e19, underflow below 1e-15 per
// element), that thread's elements are squared again in fp64, so norms of any finite fp32 or bf16 values come out. Whether a norm
// is finite is decided on the float that the caller sees.
#include <algorithm>

#include "vf_internal.cuh"
#include "vf_ops.cuh"

namespace vf {

namespace {

constexpr int THREADS = 256;
constexpr int MAX_TENSORS = 100;            // 3.2 KB of the 4 KB parameter space
constexpr int BLOCKS_PER_SM = 8;            // of the first pass

struct Table {
    const void* in[MAX_TENSORS];
    void* out[MAX_TENSORS];
    long long size[MAX_TENSORS];
    int first[MAX_TENSORS + 1];  // first chunk of each tensor
    unsigned char dtype[MAX_TENSORS];
    int n;
};

// A chunk is what a block takes at a time: V 16-byte loads per thread.
__host__ __device__ __forceinline__ int chunk_elems(int dtype, int V) { return THREADS * 16 * V / (dtype == VF_F32 ? 4 : 2); }
// The tensor that chunk c belongs to.
__device__ __forceinline__ int tensor_of(const Table& tab, int c) {
    int lo = 0, hi = tab.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (c >= tab.first[mid])
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <typename T, int N>
struct alignas(16) Vec {
    T v[N];
};

// Sum of squares of n <= 16 values, see the header.
template <typename T>
__device__ __forceinline__ double squares(const T* v, int n) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const float x = to_f32(v[i]);
        s = fmaf(x, x, s);
    }
    if (!(s < 3e38f) || s < 1e-30f) {
        double d = 0.0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const double x = (double)to_f32(v[i]);
            d = fma(x, x, d);
        }
        return d;
    }
    return (double)s;
}

// One chunk of a tensor: elements [e0, e1). `head` elements come before the first 16-byte boundary.
template <typename T, int V>
__device__ __forceinline__ double chunk_squares(const T* __restrict__ p, long long e0, long long e1) {
    constexpr int N = 16 / sizeof(T);
    const T* q = p + e0;
    const int len = (int)(e1 - e0);
    const int head = min(len, (int)(((16 - (reinterpret_cast<uintptr_t>(q) & 15)) & 15) / sizeof(T)));
    const int nv = (len - head) / N;
    const Vec<T, N>* b = reinterpret_cast<const Vec<T, N>*>(q + head);
    double d = 0.0;
    if (nv == V * THREADS) {
        Vec<T, N> v[V];
#pragma unroll
        for (int u = 0; u < V; ++u) v[u] = b[threadIdx.x + u * THREADS];
#pragma unroll
        for (int u = 0; u < V; u += 2) {  // two vectors at a time in fp32
            T w[2 * N];
            *reinterpret_cast<Vec<T, N>*>(w) = v[u];
            *reinterpret_cast<Vec<T, N>*>(w + N) = v[u + 1];
            d += squares(w, 2 * N);
        }
    } else {
        for (int i = threadIdx.x; i < nv; i += THREADS) {
            const Vec<T, N> w = b[i];
            d += squares(w.v, N);
        }
    }
    if (threadIdx.x < head) d += squares(q + threadIdx.x, 1);
    const int tail = head + nv * N + threadIdx.x;
    if (tail < len) d += squares(q + tail, 1);
    return d;
}

__device__ __forceinline__ double block_sum(double d) {
    __shared__ double w[THREADS / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = d;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) t += w[i];
    return t;
}

template <int V>
__global__ void __launch_bounds__(THREADS) clip_norm_k(const __grid_constant__ Table tab, double* part) {
    double d = 0.0;
    int t = 0;
    for (int c = blockIdx.x; c < tab.first[tab.n]; c += gridDim.x) {
        while (c >= tab.first[t + 1]) ++t;
        const long long e = chunk_elems(tab.dtype[t], V);
        const long long e0 = (c - tab.first[t]) * e, e1 = min(tab.size[t], e0 + e);
        switch (tab.dtype[t]) {
            case VF_F32: d += chunk_squares<float, V>((const float*)tab.in[t], e0, e1); break;
            case VF_BF16: d += chunk_squares<__nv_bfloat16, V>((const __nv_bfloat16*)tab.in[t], e0, e1); break;
            default: d += chunk_squares<__half, V>((const __half*)tab.in[t], e0, e1); break;
        }
    }
    const double s = block_sum(d);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// f as two factors: fp32 holds fewer than 24 bits of an f below 2^-126 (a norm of 1e38 clipped to 1), so 2^-126 is taken out of it
// there, and a product that is not subnormal keeps its bits. `low` is 1 elsewhere.
struct Factor {
    float high, low;
    __device__ __forceinline__ explicit Factor(double f) {
        low = f < 1.1754943508222875e-38 ? 1.17549435e-38f : 1.f;
        high = (float)(f / (double)low);
    }
    template <typename T>
    __device__ __forceinline__ T operator()(T x) const {
        return from_f32<T>(to_f32(x) * high * low);
    }
};

template <typename T, int V>
__device__ __forceinline__ void chunk_scale(const T* p, T* out, long long e0, long long e1, const Factor& f) {
    constexpr int N = 16 / sizeof(T);
    const T* q = p + e0;
    T* o = out + e0;
    const int len = (int)(e1 - e0);
    const int head = min(len, (int)(((16 - (reinterpret_cast<uintptr_t>(q) & 15)) & 15) / sizeof(T)));
    if (((reinterpret_cast<uintptr_t>(q) ^ reinterpret_cast<uintptr_t>(o)) & 15) != 0) {
        for (int i = threadIdx.x; i < len; i += THREADS) o[i] = f(q[i]);
        return;
    }
    const int nv = (len - head) / N;
    const Vec<T, N>* b = reinterpret_cast<const Vec<T, N>*>(q + head);
    Vec<T, N>* ob = reinterpret_cast<Vec<T, N>*>(o + head);
    if (nv == V * THREADS) {
        Vec<T, N> v[V];
#pragma unroll
        for (int u = 0; u < V; ++u) v[u] = b[threadIdx.x + u * THREADS];
#pragma unroll
        for (int u = 0; u < V; ++u) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[u].v[i] = f(v[u].v[i]);
            ob[threadIdx.x + u * THREADS] = v[u];
        }
    } else {
        for (int i = threadIdx.x; i < nv; i += THREADS) {
            Vec<T, N> w = b[i];
#pragma unroll
            for (int k = 0; k < N; ++k) w.v[k] = f(w.v[k]);
            ob[i] = w;
        }
    }
    if (threadIdx.x < head) o[threadIdx.x] = f(q[threadIdx.x]);
    const int tail = head + nv * N + threadIdx.x;
    if (tail < len) o[tail] = f(q[tail]);
}

template <int V>
__global__ void __launch_bounds__(THREADS)
clip_scale_k(const __grid_constant__ Table tab, const double* part, int nparts, float scale, float max_norm, float* norm,
             int write_norm) {
    double d = 0.0;
    for (int i = threadIdx.x; i < nparts; i += THREADS) d += part[i];
    const double n = (double)scale * sqrt(block_sum(d));
    if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    const bool clip = n > (double)max_norm && !isinf((float)n);  // NaN compares false
    const Factor f(clip ? (double)scale * ((double)max_norm / n) : (double)scale);
    if (tab.n == 0) return;
    // backwards: what the norm's pass read last is still in L2
    int c = tab.first[tab.n] - 1 - (int)blockIdx.x;
    for (int t = c < 0 ? 0 : tensor_of(tab, c); c >= 0; c -= gridDim.x) {
        while (c < tab.first[t]) --t;
        if (tab.in[t] == tab.out[t] && f.high == 1.f && f.low == 1.f) continue;
        const long long e = chunk_elems(tab.dtype[t], V);
        const long long e0 = (c - tab.first[t]) * e, e1 = min(tab.size[t], e0 + e);
        switch (tab.dtype[t]) {
            case VF_F32: chunk_scale<float, V>((const float*)tab.in[t], (float*)tab.out[t], e0, e1, f); break;
            case VF_BF16:
                chunk_scale<__nv_bfloat16, V>((const __nv_bfloat16*)tab.in[t], (__nv_bfloat16*)tab.out[t], e0, e1, f);
                break;
            default: chunk_scale<__half, V>((const __half*)tab.in[t], (__half*)tab.out[t], e0, e1, f); break;
        }
    }
}

// One sum for many partial sums, in a fixed order.
__global__ void __launch_bounds__(THREADS) clip_join_k(double* part, int nparts, double* sum) {
    double d = 0.0;
    for (int i = threadIdx.x; i < nparts; i += THREADS) d += part[i];
    const double s = block_sum(d);
    if (threadIdx.x == 0) *sum = s;
}

cudaError_t grid_limit(int* blocks) {
    int sms = 0;
    const cudaError_t e = device_sms(&sms);
    *blocks = sms * BLOCKS_PER_SM;
    return e;
}

// Fills `tab` with tensors from index *t on, as many as fit; advances *t.
void fill(const ClipList& l, int* t, Table* tab, int V) {
    tab->n = 0;
    tab->first[0] = 0;
    for (; *t < l.n && tab->n < MAX_TENSORS; ++*t) {
        if (l.size[*t] == 0) continue;
        const int k = tab->n;
        const long long e = chunk_elems(l.dtype[*t], V);
        const long long chunks = (l.size[*t] + e - 1) / e;
        if (tab->first[k] + chunks > 0x7fffffffLL) break;  // chunk numbers stay ints; the next launch takes it
        tab->in[k] = l.in[*t];
        tab->out[k] = l.out[*t];
        tab->size[k] = l.size[*t];
        tab->dtype[k] = (unsigned char)l.dtype[*t];
        tab->first[k + 1] = tab->first[k] + (int)chunks;
        tab->n = k + 1;
    }
}

}  // namespace

long long clip_work_doubles(int n, int sms) {
    // a launch ends early only when 2^31 chunks (32 TiB) are reached, so ceil(n / MAX_TENSORS) launches always do
    return (long long)std::max(1, (n + MAX_TENSORS - 1) / MAX_TENSORS) * sms * BLOCKS_PER_SM + 1;  // and clip_join_k's
}

cudaError_t launch_clip(const ClipList& l, float scale, float max_norm, float* norm, double* work, cudaStream_t s) {
    int limit = 0;
    cudaError_t e = grid_limit(&limit);
    if (e != cudaSuccess) return e;
    long long bytes = 0;
    for (int t = 0; t < l.n; ++t) bytes += l.size[t] * (l.dtype[t] == VF_F32 ? 4 : 2);
    // First pass: a fixed number of blocks, each with a partial sum. Eight loads in flight per thread pay where the list
    // is long (560 MB: 92 us against 98 us with four), four leave more blocks to a short one.
    const int V = bytes >= (64LL << 20) ? 8 : 4;
    Table tab;
    int parts = 0;
    for (int t = 0; t < l.n;) {
        fill(l, &t, &tab, V);
        if (tab.n == 0) continue;
        const int grid = std::min(tab.first[tab.n], limit);
        if (V == 8)
            clip_norm_k<8><<<grid, THREADS, 0, s>>>(tab, work + parts);
        else
            clip_norm_k<4><<<grid, THREADS, 0, s>>>(tab, work + parts);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        parts += grid;
    }
    if (parts > limit) {  // every block of the second pass adds the partial sums: not those of many launches
        clip_join_k<<<1, THREADS, 0, s>>>(work, parts, work + parts);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        work += parts;
        parts = 1;
    }
    // Second pass: 32 blocks per SM, four times what is resident. Blocks that come and go spread reads and writes better
    // (560 MB read and written: 173 us, with eight blocks per SM 188 us); one per chunk would cost 30 us in blocks alone
    // where nothing is left to write.
    bool wrote = false;
    for (int t = 0; t < l.n || !wrote;) {
        fill(l, &t, &tab, V);
        if (tab.n == 0 && wrote) continue;
        const int grid = std::max(1, std::min(tab.first[tab.n], 4 * limit));
        if (V == 8)
            clip_scale_k<8><<<grid, THREADS, 0, s>>>(tab, work, parts, scale, max_norm, norm, wrote ? 0 : 1);
        else
            clip_scale_k<4><<<grid, THREADS, 0, s>>>(tab, work, parts, scale, max_norm, norm, wrote ? 0 : 1);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        wrote = true;
    }
    return cudaSuccess;
}

}  // namespace vf
