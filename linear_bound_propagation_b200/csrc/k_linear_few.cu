// Backward pass of the dense layer for a few rows (M <= 8) on the FFMA units.
//
// With so few rows the pass is W read once (dx = g W) and dW written once (dW = g^T x): 2 N K elements against 4 M N K
// operations, bound by memory, and one loop over the rows of both serves both. A block takes a slab of rows n and a chunk
// of columns k: g of the slab is formed once in shared memory (fp32, not rounded), x of the chunk stays in registers, and
// each row of W and of dW passes through once. dx of a slab is a partial sum; a second launch adds the slabs in a fixed
// order. db and dr come from the first chunk's blocks.
#include <algorithm>

#include "vf_internal.cuh"
#include "vf_ops.cuh"

namespace vf {

namespace {

constexpr int THREADS = 256;
constexpr int MAX_M = 8;
constexpr int MAX_SLAB = 1024;  // rows of g in shared memory: 32 KB for eight rows of inputs

struct FewParams {
    const void *dy, *z, *x, *W;
    long long lddy, ldz, ldx, ldw;
    int M, N, K, act;
    void *dx, *dW, *db, *dr;
    long long lddx, lddw, lddr;
    float* part;  // [slab][M][K], or nullptr: one slab, dx is written as it is
    int slab;     // rows of a slab
    int tx;       // threads along k
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Row {
    T v[VEC];
};

template <typename T, int VEC, int MB>
__global__ void __launch_bounds__(THREADS) linear_few_grad_k(const __grid_constant__ FewParams P) {
    extern __shared__ float g[];  // [MB][slab], then [THREADS * VEC] for the sum over ty
    const int tx = threadIdx.x % P.tx, ty = threadIdx.x / P.tx, TY = THREADS / P.tx;
    const int k = (blockIdx.x * P.tx + tx) * VEC;
    const int n0 = blockIdx.y * P.slab, rows = min(P.slab, P.N - n0);
    for (int i = threadIdx.x; i < MB * rows; i += THREADS) {
        const int m = i / rows, n = n0 + i % rows;
        float v = 0.f;
        if (m < P.M) {
            v = to_f32(((const T*)P.dy)[m * P.lddy + n]);
            if (P.act != VF_ACT_NONE) v = act_grad<sizeof(T) == 2>(v, to_f32(((const T*)P.z)[m * P.ldz + n]), P.act);
            if (P.dr != nullptr && blockIdx.x == 0) ((T*)P.dr)[m * P.lddr + n] = from_f32<T>(v);
        }
        g[m * P.slab + i % rows] = v;
    }
    __syncthreads();
    if (P.db != nullptr && blockIdx.x == 0)
        for (int i = threadIdx.x; i < rows; i += THREADS) {
            float s = 0.f;
#pragma unroll
            for (int m = 0; m < MB; ++m) s += g[m * P.slab + i];
            ((T*)P.db)[n0 + i] = from_f32<T>(s);
        }
    const bool on = k < P.K;
    float x[MB][VEC], acc[MB][VEC];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        Row<T, VEC> r;
        if (P.dW != nullptr && on && m < P.M) r = *reinterpret_cast<const Row<T, VEC>*>((const T*)P.x + m * P.ldx + k);
#pragma unroll
        for (int u = 0; u < VEC; ++u) {
            x[m][u] = P.dW != nullptr && on && m < P.M ? to_f32(r.v[u]) : 0.f;
            acc[m][u] = 0.f;
        }
    }
    if (on) {
#pragma unroll 4
        for (int r = ty; r < rows; r += TY) {
            float w[VEC], d[VEC];
            if (P.dx != nullptr) {
                const Row<T, VEC> v = *reinterpret_cast<const Row<T, VEC>*>((const T*)P.W + (long long)(n0 + r) * P.ldw + k);
#pragma unroll
                for (int u = 0; u < VEC; ++u) w[u] = to_f32(v.v[u]);
            } else {
#pragma unroll
                for (int u = 0; u < VEC; ++u) w[u] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < VEC; ++u) d[u] = 0.f;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const float gm = g[m * P.slab + r];
#pragma unroll
                for (int u = 0; u < VEC; ++u) {
                    acc[m][u] = fmaf(gm, w[u], acc[m][u]);
                    d[u] = fmaf(gm, x[m][u], d[u]);
                }
            }
            if (P.dW != nullptr) {
                Row<T, VEC> o;
#pragma unroll
                for (int u = 0; u < VEC; ++u) o.v[u] = from_f32<T>(d[u]);
                *reinterpret_cast<Row<T, VEC>*>((T*)P.dW + (long long)(n0 + r) * P.lddw + k) = o;
            }
        }
    }
    if (P.dx == nullptr) return;
    float* red = g + MB * P.slab;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        if (m >= P.M) break;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < VEC; ++u) red[(ty * P.tx + tx) * VEC + u] = acc[m][u];
        __syncthreads();
        // the sums over ty of the chunk's tx * VEC columns
        for (int i = threadIdx.x; i < P.tx * VEC; i += THREADS) {
            const int c = blockIdx.x * P.tx * VEC + i;
            float s = 0.f;
            for (int t = 0; t < TY; ++t) s += red[t * P.tx * VEC + i];
            if (c < P.K) {
                if (P.part != nullptr)
                    P.part[((long long)blockIdx.y * P.M + m) * P.K + c] = s;
                else
                    ((T*)P.dx)[m * P.lddx + c] = from_f32<T>(s);
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
linear_few_join_k(const float* part, int slabs, int M, int K, T* dx, long long lddx) {
    const long long i = (long long)blockIdx.x * THREADS + threadIdx.x, n = (long long)M * K;
    if (i >= n) return;
    float s = 0.f;
#pragma unroll 8
    for (int t = 0; t < slabs; ++t) s += part[t * n + i];
    dx[i / K * lddx + i % K] = from_f32<T>(s);
}

struct Shape {
    int tx, chunks, slab, slabs;
};

// Threads along k: as many vectors as a row has, 32 to 256. Slabs: enough blocks to fill the SMs a few times over, none
// below four rows per thread row.
Shape shape_of(int N, int K, int vec) {
    Shape s;
    s.tx = 32;
    while (s.tx < THREADS && s.tx * vec < K) s.tx *= 2;
    s.chunks = (K + s.tx * vec - 1) / (s.tx * vec);
    const int ty = THREADS / s.tx;
    const int want = std::max(1, std::min((592 + s.chunks - 1) / s.chunks, (N + 4 * ty - 1) / (4 * ty)));
    s.slab = std::min(MAX_SLAB, (N + want - 1) / want);
    s.slabs = (N + s.slab - 1) / s.slab;
    return s;
}

template <typename T>
bool rows_of(const void* p, long long ld, int vec) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (sizeof(T) * vec) == 0 && ld % vec == 0);
}

template <typename T, int VEC, int MB>
cudaError_t launch_mb(const FewParams& P, const Shape& s, cudaStream_t st) {
    const size_t smem = ((size_t)MB * s.slab + THREADS * VEC) * sizeof(float);
    linear_few_grad_k<T, VEC, MB><<<dim3(s.chunks, s.slabs), THREADS, smem, st>>>(P);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_vec(const LinearGrad& f, FewParams& P, float* work, size_t have, size_t* need, cudaStream_t st) {
    const Shape s = shape_of(f.N, f.K, VEC);
    P.slab = s.slab;
    P.tx = s.tx;
    *need = f.dx != nullptr && s.slabs > 1 ? (size_t)s.slabs * f.M * f.K * sizeof(float) : 0;
    if (*need > have) return cudaSuccess;  // the caller reports it
    P.part = *need > 0 ? work : nullptr;
    cudaError_t e;
    if (f.M == 1)
        e = launch_mb<T, VEC, 1>(P, s, st);
    else if (f.M == 2)
        e = launch_mb<T, VEC, 2>(P, s, st);
    else if (f.M <= 4)
        e = launch_mb<T, VEC, 4>(P, s, st);
    else
        e = launch_mb<T, VEC, 8>(P, s, st);
    if (e != cudaSuccess || P.part == nullptr) return e;
    linear_few_join_k<T><<<(unsigned)((f.M * f.K + THREADS - 1) / THREADS), THREADS, 0, st>>>(P.part, s.slabs, (int)f.M, f.K,
                                                                                             (T*)f.dx, f.lddx);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_few(const LinearGrad& f, float* work, size_t have, size_t* need, cudaStream_t st) {
    FewParams P{f.dy,  f.act == VF_ACT_NONE ? nullptr : f.z, f.x, f.W, f.lddy, f.ldz, f.ldx, f.ldw, (int)f.M, f.N, f.K,
                f.act, f.dx, f.dW, f.db, f.dr, f.lddx, f.lddw, f.lddr, nullptr, 0, 0};
    const bool vec = f.K % 4 == 0 && (f.dx == nullptr || rows_of<T>(f.W, f.ldw, 4)) &&
                     (f.dW == nullptr || (rows_of<T>(f.x, f.ldx, 4) && rows_of<T>(f.dW, f.lddw, 4)));
    return vec ? launch_vec<T, 4>(f, P, work, have, need, st) : launch_vec<T, 1>(f, P, work, have, need, st);
}

}  // namespace

bool linear_few_supported(long long M, int N, int K) {
    return M >= 1 && M <= MAX_M && N >= 1 && K >= 1 && (long long)N <= 65535LL * MAX_SLAB;
}

size_t linear_few_workspace(long long M, int N, int K) {
    const Shape a = shape_of(N, K, 4), b = shape_of(N, K, 1);
    const int slabs = std::max(a.slabs, b.slabs);
    return slabs > 1 ? (size_t)slabs * M * K * sizeof(float) : 0;
}

cudaError_t launch_linear_few_grad(const LinearGrad& f, void* work, size_t have, size_t* need, cudaStream_t s) {
    switch (f.dtype) {
        case VF_F32: return launch_few<float>(f, (float*)work, have, need, s);
        case VF_BF16: return launch_few<__nv_bfloat16>(f, (float*)work, have, need, s);
        default: return launch_few<__half>(f, (float*)work, have, need, s);
    }
}

}  // namespace vf
