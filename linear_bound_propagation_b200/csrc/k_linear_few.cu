// The dense layer for a few rows on the FFMA units: forward for up to eight, backward for up to 16 of fp32 and eight of 16 bits.
//
// Backward.
// With so few rows the pass is W read once (dx = g W) and dW written once (dW = g^T x): 2 N K elements against 4 M N K
// operations, bound by memory and, from eight rows on, by the FFMA units. A block takes a slab of rows n and a chunk of
// columns k of one of the two; g of the slab is formed in shared memory (fp32, not rounded), a warp passes over the slab's
// rows with its accumulators (or its part of x) in registers. dx of a slab is a partial sum; a second launch adds the slabs
// in a fixed order. db and dr come from the first chunk's blocks. One block for both products kept W's loads waiting behind
// twice the registers: 8 x 4096 x 4096 bf16 52 us, apart 36 us; with the inputs' g together in shared memory (a load for
// four of them) and the blocks chosen below 24.7 us.
//
// Measured here and on the tensor cores (k_linear_tc.cu), which pad the rows to 16, with relu in us out of L2:
//   bf16   x 4096 x 4096   1: 12.7 and 29.3   4: 14.7 and 29.3   8: 25.1 and 29.3   8 x 1024 x 1024: 7.9 and 9.8
//   fp32   x 4096 x 4096   1: 23.9 and 89.5   8: 36.1 and 89.7  16: 57.4 and 90.3  16 x 1024 x 1024: 10.0 and 14.1
// One row: 2 N K elements in 23.9 us (fp32, 5.6 TB/s) and 12.7 us (bf16, 5.3 TB/s); with W out of HBM 28.0 and 22.4 us (tensor
// cores 89.4 and 30.7), eight rows of bf16 30.6 (30.9).
#include <algorithm>

#include "linear_tc.cuh"
#include "vf_internal.cuh"
#include "vf_ops.cuh"

namespace vf {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int max_rows(int elem) { return elem == 4 ? 16 : 8; }
// Columns of g in shared memory, 32 KB of them at most for `rows` rows of inputs (a power of two).
constexpr int max_slab(int rows) { return 8192 / rows; }
// M rounded up to what the kernel is built for.
int rows_built(int M) {
    int r = 1;
    while (r < M) r *= 2;
    return r;
}

struct FewParams {
    const void *dy, *z, *x, *W;
    long long lddy, ldz, ldx, ldw;
    int M, N, K, act;
    void *dx, *dW, *db, *dr;
    long long lddx, lddw, lddr;
    float* part;  // [slab][M][K], or nullptr: one slab, dx is written as it is
    int slab;     // rows of a slab
    int dx_z;     // blockIdx.z of the blocks for dx (the others: dW, db and dr), -1: none
};

// VEC consecutive elements of a row (16 bytes, or one element where rows are not aligned).
template <typename T, int VEC>
__device__ __forceinline__ void load_row(const T* p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = to_f32(p[0]);
    } else if constexpr (sizeof(T) == 4) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
        unpack8(*reinterpret_cast<const Pack8<T>*>(p), v);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        p[0] = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        Pack8<T> q;
        pack8(q, v);
        *reinterpret_cast<Pack8<T>*>(p) = q;
    }
}

// g of one row of W, all MB inputs: they lie together in shared memory, so that a warp gets four of them per load.
template <int MB>
__device__ __forceinline__ void load_g(const float* p, float (&v)[MB]) {
    if constexpr (MB >= 4) {
#pragma unroll
        for (int m = 0; m < MB; m += 4) {
            const float4 q = *reinterpret_cast<const float4*>(p + m);
            v[m] = q.x, v[m + 1] = q.y, v[m + 2] = q.z, v[m + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int m = 0; m < MB; ++m) v[m] = p[m];
    }
}
template <int MB>
__device__ __forceinline__ void store_g(float* p, const float (&v)[MB]) {
    if constexpr (MB >= 4) {
#pragma unroll
        for (int m = 0; m < MB; m += 4) *reinterpret_cast<float4*>(p + m) = make_float4(v[m], v[m + 1], v[m + 2], v[m + 3]);
    } else {
#pragma unroll
        for (int m = 0; m < MB; ++m) p[m] = v[m];
    }
}

// Inputs whose partial sums of dx the warps of a block join at a time: 16 KB of shared memory at most.
template <int VEC, int MB>
constexpr int join_rows() {
    return VEC == 8 ? (MB < 2 ? MB : 2) : (MB < 4 ? MB : 4);
}

template <typename T, int VEC, int MB>
__global__ void __launch_bounds__(THREADS, MB * VEC >= 64 || MB == 16 ? 2 : 1)
linear_few_grad_k(const __grid_constant__ FewParams P) {
    extern __shared__ __align__(16) float g[];  // [slab][MB], then [join_rows][WARPS][32 * VEC] for the sum over the warps
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int k = (blockIdx.x * 32 + lane) * VEC;
    const int n0 = blockIdx.y * P.slab, rows = min(P.slab, P.N - n0);
    const bool is_dx = (int)blockIdx.z == P.dx_z, first = !is_dx && blockIdx.x == 0;
    lin::grid_trigger();
    for (int i = threadIdx.x; i < rows; i += THREADS) {
        float v[MB], sum = 0.f;
#pragma unroll
        for (int m = 0; m < MB; ++m) v[m] = m < P.M ? to_f32(((const T*)P.dy)[m * P.lddy + n0 + i]) : 0.f;
        if (P.act != VF_ACT_NONE) {
            float z[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) z[m] = m < P.M ? to_f32(((const T*)P.z)[m * P.ldz + n0 + i]) : 0.f;
#pragma unroll
            for (int m = 0; m < MB; ++m) v[m] = act_grad<sizeof(T) == 2>(v[m], z[m], P.act);
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            sum += v[m];
            if (first && P.dr != nullptr && m < P.M) ((T*)P.dr)[m * P.lddr + n0 + i] = from_f32<T>(v[m]);
        }
        store_g<MB>(g + i * MB, v);
        if (first && P.db != nullptr) ((T*)P.db)[n0 + i] = from_f32<T>(sum);
    }
    __syncthreads();
    if (is_dx) {
        float acc[MB][VEC] = {};
        if (k < P.K) {
            const T* W = (const T*)P.W + (long long)n0 * P.ldw + k;
#pragma unroll 4
            for (int r = warp; r < rows; r += WARPS) {
                float w[VEC], gr[MB];
                load_row<T, VEC>(W + (long long)r * P.ldw, w);
                load_g<MB>(g + r * MB, gr);
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int u = 0; u < VEC; ++u) acc[m][u] = fmaf(gr[m], w[u], acc[m][u]);
            }
        }
        constexpr int R = join_rows<VEC, MB>(), COLS = 32 * VEC;
        float* red = g + MB * P.slab;
#pragma unroll
        for (int m0 = 0; m0 < MB; m0 += R) {
            if (m0 >= P.M) break;
            __syncthreads();
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int u = 0; u < VEC; ++u) red[(m * WARPS + warp) * COLS + lane * VEC + u] = acc[m0 + m][u];
            __syncthreads();
            for (int e = threadIdx.x; e < R * COLS; e += THREADS) {
                const int m = e / COLS, c = blockIdx.x * COLS + e % COLS;
                if (m0 + m >= P.M || c >= P.K) continue;
                float s = 0.f;
#pragma unroll
                for (int t = 0; t < WARPS; ++t) s += red[(m * WARPS + t) * COLS + e % COLS];
                if (P.part != nullptr)
                    P.part[((long long)blockIdx.y * P.M + m0 + m) * P.K + c] = s;
                else
                    ((T*)P.dx)[(m0 + m) * P.lddx + c] = from_f32<T>(s);
            }
        }
    } else if (P.dW != nullptr && k < P.K) {
        float x[MB][VEC];
#pragma unroll
        for (int m = 0; m < MB; ++m) load_row<T, VEC>((const T*)P.x + (m < P.M ? m : 0) * P.ldx + k, x[m]);
        T* dW = (T*)P.dW + (long long)n0 * P.lddw + k;
#pragma unroll 2
        for (int r = warp; r < rows; r += WARPS) {
            float d[VEC] = {}, gr[MB];
            load_g<MB>(g + r * MB, gr);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                if (m >= P.M) break;  // x of a row that does not exist may be infinite
#pragma unroll
                for (int u = 0; u < VEC; ++u) d[u] = fmaf(gr[m], x[m][u], d[u]);
            }
            store_row<T, VEC>(dW + (long long)r * P.lddw, d);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS)
linear_few_join_k(const float* part, int slabs, int M, int K, T* dx, long long lddx) {
    lin::grid_wait();
    const long long i = (long long)blockIdx.x * THREADS + threadIdx.x, n = (long long)M * K;
    if (i >= n) return;
    float s = 0.f;
#pragma unroll 8
    for (int t = 0; t < slabs; ++t) s += part[t * n + i];
    dx[i / K * lddx + i % K] = from_f32<T>(s);
}

struct Shape {
    int chunks, slab, slabs;
};

// Chunks of 32 vectors. Slabs: as many blocks for each product as lie beside each other on the SMs at the kernel's registers,
// but four rows a warp at least, and partial sums of dx (fp32, M rows a slab) of no more than about a quarter of W's bytes.
// M x 4096 x 4096 with 148, 296 and 592 blocks, us:
//   fp32   1: 37.3 27.5 23.6   2: 36.5 26.9 27.9   8: 40.0 35.3 39.8   12 x 1024 x 1024: 10.5 14.4 14.4
//   bf16   1: 12.4 12.8 17.0   4: 14.4 18.2 20.6   8: 24.7 27.9 34.9
Shape shape_of(int M, int N, int K, int vec, int elem) {
    Shape s;
    s.chunks = (K + 32 * vec - 1) / (32 * vec);
    const int blocks = elem == 2 || M > 8 ? 148 : M > 1 ? 296 : 592;
    const int want = std::min({std::max(1, blocks / s.chunks), (N + 4 * WARPS - 1) / (4 * WARPS), std::max(1, (int)((long long)N * elem / (16 * M)))});
    s.slab = std::min(max_slab(rows_built(M)), (N + want - 1) / want);
    s.slabs = (N + s.slab - 1) / s.slab;
    return s;
}

template <typename T>
bool rows_of(const void* p, long long ld, int vec) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % (sizeof(T) * vec) == 0 && ld % vec == 0);
}

template <typename T, int VEC, int MB>
cudaError_t launch_mb(const FewParams& P, const Shape& s, cudaStream_t st) {
    const size_t smem = ((size_t)MB * s.slab + join_rows<VEC, MB>() * THREADS * VEC) * sizeof(float);
    const bool other = P.dW != nullptr || P.db != nullptr || P.dr != nullptr;
    if (P.dx == nullptr && !other) return cudaSuccess;
    linear_few_grad_k<T, VEC, MB><<<dim3(s.chunks, s.slabs, (P.dx != nullptr) + other), THREADS, smem, st>>>(P);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_vec(const LinearGrad& f, FewParams& P, float* work, size_t have, size_t* need, cudaStream_t st) {
    const Shape s = shape_of((int)f.M, f.N, f.K, VEC, sizeof(T));
    P.slab = s.slab;
    P.dx_z = f.dx != nullptr ? 0 : -1;
    *need = f.dx != nullptr && s.slabs > 1 ? (size_t)s.slabs * f.M * f.K * sizeof(float) : 0;
    if (*need > have) return cudaSuccess;  // the caller reports it
    P.part = *need > 0 ? work : nullptr;
    cudaError_t e;
    switch (rows_built((int)f.M)) {
        case 1: e = launch_mb<T, VEC, 1>(P, s, st); break;
        case 2: e = launch_mb<T, VEC, 2>(P, s, st); break;
        case 4: e = launch_mb<T, VEC, 4>(P, s, st); break;
        case 8: e = launch_mb<T, VEC, 8>(P, s, st); break;
        default: e = launch_mb<T, VEC, max_rows(sizeof(T))>(P, s, st);  // 16, fp32 only
    }
    if (e != cudaSuccess || P.part == nullptr) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)((f.M * f.K + THREADS - 1) / THREADS));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_few_join_k<T>, (const float*)P.part, s.slabs, (int)f.M, f.K, (T*)f.dx, f.lddx);
}

template <typename T>
cudaError_t launch_few(const LinearGrad& f, float* work, size_t have, size_t* need, cudaStream_t st) {
    FewParams P{f.dy,  f.act == VF_ACT_NONE ? nullptr : f.z, f.x, f.W, f.lddy, f.ldz, f.ldx, f.ldw, (int)f.M, f.N, f.K,
                f.act, f.dx, f.dW, f.db, f.dr, f.lddx, f.lddw, f.lddr, nullptr, 0, 0};
    constexpr int V = 16 / sizeof(T);
    const bool vec = f.K % V == 0 && (f.dx == nullptr || rows_of<T>(f.W, f.ldw, V)) &&
                     (f.dW == nullptr || (rows_of<T>(f.x, f.ldx, V) && rows_of<T>(f.dW, f.lddw, V)));
    return vec ? launch_vec<T, V>(f, P, work, have, need, st) : launch_vec<T, 1>(f, P, work, have, need, st);
}

// ------------------------------------------------------------------------------------------------------- forward

constexpr int ROWS = 4;  // rows of W per group of warps

// y = act(x W^T + b + r) for M <= MB rows of x: W is read once, 2 M operations for each element, so memory bounds it. A group
// of warps takes four rows of W and shares the reduction; a lane's part of x, loaded from L1, serves the four rows, and the
// next step's part of W is on its way meanwhile. Sums are fp32 in a fixed order. 1 x 4096 x 4096 fp32 8.4 us out of L2, 18.6 us out
// of HBM.
template <typename T, int VEC, int MB>
__global__ void __launch_bounds__(THREADS, 2) linear_few_k(const __grid_constant__ LinearFwd f, int glog) {
    constexpr int C = MB * ROWS;
    __shared__ float part[WARPS][C];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, M = (int)f.M;
    // 2^glog warps share the reduction of four rows
    const int group = warp >> glog, share = warp & ((1 << glog) - 1), step = (32 << glog) * VEC;
    const long long n0 = (((long long)blockIdx.x << (3 - glog)) + group) * ROWS;
    const T* w[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) w[r] = (const T*)f.W + min(n0 + r, f.N - 1LL) * f.ldw;
    float acc[C] = {}, a[ROWS][VEC] = {}, b[ROWS][VEC] = {};  // acc[m * ROWS + r]
    long long k = (share * 32 + lane) * VEC;
    if (k < f.K)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) load_row<T, VEC>(w[r] + k, a[r]);
    while (k < f.K) {
        const T* x = (const T*)f.x + k;
        k += step;
        if (k < f.K)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) load_row<T, VEC>(w[r] + k, b[r]);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            float v[VEC];
            load_row<T, VEC>(x, v);
            if (m + 1 < M) x += f.ldx;  // rows that do not exist repeat the last; their sums are not stored
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int u = 0; u < VEC; ++u) acc[m * ROWS + r] = fmaf(v[u], a[r][u], acc[m * ROWS + r]);
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int u = 0; u < VEC; ++u) a[r][u] = b[r][u];
    }
    // Sums over the lanes: at each step a lane hands half of its sums to its partner, until each has one.
    int first = 0, c = C;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (c > 1) {
            c /= 2;
            const bool upper = (lane & o) != 0;
            first += upper ? c : 0;
#pragma unroll
            for (int i = 0; i < C / 2; ++i)
                if (i < c) {
                    const float give = upper ? acc[i] : acc[i + c], keep = upper ? acc[i + c] : acc[i];
                    acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
        } else {
            acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
        }
    }
    static_assert(C <= 32, "a lane ends with one sum");
    part[warp][first] = acc[0];  // the lanes that share a sum hold the same
    __syncthreads();
    const int g = threadIdx.x / C, m = threadIdx.x % C / ROWS;
    const long long n = (((long long)blockIdx.x << (3 - glog)) + g) * ROWS + threadIdx.x % ROWS;
    if (g >= WARPS >> glog || m >= M || n >= f.N) return;
    float z = 0.f;
    for (int t = 0; t < 1 << glog; ++t) z += part[(g << glog) + t][threadIdx.x % C];
    if (f.b != nullptr) z += to_f32(((const T*)f.b)[n]);
    if (f.r != nullptr) z += to_f32(((const T*)f.r)[m * f.ldr + n]);
    if (f.z != nullptr) ((T*)f.z)[m * f.ldz + n] = from_f32<T>(z);
    ((T*)f.y)[m * f.ldy + n] = from_f32<T>(act_value<sizeof(T) == 2>(z, f.act));
}

// All eight warps share a reduction, or fewer where there would be more than two blocks per SM and a warp fewer than four steps:
// 1 x 4096 x 1024 bf16 6.6 us with eight, 4.0 us with two (W out of HBM 9.7 and 6.1); 8 x 4096 x 4096 fp32 18.4 us with eight,
// 18.8 us with two (29.2 and 37).
template <typename T, int VEC>
cudaError_t launch_rows(const LinearFwd& f, cudaStream_t s) {
    const long long rows = (f.N + ROWS - 1LL) / ROWS;
    int glog = 3;
    while (glog > 0 && ((rows << glog) + WARPS - 1) / WARPS > 148 * 2 && f.K < 4 * (32 << glog) * VEC) --glog;
    const unsigned grid = (unsigned)(((rows << glog) + WARPS - 1) / WARPS);
    switch (rows_built((int)f.M)) {
        case 1: linear_few_k<T, VEC, 1><<<grid, THREADS, 0, s>>>(f, glog); break;
        case 2: linear_few_k<T, VEC, 2><<<grid, THREADS, 0, s>>>(f, glog); break;
        case 4: linear_few_k<T, VEC, 4><<<grid, THREADS, 0, s>>>(f, glog); break;
        default: linear_few_k<T, VEC, 8><<<grid, THREADS, 0, s>>>(f, glog);
    }
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_few_forward(const LinearFwd& f, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool vec = f.K % V == 0 && rows_of<T>(f.x, f.ldx, V) && rows_of<T>(f.W, f.ldw, V);
    return vec ? launch_rows<T, V>(f, s) : launch_rows<T, 1>(f, s);
}

}  // namespace

// Up to eight rows, in 16 bits up to 2^24 multiplications. M x N x K, us here and on the tensor cores (k_linear_direct.cu for
// fp32, k_linear_tc.cu for 16 bits; replayed from a graph, W in L2, in parentheses with W out of HBM):
//   fp32  1x1024x1024 2.6 and 7.2 (3.4 and 8.6)   1x4096x4096 8.4 and 21.5 (18.6 and 27.6)   8x4096x4096 18.4 and 21.6 (29.2 and 28.0)
//   bf16  1x1024x1024 3.0 and 6.1 (3.7 and 6.8)   1x4096x1024 4.2 and 6.1 (6.5 and 7.9)   8x2048x1024 4.6 and 6.1 (6.5 and 7.3)
//         8x4096x512 4.7 and 5.1 (6.2 and 6.4)   1x4096x4096 9.4 and 9.6 (14.5 and 14.3)   8x4096x1024 6.5 and 6.2 (9.0 and 7.9)
//         2x4096x4096 11.1 and 8.9 (16.5 and 14.2)   8x4096x4096 18.2 and 8.6 (24.1 and 13.8)
// The rule does not look at the alignment, off which this kernel loads single elements and the other side (k_linear_direct.cu in
// every type) is the faster one: bf16 4x4093x1023 12.4 and 6.1, 8x2040x1023 8.0 and 6.1, fp32 8x4093x1023 11.7 and 10.5.
bool linear_few_forward(int dtype, long long M, int N, int K) {
    return M >= 1 && M <= 8 && N >= 1 && K >= 1 && (dtype == VF_F32 || (double)M * N * K <= 16777216.0);
}

cudaError_t launch_linear_few(const LinearFwd& f, cudaStream_t s) {
    switch (f.dtype) {
        case VF_F32: return launch_few_forward<float>(f, s);
        case VF_BF16: return launch_few_forward<__nv_bfloat16>(f, s);
        default: return launch_few_forward<__half>(f, s);
    }
}

bool linear_few_supported(int dtype, long long M, int N, int K) {
    return M >= 1 && M <= max_rows(dtype == VF_F32 ? 4 : 2) && N >= 1 && K >= 1 &&
           (long long)N <= 65535LL * max_slab(rows_built((int)M));
}

size_t linear_few_workspace(int dtype, long long M, int N, int K) {
    const int e = dtype == VF_F32 ? 4 : 2;
    const int slabs = std::max(shape_of((int)M, N, K, 16 / e, e).slabs, shape_of((int)M, N, K, 1, e).slabs);
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
