// Dense layer with bias, residual and activation, and its backward pass, on the FFMA units.
//
//   forward   y[m, n] = act(z[m, n]),  z[m, n] = sum_k x[m, k] W[n, k] + b[n] + r[m, n]
//   backward  g = dy act'(z);  dx[m, k] = sum_n g[m, n] W[n, k];  dW[n, k] = sum_m g[m, n] x[m, k];
//             db[n] = sum_m g[m, n];  dr = g
//
// All three products are  C[j, i] = sum_t A(i, t) B(j, t)  with i the contiguous index of the output. Operands are read
// through two strides each, so any row stride and alignment is served and nothing is staged in global memory.
#include <algorithm>

#include "vf_internal.cuh"
#include "vf_ops.cuh"

namespace vf {

namespace {

constexpr int TB = 32;        // output tile edge
constexpr int TT = 32;        // reduction slice
constexpr int THREADS = 256;  // 2 x 2 outputs per thread

// Element (row, t) of an operand at p[row * sr + t * st]; one of the strides is 1. z != nullptr: the element is
// multiplied by act'(z[row * zr + t * zt]).
template <typename T>
struct Operand {
    const T* p;
    long long sr, st;
    const T* z;
    long long zr, zt;
    long long rows;
};

template <typename T>
struct Product {
    Operand<T> A, B;  // A: rows i, B: rows j
    long long I, J, Tn;
    T* out;  // out[j * ldo + i]
    long long ldo;
    const T* bias;  // [I] or nullptr
    const T* res;   // [j * ldr + i] or nullptr
    long long ldr;
    T* zout;  // or nullptr
    long long ldz;
    long long tiles_i, tiles;
};

template <typename T>
__device__ __forceinline__ void load_slice(const Operand<T>& o, long long r0, long long t0, long long Tn, int act,
                                           float (*s)[TB + 1]) {
    const bool along_t = o.st == 1;
#pragma unroll
    for (int e = 0; e < TB * TT / THREADS; ++e) {
        const int idx = threadIdx.x + e * THREADS;
        const int a = idx & 31, c = idx >> 5;  // a: along the contiguous index
        const int r = along_t ? c : a, t = along_t ? a : c;
        float v = 0.f;
        if (r0 + r < o.rows && t0 + t < Tn) {
            v = to_f32(o.p[(r0 + r) * o.sr + (t0 + t) * o.st]);
            if (o.z != nullptr) v = act_grad<sizeof(T) == 2>(v, to_f32(o.z[(r0 + r) * o.zr + (t0 + t) * o.zt]), act);
        }
        s[t][r] = v;
    }
}

template <typename T>
__device__ void product_tile(const Product<T>& p, long long tile, int act_in, int act_out) {
    __shared__ float As[TT][TB + 1], Bs[TT][TB + 1];
    const long long i0 = (tile % p.tiles_i) * TB, j0 = (tile / p.tiles_i) * TB;
    const int ti = threadIdx.x & 15, tj = threadIdx.x >> 4;  // outputs i = ti, ti + 16; j = tj, tj + 16
    float acc[2][2] = {};
    for (long long t0 = 0; t0 < p.Tn; t0 += TT) {
        load_slice(p.A, i0, t0, p.Tn, act_in, As);
        load_slice(p.B, j0, t0, p.Tn, act_in, Bs);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float a0 = As[t][ti], a1 = As[t][ti + 16], b0 = Bs[t][tj], b1 = Bs[t][tj + 16];
            acc[0][0] = fmaf(a0, b0, acc[0][0]);
            acc[0][1] = fmaf(a0, b1, acc[0][1]);
            acc[1][0] = fmaf(a1, b0, acc[1][0]);
            acc[1][1] = fmaf(a1, b1, acc[1][1]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const long long i = i0 + ti + 16 * u;
        if (i >= p.I) continue;
        const float bias = p.bias != nullptr ? to_f32(p.bias[i]) : 0.f;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const long long j = j0 + tj + 16 * v;
            if (j >= p.J) continue;
            float z = acc[u][v] + bias;
            if (p.res != nullptr) z += to_f32(p.res[j * p.ldr + i]);
            if (p.zout != nullptr) p.zout[j * p.ldz + i] = from_f32<T>(z);
            p.out[j * p.ldo + i] = from_f32<T>(act_value<sizeof(T) == 2>(z, act_out));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(THREADS) linear_ffma_k(Product<T> p, int act) {
    for (long long t = blockIdx.x; t < p.tiles; t += gridDim.x) product_tile(p, t, VF_ACT_NONE, act);
}

// Column sums of g (32 columns per block, eight rows in flight, joined in a fixed order) and dr = g.
template <typename T>
__device__ void column_tile(const Operand<T>& g, long long N, long long M, long long tile, int act, T* db, T* dr,
                            long long lddr) {
    __shared__ float part[THREADS / 32][33];
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
    const long long n = tile * 32 + c;
    float s = 0.f;
    if (n < N)
        for (long long m = q; m < M; m += THREADS / 32) {
            float v = to_f32(g.p[m * g.st + n]);
            if (g.z != nullptr) v = act_grad<sizeof(T) == 2>(v, to_f32(g.z[m * g.zt + n]), act);
            if (dr != nullptr) dr[m * lddr + n] = from_f32<T>(v);
            s += v;
        }
    part[q][c] = s;
    __syncthreads();
    if (q == 0 && n < N && db != nullptr) {
        float t = 0.f;
#pragma unroll
        for (int u = 0; u < THREADS / 32; ++u) t += part[u][c];
        db[n] = from_f32<T>(t);
    }
    __syncthreads();
}

// One launch for the whole backward pass: tiles of dx, then of dW, then column tiles for db and dr.
template <typename T>
__global__ void __launch_bounds__(THREADS)
linear_grad_ffma_k(Product<T> dx, Product<T> dW, long long col_tiles, T* db, T* dr, long long lddr, int act) {
    const long long all = dx.tiles + dW.tiles + col_tiles;
    for (long long t = blockIdx.x; t < all; t += gridDim.x) {
        if (t < dx.tiles)
            product_tile(dx, t, act, VF_ACT_NONE);
        else if (t < dx.tiles + dW.tiles)
            product_tile(dW, t - dx.tiles, act, VF_ACT_NONE);
        else
            column_tile(dW.B, dW.J, dW.Tn, t - dx.tiles - dW.tiles, act, db, dr, lddr);
    }
}

template <typename T>
void set_tiles(Product<T>& p, bool on) {
    p.tiles_i = (p.I + TB - 1) / TB;
    p.tiles = on ? p.tiles_i * ((p.J + TB - 1) / TB) : 0;
}

constexpr long long MAX_GRID = 1LL << 20;

template <typename T>
cudaError_t fwd(const LinearFwd& f, cudaStream_t s) {
    Product<T> p{};
    p.I = f.N;
    p.J = f.M;
    p.Tn = f.K;
    p.A = Operand<T>{(const T*)f.W, f.ldw, 1, nullptr, 0, 0, f.N};
    p.B = Operand<T>{(const T*)f.x, f.ldx, 1, nullptr, 0, 0, f.M};
    p.out = (T*)f.y;
    p.ldo = f.ldy;
    p.bias = (const T*)f.b;
    p.res = (const T*)f.r;
    p.ldr = f.ldr;
    p.zout = (T*)f.z;
    p.ldz = f.ldz;
    set_tiles(p, true);
    if (p.tiles == 0) return cudaSuccess;
    linear_ffma_k<T><<<(unsigned)std::min(p.tiles, MAX_GRID), THREADS, 0, s>>>(p, f.act);
    return cudaGetLastError();
}

template <typename T>
cudaError_t grad(const LinearGrad& f, cudaStream_t s) {
    const T* z = f.act == VF_ACT_NONE ? nullptr : (const T*)f.z;
    Product<T> dx{}, dW{};
    dx.I = f.K;
    dx.J = f.M;
    dx.Tn = f.N;
    dx.A = Operand<T>{(const T*)f.W, 1, f.ldw, nullptr, 0, 0, f.K};
    dx.B = Operand<T>{(const T*)f.dy, f.lddy, 1, z, f.ldz, 1, f.M};
    dx.out = (T*)f.dx;
    dx.ldo = f.lddx;
    dW.I = f.K;
    dW.J = f.N;
    dW.Tn = f.M;
    dW.A = Operand<T>{(const T*)f.x, 1, f.ldx, nullptr, 0, 0, f.K};
    dW.B = Operand<T>{(const T*)f.dy, 1, f.lddy, z, 1, f.ldz, f.N};
    dW.out = (T*)f.dW;
    dW.ldo = f.lddw;
    set_tiles(dx, f.dx != nullptr);
    set_tiles(dW, f.dW != nullptr);
    const long long cols = (f.db != nullptr || f.dr != nullptr) ? ((long long)f.N + 31) / 32 : 0;
    const long long all = dx.tiles + dW.tiles + cols;
    if (all == 0) return cudaSuccess;
    linear_grad_ffma_k<T><<<(unsigned)std::min(all, MAX_GRID), THREADS, 0, s>>>(dx, dW, cols, (T*)f.db, (T*)f.dr,
                                                                               f.lddr, f.act);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_ffma(const LinearFwd& p, cudaStream_t s) {
    switch (p.dtype) {
        case VF_F32: return fwd<float>(p, s);
        case VF_BF16: return fwd<__nv_bfloat16>(p, s);
        default: return fwd<__half>(p, s);
    }
}

cudaError_t launch_linear_grad_ffma(const LinearGrad& p, cudaStream_t s) {
    switch (p.dtype) {
        case VF_F32: return grad<float>(p, s);
        case VF_BF16: return grad<__nv_bfloat16>(p, s);
        default: return grad<__half>(p, s);
    }
}

}  // namespace vf
