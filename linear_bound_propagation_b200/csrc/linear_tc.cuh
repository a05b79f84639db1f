// Shared by the tensor-core kernels of the dense layer (k_linear_tc.cu, k_linear_direct.cu): matrix instructions and their
// descriptors, TMEM, clusters, the epilogue's arithmetic and the join of split reductions.
#pragma once
#include <cuda.h>

#include "tc_ptx.cuh"
#include "vf_ops.cuh"

namespace vf {
namespace lin {

using namespace tc;

// 16-bit operands: steps of the reduction that one accumulator in TMEM adds up before it is added to the others in registers,
// rounding to nearest. An MMA (16 steps) cuts what it adds, by 1.9e-7 of the sum in float16 and 1.1e-7 in bf16 on average for
// positive terms: 1.2e-5 and 7e-6 of the result over 128 of them, a twentieth of float16's half step. Kept there for the whole
// reduction, 60000 terms came out 9.6e-5 low and the weight gradient over 2^18 rows 1.7e-3. 8192 x 4096 x 4096 bf16, gelu and z:
// 192 us; with runs of 1024 steps, whose second waits for the tile before to be written, 202 us; without runs 187 us.
constexpr int CHUNK_16 = 2048;

constexpr int BM = 128;  // rows of an MMA's A operand: lanes of TMEM, consecutive elements of an output row

struct TcProduct {
    long long I, J;      // output columns (contiguous) and rows
    int nk;              // blocks of the reduction
    int a_mn, b_mn;      // operand contiguous along i (j) instead of t
    int tiles_i;
    int tiles;
    void* out;
    long long ldo;
    const void* bias;
    const void* res;
    long long ldr;
    void* zout;
    long long ldz;
    int act;
    int vec;             // output, residual and z rows all allow 16-byte accesses (and TMA)
    int plog;            // k_linear_tc.cu: the reduction is cut into 2^plog parts, each a tile of its own
    float* sums;         // their fp32 sums, [part][J][I]
};

// Start of the r-th of 2^log parts of n blocks.
__device__ __forceinline__ int share(int n, int r, int log) { return (int)(((long long)n * r) >> log); }

// D (tmem) (+)= A (smem) x B (smem), kind::f16.
template <int CG>
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// Position in the ring of stages: slot and how often the ring has been passed. Kept as counters: the roles below are
// single threads, for which a division per block would cost more than the block's MMAs.
struct Ring {
    int slot = 0;
    uint32_t lap = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++slot == stages) {
            slot = 0;
            ++lap;
        }
    }
};

// Operand of rows x BK elements in shared memory. Contiguous along t: rows of BK elements (128 or 64 bytes, swizzled
// over as many bytes), 8-row groups one after the other. Contiguous along i or j: atoms of 64 elements x BK steps of t,
// 128-byte rows swizzled over 128 bytes, 8-step groups 1024 bytes apart, atoms BK * 128 bytes apart.
template <int BK>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr, int mn) {
    const uint64_t base = (uint64_t)((saddr >> 4) & 0x3FFF) | (1ull << 46);
    if (mn) return base | ((uint64_t)(BK * 128 / 16) << 16) | (64ull << 32) | (2ull << 61);
    return base | (1ull << 16) | ((uint64_t)(8 * BK * 2 / 16) << 32) | ((BK == 64 ? 2ull : 4ull) << 61);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]);
template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

// Bounded wait like mbar_wait, without its suspend-time hint: the roles wait for one another every few hundred cycles.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_test(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_test(bar, parity)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > WAIT_CYCLES) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// One lane of a converged warp. tcgen05 and TMA instructions take their operands from uniform registers: behind
// elect.sync the compiler knows that a single lane runs and issues them back to back; behind `lane == 0` every MMA took
// about 110 cycles to issue.
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(on));
    return on != 0;
}

// Programmatic dependent launch: grid_wait returns when the launches before have completed and their writes are seen;
// grid_trigger lets the next launch begin its prologue.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t saddr, uint32_t rank, float v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

template <typename T, int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    constexpr bool FAST = sizeof(T) == 2;
    switch (act) {
        case VF_ACT_RELU:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = act_value<FAST>(v[u], VF_ACT_RELU);
            break;
        case VF_ACT_GELU:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = act_value<FAST>(v[u], VF_ACT_GELU);
            break;
        case VF_ACT_SILU:
#pragma unroll
            for (int u = 0; u < N; ++u) v[u] = act_value<FAST>(v[u], VF_ACT_SILU);
            break;
        default: break;
    }
}

// Rows that allow 16-byte accesses: eight consecutive outputs i .. i + 7 of row j per thread. The residual is loaded
// ahead (res8) so that several rows' loads are in flight.
template <typename T>
__device__ __forceinline__ void res8(const TcProduct& p, long long i, long long j, Pack8<T>& w) {
    zero8(w);
    if (p.res != nullptr && j < p.J) load_raw8((const T*)p.res + j * p.ldr + i, (int)min(8LL, p.I - i), true, w);
}
template <typename T>
__device__ __forceinline__ void finish8(const TcProduct& p, long long i, long long j, float (&v)[8], const float (&bias)[8],
                                        const Pack8<T>& r) {
    const int n = (int)min(8LL, p.I - i);
    float x[8];
    unpack8(r, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] += bias[u] + x[u];
    Pack8<T> w;
    if (p.zout != nullptr) {
        pack8(w, v);
        store_raw8((T*)p.zout + j * p.ldz + i, n, true, w);
    }
    activate<T>(v, p.act);
    pack8(w, v);
    store_raw8((T*)p.out + j * p.ldo + i, n, true, w);
}

// One element i of N rows j .. j + N - 1 per thread, a warp's lanes on consecutive elements: fp32 rows (a warp's access
// is a whole 128-byte line) and rows that do not allow 16-byte accesses.
// The residual's N rows of one element. Addresses are clamped into the tensor instead of guarded, so that all loads are
// issued before one is used; what lies outside is never stored.
template <typename T, int N>
__device__ __forceinline__ void res_lane(const TcProduct& p, long long i, long long j, float (&r)[N]) {
    if (p.res == nullptr) {
#pragma unroll
        for (int u = 0; u < N; ++u) r[u] = 0.f;
        return;
    }
    const T* q = (const T*)p.res + min(i, p.I - 1);
    T v[N];
#pragma unroll
    for (int u = 0; u < N; ++u) v[u] = q[min(j + u, p.J - 1) * p.ldr];
#pragma unroll
    for (int u = 0; u < N; ++u) r[u] = to_f32(v[u]);
}
template <typename T, int N>
__device__ __forceinline__ void finish_lane(const TcProduct& p, long long i, long long j, float (&v)[N], float bias,
                                            const float (&r)[N]) {
    if (i >= p.I) return;
    const int n = (int)min((long long)N, p.J - j);
#pragma unroll
    for (int u = 0; u < N; ++u) v[u] += bias + r[u];
    if (p.zout != nullptr) {
        T* z = (T*)p.zout + j * p.ldz + i;
#pragma unroll
        for (int u = 0; u < N; ++u)
            if (u < n) z[u * p.ldz] = from_f32<T>(v[u]);
    }
    activate<T>(v, p.act);
    T* o = (T*)p.out + j * p.ldo + i;
#pragma unroll
    for (int u = 0; u < N; ++u)
        if (u < n) o[u * p.ldo] = from_f32<T>(v[u]);
}

// x = h + m + l: three bf16, each what is left rounded to nearest, of 8 significand bits. The subtractions are exact, |m| is at most
// 2^-8 and |l| at most 2^-17 of x's leading power of two, so l holds the rest. (Pieces cut instead of rounded leave twice as
// much in m and l, all of x's sign: products without m l and l m then came out low by up to 4.7e-7.) What bf16 would round to
// infinity is cut. An infinity or NaN goes to l alone: a piece that is not finite meets h of the other operand, which is zero
// only where that is zero, so the product is the one of fp32 (infinity times infinity excepted: NaN), and none of another sign.
// Of values below 2^-110 the pieces hold what lies above 2^-133, bf16's last place (the MMAs take its subnormal numbers as they are).
constexpr float LARGEST_ROUNDED = 0x1.fefffep127f;  // the largest fp32 value that bf16 rounds to a finite one
__device__ __forceinline__ uint32_t round2(float a, float b) {
    const __nv_bfloat162 w = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&w);
}
// The pieces as floats.
__device__ __forceinline__ void split3(float x, float& h, float& m, float& l) {
    h = __uint_as_float(round2(x, 0.f) << 16);
    const bool finite = fabsf(x) < __uint_as_float(0x7f800000u);
    if (!(fabsf(x) <= LARGEST_ROUNDED)) h = finite ? __uint_as_float(__float_as_uint(x) & 0xffff0000u) : 0.f;
    const float r = x - h;
    m = finite ? __uint_as_float(round2(r, 0.f) << 16) : 0.f;
    l = __uint_as_float(round2(r - m, 0.f) << 16);
}
// The upper halves of two floats.
__device__ __forceinline__ uint32_t upper2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ void split3x8(const float (&v)[8], uint4& h, uint4& m, uint4& l) {
    uint32_t hw[4], mw[4], lw[4];
    float big = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) big = max_nan(big, fabsf(v[u]));
    if (big <= LARGEST_ROUNDED) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float a = v[2 * u], b = v[2 * u + 1];
            hw[u] = round2(a, b);
            const float ra = a - __uint_as_float(hw[u] << 16), rb = b - __uint_as_float(hw[u] & 0xffff0000u);
            mw[u] = round2(ra, rb);
            lw[u] = round2(ra - __uint_as_float(mw[u] << 16), rb - __uint_as_float(mw[u] & 0xffff0000u));
        }
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float ha, ma, la, hb, mb, lb;
            split3(v[2 * u], ha, ma, la);
            split3(v[2 * u + 1], hb, mb, lb);
            hw[u] = upper2(ha, hb);
            mw[u] = upper2(ma, mb);
            lw[u] = upper2(la, lb);
        }
    }
    h = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    m = make_uint4(mw[0], mw[1], mw[2], mw[3]);
    l = make_uint4(lw[0], lw[1], lw[2], lw[3]);
}

// Split reductions. Each of the 2^log CTAs of a cluster finishes its share of the tile's BN columns; its shared memory at
// `inbox` (BN x 512 bytes, used for nothing else) receives the others' partial sums of these columns, one slab of
// share x 128 floats per sender. The cluster meets twice: every CTA has begun (arrive at the start, wait before the first
// push), and every push has landed. Nothing is read from another CTA, so each leaves when it has finished.
template <int BN>
__device__ __forceinline__ void push_column(uint32_t inbox, int c, int lane128, int rank, int log, float v) {
    constexpr int LOG_BN = BN == 16 ? 4 : BN == 32 ? 5 : BN == 64 ? 6 : BN == 128 ? 7 : 8;
    const int w = BN >> log;  // columns of a share; BN is at least 16, the cluster at most 8
    const int owner = c >> (LOG_BN - log), cl = c & (w - 1);
    st_cluster(inbox + ((rank * w + cl) * BM + lane128) * 4, owner, v);
}
// Called by every thread, converged, after its pushes; `ew` is the warp's place among the NW that work.
template <typename T, int BN, int NW>
__device__ __forceinline__ void join_cluster(const TcProduct& p, int i0, int j0, const float* inbox, int rank, int log, int ew) {
    const int S = 1 << log, lane = threadIdx.x & 31, e = ew * 32 + lane, w = BN >> log;
    const long long iv = (long long)i0 + (e & 15) * 8;
    float bias[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        bias[k] = (p.vec && p.bias != nullptr && iv + k < p.I) ? to_f32(((const T*)p.bias)[iv + k]) : 0.f;
    __syncwarp();
    cluster_sync_all();
    if (ew < 0 || ew >= NW) return;
    if (p.vec) {  // eight lanes of a column per thread
        for (int c = e >> 4; c < w; c += 2 * NW) {
            const long long j = (long long)j0 + rank * w + c;
            if (iv >= p.I || j >= p.J) continue;
            Pack8<T> r;
            res8<T>(p, iv, j, r);
            float o[8] = {};
            for (int k = 0; k < S; ++k) {  // rank order
                const float4* x = reinterpret_cast<const float4*>(inbox + (k * w + c) * BM + (e & 15) * 8);
                const float4 a = x[0], b = x[1];
                o[0] += a.x, o[1] += a.y, o[2] += a.z, o[3] += a.w;
                o[4] += b.x, o[5] += b.y, o[6] += b.z, o[7] += b.w;
            }
            finish8<T>(p, iv, j, o, bias, r);
        }
    } else {  // four lanes, 32 apart, of a column per thread
        for (int c = ew; c < w; c += NW) {
            const long long j = (long long)j0 + rank * w + c;
            if (j >= p.J) continue;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const long long i = (long long)i0 + k * 32 + lane;
                float o[1] = {0.f};
                for (int r = 0; r < S; ++r) o[0] += inbox[(r * w + c) * BM + k * 32 + lane];
                const float bl = (p.bias != nullptr && i < p.I) ? to_f32(((const T*)p.bias)[i]) : 0.f;
                float res[1];
                res_lane<T>(p, i, j, res);
                finish_lane<T>(p, i, j, o, bl, res);
            }
        }
    }
}

}  // namespace lin
}  // namespace vf
