// Shared by the tensor-core kernels of the dense layer (k_linear_tc.cu, k_linear_direct.cu): matrix instructions and their
// descriptors, TMEM, clusters, the epilogue's arithmetic and the join of split reductions.
#pragma once
#include <cuda.h>

#include "tc_ptx.cuh"
#include "vf_ops.cuh"

namespace vf {
namespace lin {

using namespace tc;

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

// Bounded wait like mbar_wait, without the suspend-time hint: with it a waiting warp woke late.
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

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster4(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

template <typename T>
struct alignas(16) Pack8 {
    T v[8];
};

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
#pragma unroll
    for (int u = 0; u < 8; ++u) w.v[u] = from_f32<T>(0.f);
    if (p.res == nullptr || j >= p.J) return;
    const T* r = (const T*)p.res + j * p.ldr + i;
    if (i + 8 <= p.I) {
        w = *reinterpret_cast<const Pack8<T>*>(r);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i + u < p.I) w.v[u] = r[u];
    }
}
template <typename T>
__device__ __forceinline__ void put8(T* o, int n, const float (&v)[8]) {
    Pack8<T> w;
#pragma unroll
    for (int u = 0; u < 8; ++u) w.v[u] = from_f32<T>(v[u]);
    if (n >= 8) {
        *reinterpret_cast<Pack8<T>*>(o) = w;
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (u < n) o[u] = w.v[u];
    }
}
template <typename T>
__device__ __forceinline__ void finish8(const TcProduct& p, long long i, long long j, float (&v)[8], const float (&bias)[8],
                                        const Pack8<T>& r) {
    const int n = (int)min(8LL, p.I - i);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] += bias[u] + to_f32(r.v[u]);
    if (p.zout != nullptr) put8<T>((T*)p.zout + j * p.ldz + i, n, v);
    activate<T>(v, p.act);
    put8<T>((T*)p.out + j * p.ldo + i, n, v);
}

// One element i of N rows j .. j + N - 1 per thread, a warp's lanes on consecutive elements: fp32 rows (a warp's access
// is a whole 128-byte line) and rows that do not allow 16-byte accesses.
template <typename T, int N>
__device__ __forceinline__ void res_lane(const TcProduct& p, long long i, long long j, float (&r)[N]) {
#pragma unroll
    for (int u = 0; u < N; ++u)
        r[u] = (p.res != nullptr && i < p.I && j + u < p.J) ? to_f32(((const T*)p.res)[(j + u) * p.ldr + i]) : 0.f;
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

// x = h + m + l: three bf16 by truncation, 8 significand bits each (the subtractions are exact). What is not finite gives
// a piece that is not finite, and so products that are not.
__device__ __forceinline__ void split3(float x, float& r, float& l) {
    r = x - __uint_as_float(__float_as_uint(x) & 0xffff0000u);
    l = r - __uint_as_float(__float_as_uint(r) & 0xffff0000u);
}
// The upper halves of two floats: their leading bf16 pieces.
__device__ __forceinline__ uint32_t upper2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ void split3x8(const float (&v)[8], uint4& h, uint4& m, uint4& l) {
    float r[8], t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) split3(v[u], r[u], t[u]);
    h = make_uint4(upper2(v[0], v[1]), upper2(v[2], v[3]), upper2(v[4], v[5]), upper2(v[6], v[7]));
    m = make_uint4(upper2(r[0], r[1]), upper2(r[2], r[3]), upper2(r[4], r[5]), upper2(r[6], r[7]));
    l = make_uint4(upper2(t[0], t[1]), upper2(t[2], t[3]), upper2(t[4], t[5]), upper2(t[6], t[7]));
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[8]) {
    if (vec && n >= 8) {
        const Pack8<T> w = *reinterpret_cast<const Pack8<T>*>(p);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = to_f32(w.v[u]);
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = u < n ? to_f32(p[u]) : 0.f;
    }
}

// Joins the 2^log partial tiles of a cluster (each CTA's in its shared memory at `part`: BN columns of 128 floats), each
// CTA finishing its share of the columns. Called by every thread, converged; `ew` is the warp's place among the NW that
// work (outside 0..NW-1: only the barrier). The caller joins the cluster once more before it leaves.
template <typename T, int BN, int NW>
__device__ __forceinline__ void join_cluster(const TcProduct& p, int i0, int j0, uint32_t part, int rank, int log, int ew) {
    const int S = 1 << log, lane = threadIdx.x & 31, e = ew * 32 + lane;
    const int c0 = share(BN, rank, log), c1 = share(BN, rank + 1, log);
    const long long iv = (long long)i0 + (e & 15) * 8;
    float bias[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        bias[k] = (p.vec && p.bias != nullptr && iv + k < p.I) ? to_f32(((const T*)p.bias)[iv + k]) : 0.f;
    __syncwarp();
    cluster_sync_all();
    if (ew < 0 || ew >= NW) return;
    // the loads of four ranks are issued before the first is used
    if (p.vec) {  // eight lanes of a column per thread
        for (int c = c0 + (e >> 4); c < c1; c += 2 * NW) {
            const long long j = (long long)j0 + c;
            if (iv >= p.I || j >= p.J) continue;
            Pack8<T> r;
            res8<T>(p, iv, j, r);
            float o[8] = {};
#pragma unroll
            for (int k0 = 0; k0 < 8; k0 += 4) {
                if (k0 >= S) break;
                float4 x[4][2];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k0 + k < S) {
                        x[k][0] = ld_cluster4(part + (c * BM + (e & 15) * 8) * 4, k0 + k);
                        x[k][1] = ld_cluster4(part + (c * BM + (e & 15) * 8 + 4) * 4, k0 + k);
                    }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k0 + k < S) {
                        o[0] += x[k][0].x, o[1] += x[k][0].y, o[2] += x[k][0].z, o[3] += x[k][0].w;
                        o[4] += x[k][1].x, o[5] += x[k][1].y, o[6] += x[k][1].z, o[7] += x[k][1].w;
                    }
            }
            finish8<T>(p, iv, j, o, bias, r);
        }
    } else {  // four lanes, 32 apart, of a column per thread
        for (int c = c0 + ew; c < c1; c += NW) {
            const long long j = (long long)j0 + c;
            if (j >= p.J) continue;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const long long i = (long long)i0 + k * 32 + lane;
                float x[8], o[1] = {0.f};
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < S) x[r] = ld_cluster(part + (c * BM + k * 32 + lane) * 4, r);
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < S) o[0] += x[r];
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
