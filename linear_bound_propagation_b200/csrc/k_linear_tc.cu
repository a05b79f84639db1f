// Dense layer and its backward pass on the 5th-generation tensor cores (sm_100a): tcgen05.mma kind::f16, operands
// staged by TMA, fp32 accumulators in TMEM.
//
// Every product here is  C[j, i] = sum_t A(i, t) B(j, t)  with i the contiguous index of the output:
//   forward  y[m, n]  : i = n, j = m, t = k;  A = W and B = x, both contiguous along t
//   dx[m, k]          : i = k, j = m, t = n;  A = W contiguous along i, B = g contiguous along t
//   dW[n, k]          : i = k, j = n, t = m;  A = x contiguous along i, B = g contiguous along j
// The tensor cores take either order of either operand (the descriptors' major bits), so nothing is transposed. i runs
// along the MMA's M (128 TMEM lanes), j along its N: the small dimension of a call of few rows is the one that can be
// as narrow as 16 columns, and a warp's 32 lanes hold consecutive elements of an output row.
//
// fp32 (PL = 3): x = h + m + l, three bf16 pieces of 8 significand bits each, rounded to nearest, so the pieces hold all 24
// bits and bf16's exponent range is fp32's. Six of the nine products are formed (h h, h m, m h, m m, h l, l h); the
// three left out are at most 2^-24 of the product together, of either sign. An MMA cuts what it adds to its accumulator
// (linear_tc.cuh), so the five small products go to an accumulator of their own, and both are added to registers, rounding to
// nearest: h h every 256 steps, the small ones every COR_CHUNKS chunks. Error against 64 bits (2-norm, in parentheses a plain
// fp32 product): signed normal values 2.3e-7 (5.7e-7) at a reduction of 1024 and 2.4e-7 (1.1e-6) at 4096; positive ones 3.8e-7
// (4.9e-7 and 9.9e-7) at either, nearly all of it low by 3.8e-7.
//
// Roles (one CTA per SM, or a pair of CTAs on two SMs for 256 x 256 tiles; persistent over the tiles): warp 0 TMA
// producer, warp 1 MMA issuer, warps 2 and up epilogue (lane quarter warp % 4 of TMEM, four warps to a share of the
// tile's columns; warp 2 owns the TMEM allocation).
// When the tiles are too few to fill the SMs, the reduction is split over a cluster of 2, 4 or 8 CTAs, which
// join their partial tiles through distributed shared memory in rank order. All waits are bounded: on expiry an abort
// flag stops every role, copies and MMAs in flight are waited for (also bounded), TMEM is freed and a device flag set.
#include <cuda.h>

#include <algorithm>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include "linear_tc.cuh"
#include "vf_internal.cuh"
#include "vf_ops.cuh"

namespace vf {

namespace {

using namespace tc;
using namespace lin;

__device__ int g_ops_timeout;

// Epilogue warps: 16 behind the 256-column tiles, each with a quarter of the columns of its 32 lanes, 8 with half of them,
// or 4 with all of a narrow tile's.
template <int BN>
constexpr int epi_warps() {
    return BN == 256 ? 16 : BN >= 64 ? 8 : 4;
}
template <int BN>
constexpr int threads_of() {
    return 64 + 32 * epi_warps<BN>();
}
constexpr int MAX_STAGES = 8;
constexpr int SMEM_LIMIT = 232448;  // 227 KB, static shared memory included
constexpr int COR_CHUNKS = 8;  // fp32: chunks between two additions of the small products' accumulator

template <int PL>
constexpr int block_k() {
    return PL == 3 ? 32 : 64;
}

struct TcParams {
    TcProduct p[2];      // the longer reduction first
    int gap;             // tiles of p[1] that take about as long as one of p[0]
    int workers;         // CTAs, pairs or clusters that walk the tiles
    int split, split_log;  // CTAs per tile (cluster size), a power of two
    int stages;
    const float* unscale;  // float16: what the sums are multiplied by, a power of two; or nullptr
    int test_stall;        // tests only: the first CTA never makes its first copies, so that a bounded wait expires
    // column sums of g, joined here: db[n] = sum_q part[q * N + n]
    const float* part;
    int nparts, N;
    void* db;
};

// Tile number u of a product: its part of the reduction, its place among the tiles, and its blocks kb0 .. kb1 - 1 of the
// reduction (of a part, or of a CTA's share where a cluster splits it).
struct Place {
    int part, i, j, kb0, kb1;
    __device__ __forceinline__ Place(const TcParams& P, const TcProduct& p, int u, int rank) {
        part = u & ((1 << p.plog) - 1);
        u >>= p.plog;
        j = u / p.tiles_i;
        i = u - j * p.tiles_i;
        const int r = P.split > 1 ? rank : part, log = P.split > 1 ? P.split_log : p.plog;
        kb0 = share(p.nk, r, log);
        kb1 = share(p.nk, r + 1, log);
    }
};

// Tensor maps of a launch: operands, and where rows allow TMA the outputs, the residual and z of p[0].
struct Maps {
    CUtensorMap a[2], b[2], out[2], res, z;
};

// The tiles of worker w, the same for every role: its turns through p[0], then through p[1], where the workers that the
// last, partial turn through p[0] left out begin with `gap` tiles of p[1] each.
struct Walk {
    int w, workers, n0, n1, gap, rem, t, phase;
    __device__ __forceinline__ Walk(const TcParams& P, int worker)
        : w(worker), workers(P.workers), n0(P.p[0].tiles), n1(P.p[1].tiles), gap(P.gap), t(worker), phase(0) {
        rem = n0 % workers;
    }
    // false: no more tiles
    __device__ __forceinline__ bool next(int& prod, int& tile) {
        if (phase == 0) {
            if (t < n0) {
                prod = 0;
                tile = t;
                t += workers;
                return true;
            }
            phase = rem > 0 && w >= rem ? 1 : 2;
            t = phase == 1 ? (w - rem) * gap : w + (rem > 0 ? (workers - rem) * gap : 0);
        }
        prod = 1;
        tile = t;
        if (t >= n1 && phase == 2) return false;
        if (phase == 1) {
            if (t >= n1) return false;  // later turns begin further on still
            if (++t == (w - rem + 1) * gap) {
                phase = 2;
                t = w + (workers - rem) * gap;
            }
        } else {
            t += workers;
        }
        return true;
    }
};

// Tile of an output, a residual or z between shared memory and a 2-D map. Stores belong to the issuing thread's groups.
__device__ __forceinline__ void store_tile(const CUtensorMap* map, const void* src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// At most one store of this thread has its shared memory still to read.
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Two CTAs of a pair (CG = 2) compute one tile: the first issues the MMAs for both, so barriers that its issuer waits on
// live in its shared memory, and commits arrive in both.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
template <int CG>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
    if (CG == 1)
        mbar_arrive(bar);
    else
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar)) : "memory");
}
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if (CG == 1)
        mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void load_operand(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
            "[%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
            "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
            : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// Epilogue through TMA (tiles of 64 columns and more whose rows allow it): a warp handles its 32 lanes in rounds of
// ROUND columns, with two buffers for the residual on its way in and two for z and y on their way out, 64 KB in all.
// Split reductions have their inbox in the same place, and narrow tiles this alone.
template <int BN>
constexpr int epi_bytes() {
    return BN >= 64 ? 65536 : BN * 512;
}
template <typename T, int BN>
constexpr int epi_round() {
    return 65536 / epi_warps<BN>() / 4 / 32 / (int)sizeof(T);
}
// A pair of CTAs takes the 256-column tiles: each loads half of both operands, which halves what a CTA reads per MMA.
template <int BN>
constexpr int pair_of() {
    return BN == 256 ? 2 : 1;
}
// Blocks per stage. The issuing thread spends about 350 cycles per stage on its barriers, more than the four MMAs of a narrow
// 16-bit tile take: there a stage holds two blocks.
template <int PL, int BN>
constexpr int stage_blocks() {
    return PL == 1 && BN <= 32 ? 2 : 1;
}
template <int PL, int BN>
constexpr int stage_bytes() {
    return stage_blocks<PL, BN>() * PL * (BM + BN / pair_of<BN>()) * block_k<PL>() * 2;
}
// Stages between two additions of an accumulator to registers: 256 steps of the reduction in fp32, CHUNK_16 in 16 bits.
template <int PL, int BN>
constexpr int chunk_stages() {
    return (PL == 3 ? 256 : CHUNK_16) / (block_k<PL>() * stage_blocks<PL, BN>());
}

// N columns of this lane, 32 elements apart. The 16-bit conversions work on pairs.
template <int N>
__device__ __forceinline__ void put_lane(float* o, const float (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; ++c) o[c * 32] = v[c];
}
template <int N>
__device__ __forceinline__ void put_lane(__nv_bfloat16* o, const float (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const __nv_bfloat162 w = __floats2bfloat162_rn(v[c], v[c + 1]);
        o[c * 32] = w.x;
        o[c * 32 + 32] = w.y;
    }
}
template <int N>
__device__ __forceinline__ void put_lane(__half* o, const float (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const __half2 w = __floats2half2_rn(v[c], v[c + 1]);
        o[c * 32] = w.x;
        o[c * 32 + 32] = w.y;
    }
}

// One round of a warp: 32 lanes x N columns to shared memory, a column's 32 elements together, and on to rows
// y .. y + N - 1 of the map. Two buffers take turns: the store before last has read the one written here.
template <typename T, int N>
__device__ __forceinline__ void put_round(T* buf, const float (&v)[N], const CUtensorMap* map, int x, int y, int lane) {
    if (lane == 0) store_wait_read();
    __syncwarp();
    put_lane<N>(buf + lane, v);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) store_tile(map, buf, x, y);
}

template <typename T, int PL, int BN>
__global__ void __launch_bounds__(threads_of<BN>(), 1)
linear_tc_k(const __grid_constant__ Maps maps, const __grid_constant__ TcParams P) {
    constexpr int BK = block_k<PL>();
    constexpr int CG = pair_of<BN>();
    constexpr int BL = BN / CG;                              // rows of B that a CTA loads
    constexpr int A_PLANE = BM * BK * 2, B_PLANE = BL * BK * 2;
    constexpr int STAGE = stage_bytes<PL, BN>();
    constexpr int KS = stage_blocks<PL, BN>(), BLOCK = STAGE / KS;  // blocks of a stage lie one after the other
    constexpr int NB = (PL == 1 || BN <= 128) ? 2 : 1;       // accumulator sets in TMEM
    constexpr int CHUNK = chunk_stages<PL, BN>();
    constexpr int ACC_COLS = NB * BN;
    constexpr int USED_COLS = PL == 3 ? 2 * ACC_COLS : ACC_COLS;
    constexpr int TMEM_COLS = USED_COLS < 32 ? 32 : USED_COLS;
    constexpr int EW = epi_warps<BN>(), EPI_THREADS = 32 * EW;
    constexpr int PART = BN / (EW / 4);                      // columns of an epilogue warp
    constexpr int LD = PART < 16 ? 8 : 16;                   // columns per TMEM load
    constexpr bool EPI_TMA = BN >= 64;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2], cor_empty[2], done_bar;
    __shared__ uint64_t res_full[EW][2];
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NS = P.stages;
    const int S = CG == 1 ? P.split : 1;
    const int crank = (CG > 1 || S > 1) ? (int)cluster_rank() : 0;
    const int rank = CG == 1 ? crank : 0;   // share of a split reduction
    const int pr = CG == 2 ? crank : 0;     // place in a pair
    const int worker = CG == 2 ? blockIdx.x >> 1 : blockIdx.x >> P.split_log;

    // The producer needs the barriers only; TMEM is allocated beside its first loads.
    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], EW * CG);  // one arrival per epilogue warp
            mbar_init(&cor_empty[s], EW * CG);
        }
        for (int s = 0; s < 2 * EW; ++s) mbar_init(&res_full[s >> 1][s & 1], 1);
        mbar_init(&done_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1 && elect_one()) {
        for (int w = 0; w < 2; ++w)
            if (P.p[w].tiles > 0) {
                prefetch_map(&maps.a[w]);
                prefetch_map(&maps.b[w]);
            }
    }
    if (CG == 2) {
        __syncwarp();
        cluster_sync_all();  // the other CTA's barriers exist
    } else {
        __syncthreads();
        if (S > 1) cluster_arrive();
    }
    grid_wait();  // what the launch before wrote may be read from here on
    uint32_t tmem = 0;
    if (warp > 0) {
        if (warp == 2) {
            if (CG == 2) {
                asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                                 smem_u32(&tmem_base_sh)),
                             "r"(TMEM_COLS)
                             : "memory");
                asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
            } else {
                asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                                 smem_u32(&tmem_base_sh)),
                             "r"(TMEM_COLS)
                             : "memory");
                asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
            }
        }
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" ::"r"(32 + EPI_THREADS) : "memory");
        tc_fence_after();
        tmem = tmem_base_sh;
    }
    volatile int* abort_flag = &abort_sh;
    bool pushed = false;  // this warp has met the cluster's first barrier

    if (warp == 0) {
        if (elect_one()) {
            // ------------------------------------------------------------------------------- TMA producer
            Ring g;
            Walk walk(P, worker);
            int w, u;
            while (!*abort_flag && walk.next(w, u)) {
                const TcProduct& p = P.p[w];
                const Place at(P, p, u, rank);
                const int i0 = at.i * (BM * CG) + pr * BM, j0 = at.j * BN + pr * BL;
                const CUtensorMap* ma = &maps.a[w];
                const CUtensorMap* mb = &maps.b[w];
                const int kb0 = at.kb0, kb1 = at.kb1;
                const bool a_mn = p.a_mn, b_mn = p.b_mn;
                for (int kb = kb0; kb < kb1; ++kb, g.next(NS)) {
                    if (g.lap > 0 && !wait_phase(&empty[g.slot], (g.lap - 1) & 1, abort_flag)) break;
                    uint8_t* st = base + (size_t)g.slot * STAGE;
                    uint32_t bar = smem_u32(&full[g.slot]);
                    if (CG == 1 || pr == 0) mbar_expect_tx(&full[g.slot], STAGE * CG);
                    if (CG == 2) bar = leader_addr(&full[g.slot]);
                    if (P.test_stall && blockIdx.x == 0 && g.lap == 0 && g.slot == 0) continue;
#pragma unroll
                    for (int q = 0; q < PL * KS; ++q) {
                        // plane q % PL of block q / PL (one of the two is always one)
                        uint8_t* a = st + (q / PL) * BLOCK + (q % PL) * A_PLANE;
                        uint8_t* b = st + (q / PL) * BLOCK + PL * A_PLANE + (q % PL) * B_PLANE;
                        const int t0 = (kb * KS + q / PL) * BK;
                        if (a_mn) {
#pragma unroll
                            for (int c = 0; c < BM / 64; ++c)
                                load_operand<CG>(a + c * BK * 128, ma, bar, i0 + c * 64, t0, q % PL);
                        } else {
                            load_operand<CG>(a, ma, bar, t0, i0, q % PL);
                        }
                        if (BL >= 64 && b_mn) {
#pragma unroll
                            for (int c = 0; c < BL / 64; ++c)
                                load_operand<CG>(b + c * BK * 128, mb, bar, j0 + c * 64, t0, q % PL);
                        } else {
                            load_operand<CG>(b, mb, bar, t0, j0, q % PL);
                        }
                    }
                }
            }
            if (*abort_flag) {  // wait (bounded) for copies that nobody will consume: the last lap's
                if (CG == 2) {  // their barriers may be the other CTA's: a millisecond is enough for any of them
                    const long long t0 = clock64();
                    while (clock64() - t0 < 2000000) {
                    }
                }
                for (int h = 0; h < NS && CG == 1; ++h) {
                    const uint32_t laps = g.lap + (h < g.slot ? 1 : 0);  // copies issued into slot h
                    const long long t0 = clock64();
                    while (laps > 0 && !mbar_test(&full[h], (laps - 1) & 1) && clock64() - t0 < WAIT_CYCLES) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (pr == 0 && elect_one()) {
            // --------------------------------------------------------------------------------- MMA issuer
            Ring g, chunk, cor;  // stages; accumulator sets (a chunk each); sets of the small products (COR_CHUNKS chunks)
            bool ok = true;
            Walk walk(P, worker);
            int w, u;
            while (ok && !*abort_flag && walk.next(w, u)) {
                const TcProduct& p = P.p[w];
                const Place at(P, p, u, rank);
                const int kb0 = at.kb0, kb1 = at.kb1;
                const int a_mn = p.a_mn, b_mn = p.b_mn;
                const uint32_t fmt = (PL == 3 || std::is_same<T, __nv_bfloat16>::value) ? 1u : 0u;
                const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)a_mn << 15) |
                                       ((uint32_t)b_mn << 16) | ((uint32_t)(BN >> 3) << 17) |
                                       ((uint32_t)(BM * CG >> 4) << 24);
                // descriptors of the ring's first slot, and their steps (16-byte units) per K = 16, plane and slot
                const uint64_t a0 = operand_desc<BK>(smem_u32(base), a_mn);
                const uint64_t b0 = operand_desc<BK>(smem_u32(base) + PL * A_PLANE, b_mn);
                const uint32_t step_a = (a_mn ? 2048 : 32) / 16, step_b = (b_mn ? 2048 : 32) / 16;
                int in_chunk = 0, in_cor = 0;
                for (int kb = kb0; kb < kb1; ++kb, g.next(NS)) {
                    if (!(ok = wait_phase(&full[g.slot], g.lap & 1, abort_flag))) break;
                    const uint32_t d = tmem + (uint32_t)chunk.slot * BN;
                    const uint64_t ah = a0 + (uint32_t)(g.slot * (STAGE / 16)), bh = b0 + (uint32_t)(g.slot * (STAGE / 16));
                    if (PL == 3) {
                        if (in_cor == 0 && in_chunk == 0 && cor.lap > 0 &&
                            !(ok = wait_phase(&cor_empty[cor.slot], (cor.lap - 1) & 1, abort_flag)))
                            break;
                        tc_fence_after();
                        const uint32_t dc = tmem + ACC_COLS + (uint32_t)cor.slot * BN;
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk) {
                            const uint64_t h = ah + kk * step_a, m = h + A_PLANE / 16, l = m + A_PLANE / 16;
                            const uint64_t H = bh + kk * step_b, M = H + B_PLANE / 16, L = M + B_PLANE / 16;
                            mma_f16_ss<CG>(dc, l, H, idesc, (in_cor > 0 || in_chunk > 0 || kk > 0) ? 1u : 0u);
                            mma_f16_ss<CG>(dc, h, L, idesc, 1u);
                            mma_f16_ss<CG>(dc, m, M, idesc, 1u);
                            mma_f16_ss<CG>(dc, m, H, idesc, 1u);
                            mma_f16_ss<CG>(dc, h, M, idesc, 1u);
                        }
                    }
                    if (in_chunk == 0 && chunk.lap > 0 &&
                        !(ok = wait_phase(&acc_empty[chunk.slot], (chunk.lap - 1) & 1, abort_flag)))
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < KS * BK / 16; ++kk) {
                        const uint32_t blk = kk / (BK / 16) * (BLOCK / 16), in = kk % (BK / 16);
                        mma_f16_ss<CG>(d, ah + blk + in * step_a, bh + blk + in * step_b, idesc,
                                       (in_chunk > 0 || kk > 0) ? 1u : 0u);
                    }
                    commit<CG>(&empty[g.slot]);
                    ++in_chunk;
                    if (kb + 1 == kb1 || in_chunk == CHUNK) {
                        commit<CG>(&acc_full[chunk.slot]);
                        chunk.next(NB);
                        in_chunk = 0;
                        if (PL == 3 && (kb + 1 == kb1 || ++in_cor == COR_CHUNKS)) {
                            cor.next(NB);
                            in_cor = 0;
                        }
                    }
                }
            }
            // TMEM is never freed, nor the stages reused, under MMAs in flight: one last commit tracks them all
            if (CG == 1)
                mma_commit(&done_bar);
            else
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                                 smem_u32(&done_bar))
                             : "memory");
            const long long t0 = clock64();
            while (!mbar_test(&done_bar, 0) && clock64() - t0 < WAIT_CYCLES) {
            }
        }
    } else {
        // ------------------------------------------------------------------------------------- epilogue
        const int e = warp - 2, q = warp & 3, part_no = e >> 2;
        const uint32_t lane_base = ((uint32_t)(q * 32) << 16) + part_no * PART;
        if (P.db != nullptr)
            for (long long n = (long long)blockIdx.x * EPI_THREADS + threadIdx.x - 64; n < P.N;
                 n += (long long)gridDim.x * EPI_THREADS) {
                float s = 0.f;
#pragma unroll 16
                for (int k = 0; k < P.nparts; ++k) s += P.part[(long long)k * P.N + n];
                ((T*)P.db)[n] = from_f32<T>(s);
            }
        constexpr int ROUND = epi_round<T, BN>(), RL = ROUND < 16 ? 8 : 16;
        const float unscale = std::is_same<T, __half>::value && P.unscale != nullptr ? *P.unscale : 1.f;
        T* buf = reinterpret_cast<T*>(base + (size_t)NS * STAGE + (EPI_TMA ? e * (65536 / EW) : 0));  // 4 x 32 x ROUND
        Ring chunk, cor;      // as the MMA issuer counts them
        Ring rin;             // residual rounds consumed
        int pending = 0;      // residual rounds loaded and not yet consumed
        int ob = 0;           // output buffer in turn
        Walk walk(P, worker);
        int w, u;
        while (walk.next(w, u)) {
            const TcProduct& p = P.p[w];
            const Place at(P, p, u, rank);
            const int i0 = at.i * (BM * CG) + pr * BM + q * 32, j0 = at.j * BN + part_no * PART;
            const long long i = (long long)i0 + lane;
            const bool by_tma = EPI_TMA && S == 1 && p.vec && p.plog == 0;
            const int rounds = by_tma && i0 < p.I && j0 < p.J ? (int)min((long long)PART / ROUND, (p.J - j0 + ROUND - 1) / ROUND) : 0;
            // the residual comes in while the products run
            if (by_tma && p.res != nullptr) {
                for (int k = 0; k < 2 && k < rounds; ++k, ++pending)
                    if (lane == 0) {
                        uint64_t* bar = &res_full[e][(rin.slot + k) & 1];
                        mbar_expect_tx(bar, 32 * ROUND * sizeof(T));
                        tma_load_2d(buf + ((rin.slot + k) & 1) * 32 * ROUND, &maps.res, bar, i0, j0 + k * ROUND);
                    }
            }
            const float bias = (p.bias != nullptr && i < p.I) ? to_f32(((const T*)p.bias)[i]) : 0.f;
            float r[LD];
            if (S == 1 && !by_tma) res_lane<T>(p, i, j0, r);
            const int kb0 = at.kb0, kb1 = at.kb1;
            uint32_t acc_t = 0;  // TMEM columns that hold this warp's part of the finished tile
            bool alive = true;
            const int nc = (kb1 - kb0 + CHUNK - 1) / CHUNK;
            if (PL == 3 || nc > 1) {
                float acc[PART];
#pragma unroll
                for (int c = 0; c < PART; ++c) acc[c] = 0.f;
                for (int ch = 0; ch < nc; ++ch) {
                    if (!__all_sync(0xffffffffu, wait_phase(&acc_full[chunk.slot], chunk.lap & 1, abort_flag))) {
                        alive = false;
                        break;
                    }
                    tc_fence_after();
                    acc_t = tmem + lane_base + chunk.slot * BN;
#pragma unroll
                    for (int c = 0; c < PART; c += LD) {
                        uint32_t v[LD];
                        tmem_ld<LD>(acc_t + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < LD; ++k) acc[c + k] += __uint_as_float(v[k]);
                    }
                    if (ch + 1 < nc) {  // the last chunk's columns are released after the epilogue
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_leader<CG>(&acc_empty[chunk.slot]);
                        chunk.next(NB);
                        if (PL == 3 && (ch + 1) % COR_CHUNKS == 0) {
                            const uint32_t cor_t = tmem + lane_base + ACC_COLS + cor.slot * BN;
#pragma unroll
                            for (int c = 0; c < PART; c += LD) {
                                uint32_t v[LD];
                                tmem_ld<LD>(cor_t + c, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < LD; ++k) acc[c + k] += __uint_as_float(v[k]);
                            }
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_leader<CG>(&cor_empty[cor.slot]);
                            cor.next(NB);
                        }
                    }
                }
                if (!alive) break;
                const uint32_t cor_t = tmem + lane_base + ACC_COLS + cor.slot * BN;
#pragma unroll
                for (int c = 0; c < PART; c += LD) {  // the finished sums go back to TMEM for the rolled loops below
                    if (PL == 3) {
                        uint32_t v[LD];
                        tmem_ld<LD>(cor_t + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < LD; ++k) acc[c + k] += __uint_as_float(v[k]);
                    }
#pragma unroll
                    for (int k = 0; k < LD; k += 8) tmem_st8(acc_t + c + k, acc + c + k);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                if (PL == 3) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_leader<CG>(&cor_empty[cor.slot]);
                    cor.next(NB);
                }
            } else {
                if (!__all_sync(0xffffffffu, wait_phase(&acc_full[chunk.slot], chunk.lap & 1, abort_flag))) break;
                tc_fence_after();
                acc_t = tmem + lane_base + chunk.slot * BN;
            }
            if (S > 1) {
                cluster_wait();  // all of the cluster's CTAs have begun
#pragma unroll 1
                for (int c = 0; c < PART; c += 8) {
                    uint32_t v[8];
                    tmem_ld<8>(acc_t + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        push_column<BN>(smem_u32(base + (size_t)NS * STAGE), part_no * PART + c + k, q * 32 + lane, rank,
                                        P.split_log, __uint_as_float(v[k]) * unscale);
                }
                pushed = true;
            } else if (by_tma) {
#pragma unroll 1
                for (int k = 0; k < rounds; ++k) {
                    uint32_t v[ROUND];
#pragma unroll
                    for (int c = 0; c < ROUND; c += RL)
                        tmem_ld<RL>(acc_t + k * ROUND + c, reinterpret_cast<uint32_t(&)[RL]>(v[c]));
                    tmem_wait_ld();
                    float o[ROUND];
#pragma unroll
                    for (int c = 0; c < ROUND; ++c) o[c] = fmaf(__uint_as_float(v[c]), unscale, bias);
                    if (p.res != nullptr) {
                        alive = __all_sync(0xffffffffu, wait_phase(&res_full[e][rin.slot], rin.lap & 1, abort_flag));
                        if (!alive) break;
                        const T* rb = buf + rin.slot * 32 * ROUND + lane;
#pragma unroll
                        for (int c = 0; c < ROUND; ++c) o[c] += to_f32(rb[c * 32]);
                        __syncwarp();
                        --pending;
                        if (k + 2 < rounds) {
                            if (lane == 0) {
                                fence_proxy_async_smem();
                                mbar_expect_tx(&res_full[e][rin.slot], 32 * ROUND * sizeof(T));
                                tma_load_2d(buf + rin.slot * 32 * ROUND, &maps.res, &res_full[e][rin.slot], i0,
                                            j0 + (k + 2) * ROUND);
                            }
                            ++pending;
                        }
                        rin.next(2);
                    }
                    if (p.zout != nullptr) {
                        put_round<T, ROUND>(buf + (2 + ob) * 32 * ROUND, o, &maps.z, i0, j0 + k * ROUND, lane);
                        ob ^= 1;
                    }
                    activate<T>(o, p.act);
                    put_round<T, ROUND>(buf + (2 + ob) * 32 * ROUND, o, &maps.out[w], i0, j0 + k * ROUND, lane);
                    ob ^= 1;
                }
                if (!alive) break;
            } else if (p.plog > 0) {
                float* o = p.sums + ((long long)at.part * p.J + j0) * p.I + i;
                const int n = (int)min((long long)PART, p.J - j0);
#pragma unroll 1
                for (int c = 0; c < PART; c += LD, o += LD * p.I) {
                    uint32_t v[LD];
                    tmem_ld<LD>(acc_t + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < LD; ++k)
                        if (i < p.I && c + k < n) o[k * p.I] = __uint_as_float(v[k]) * unscale;
                }
            } else {
                float rn[LD];
#pragma unroll 1
                for (int c = 0; c < PART; c += LD) {
                    uint32_t v[LD];
                    tmem_ld<LD>(acc_t + c, v);
                    if (c + LD < PART) res_lane<T>(p, i, (long long)j0 + c + LD, rn);
                    tmem_wait_ld();
                    float o[LD];
#pragma unroll
                    for (int k = 0; k < LD; ++k) o[k] = __uint_as_float(v[k]) * unscale;
                    if ((long long)j0 + c < p.J) finish_lane<T>(p, i, (long long)j0 + c, o, bias, r);
#pragma unroll
                    for (int k = 0; k < LD; ++k) r[k] = rn[k];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader<CG>(&acc_empty[chunk.slot]);
            chunk.next(NB);
        }
        // stores have read their buffers and reached memory, and no load into them is left behind
        if (lane == 0) {
            store_wait_all();
            for (; pending > 0; --pending, rin.next(2)) {
                const long long t0 = clock64();
                while (!mbar_test(&res_full[e][rin.slot], rin.lap & 1) && clock64() - t0 < WAIT_CYCLES) {
                }
            }
        }
    }

    if (S > 1) {
        Walk walk(P, worker);
        int w, u;
        walk.next(w, u);
        const TcProduct& p = P.p[w];
        const Place at(P, p, u, rank);
        __syncwarp();
        if (!pushed) cluster_wait();
        join_cluster<T, BN, EW>(p, at.i * BM, at.j * BN,
                               reinterpret_cast<const float*>(base + (size_t)NS * STAGE), rank, P.split_log, warp - 2);
    }
    tc_fence_before();
    if (CG > 1) {
        __syncwarp();
        cluster_sync_all();  // no CTA leaves while the other reads its shared memory or arrives on its barriers
    } else {
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        if (CG == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
    if (threadIdx.x == 0 && abort_sh) atomicExch(&g_ops_timeout, 1);
}

// ----------------------------------------------------------------------------------- operands in tensor-core form

// Eight values of a row to the planes of the operand at dst (planes `plane` elements apart; PL = 1: the type itself).
template <typename T>
__device__ __forceinline__ void store_operand(uint16_t* dst, long long plane, const float (&v)[8]) {
    if (sizeof(T) == 4) {
        uint4 h, m, l;
        split3x8(v, h, m, l);
        *reinterpret_cast<uint4*>(dst) = h;
        *reinterpret_cast<uint4*>(dst + plane) = m;
        *reinterpret_cast<uint4*>(dst + 2 * plane) = l;
    } else {
        Pack8<T> w;
        pack8(w, v);
        *reinterpret_cast<Pack8<T>*>(dst) = w;
    }
}

// A matrix to lay out: rows x cols, to `planes` planes of rows x ldp (ldp a multiple of 64).
struct PackJob {
    const void* src;
    long long ld, rows;
    int cols, vec;
    uint16_t* dst;
    long long ldp;
    long long blocks;  // of 8 * steps rows x PACK_COLS columns
    int blocks_c, steps;
};
constexpr int PACK_COLS = 256, PACK_THREADS = 256;

template <typename T>
__device__ void pack_block(const PackJob& j, long long blk) {
    const long long r0 = blk / j.blocks_c * (8 * j.steps) + (threadIdx.x >> 5);
    const int c = (int)(blk % j.blocks_c) * PACK_COLS + (threadIdx.x & 31) * 8;
    if (c >= j.cols) return;
    const long long plane = j.rows * j.ldp;
#pragma unroll 4
    for (int k = 0; k < j.steps; ++k) {
        const long long r = r0 + k * 8;
        if (r >= j.rows) break;
        Pack8<T> x;
        float v[8];
        load_raw8((const T*)j.src + r * j.ld + c, j.cols - c, j.vec, x);
        unpack8(x, v);
        store_operand<T>(j.dst + r * j.ldp + c, plane, v);
    }
}

// g = dy act'(z) of 8 * steps rows x PACK_COLS columns: to the operand (dst, unless g is dy itself), to dr, and its column sums
// over the rows, in fp32, to part[row block][N]. In 16 bits g of gelu and silu is rounded to the element type (float16: scaled
// first, below): the error of dx and dW then is 1.4 times that of their own rounding (bf16 8192 x 4096 x 4096 2.3e-3 against
// 1.7e-3, float16 2.9e-4 against 2.1e-4); a second 16-bit piece of g would double the products' time.
struct GradJob {
    const void* dy;
    long long lddy;
    const void* z;
    long long ldz;
    long long M;
    int N, act, vec, vec_r;
    uint16_t* dst;  // or nullptr
    long long ldp;
    void* dr;  // or nullptr
    long long lddr;
    float* part;  // or nullptr
    long long blocks;
    int blocks_c, steps;
    // float16: the largest finite |dy| of each block of linear_peak_k, and where the inverse of the operand's scale goes; or nullptr
    const unsigned* peaks;
    int npeaks;
    float* unscale;
};
constexpr int MAX_PEAKS = 592;  // blocks of that pass at most: four per SM

// U rows of dy and z on their way into registers while the U before are worked on.
template <typename T, int ACT, int U>
struct GradRows {
    Pack8<T> d[U], z[U];
    __device__ __forceinline__ void load(const GradJob& j, long long r0, int k0, int c) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const long long r = r0 + (k0 + k) * 8;
            const int n = k0 + k < j.steps && r < j.M ? j.N - c : 0;
            load_raw8((const T*)j.dy + r * j.lddy + c, n, j.vec, d[k]);
            if (ACT != VF_ACT_NONE) load_raw8((const T*)j.z + r * j.ldz + c, n, j.vec, z[k]);
        }
    }
    __device__ __forceinline__ void work(const GradJob& j, long long r0, int k0, int c, float scale, float (&s)[8]) {
        const int n = j.N - c;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const long long r = r0 + (k0 + k) * 8;
            if (k0 + k >= j.steps || r >= j.M) break;
            float v[8], x[8];
            unpack8(d[k], v);
            if (ACT != VF_ACT_NONE) unpack8(z[k], x);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (ACT != VF_ACT_NONE) v[u] = act_grad<sizeof(T) == 2>(v[u], x[u], ACT);
                s[u] += v[u];
            }
            constexpr bool SCALED = std::is_same<T, __half>::value;
            if (!SCALED && j.dst != nullptr) store_operand<T>(j.dst + r * j.ldp + c, j.M * j.ldp, v);
            if (j.dr != nullptr) {
                Pack8<T> p;
                pack8(p, v);
                store_raw8((T*)j.dr + r * j.lddr + c, n, j.vec_r, p);
            }
            if (SCALED && j.dst != nullptr) {
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] *= scale;
                store_operand<T>(j.dst + r * j.ldp + c, j.M * j.ldp, v);
            }
        }
    }
};
template <typename T, int ACT>
__device__ __forceinline__ void grad_rows(const GradJob& j, long long r0, int c, float scale, float (&s)[8]) {
    constexpr int U = sizeof(T) == 2 ? 2 : 1;
    GradRows<T, ACT, U> a, b;
    a.load(j, r0, 0, c);
#pragma unroll 1
    for (int k = 0; k < j.steps; k += 2 * U) {
        b.load(j, r0, k + U, c);
        a.work(j, r0, k, c, scale, s);
        a.load(j, r0, k + 2 * U, c);
        b.work(j, r0, k + U, c, scale, s);
    }
}

// Largest of a block's values, in every thread.
__device__ __forceinline__ unsigned block_peak(unsigned m) {
    __shared__ unsigned w[PACK_THREADS / 32];
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PACK_THREADS / 32; ++k) m = max(m, w[k]);
    return m;
}

// float16 has 11 bits from 2^-14 to 2^16 only: gradients of 1e-6 would keep four of them, and 65504 times a slope above one
// would be infinite. So where g has to be rounded (gelu, silu: slopes up to 1.13) it is first multiplied by the power of two that
// brings dy's largest magnitude to 2^13 .. 2^14, which needs a pass over dy before, and the products' sums by its inverse. What
// is lost then lies below 2^-38 of the largest. bf16 has fp32's range and needs none.
// This pass: the largest finite |dy| of each block's rows, as the bits of a float16.
__global__ void __launch_bounds__(PACK_THREADS) linear_peak_k(const __grid_constant__ GradJob j, unsigned* peaks) {
    constexpr int U = 4;
    grid_trigger();
    grid_wait();
    unsigned m = 0;
    for (long long blk = blockIdx.x; blk < j.blocks; blk += gridDim.x) {
        const int c = (int)(blk % j.blocks_c) * PACK_COLS + (threadIdx.x & 31) * 8;
        if (c >= j.N) continue;
        const long long r0 = blk / j.blocks_c * (8 * j.steps) + (threadIdx.x >> 5);
#pragma unroll 1
        for (int k = 0; k < j.steps; k += U) {
            GradRows<__half, VF_ACT_NONE, U> rows;
            rows.load(j, r0, k, c);
#pragma unroll
            for (int q = 0; q < U; ++q)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const unsigned lo = rows.d[q].w[u] & 0x7fff, hi = rows.d[q].w[u] >> 16 & 0x7fff;
                    m = max(m, max(lo < 0x7c00 ? lo : 0, hi < 0x7c00 ? hi : 0));
                }
        }
    }
    m = block_peak(m);
    if (threadIdx.x == 0) peaks[blockIdx.x] = m;
}
// The scale, from the blocks' largest; the first block hands its inverse on.
__device__ __forceinline__ float grad_scale(const GradJob& j, long long blk) {
    unsigned m = 0;
    for (int k = threadIdx.x; k < j.npeaks; k += PACK_THREADS) m = max(m, j.peaks[k]);
    m = block_peak(m);
    const float peak = __half2float(__ushort_as_half((unsigned short)m));  // 0, or 2^-24 to 65504: a normal number
    const int e = m == 0 ? 0 : 13 + 127 - (int)(__float_as_uint(peak) >> 23);
    if (blk == 0 && threadIdx.x == 0) *j.unscale = __uint_as_float((unsigned)(127 - e) << 23);
    return __uint_as_float((unsigned)(127 + e) << 23);
}

template <typename T>
__device__ void grad_block(const GradJob& j, long long blk) {
    __shared__ float sums[8][PACK_COLS];
    const float scale = std::is_same<T, __half>::value && j.peaks != nullptr ? grad_scale(j, blk) : 1.f;
    const int w = threadIdx.x >> 5;
    const long long rb = blk / j.blocks_c;
    const int c0 = (int)(blk % j.blocks_c) * PACK_COLS, cl = (threadIdx.x & 31) * 8, c = c0 + cl;
    float s[8] = {};
    if (c < j.N) {
        const long long r0 = rb * (8 * j.steps) + w;
        switch (j.act) {
            case VF_ACT_RELU: grad_rows<T, VF_ACT_RELU>(j, r0, c, scale, s); break;
            case VF_ACT_GELU: grad_rows<T, VF_ACT_GELU>(j, r0, c, scale, s); break;
            case VF_ACT_SILU: grad_rows<T, VF_ACT_SILU>(j, r0, c, scale, s); break;
            default: grad_rows<T, VF_ACT_NONE>(j, r0, c, scale, s);
        }
    }
    if (j.part == nullptr) return;
#pragma unroll
    for (int u = 0; u < 8; ++u) sums[w][cl + u] = s[u];
    __syncthreads();
    const int n = c0 + threadIdx.x;
    if (n < j.N) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += sums[k][threadIdx.x];
        j.part[rb * j.N + n] = t;
    }
}

template <typename T>
__global__ void __launch_bounds__(PACK_THREADS, 3)
linear_operands_k(const __grid_constant__ GradJob g, const __grid_constant__ PackJob a, const __grid_constant__ PackJob b) {
    grid_trigger();
    grid_wait();
    const long long t = blockIdx.x;
    if (t < g.blocks)
        grad_block<T>(g, t);
    else if (t < g.blocks + a.blocks)
        pack_block<T>(a, t - g.blocks);
    else
        pack_block<T>(b, t - g.blocks - a.blocks);
}

// The sums of a reduction cut into parts, added in order.
struct JoinJob {
    const float* sums;
    long long I, n;  // n = I * J
    int parts;
    void* out;
    long long ldo;
    int blocks;
};
constexpr int JOIN_THREADS = 256;

template <typename T>
__global__ void __launch_bounds__(JOIN_THREADS)
linear_join_k(const __grid_constant__ JoinJob a, const __grid_constant__ JoinJob b) {
    grid_wait();
    const JoinJob& j = (int)blockIdx.x < a.blocks ? a : b;
    const long long e = ((long long)blockIdx.x - ((int)blockIdx.x < a.blocks ? 0 : a.blocks)) * JOIN_THREADS + threadIdx.x;
    if (e >= j.n) return;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < j.parts; ++k) s += j.sums[k * j.n + e];
    ((T*)j.out)[e / j.I * j.ldo + e % j.I] = from_f32<T>(s);
}

// ------------------------------------------------------------------------------------------------- host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {  // thread-safe one-time lookup
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// A matrix in tensor-core form: 16-bit planes of rows x cols, rows ld elements apart, 16-byte aligned.
struct Operand16 {
    const void* ptr;
    long long rows, ld;
    int cols;
};

// mn: the operand is contiguous along its own index; its box is 64 columns x bk rows (steps of t). Else box of bk
// columns x `box` rows, swizzled over the bk * 2 bytes of a row.
bool make_map(CUtensorMap* map, const Operand16& o, int planes, bool mn, int bk, int box, bool bf16) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows, (cuuint64_t)planes};
    cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)o.rows * o.ld * 2};
    if (planes == 1 && strides[1] >= (1ull << 40)) strides[1] = strides[0];  // of the one plane: never used
    cuuint32_t boxes[3] = {(cuuint32_t)(mn ? 64 : bk), (cuuint32_t)(mn ? bk : box), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUtensorMapSwizzle swz = (mn || bk == 64) ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(o.ptr),
              dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of an output, a residual or z for the epilogue's rounds: boxes of 32 columns x `rows` rows.
template <typename T>
bool make_rows(CUtensorMap* map, const void* ptr, long long cols, long long rows, long long ld, int box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * sizeof(T)};
    cuuint32_t boxes[2] = {32, (cuuint32_t)box}, estr[2] = {1, 1};
    const CUtensorMapDataType t = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return fn(map, t, 2, const_cast<void*>(ptr), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of a block are 8 * steps: 256, or fewer (down to 8) until there are three blocks per SM, and on to six as long as no
// more than 64 partial column sums result. 8192 x 4096, g, dr and db of a gelu: 512 blocks, little over three per SM, 52.9 us
// in bf16 and 111.8 in fp32; 1024 blocks 48.0 and 96.4. Depends on the sizes alone, so that column sums are added in the
// same order on every device.
int pack_steps(long long rows, int blocks_c) {
    auto blocks = [&](int steps) { return (rows + 8 * steps - 1) / (8 * steps); };
    int steps = 32;
    while (steps > 1 && (blocks(steps) * blocks_c < 444 || (blocks(steps) * blocks_c < 888 && blocks(steps / 2) <= 64))) steps /= 2;
    return steps;
}

long long round_up(long long v, long long m) { return (v + m - 1) / m * m; }

// Bytes of the laid-out form of a rows x cols matrix.
size_t operand_bytes(int dtype, long long rows, long long cols) {
    return (size_t)round_up((dtype == VF_F32 ? 6 : 2) * rows * round_up(cols, 64), 256);
}

// Carves the workspace; hands out nullptr-based offsets too when base is nullptr.
struct Carver {
    uint8_t* base;
    size_t used = 0;
    uint8_t* take(size_t bytes) {
        uint8_t* p = base + used;
        used += (size_t)round_up((long long)bytes, 256);
        return p;
    }
};

// The operand as it is where TMA can read it (16-bit type, 16-byte rows), else a job that lays it out.
Operand16 operand(int dtype, const void* src, long long ld, long long rows, int cols, Carver& w, PackJob* job) {
    const int e = dtype == VF_F32 ? 4 : 2;
    *job = PackJob{};
    if (e == 2 && aligned16(src, ld, e)) return Operand16{src, rows, ld, cols};
    job->src = src;
    job->ld = ld;
    job->rows = rows;
    job->cols = cols;
    job->vec = aligned16(src, ld, e);
    job->ldp = round_up(cols, 64);
    job->dst = (uint16_t*)w.take(operand_bytes(dtype, rows, cols));
    job->blocks_c = (cols + PACK_COLS - 1) / PACK_COLS;
    job->steps = pack_steps(rows, job->blocks_c);
    job->blocks = (rows + 8 * job->steps - 1) / (8 * job->steps) * job->blocks_c;
    return Operand16{job->dst, rows, job->ldp, cols};
}

cudaError_t launch_operands(int dtype, const GradJob& g, const PackJob& a, const PackJob& b, cudaStream_t s) {
    const long long blocks = g.blocks + a.blocks + b.blocks;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(PACK_THREADS);
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    switch (dtype) {
        case VF_F32: return cudaLaunchKernelEx(&cfg, linear_operands_k<float>, g, a, b);
        case VF_BF16: return cudaLaunchKernelEx(&cfg, linear_operands_k<__nv_bfloat16>, g, a, b);
        default: return cudaLaunchKernelEx(&cfg, linear_operands_k<__half>, g, a, b);
    }
}

cudaError_t launch_peaks(const GradJob& g, unsigned* peaks, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)g.npeaks);
    cfg.blockDim = dim3(PACK_THREADS);
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_peak_k, g, peaks);
}

struct Side {
    Operand16 o;
    bool mn;
};

int blocks_of(int dtype, long long t) {
    const int bk = dtype == VF_F32 ? block_k<3>() : block_k<1>();
    return (int)((t + bk - 1) / bk);
}

// A launch as planned: tile width, cluster size, parts of each product's reduction (log 2) and estimated time in SM cycles.
struct Plan {
    int bn, split, plog[2];
    double cost;
};

// Products of a call: output extents and blocks of the reduction, the longer reduction first.
struct Extents {
    long long I[2], J[2];
    int nk[2], count;
    bool mn[2];  // B contiguous along j: tiles of 64 columns and more
};

// Estimated cycles of one tile: a block of the reduction costs what its MMAs take (fp32: twelve of 32 to 128 cycles;
// 16-bit: four, or the issuing thread's loop), a tile at least its epilogue, 30 cycles a column; measured on this kernel.
double tile_cycles(int nk, bool f32, int bn) {
    const double tb = f32 ? (bn == 256 ? 1536 : bn == 128 ? 1000 : bn == 64 ? 860 : 700) : (bn == 256 ? 560 : bn >= 64 ? 480 : 290);
    return std::max(nk * tb, 30.0 * bn);
}

// The cheapest launch by estimate: tiles per worker times their cycles, plus an epilogue, 6000 cycles before and after,
// 4000 for a join over a cluster; parts cost another launch and their sums' way through L2 (1300 bytes a cycle). Parts
// are taken until a tile is no longer than the average worker's load, eight blocks of the reduction each at least.
Plan plan(const Extents& x, bool f32, bool parts, int sms) {
    Plan best{64, 1, {0, 0}, 1e300};
    long long J = 1, I = 1;
    bool mn = false;
    for (int k = 0; k < x.count; ++k) {
        J = std::max(J, x.J[k]);
        I = std::max(I, x.I[k]);
        mn = mn || x.mn[k];
    }
    for (int bn = 16; bn <= 256; bn *= 2) {
        if (bn < 64 && (mn || J > bn)) continue;
        if (bn > 64 && (J <= bn / 2 || (bn == 256 && I <= BM))) continue;
        const int cg = bn == 256 ? 2 : 1, workers = sms / cg;
        auto tiles_of = [&](int k) { return (x.I[k] + BM * cg - 1) / (BM * cg) * ((x.J[k] + bn - 1) / bn); };
        auto consider = [&](int split, const int (&plog)[2]) {
            double total = 0, longest = 0, join = 0;
            long long tiles = 0;
            for (int k = 0; k < x.count; ++k) {
                const int cut = split << plog[k];
                const double t = tile_cycles((x.nk[k] + cut - 1) / cut, f32, bn);
                const long long n = tiles_of(k) * cut;
                tiles += n;
                total += t * n;
                longest = std::max(longest, t);
                if (plog[k] > 0) join += (double)(x.I[k] * x.J[k]) * (8 << plog[k]) / 1300;
            }
            double cost = tiles <= workers     ? longest
                          : x.count == 1 ? (double)((tiles + workers - 1) / workers) * longest
                                         : std::max(total / workers, longest) + 0.3 * longest;
            cost += 30.0 * bn + 6000 + (split > 1 ? 4000 : 0) + (join > 0 ? 8000 + join : 0);
            if (cost < best.cost) best = Plan{bn, split, {plog[0], plog[1]}, cost};
        };
        long long tiles = 0;
        int min_nk = 1 << 30;
        double load = 0;
        for (int k = 0; k < x.count; ++k) {
            tiles += tiles_of(k);
            min_nk = std::min(min_nk, x.nk[k]);
            load += tile_cycles(x.nk[k], f32, bn) * tiles_of(k) / workers;
        }
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (cg > 1 || tiles * split > sms || min_nk < 4 * split)) break;
            consider(split, {0, 0});
        }
        if (parts) {
            int plog[2] = {0, 0};
            for (int k = 0; k < x.count; ++k)
                while (plog[k] < 4 && x.nk[k] >> plog[k] >= 16 && tile_cycles(x.nk[k] >> plog[k], f32, bn) > load) ++plog[k];
            if (plog[0] + plog[1] > 0) consider(1, plog);
        }
    }
    return best;
}

// One launch for all products, or one for each.
struct Plans {
    bool apart;
    Plan a, b;  // of all, or of the first and the second
};
Plans plans(const Extents& x, bool f32, bool parts, int sms) {
    Plans r{false, plan(x, f32, parts, sms), {}};
    if (x.count < 2) return r;
    Extents y = x, z = x;
    y.count = z.count = 1;
    z.I[0] = x.I[1];
    z.J[0] = x.J[1];
    z.nk[0] = x.nk[1];
    z.mn[0] = x.mn[1];
    const Plan a = plan(y, f32, parts, sms), b = plan(z, f32, parts, sms);
    return a.cost + b.cost + 4000 < r.a.cost ? Plans{true, a, b} : r;
}
int plog_of(const Plans& p, int k) { return p.apart && k == 1 ? p.b.plog[0] : p.a.plog[k]; }

// The backward pass's products, dx and dW as far as wanted.
Extents grad_extents(int dtype, long long M, int N, int K, bool dx, bool dW) {
    Extents x{};
    if (dx) {
        x.I[0] = K;
        x.J[0] = M;
        x.nk[0] = blocks_of(dtype, N);
        x.count = 1;
    }
    if (dW) {
        const int k = x.count++;
        x.I[k] = K;
        x.J[k] = N;
        x.nk[k] = blocks_of(dtype, M);
        x.mn[k] = true;
    }
    if (x.count == 2 && x.nk[1] > x.nk[0]) {
        std::swap(x.I[0], x.I[1]);
        std::swap(x.J[0], x.J[1]);
        std::swap(x.nk[0], x.nk[1]);
        std::swap(x.mn[0], x.mn[1]);
    }
    return x;
}
size_t sums_bytes(const Extents& x, const Plans& p) {
    size_t n = 0;
    for (int k = 0; k < x.count; ++k)
        if (plog_of(p, k) > 0) n += (size_t)round_up(((x.I[k] * x.J[k]) << plog_of(p, k)) * 4, 256);
    return n;
}

// Clusters of cfg's size that run at once on the current device (asked once per kernel, size and device).
cudaError_t cluster_limit(const void* kern, const cudaLaunchConfig_t* cfg, int* fit) {
    static std::mutex mu;
    static std::map<std::tuple<const void*, unsigned, int>, int> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const auto key = std::make_tuple(kern, cfg->attrs[0].val.clusterDim.x, dev);
    std::lock_guard<std::mutex> lock(mu);
    const auto it = known.find(key);
    if (it != known.end()) {
        *fit = it->second;
        return cudaSuccess;
    }
    e = cudaOccupancyMaxActiveClusters(fit, kern, cfg);
    if (e == cudaSuccess) known[key] = *fit;
    return e;
}

template <typename T, int PL, int BN>
cudaError_t launch_bn(TcParams& P, const Side (&A)[2], const Side (&B)[2], int count, int split, int sms,
                      cudaStream_t s) {
    constexpr int BK = block_k<PL>(), CG = pair_of<BN>();
    const bool bf16 = PL == 3 || std::is_same<T, __nv_bfloat16>::value;
    Maps m;
    memset(&m, 0, sizeof(m));
    long long tiles = 0;
    for (int k = 0; k < count; ++k) {
        TcProduct& p = P.p[k];
        p.a_mn = A[k].mn;
        p.b_mn = B[k].mn;
        p.nk = (p.nk + stage_blocks<PL, BN>() - 1) / stage_blocks<PL, BN>();  // stages from here on
        p.tiles_i = (int)((p.I + BM * CG - 1) / (BM * CG));
        const long long n = ((long long)p.tiles_i * ((p.J + BN - 1) / BN)) << p.plog;
        if (n > 0x3fffffffLL) return cudaErrorInvalidValue;  // tile numbers are ints
        p.tiles = (int)n;
        tiles += n;
        if (!make_map(&m.a[k], A[k].o, PL, A[k].mn, BK, BM, bf16) || !make_map(&m.b[k], B[k].o, PL, B[k].mn, BK, BN / CG, bf16))
            return cudaErrorInvalidValue;
        constexpr int R = epi_round<T, BN>();
        if (BN >= 64 && p.vec && p.plog == 0 &&
            (!make_rows<T>(&m.out[k], p.out, p.I, p.J, p.ldo, R) ||
             (p.res != nullptr && !make_rows<T>(&m.res, p.res, p.I, p.J, p.ldr, R)) ||
             (p.zout != nullptr && !make_rows<T>(&m.z, p.zout, p.I, p.J, p.ldz, R))))
            return cudaErrorInvalidValue;
    }
    auto kern = linear_tc_k<T, PL, BN>;
    cudaError_t e = allow_dyn_smem((const void*)kern, SMEM_LIMIT - 1024);
    if (e != cudaSuccess) return e;
    const int need = stage_bytes<PL, BN>();
    P.stages = std::min(MAX_STAGES, (SMEM_LIMIT - 1024 - 1024 - epi_bytes<BN>()) / need);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(threads_of<BN>());
    cfg.dynamicSmemBytes = 1024 + (size_t)P.stages * need + epi_bytes<BN>();
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    // The planned cluster, as long as all clusters run at once (a cluster's CTAs share a GPC, so fewer may fit than the SMs
    // suggest).
    P.split = 1;
    P.split_log = 0;
    while (CG == 1 && P.split < split) {
        at[0].val.clusterDim.x = P.split * 2;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)(tiles * P.split * 2));
        int fit = 0;
        if ((e = cluster_limit((const void*)kern, &cfg, &fit)) != cudaSuccess) return e;
        if (fit < tiles) break;
        P.split *= 2;
        ++P.split_log;
    }
    P.test_stall = getenv("VF_TEST_OPS_STALL") != nullptr;
    P.workers = (int)std::min<long long>(tiles, P.split > 1 ? tiles : sms / CG);
    if (tiles == 0) P.workers = std::min((P.N + 127) / 128, sms);
    P.gap = 1;
    if (P.split == 1 && count == 2) {
        // as long as a tile of p[0], but no more than evens out over the workers that its last turn leaves idle
        const int rem = P.p[0].tiles % P.workers;
        const double a = tile_cycles(P.p[0].nk >> P.p[0].plog, PL == 3, BN), b = tile_cycles(P.p[1].nk >> P.p[1].plog, PL == 3, BN);
        P.gap = std::max(1, std::min((int)(a / b + 0.5), (P.p[1].tiles + P.workers - rem - 1) / (P.workers - rem)));
    }
    cfg.gridDim = dim3((unsigned)(P.workers * CG * P.split));
    at[0].val.clusterDim.x = CG * P.split;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, m, P);
}

template <typename T, int PL>
cudaError_t launch_as(TcParams& P, const Side (&A)[2], const Side (&B)[2], int count, const Plan& plan, int sms,
                      cudaStream_t s) {
    switch (plan.bn) {
        case 16: return launch_bn<T, PL, 16>(P, A, B, count, plan.split, sms, s);
        case 32: return launch_bn<T, PL, 32>(P, A, B, count, plan.split, sms, s);
        case 64: return launch_bn<T, PL, 64>(P, A, B, count, plan.split, sms, s);
        case 128: return launch_bn<T, PL, 128>(P, A, B, count, plan.split, sms, s);
        default: return launch_bn<T, PL, 256>(P, A, B, count, plan.split, sms, s);
    }
}

template <typename T, int PL>
cudaError_t launch_pl(TcParams& P, const Side (&A)[2], const Side (&B)[2], int count, const Plans& plans, int sms,
                      cudaStream_t s) {
    JoinJob join[2] = {};
    for (int k = 0; k < count; ++k) {
        TcProduct& p = P.p[k];
        p.plog = plog_of(plans, k);
        if (p.plog > 0) join[k] = JoinJob{p.sums, p.I, p.I * p.J, 1 << p.plog, p.out, p.ldo, (int)((p.I * p.J + JOIN_THREADS - 1) / JOIN_THREADS)};
    }
    cudaError_t e;
    if (!plans.apart) {
        e = launch_as<T, PL>(P, A, B, count, plans.a, sms, s);
    } else {
        TcParams Q{};
        Q.p[0] = P.p[1];
        Q.unscale = P.unscale;
        const Side A1[2] = {A[1], {}}, B1[2] = {B[1], {}};
        P.p[1] = TcProduct{};
        e = launch_as<T, PL>(P, A, B, 1, plans.a, sms, s);
        if (e == cudaSuccess) e = launch_as<T, PL>(Q, A1, B1, 1, plans.b, sms, s);
    }
    const int blocks = join[0].blocks + join[1].blocks;
    if (e != cudaSuccess || blocks == 0) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_join_k<T>, join[0], join[1]);
}

cudaError_t launch_products(int dtype, TcParams& P, const Side (&A)[2], const Side (&B)[2], int count, const Plans& plans,
                            int sms, cudaStream_t s) {
    switch (dtype) {
        case VF_F32: return launch_pl<float, 3>(P, A, B, count, plans, sms, s);
        case VF_BF16: return launch_pl<__nv_bfloat16, 1>(P, A, B, count, plans, sms, s);
        default: return launch_pl<__half, 1>(P, A, B, count, plans, sms, s);
    }
}

int col_blocks(int N) { return (N + PACK_COLS - 1) / PACK_COLS; }
long long row_blocks(long long M, int N) {
    const int rows = 8 * pack_steps(M, col_blocks(N));
    return (M + rows - 1) / rows;
}

}  // namespace

bool linear_tc_supported(long long M, int N, int K) { return M > 0 && N > 0 && K > 0; }

bool linear_tc_in_place(const LinearFwd& f) {
    return f.dtype != VF_F32 && aligned16(f.x, f.ldx, 2) && aligned16(f.W, f.ldw, 2);
}

size_t linear_tc_workspace(int dtype, long long M, int N, int K, bool grad) {
    size_t n = operand_bytes(dtype, M, K) + operand_bytes(dtype, N, K);
    if (!grad) return n;
    n += operand_bytes(dtype, M, N) + (size_t)round_up(row_blocks(M, N) * N * 4, 256);
    if (dtype == VF_F16) n += (size_t)round_up((MAX_PEAKS + 1) * 4, 256);
    int sms = 0;
    if (device_sms(&sms) != cudaSuccess) return n;
    size_t sums = 0;
    for (int want = 1; want < 4; ++want) {  // dx, dW, both
        const Extents x = grad_extents(dtype, M, N, K, want & 1, (want & 2) != 0);
        sums = std::max(sums, sums_bytes(x, plans(x, dtype == VF_F32, true, sms)));
    }
    return n + sums;
}

cudaError_t launch_linear_tc(const LinearFwd& f, void* work, size_t have, size_t* need, cudaStream_t s) {
    const int e = f.dtype == VF_F32 ? 4 : 2;
    Carver w{(uint8_t*)work};
    PackJob jx, jw;
    Side A[2] = {}, B[2] = {};
    A[0] = Side{operand(f.dtype, f.W, f.ldw, f.N, f.K, w, &jw), false};
    B[0] = Side{operand(f.dtype, f.x, f.ldx, f.M, f.K, w, &jx), false};
    *need = w.used;
    if (w.used > have) return cudaSuccess;  // the caller reports it
    cudaError_t err = launch_operands(f.dtype, GradJob{}, jw, jx, s);
    if (err != cudaSuccess) return err;
    TcParams P{};
    TcProduct& p = P.p[0];
    p.I = f.N;
    p.J = f.M;
    p.nk = blocks_of(f.dtype, f.K);
    p.out = f.y;
    p.ldo = f.ldy;
    p.bias = f.b;
    p.res = f.r;
    p.ldr = f.ldr;
    p.zout = f.z;
    p.ldz = f.ldz;
    p.act = f.act;
    p.vec = aligned16(f.y, f.ldy, e) && (f.r == nullptr || aligned16(f.r, f.ldr, e)) &&
            (f.z == nullptr || aligned16(f.z, f.ldz, e));
    Extents x{};
    x.I[0] = p.I;
    x.J[0] = p.J;
    x.nk[0] = p.nk;
    x.count = 1;
    int sms = 0;
    if ((err = device_sms(&sms)) != cudaSuccess) return err;
    return launch_products(f.dtype, P, A, B, 1, plans(x, f.dtype == VF_F32, false, sms), sms, s);
}

cudaError_t launch_linear_grad_tc(const LinearGrad& f, void* work, size_t have, size_t* need, cudaStream_t s) {
    const int e = f.dtype == VF_F32 ? 4 : 2;
    Carver w{(uint8_t*)work};
    const bool products = f.dx != nullptr || f.dW != nullptr;
    GradJob gj{};
    gj.dy = f.dy;
    gj.lddy = f.lddy;
    gj.z = f.z;
    gj.ldz = f.ldz;
    gj.M = f.M;
    gj.N = f.N;
    gj.act = f.act;
    gj.vec = aligned16(f.dy, f.lddy, e) && (f.act == VF_ACT_NONE || aligned16(f.z, f.ldz, e));
    gj.dr = f.dr;
    gj.lddr = f.lddr;
    gj.vec_r = f.dr != nullptr && aligned16(f.dr, f.lddr, e);
    Operand16 g{};
    const bool scaled = products && f.dtype == VF_F16 && (f.act == VF_ACT_GELU || f.act == VF_ACT_SILU);
    if (products) {
        if (e == 2 && f.act == VF_ACT_NONE && aligned16(f.dy, f.lddy, e)) {
            g = Operand16{f.dy, f.M, f.lddy, f.N};  // dy is g, and TMA can read it
        } else if (e == 2 && gj.vec_r && !scaled) {
            g = Operand16{f.dr, f.M, f.lddr, f.N};  // dr is g
        } else {
            gj.ldp = round_up(f.N, 64);
            gj.dst = (uint16_t*)w.take(operand_bytes(f.dtype, f.M, f.N));
            g = Operand16{gj.dst, f.M, gj.ldp, f.N};
        }
    }
    if (f.db != nullptr) gj.part = (float*)w.take((size_t)row_blocks(f.M, f.N) * f.N * 4);
    if (gj.dst != nullptr || gj.dr != nullptr || gj.part != nullptr) {
        gj.blocks_c = col_blocks(f.N);
        gj.steps = pack_steps(f.M, gj.blocks_c);
        gj.blocks = row_blocks(f.M, f.N) * gj.blocks_c;
    }
    unsigned* peaks = nullptr;
    if (scaled) {
        peaks = (unsigned*)w.take((MAX_PEAKS + 1) * 4);
        gj.npeaks = (int)std::min<long long>(gj.blocks, MAX_PEAKS);
    }
    PackJob jw{}, jx{};
    Side A[2] = {}, B[2] = {};
    TcParams P{};
    int count = 0;
    if (f.dx != nullptr) {
        A[count] = Side{operand(f.dtype, f.W, f.ldw, f.N, f.K, w, &jw), true};
        B[count] = Side{g, false};
        TcProduct& p = P.p[count++];
        p.I = f.K;
        p.J = f.M;
        p.nk = blocks_of(f.dtype, f.N);
        p.out = f.dx;
        p.ldo = f.lddx;
        p.vec = aligned16(f.dx, f.lddx, e);
    }
    if (f.dW != nullptr) {
        A[count] = Side{operand(f.dtype, f.x, f.ldx, f.M, f.K, w, &jx), true};
        B[count] = Side{g, true};
        TcProduct& p = P.p[count++];
        p.I = f.K;
        p.J = f.N;
        p.nk = blocks_of(f.dtype, f.M);
        p.out = f.dW;
        p.ldo = f.lddw;
        p.vec = aligned16(f.dW, f.lddw, e);
    }
    if (count == 2 && P.p[1].nk > P.p[0].nk) {
        std::swap(P.p[0], P.p[1]);
        std::swap(A[0], A[1]);
        std::swap(B[0], B[1]);
    }
    int sms = 0;
    cudaError_t err = device_sms(&sms);
    if (err != cudaSuccess) return err;
    const Plans how = plans(grad_extents(f.dtype, f.M, f.N, f.K, f.dx != nullptr, f.dW != nullptr), f.dtype == VF_F32, true, sms);
    for (int k = 0; k < count; ++k)
        if (plog_of(how, k) > 0) P.p[k].sums = (float*)w.take((size_t)((P.p[k].I * P.p[k].J) << plog_of(how, k)) * 4);
    *need = w.used;
    if (w.used > have) return cudaSuccess;  // the caller reports it
    if (scaled) {
        if ((err = launch_peaks(gj, peaks, s)) != cudaSuccess) return err;
        gj.peaks = peaks;
        P.unscale = gj.unscale = (float*)(peaks + MAX_PEAKS);
    }
    err = launch_operands(f.dtype, gj, jw, jx, s);
    if (err != cudaSuccess) return err;
    if (count == 0 && f.db == nullptr) return cudaSuccess;
    P.part = gj.part;
    P.nparts = (int)row_blocks(f.M, f.N);
    P.N = f.N;
    P.db = f.db;
    return launch_products(f.dtype, P, A, B, count, how, sms, s);
}

cudaError_t device_sms(int* sms) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// Reads and clears the flags of expired waits (the device is idle when this is called).
cudaError_t ops_take_timeout(int* flag) {
    int direct = 0;
    cudaError_t e = direct_take_timeout(&direct);
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(flag, g_ops_timeout, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *flag != 0) e = cudaMemcpyToSymbol(g_ops_timeout, &zero, sizeof(int));
    *flag |= direct;
    return e;
}

}  // namespace vf
