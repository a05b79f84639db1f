// Dense layer on the tensor cores, operands laid out on the way into shared memory: one launch, no workspace, any strides and
// alignment. The product and the fp32 scheme are those of k_linear_tc.cu.
//
// k_linear_tc.cu feeds 16-bit rows that TMA can read, and everything else from a laid-out copy that another launch
// makes. Where every tile has an SM to itself that copy costs more than it saves: an operand is read by a few CTAs only.
// Here 16 warps load the next block of 64 steps of both operands into registers while the block before is on its way
// into the tensor cores, split fp32 into its three pieces, and store them in the swizzled form that the MMAs read; one more
// warp issues the MMAs. The same warps then finish the tile: directly, or, with the reduction split over a cluster, after
// joining the partial tiles.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "linear_tc.cuh"
#include "vf_internal.cuh"

namespace vf {

namespace {

using namespace tc;
using namespace lin;

__device__ int g_direct_timeout;

constexpr int BK = 64;             // steps of the reduction per block: 128-byte rows in shared memory
constexpr int WORKERS = 512;       // loading and finishing threads
constexpr int THREADS = WORKERS + 32;
// Blocks added up in one accumulator, as in k_linear_tc.cu.
constexpr int chunk_blocks(int pl) { return (pl == 3 ? 256 : CHUNK_16) / BK; }
// Accumulators (fp32: of h h products), one after the other, all added in registers at the end; TMEM has 512 columns, and fp32's small
// products take one accumulator more.
constexpr int accumulators(int pl, int bn) { return pl == 3 && bn == 64 ? 4 : 8; }

// rows x Tn operand at p: element (r, t) at p[r * ld + t].
struct Source {
    const void* p;
    long long ld;
    int rows;
};

struct DirectParams {
    TcProduct p;
    Source a, b;
    int Tn;  // length of the reduction
    int split_log, stages;
};

// What a thread holds of a block of one operand: N times eight elements. A staged operand is made of 128-byte lines of
// BK elements, one per row. VEC (rows of 16-byte alignment): eight elements that lie together, a line by eight neighbouring
// threads, groups of 64 lines. Else single elements, a line by the lanes of a warp, half by half, groups of 16 lines.
template <typename T, int N, bool VEC>
struct Held {
    Pack8<T> v[N];
};
template <typename T, int N>
struct Held<T, N, false> {
    T e[8 * N];  // a register each: nothing waits for a load before the block is laid out
};

template <typename T, int N, int LINES, bool VEC>
struct Loader {
    static constexpr int STEP = VEC ? 64 : 16;
    const T* p;           // this thread's first element of the next block
    long long line_step;  // elements between its lines
    int left;             // rows from its first line to the operand's last
    int t;                // step of its first element in a block
    Held<T, N, VEC> h[2];
    __device__ __forceinline__ Loader(const Source& s, int r0, int kb0) {
        const int line = VEC ? threadIdx.x >> 3 : threadIdx.x >> 5;
        t = VEC ? (threadIdx.x & 7) * 8 : threadIdx.x & 31;
        left = line < LINES ? s.rows - r0 - line : 0;
        p = (const T*)s.p + (long long)(r0 + line) * s.ld + (long long)kb0 * BK + t;
        line_step = STEP * s.ld;
    }
    // The next block; `steps` of its BK exist.
    __device__ __forceinline__ void load(int b, int steps) {
        const T* q = p;
#pragma unroll
        for (int g = 0; g < (VEC ? N : 4 * N); ++g, q += line_step) {
            if (LINES < STEP * (g + 1) && (int)(VEC ? threadIdx.x >> 3 : threadIdx.x >> 5) + STEP * g >= LINES) break;
            const int n = left > STEP * g ? steps - t : 0;
            if constexpr (VEC) {
                load_raw8(q, n, true, h[b].v[g]);
            } else {
                h[b].e[2 * g] = n > 0 ? q[0] : from_f32<T>(0.f);
                h[b].e[2 * g + 1] = n > 32 ? q[32] : from_f32<T>(0.f);
            }
        }
        p += BK;
    }
};

// Eight elements c * 8 .. of a line of 128 bytes: 128-byte swizzle, 16 bytes at a time.
__device__ __forceinline__ int swizzled(int line, int c) { return line * 128 + ((c ^ (line & 7)) << 4); }

template <typename T, int PL, int N, int LINES, bool VEC>
__device__ __forceinline__ void store_block(uint8_t* dst, int plane, const Held<T, N, VEC>& h) {
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int line = (int)(threadIdx.x >> 3) + 64 * k;
            if (LINES < 64 * (k + 1) && line >= LINES) break;
            uint8_t* o = dst + swizzled(line, threadIdx.x & 7);
            if (PL == 3) {
                float v[8];
                unpack8(h.v[k], v);
                uint4 hi, mid, lo;
                split3x8(v, hi, mid, lo);
                *reinterpret_cast<uint4*>(o) = hi;
                *reinterpret_cast<uint4*>(o + plane) = mid;
                *reinterpret_cast<uint4*>(o + 2 * plane) = lo;
            } else {
                *reinterpret_cast<Pack8<T>*>(o) = h.v[k];
            }
        }
    } else {
#pragma unroll
        for (int x = 0; x < 8 * N; ++x) {
            const int line = (int)(threadIdx.x >> 5) + 16 * (x >> 1), e = (threadIdx.x & 31) + (x & 1) * 32;
            if (LINES < 16 * ((x >> 1) + 1) && line >= LINES) break;
            uint8_t* o = dst + swizzled(line, e >> 3) + (e & 7) * 2;
            if (PL == 3) {
                const float v = to_f32(h.e[x]);
                float hi, mid, lo;
                split3(v, hi, mid, lo);
                *reinterpret_cast<uint16_t*>(o) = (uint16_t)(__float_as_uint(hi) >> 16);
                *reinterpret_cast<uint16_t*>(o + plane) = (uint16_t)(__float_as_uint(mid) >> 16);
                *reinterpret_cast<uint16_t*>(o + 2 * plane) = (uint16_t)(__float_as_uint(lo) >> 16);
            } else {
                *reinterpret_cast<T*>(o) = h.e[x];
            }
        }
    }
}

template <int PL, int BN>
constexpr int direct_stage() {
    return PL * (BM + BN) * 128;
}

template <typename T, int PL, int BN, bool VA, bool VB>
__global__ void __launch_bounds__(THREADS, 1) linear_direct_k(const __grid_constant__ DirectParams P) {
    constexpr int A_PLANE = BM * 128, B_PLANE = BN * 128;
    constexpr int STAGE = direct_stage<PL, BN>();
    constexpr int CHUNK = chunk_blocks(PL);
    constexpr int COR = accumulators(PL, BN) * BN;                 // columns of the small products
    constexpr int TMEM_COLS = PL == 3 ? (BN == 16 ? 256 : 512) : COR;
    constexpr int FW = BN >= 32 ? 16 : 8;                          // finishing warps
    constexpr int PART = BN / (FW / 4);                            // columns of one
    constexpr int NA = BM * 8 / WORKERS;                           // times eight elements of A per thread
    constexpr int NBC = (BN * 8 + WORKERS - 1) / WORKERS;          // of B
    constexpr int LD = PART < 16 ? 8 : 16;  // per TMEM load
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[4], empty[4], acc_full, done_bar;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = 1 << P.split_log, NS = P.stages;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const int worker = blockIdx.x >> P.split_log;
    grid_wait();
    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], WORKERS / 32);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&done_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == WORKERS / 32) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_sh)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const TcProduct& p = P.p;
    const int i0 = worker % p.tiles_i * BM, j0 = worker / p.tiles_i * BN;
    const int kb0 = share(p.nk, rank, P.split_log), kb1 = share(p.nk, rank + 1, P.split_log);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (S > 1) cluster_arrive();
    const uint32_t tmem = tmem_base_sh;
    volatile int* abort_flag = &abort_sh;
    const uint32_t inbox = smem_u32(base) + NS * STAGE;
    bool pushed = false;  // this warp has met the cluster's first barrier

    if (warp == WORKERS / 32) {
        if (elect_one()) {
            const uint32_t fmt = (PL == 3 || std::is_same<T, __nv_bfloat16>::value) ? 1u : 0u;
            const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(BN >> 3) << 17) |
                                   ((uint32_t)(BM >> 4) << 24);
            const uint64_t a0 = operand_desc<BK>(smem_u32(base), 0);
            const uint64_t b0 = operand_desc<BK>(smem_u32(base) + PL * A_PLANE, 0);
            Ring g;
            for (int kb = kb0; kb < kb1; ++kb, g.next(NS)) {
                if (!wait_phase(&full[g.slot], g.lap & 1, abort_flag)) break;
                tc_fence_after();
                const uint64_t ah = a0 + (uint32_t)(g.slot * (STAGE / 16)), bh = b0 + (uint32_t)(g.slot * (STAGE / 16));
                const int at = kb - kb0;
                const uint32_t d = tmem + at / CHUNK * BN;
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk) {
                    const uint64_t h = ah + kk * 2, H = bh + kk * 2;  // 32 bytes along a line
                    if (PL == 3) {
                        const uint32_t more = at > 0 || kk > 0 ? 1u : 0u;
                        const uint64_t m = h + A_PLANE / 16, l = m + A_PLANE / 16;
                        const uint64_t M = H + B_PLANE / 16, L = M + B_PLANE / 16;
                        mma_f16_ss<1>(tmem + COR, l, H, idesc, more);
                        mma_f16_ss<1>(tmem + COR, h, L, idesc, 1u);
                        mma_f16_ss<1>(tmem + COR, m, M, idesc, 1u);
                        mma_f16_ss<1>(tmem + COR, m, H, idesc, 1u);
                        mma_f16_ss<1>(tmem + COR, h, M, idesc, 1u);
                    }
                    mma_f16_ss<1>(d, h, H, idesc, at % CHUNK > 0 || kk > 0 ? 1u : 0u);
                }
                mma_commit(&empty[g.slot]);
            }
            mma_commit(&acc_full);
            mma_commit(&done_bar);  // TMEM is never freed under MMAs in flight
            const long long t0 = clock64();
            while (!mbar_test(&done_bar, 0) && clock64() - t0 < WAIT_CYCLES) {
            }
        }
    } else {
        Loader<T, NA, BM, VA> a(P.a, i0, kb0);
        Loader<T, NBC, BN, VB> b(P.b, j0, kb0);
        Ring g;
        bool ok = true;
        auto stage = [&](int kb, int h) {
            if (kb + 1 < kb1) {  // in flight while this block is laid out and multiplied
                a.load(h ^ 1, P.Tn - (kb + 1) * BK);
                b.load(h ^ 1, P.Tn - (kb + 1) * BK);
            }
            if (g.lap > 0) ok = wait_phase(&empty[g.slot], (g.lap - 1) & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            uint8_t* st = base + (size_t)g.slot * STAGE;
            store_block<T, PL, NA, BM, VA>(st, A_PLANE, a.h[h]);
            store_block<T, PL, NBC, BN, VB>(st + PL * A_PLANE, B_PLANE, b.h[h]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[g.slot]);
            g.next(NS);
        };
        a.load(0, P.Tn - kb0 * BK);
        b.load(0, P.Tn - kb0 * BK);
        for (int kb = kb0; kb < kb1 && ok; kb += 2) {
            stage(kb, 0);
            if (kb + 1 < kb1 && ok) stage(kb + 1, 1);
        }
        // the finished tile: TMEM to its rows, or to shared memory for the join
        const int q = warp & 3, part_no = warp >> 2;
        const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + part_no * PART;
        const long long i = (long long)i0 + q * 32 + lane;
        const int jw = j0 + part_no * PART;
        const float bias = (S == 1 && p.bias != nullptr && i < p.I) ? to_f32(((const T*)p.bias)[i]) : 0.f;
        float r[LD], rn[LD];
        if (S == 1 && warp < FW) res_lane<T>(p, i, jw, r);
        ok = wait_phase(&acc_full, 0, abort_flag);
        if (__all_sync(0xffffffffu, ok) && warp < FW) {
            tc_fence_after();
            if (S > 1) cluster_wait();  // all of the cluster's CTAs have begun
            pushed = true;
#pragma unroll 1
            for (int c = 0; c < PART; c += LD) {
                uint32_t v[LD];
                float o[LD];
                tmem_ld<LD>(acc + (PL == 3 ? COR : 0) + c, v);  // the small products, or the first accumulator
                if (S == 1 && c + LD < PART) res_lane<T>(p, i, (long long)jw + c + LD, rn);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < LD; ++k) o[k] = kb1 > kb0 ? __uint_as_float(v[k]) : 0.f;  // a share may hold no blocks
#pragma unroll 1
                for (int a = PL == 3 ? 0 : 1; a < (kb1 - kb0 + CHUNK - 1) / CHUNK; ++a) {
                    tmem_ld<LD>(acc + a * BN + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < LD; ++k) o[k] += __uint_as_float(v[k]);
                }
                if (S > 1) {
#pragma unroll
                    for (int k = 0; k < LD; ++k)
                        push_column<BN>(inbox, part_no * PART + c + k, q * 32 + lane, rank, P.split_log, o[k]);
                } else {
                    if ((long long)jw + c < p.J) finish_lane<T>(p, i, (long long)jw + c, o, bias, r);
#pragma unroll
                    for (int k = 0; k < LD; ++k) r[k] = rn[k];
                }
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    if (S > 1) {
        if (!pushed) cluster_wait();
        join_cluster<T, BN, WORKERS / 32>(p, i0, j0, reinterpret_cast<const float*>(base + NS * STAGE), rank, P.split_log,
                                          warp);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == WORKERS / 32) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
    if (threadIdx.x == 0 && abort_sh) atomicExch(&g_direct_timeout, 1);
}

// ------------------------------------------------------------------------------------------------- host side

constexpr int SMEM_LIMIT = 232448 - 1024;  // dynamic: 227 KB less the static part

int blocks_of(long long t) { return (int)((t + BK - 1) / BK); }

int columns(long long M) { return M > 32 ? 64 : M > 16 ? 32 : 16; }

// Cluster size (log 2) of the split reduction of `tiles` tiles over nk blocks. In units of one block's time: a CTA costs
// about five blocks before and after its products and two more for the join; the estimate is the longest CTA or the SMs'
// share of the total (clusters of eight leave SMs unused). `most`: blocks that a CTA can add up.
int split_log(long long tiles, int nk, int most, int sms) {
    int best = 0;
    double best_cost = 1e30;
    for (int log = 0; log <= 3; ++log) {
        const int S = 1 << log, part = (nk + S - 1) / S;
        if (part > most) continue;
        const double cta = 5.0 + part + (log > 0 ? 2.0 : 0.0);
        const double cost = std::max(cta, cta * S * tiles / sms * (log == 3 ? 1.3 : 1.1));
        if (cost < best_cost) {
            best_cost = cost;
            best = log;
        }
    }
    return best;
}

template <typename T, int PL, int BN, bool VA, bool VB>
cudaError_t launch_bn(DirectParams& P, int sms, cudaStream_t s) {
    TcProduct& p = P.p;
    p.nk = blocks_of(P.Tn);
    p.tiles_i = (int)((p.I + BM - 1) / BM);
    p.tiles = (int)(p.tiles_i * ((p.J + BN - 1) / BN));
    auto kern = linear_direct_k<T, PL, BN, VA, VB>;
    cudaError_t e = allow_dyn_smem((const void*)kern, SMEM_LIMIT);
    if (e != cudaSuccess) return e;
    const int need = direct_stage<PL, BN>();
    P.stages = std::min(4, (SMEM_LIMIT - 1024 - BN * 512) / need);
    P.split_log = split_log(p.tiles, p.nk, chunk_blocks(PL) * accumulators(PL, BN), sms);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS);
    cfg.gridDim = dim3((unsigned)(p.tiles << P.split_log));
    cfg.dynamicSmemBytes = 1024 + (size_t)P.stages * need + BN * 512;  // and the inbox
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1u << P.split_log;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, P);
}

template <typename T, int PL, bool VA, bool VB>
cudaError_t launch_pl(DirectParams& P, cudaStream_t s) {
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return e;
    switch (columns(P.p.J)) {
        case 16: return launch_bn<T, PL, 16, VA, VB>(P, sms, s);
        case 32: return launch_bn<T, PL, 32, VA, VB>(P, sms, s);
        default: return launch_bn<T, PL, 64, VA, VB>(P, sms, s);
    }
}

template <typename T, int PL>
cudaError_t launch_vec(DirectParams& P, bool va, bool vb, cudaStream_t s) {
    // both: fp32 only, 16-bit rows of 16-byte alignment are read by TMA in place (k_linear_tc.cu)
    if constexpr (PL == 3)
        if (va && vb) return launch_pl<T, PL, true, true>(P, s);
    if (va && !vb) return launch_pl<T, PL, true, false>(P, s);
    if (vb && !va) return launch_pl<T, PL, false, true>(P, s);
    return launch_pl<T, PL, false, false>(P, s);
}

int elem(int dtype) { return dtype == VF_F32 ? 4 : 2; }

}  // namespace

// Every tile has an SM to itself, with the reduction cut into as many parts as the accumulators ask for, up to eight.
// Against a laid-out copy and k_linear_tc.cu (M x N x K, us out of L2, here and there): fp32 16x512x512 6.1 and 9.0, 1024x256x784
// 11.0 and 13.8, 512x1024x1024 15.0 and 18.2, 16x4096x4096 21.1 and 53.9; many waves of tiles, 297x3712x1472 118 and 35.
// Rows that are not 16-byte aligned are loaded element by element. In fp32 that costs more than the copy where several
// columns of tiles load the same W and a CTA takes many such lines: x and W unaligned, 256x256x256 9.0 and 10.0,
// 1024x256x784 16.1 and 14.4, 512x1024x1024 26.5 and 18.5; one column of tiles, 16x2048x4096, 38.5 and 36.5. In 16 bits the
// two are close (bf16 1024x256x784 10.1 and 10.4, 777x1001x512 13.2 and 10.0), and a call that waits for the host is shorter
// with one launch (9.9 and 14.3).
bool linear_direct_fits(int dtype, long long M, int N, int K, bool x_aligned, bool w_aligned) {
    int sms = 0, parts = 1;
    if (device_sms(&sms) != cudaSuccess) return false;
    const int bn = columns(M), nk = blocks_of(K), pl = dtype == VF_F32 ? 3 : 1, most = chunk_blocks(pl) * accumulators(pl, bn);
    while (parts * most < nk && parts <= 8) parts *= 2;
    const long long tiles = ((long long)N + BM - 1) / BM * ((M + bn - 1) / bn);
    if (parts > 8 || tiles * parts > sms) return false;
    if (dtype != VF_F32 || M <= bn) return true;
    const int S = 1 << split_log(tiles, nk, most, sms);
    return ((x_aligned ? 0 : bn) + (w_aligned ? 0 : BM)) * ((nk + S - 1) / S) < 512;
}

cudaError_t launch_linear_direct(const LinearFwd& f, cudaStream_t s) {
    const int e = elem(f.dtype);
    DirectParams P{};
    P.a = Source{f.W, f.ldw, f.N};
    P.b = Source{f.x, f.ldx, (int)f.M};
    P.Tn = f.K;
    TcProduct& p = P.p;
    p.I = f.N;
    p.J = f.M;
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
    const bool va = aligned16(f.W, f.ldw, e), vb = aligned16(f.x, f.ldx, e);
    switch (f.dtype) {
        case VF_F32: return launch_vec<float, 3>(P, va, vb, s);
        case VF_BF16: return launch_vec<__nv_bfloat16, 1>(P, va, vb, s);
        default: return launch_vec<__half, 1>(P, va, vb, s);
    }
}

cudaError_t direct_take_timeout(int* flag) {
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_direct_timeout, sizeof(int));
    if (e != cudaSuccess || *flag == 0) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_direct_timeout, &zero, sizeof(int));
}

}  // namespace vf
