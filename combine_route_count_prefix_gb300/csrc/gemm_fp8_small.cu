// gemm_fp8_small.cu -- grouped products of block-scaled e4m3 operands for few
// rows per expert.
//
// With few rows the time is the time to read the weights.  So the weights are
// the MMA's M side (128 channels: every tensor-core row busy whatever the row
// count) and the expert's rows its N side (as many as present, rounded up to
// 16), and a deep ring of TMA copies keeps the weights coming.  As in the
// large form every 128-deep block of K has an accumulator of its own, which
// the epilogue reads back, scales (the row's scale varies along the columns
// here) and adds to fp32 sums in registers.
//
// Kernel shape (one persistent CTA per SM, 12 warps):
//   warp 0       TMA producer of the weights: NG x 128 channels, 128 bytes of K
//                each, per block, into the ring
//   warp 2       TMA producer of the block's TB rows, into the same stages.  In a
//                call's later kernels only these (and their scales) depend on
//                the kernel before, so the weights start to come while it ends
//   warps 1, 3   MMA issuers, one per 128-channel group, or taking turns on the
//                blocks of the one group (issuing a tcgen05.mma takes a thread
//                about 130 cycles whatever its N); warp 1 owns TMEM
//   warps 4..11  epilogue: TMEM lane quadrant (32 channels) x half of the rows
// Tiles are (expert, TB rows, NG x 128 channels), channel block fastest.
// SwiGLU form (NG = 2): the groups are 128 SiLU-half channels and their
// multipliers, so a tile holds 128 complete channels of g and quantises them
// as one block.
// Where the tiles are fewer than the SMs, a cluster of S CTAs shares a tile:
// each takes a range of K, and the partial sums are added in rank order (so
// repeats are bitwise equal) through distributed shared memory, every CTA
// finishing the rows c = rank mod S.
// What bounds it: the weights' bytes from HBM where there are many (an FFN of
// 128 experts of 7168 x 4096, 8 rows each: 829 us, 6.8 TB/s), the fixed steps
// where there are few (16 rows, 4096 x 7168: 8.9 us a kernel, of which 2.2 go to
// the set-up, 1.2 to the first data, 1.4 to the join of a shared tile and 0.9
// to the exit; the weights' bytes alone take 4.4).
// Every wait is bounded (about two seconds) and sets MOE_DEV_TIMEOUT.
#include "common.cuh"
#include "fp8.cuh"
#include "tcgen05.cuh"

#include <algorithm>
#include <cuda.h>

namespace moe {
namespace {

using namespace tc;

constexpr int BW = 128;                  // channels per group = MMA M
constexpr int BK = 128;                  // bytes of K per block: one scale
constexpr int W_BYTES = BW * BK;
constexpr int EPI_WARP0 = 4;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr size_t kBarrierBytes = 512;
constexpr int kMaxSplit = 8;             // CTAs of a portable cluster

enum { EPI_F32 = 0, EPI_BF16 = 1, EPI_SWIGLU = 2 };

template <int EPI, int TB_>
struct Cfg {
    static constexpr int TB = TB_;                       // rows per tile
    static constexpr int NG = EPI == EPI_SWIGLU ? 2 : 1;
    static constexpr int CW = TB / 2;                    // rows per epilogue warp
    static constexpr int NBUF = 4;                       // accumulators
    static constexpr uint32_t TMEM_COLS = NBUF * NG * TB < 32 ? 32 : NBUF * NG * TB;
    static constexpr int STAGE_BYTES = NG * W_BYTES + TB * BK;
    // partial sums of a shared tile; the 64-row SwiGLU tile has no room for them
    static constexpr bool SPLIT = TB == 32 || NG == 1;
    static constexpr size_t PART_BYTES = SPLIT ? (size_t)NG * TB * BW * sizeof(float) : 0;
    static constexpr size_t SCALE_BYTES = (size_t)EPI_WARPS * 2 * NG * CW * sizeof(float);
    static constexpr size_t RED_BYTES = (size_t)2 * 4 * TB * sizeof(float);
    static constexpr size_t FIXED = 1024 + kBarrierBytes + PART_BYTES + SCALE_BYTES + RED_BYTES +
                                    2 * (kMaxExperts + 1) * sizeof(int32_t);
    static constexpr int FIT = (int)((232448 - FIXED) / STAGE_BYTES);
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr size_t RING_BYTES = (size_t)STAGES * STAGE_BYTES;
    static constexpr size_t SMEM_BYTES = RING_BYTES + FIXED;
    static_assert(STAGES >= 4, "ring depth");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(TMEM_COLS <= 512, "TMEM budget");
    static_assert((2 * STAGES + 2 * NBUF + 5) * 8 + 16 <= (int)kBarrierBytes, "barriers");
};

struct SmallDev {
    const int32_t *offsets;
    int E;
    int n_wblocks;       // channel blocks (128 channels of C, or of g)
    int num_kb;
    int N;
    int w_blocks;        // ceil(N / 128)
    int64_t cap_rows;
    const float *a_scales;
    const float *w_scales;
    void *c;
    uint8_t *q2;
    float *s2;
    int32_t *status;
    int reset_status;    // first kernel of its call
    int split;           // CTAs per tile (the cluster's size)
    int early;           // offsets and weights were final before the previous kernel began
};

struct Tile {
    int e, row0, rows, wb;
};

__device__ __forceinline__ Tile decode(int64_t tile, const SmallDev &p, int TB, const int32_t *s_blk,
                                       const int32_t *s_off) {
    const int mblk = (int)(tile / p.n_wblocks);
    Tile t;
    t.wb = (int)(tile % p.n_wblocks);
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {   // last expert whose first row block is <= mblk
        const int mid = (lo + hi + 1) >> 1;
        if (s_blk[mid] <= mblk) lo = mid; else hi = mid - 1;
    }
    t.e = lo;
    t.row0 = s_off[lo] + (mblk - s_blk[lo]) * TB;
    t.rows = min(TB, s_off[lo + 1] - t.row0);
    return t;
}

// Arrival on the barrier at `bar`'s offset in CTA `rank`, ordering this
// thread's earlier shared-memory accesses across the cluster.
__device__ __forceinline__ void arrive_cluster(uint64_t *bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(bar, rank))
                 : "memory");
}
// The bounded wait that also acquires what other CTAs of the cluster released.
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort_flag,
                                             int32_t *status) {
    const uint64_t t0 = globaltimer();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(kWaitSliceNs)
            : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > kTimeoutNs) {
            *abort_flag = 1;
            if (status) atomicOr(status, MOE_DEV_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// a0 += s0 * d0, a1 += s1 * d1, one instruction.  Volatile, to stay behind the
// wait that makes the loaded d valid.
__device__ __forceinline__ void fma2(float &a0, float &a1, float s0, float s1, uint32_t d0, uint32_t d1) {
    asm volatile("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\t"
        "mov.b64 {%0, %1}, c;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "r"(d0), "r"(d1), "f"(s0), "f"(s1));
}

template <int EPI, int TB_>
__global__ void __launch_bounds__(THREADS, 1)
k_gemm_fp8_small(const __grid_constant__ CUtensorMap tmRows, const __grid_constant__ CUtensorMap tmW,
                 SmallDev p) {
    using C = Cfg<EPI, TB_>;
    constexpr int TB = C::TB, NG = C::NG, CW = C::CW, NBUF = C::NBUF, STAGES = C::STAGES;
    // aligned by its declaration, so that every address in it is a constant
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::RING_BYTES);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;
    uint64_t *acc_empty = acc_full + NBUF;
    uint64_t *drain = acc_empty + NBUF;
    uint64_t *part_full = drain + 1;       // every warp of the cluster's epilogues has written its partials
    uint64_t *part_free = part_full + 1;   // ... and has read everyone's
    uint64_t *red_bar = part_free + 1;     // [2]: the four quadrants of a row half
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(red_bar + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *s_part = reinterpret_cast<float *>(smem + C::RING_BYTES + kBarrierBytes);   // [NG][TB][BW]
    float *s_scale = s_part + C::PART_BYTES / sizeof(float);                           // [warp][2][NG][CW]
    float *s_red = s_scale + C::SCALE_BYTES / sizeof(float);                           // [2][4][TB]
    int32_t *s_off = reinterpret_cast<int32_t *>(s_red + C::RED_BYTES / sizeof(float));
    int32_t *s_blk = s_off + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.split;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], NG);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&acc_full[b], NG);
            mbar_init(&acc_empty[b], EPI_WARPS);
        }
        mbar_init(drain, 2);
        mbar_init(part_full, S * EPI_WARPS);
        mbar_init(part_free, S * EPI_WARPS);
        mbar_init(&red_bar[0], 4);
        mbar_init(&red_bar[1], 4);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmRows) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmW) : "memory");
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (!p.early) pdl_wait();   // everything below may read what earlier kernels wrote
    // Block 0 starts no later than any other, and no wait gives up before two
    // seconds have passed, so no bit set by this call is lost.
    if (p.reset_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    for (int i = threadIdx.x; i <= p.E; i += blockDim.x) s_off[i] = p.offsets[i];
    __syncthreads();
    if (warp == 0) {
        // s_blk[e] = TB-row blocks of the experts before e (warp scan)
        int carry = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            const int c = e < p.E ? (s_off[e + 1] - s_off[e] + TB - 1) / TB : 0;
            int x = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (e < p.E) s_blk[e] = carry + x - c;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) s_blk[p.E] = carry;
    }
    tc_fence_before();
    __syncthreads();
    // every CTA's barriers exist before any remote arrival: awaited only there
    if (S > 1) cluster_arrive();
    bool met = S == 1;   // this thread has waited for it
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int64_t total_tiles = (int64_t)s_blk[p.E] * p.n_wblocks;
    const int64_t first = blockIdx.x / S, step = gridDim.x / S;
    // this CTA's blocks of K
    const int kb0 = (int)((int64_t)p.num_kb * rank / S), kb1 = (int)((int64_t)p.num_kb * (rank + 1) / S);

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ weight producer
            int stage = 0;
            uint32_t phase = 0;
            int64_t armed = 0;   // stage uses
            bool ok = true;
            for (int64_t tile = first; ok && tile < total_tiles; tile += step) {
                const Tile t = decode(tile, p, TB, s_blk, s_off);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_bounded(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);   // the rows' bytes too
                    ++armed;
                    uint8_t *dst = smem + (size_t)stage * C::STAGE_BYTES;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        tma_load_3d(dst + g * W_BYTES, &tmW, &full[stage], kb * BK,
                                    g * (p.N / 2) + t.wb * BW, t.e);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            for (int64_t u = armed > STAGES ? armed - STAGES : 0; u < armed; ++u)
                ok = wait_bounded(&full[u % STAGES], (uint32_t)(u / STAGES) & 1u, abort_flag, p.status, false) && ok;
            if (!ok) {   // after a give-up, leave row copies still in flight time to land
                const uint64_t t0 = globaltimer();
                while (globaltimer() - t0 < 100000ull) __nanosleep(2000);
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            // ------------------------------------------------ row producer
            if (p.early) pdl_wait();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t tile = first; ok && tile < total_tiles; tile += step) {
                const Tile t = decode(tile, p, TB, s_blk, s_off);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_bounded(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    // rows past the tile's (another expert's, or zero fill) only
                    // reach accumulator columns that are never read
                    tma_load_2d(smem + (size_t)stage * C::STAGE_BYTES + NG * W_BYTES, &tmRows,
                                &full[stage], kb * BK, t.row0);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
        }
    } else if (warp == 1 || warp == 3) {
        if (lane == 0) {
            // ------------------------------------------------ MMA issuers
            const int me = warp >> 1;            // NG = 2: the group; NG = 1: every second block
            const int g = NG == 2 ? me : 0;
            int stage = 0;
            uint32_t phase = 0;
            int accb = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int64_t tile = first; ok && tile < total_tiles; tile += step) {
                const Tile t = decode(tile, p, TB, s_blk, s_off);
                const uint32_t idesc = idesc_e4m3(BW, ((t.rows + 15) / 16) * 16);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (NG == 2 || (accb & 1) == me) {
                        // The accumulator first: it is free once the block NBUF before
                        // has been added, so the stage's use before this one, which
                        // may have been the other issuer's, has landed by then and
                        // the second wait cannot take that phase for its own.
                        static_assert(STAGES >= NBUF, "a stage's last use is behind the accumulator's");
                        if (!wait_bounded(&acc_empty[accb], acc_phase ^ 1u, abort_flag, p.status) ||
                            !wait_bounded(&full[stage], phase, abort_flag, p.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d_tmem = tmem_base + (uint32_t)((accb * NG + g) * TB);
                        const uint32_t base = smem_u32(smem + (size_t)stage * C::STAGE_BYTES);
#pragma unroll
                        for (int k = 0; k < BK / 32; ++k)
                            mma_f8(d_tmem, desc_sw128(base + g * W_BYTES + 32 * k),
                                   desc_sw128(base + NG * W_BYTES + 32 * k), idesc, k > 0 ? 1u : 0u);
                        mma_commit(&acc_full[accb]);
                        mma_commit(&empty[stage]);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (++accb == NBUF) { accb = 0; acc_phase ^= 1u; }
                }
            }
            mma_commit(drain);
            wait_bounded(drain, 0, abort_flag, p.status, false);
        }
    } else if (warp >= EPI_WARP0) {
        // ---------------------------------------------------- epilogue warps
        if (p.early) pdl_wait();
        const int q = warp & 3;
        const int hf = (warp - EPI_WARP0) >> 2;
        const int c0 = hf * CW;                   // first row of this warp
        constexpr int LDW = CW < 32 || NG == 2 ? 16 : 32;   // columns per TMEM load
        constexpr int SPT = (CW + 31) / 32;       // row scales per lane
        float *my_scale = s_scale + (size_t)(warp - EPI_WARP0) * 2 * NG * CW;
        int accb = 0;
        uint32_t acc_phase = 0, tile_par = 0;
        int buf = 0;
        for (int64_t tile = first; tile < total_tiles; tile += step) {
            const Tile t = decode(tile, p, TB, s_blk, s_off);
            const int nj = (t.rows - c0 + LDW - 1) / LDW;   // column groups holding rows (may be <= 0)
            float acc[NG][CW];
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int i = 0; i < CW; ++i) acc[g][i] = 0.0f;
            const float *sw = p.w_scales + ((int64_t)t.e * p.w_blocks + t.wb) * p.num_kb;
            const float *sa[SPT];
            float sa_n[SPT], sw_n[NG];
#pragma unroll
            for (int u = 0; u < SPT; ++u) {
                // a row that exists, so that every lane may read its scales
                const int c = c0 + lane + 32 * u;
                const int64_t row = min((int64_t)t.row0 + (c < t.rows ? c : 0), p.cap_rows - 1);
                sa[u] = p.a_scales + row * p.num_kb;
                sa_n[u] = __ldg(sa[u] + kb0);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g)
                sw_n[g] = __ldg(sw + (int64_t)g * (p.w_blocks / 2) * p.num_kb + kb0);
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                float *sb = my_scale + buf * (NG * CW);
#pragma unroll
                for (int u = 0; u < SPT; ++u)
                    if (lane + 32 * u < CW)
#pragma unroll
                        for (int g = 0; g < NG; ++g) sb[g * CW + lane + 32 * u] = sa_n[u] * sw_n[g];
                __syncwarp();
                // in registers before the wait, where they fit
                constexpr int EARLY = CW <= 16 ? NG * CW : 4;
                float se[EARLY];
                if constexpr (CW <= 16)
#pragma unroll
                    for (int i = 0; i < NG * CW; i += 4)
                        *reinterpret_cast<float4 *>(se + i) = *reinterpret_cast<const float4 *>(sb + i);
                if (kb + 1 < kb1) {   // the next block's scales, while this one is awaited
#pragma unroll
                    for (int u = 0; u < SPT; ++u) sa_n[u] = __ldg(sa[u] + kb + 1);
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        sw_n[g] = __ldg(sw + (int64_t)g * (p.w_blocks / 2) * p.num_kb + kb + 1);
                }
                const bool w = wait_bounded_inline(&acc_full[accb], acc_phase, abort_flag, p.status);
                if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                tc_fence_after();
                const uint32_t taddr =
                    tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(accb * NG * TB + c0);
#pragma unroll
                for (int j = 0; j < CW / LDW; ++j) {
                    if (j < nj) {
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            uint32_t r[LDW];
                            if constexpr (LDW == 32) tmem_ld32(taddr + g * TB + LDW * j, r);
                            else tmem_ld16(taddr + g * TB + LDW * j, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < LDW; i += 4) {
                                const float4 s = *reinterpret_cast<const float4 *>(
                                    (CW <= 16 ? se : sb) + g * CW + LDW * j + i);
                                float *a = &acc[g][LDW * j + i];
                                fma2(a[0], a[1], s.x, s.y, r[i], r[i + 1]);
                                fma2(a[2], a[3], s.z, s.w, r[i + 2], r[i + 3]);
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[accb]);
                buf ^= 1;
                if (++accb == NBUF) { accb = 0; acc_phase ^= 1u; }
            }
            if (!ok) break;

            // sum i of this warp belongs to row c0 + i of the tile, or, after the
            // cluster's sums are joined, to row rank + S * (2 i + hf)
            if constexpr (C::SPLIT) {
                if (S > 1) {
                    if (!met) cluster_wait();
                    met = true;
                    if (!__all_sync(0xffffffffu, wait_cluster(part_free, tile_par ^ 1u, abort_flag, p.status)))
                        break;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int i = 0; i < CW; ++i)
                            if (c0 + i < t.rows) s_part[(g * TB + c0 + i) * BW + q * 32 + lane] = acc[g][i];
                    __syncwarp();
                    if (lane < S) arrive_cluster(part_full, (uint32_t)lane);
                    if (!__all_sync(0xffffffffu, wait_cluster(part_full, tile_par, abort_flag, p.status)))
                        break;
                    // a row's S partial sums are fetched together, then added in rank order
#pragma unroll
                    for (int i = 0; i < CW; ++i) {
                        const int c = rank + S * (2 * i + hf);
                        if (c >= t.rows) break;
                        float v[NG][kMaxSplit];
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int s = 0; s < kMaxSplit; ++s)
                                v[g][s] = s < S ? ld_cluster(cluster_addr(s_part + (g * TB + c) * BW + q * 32 + lane,
                                                                          (uint32_t)s))
                                                : 0.0f;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            acc[g][i] = v[g][0];
#pragma unroll
                            for (int s = 1; s < kMaxSplit; ++s) acc[g][i] += v[g][s];
                        }
                    }
                    __syncwarp();
                    if (lane < S) arrive_cluster(part_free, (uint32_t)lane);
                }
            }
            const int cs = S > 1 ? 2 * S : 1;                     // row of sum i: cf + cs * i
            const int cf = S > 1 ? rank + S * hf : c0;
            const int ch = t.wb * BW + q * 32 + lane;
            if constexpr (EPI == EPI_SWIGLU) {
                float *red = s_red + (size_t)tile_par * 4 * TB;   // [4][TB]
#pragma unroll
                for (int i = 0; i < CW; ++i) {
                    const int c = cf + cs * i;
                    if (c >= t.rows) break;
                    const float g = swiglu(acc[0][i], acc[NG - 1][i]);
                    acc[0][i] = g;
                    // magnitudes order as unsigned integers; a NaN counts as 0
                    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(g), 0.0f)));
                    if (lane == 0) red[q * TB + c] = __uint_as_float(m);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&red_bar[hf]);
                if (!__all_sync(0xffffffffu, wait_bounded(&red_bar[hf], tile_par, abort_flag, p.status)))
                    break;
                const int Nh = p.N / 2;
#pragma unroll
                for (int i = 0; i < CW; ++i) {
                    const int c = cf + cs * i;
                    if (c >= t.rows) break;
                    const int64_t row = (int64_t)t.row0 + c;
                    if (row >= p.cap_rows) break;
                    const volatile float *m = red + c;
                    float s, inv;
                    block_scale(fmaxf(fmaxf(m[0], m[TB]), fmaxf(m[2 * TB], m[3 * TB])), s, inv);
                    p.q2[row * Nh + ch] = (uint8_t)e4m3x2(acc[0][i] * inv, 0.0f);
                    if (q == 0 && lane == 0) p.s2[row * (Nh / kFp8Block) + t.wb] = s;
                }
            } else if (ch < p.N) {
#pragma unroll
                for (int i = 0; i < CW; ++i) {
                    const int c = cf + cs * i;
                    if (c >= t.rows) break;
                    const int64_t row = (int64_t)t.row0 + c;
                    if (row >= p.cap_rows) break;
                    if (EPI == EPI_BF16)
                        static_cast<__nv_bfloat16 *>(p.c)[row * p.N + ch] = __float2bfloat16_rn(acc[0][i]);
                    else
                        static_cast<float *>(p.c)[row * p.N + ch] = acc[0][i];
                }
            }
            tile_par ^= 1u;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (!met) cluster_wait();
    if (S > 1) cluster_sync();   // peers may still read this CTA's partial sums
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, C::TMEM_COLS);
}

template <int EPI, int TB>
moe_status launch(const Fp8GemmArgs &a, SmallDev d, cudaStream_t stream) {
    using C = Cfg<EPI, TB>;
    if (!set_smem_limit((const void *)k_gemm_fp8_small<EPI, TB>, C::SMEM_BYTES)) return MOE_ERR_CUDA;
    CUtensorMap mr, mw;
    const uint64_t rdims[2] = {(uint64_t)a.Kd, (uint64_t)a.cap_rows};
    const uint64_t rstr[1] = {(uint64_t)a.Kd};
    const uint32_t rbox[2] = {BK, TB};
    const uint64_t wdims[3] = {(uint64_t)a.Kd, (uint64_t)a.N, (uint64_t)a.E};
    const uint64_t wstr[2] = {(uint64_t)a.Kd, (uint64_t)a.Kd * a.N};
    const uint32_t wbox[3] = {BK, BW, 1};
    if (!make_tensor_map(&mr, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, a.a, 2, rdims,
                         rstr, rbox) ||
        !make_tensor_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, a.w, 3, wdims,
                         wstr, wbox))
        return MOE_ERR_CUDA;
    d.split = gemm_fp8_small_split(a);
    const char *names[3] = {"gemm_fp8_small_f32", "gemm_fp8_small_bf16", "gemm_fp8_small_swiglu"};
    const unsigned grid = (unsigned)(num_sms() / d.split * d.split);
    if (d.split == 1)
        MOE_LAUNCH(names[EPI], (k_gemm_fp8_small<EPI, TB>), grid, THREADS, C::SMEM_BYTES, stream, mr, mw, d);
    else
        MOE_LAUNCH_CLUSTER(names[EPI], (k_gemm_fp8_small<EPI, TB>), grid, THREADS, C::SMEM_BYTES, stream,
                           (unsigned)d.split, mr, mw, d);
    return MOE_OK;
}

template <int EPI>
moe_status launch_epi(const Fp8GemmArgs &a, const SmallDev &d, cudaStream_t stream) {
    return gemm_fp8_small_tile_rows(a) == 64 ? launch<EPI, 64>(a, d, stream) : launch<EPI, 32>(a, d, stream);
}

}  // namespace

// 32 rows where they average at most 16 an expert: few experts then have more.
int gemm_fp8_small_tile_rows(const Fp8GemmArgs &a) { return a.cap_rows > 16 * a.E ? 64 : 32; }

int gemm_fp8_small_split(const Fp8GemmArgs &a) {
    const int tb = gemm_fp8_small_tile_rows(a);
    if (a.q2 && !(tb == 32 ? Cfg<EPI_SWIGLU, 32>::SPLIT : Cfg<EPI_SWIGLU, 64>::SPLIT)) return 1;
    // Tiles at most this call can have: share them among clusters of 2, 4 or 8
    // CTAs while that still leaves no SM with a second tile.
    const int64_t wblocks = (a.N + BW - 1) / BW / (a.q2 ? 2 : 1), num_kb = (a.Kd + BK - 1) / BK;
    const int64_t tiles = (std::min<int64_t>(a.E, a.cap_rows) + a.cap_rows / tb) * wblocks;
    int split = 1;
    while (split < kMaxSplit && tiles * split * 2 <= num_sms() && split * 2 <= num_kb) split *= 2;
    return split;
}

moe_status launch_gemm_fp8_small(const Fp8GemmArgs &a, cudaStream_t stream) {
    SmallDev d;
    d.offsets = a.offsets;
    d.E = (int)a.E;
    d.num_kb = (int)((a.Kd + BK - 1) / BK);
    d.N = (int)a.N;
    d.w_blocks = (int)((a.N + kFp8Block - 1) / kFp8Block);
    d.n_wblocks = a.q2 ? d.w_blocks / 2 : d.w_blocks;
    d.cap_rows = a.cap_rows;
    d.a_scales = a.a_scales;
    d.w_scales = a.w_scales;
    d.c = a.c;
    d.q2 = static_cast<uint8_t *>(a.q2);
    d.s2 = a.s2;
    d.status = a.status;
    d.reset_status = a.reset_status;
    d.split = 1;
    d.early = a.early;
    if (a.q2) return launch_epi<EPI_SWIGLU>(a, d, stream);
    return a.out_bf16 ? launch_epi<EPI_BF16>(a, d, stream) : launch_epi<EPI_F32>(a, d, stream);
}

}  // namespace moe
