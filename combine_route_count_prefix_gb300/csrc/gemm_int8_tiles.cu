// gemm_int8_tiles.cu -- int8 products of tens to a few hundred rows a group, with one
// scale per row and one per output channel.
//
//   C[r, n] = (float(sum_k q[r, k] * W[e, n, k]) * w_scale[e, n]) * row_scale[r] + bias[e, n]
//
// The arithmetic is that of gemm_small.cu: the weights are the M side (128 output
// channels), widened from bytes to fp16 straight into tensor memory, the rows the N
// side, fp32 sums of at most 1024 products are exact, totals are int32.  What a call of
// this size waits for is not the products, though, but the steps before and behind them (64
// int8 rows of 7168 x 2048, 10.3 us, of which the weights' 2.2: start, offsets and first
// blocks 2.8, 8 blocks of K 2.6, last sums 0.7, exchange 1.1, stores 1.2, end and next start 1.9),
// so here
//   - int8 rows in tiles of 64 come as they are, and the warps that widen a block of weights
//     widen its rows, into the swizzled layout the MMA reads: no kernel makes images of
//     them first (64 rows of 7168 x 2048 12.2 -> 10.6 us).  For tiles of 128 it saved nothing
//     (4096 x 7168 19.0 / 18.8, 1536 x 2048 12.3 / 12.1): every CTA widens the rows again, and
//     shared memory carries each of them three times;
//   - three sets of four warps widen a block each, in turn, so that the way from a block's
//     arrival to its MMAs (half a microsecond) is not the time a block takes;
//   - where the tiles are fewer than SMs, a cluster of up to eight CTAs shares a tile's inner
//     dimension.  Its CTAs swap their parts through distributed shared memory with stores
//     that the receiver's barrier counts (against plain stores, a fence and an arrival,
//     4096 x 7168, 64 rows 14.8 -> 14.5 us; against sums added in L2, 128 rows of 1536 x 2048
//     13.0 -> 11.4),
//     four rows in turn to each, so the exchange, the scaling and the stores are shared out,
//     and nothing has to be cleared before the call.
//
// One CTA per SM, 16 warps:
//   warp 0       weight producer: TMA tiles of 128 channels x 128 bytes
//   warp 2       row producer: TMA tiles of TB rows x 128 bytes, or of two times 64 fp16 values
//   warps 1, 3   MMA issuers, each half of a block's K into its own accumulator
//   warps 4..15  three sets of converters: a thread a channel, shared -> tensor memory (lane
//                quadrant warp % 4), before it a share of the rows, shared -> shared
//   warps 8..15  epilogue too: 32 channels (lane quadrant warp % 4), half (warp - 8) / 4 of the
//                tile's rows
// Tiles are (group, TB rows, 128 channels), channels fastest.  The next chunk's first
// blocks are widened before this chunk's sums are taken, so that the MMAs go on meanwhile.
// Every wait is bounded (about two seconds) and sets MOE_DEV_TIMEOUT.
#include "common.cuh"
#include "groups.cuh"
#include "stream_i8.cuh"
#include "tcgen05.cuh"

#include <cudaTypedefs.h>

#include <algorithm>

namespace moe {
namespace {

using namespace tc;
using si8::widen_hi;
using si8::widen_lo;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int BW = 128;                  // output channels of a tile = MMA M
constexpr int BK = 128;                  // k-block
constexpr int BKH = 64;                  // one 128-byte swizzle atom of fp16 rows
constexpr int kSets = 3;                 // sets of converters
constexpr int W8_BYTES = BW * BK;
constexpr int CONV_WARP0 = 4, EPI_WARP0 = 8, EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr uint32_t TMEM_COLS = 512;
constexpr int ISSUERS = 2;
constexpr uint32_t ACC_COLS = 128;       // per issuer
constexpr uint32_t A_COL0 = ISSUERS * ACC_COLS;
constexpr uint32_t A_STAGE_COLS = BK / 2;
constexpr size_t kBarrierBytes = 512;
constexpr int kMaxSplits = 8;            // CTAs of a cluster

// ROWS8: the rows come as bytes and are widened here.
template <int TB_, bool ROWS8>
struct Cfg {
    static constexpr int TB = TB_;
    static constexpr int NBUF = (int)ACC_COLS / TB;     // accumulators per issuer
    static constexpr int CHUNK_KB = TB == 64 ? 8 : 16;  // k-blocks per exact chunk
    static constexpr int SA = TB == 64 ? 4 : 3;         // operand stages: TMEM A + widened rows
    static constexpr int S8 = TB == 64 ? 4 : 3;         // weight stages
    static constexpr int SR = 4;                        // stages of rows as bytes
    static constexpr int kAhead = SA - 1;               // k-blocks widened before a chunk's sums are taken
    static_assert(SA >= kSets, "a set's next block is at most one turn of a ring on");
    // What lets a set wait for a copy by its parity: behind ab_empty, and in rings no shorter than that one,
    // the block before in the slot has been multiplied, so its copy's phase is over and only this block's is open.
    static_assert(S8 >= SA && (!ROWS8 || SR >= SA), "a copy's phase is over when its stage is asked for again");
    static constexpr int R8_BYTES = TB * BK;
    static constexpr int B_HALF_BYTES = TB * BKH * 2;
    static constexpr int B_BYTES = 2 * B_HALF_BYTES;
    static constexpr int EPI_COLS = TB / 2;             // tile rows per epilogue warp
    static constexpr int PART_BYTES = EPI_WARPS * (EPI_COLS / 4) * 512;   // sums, as they are swapped
    static constexpr size_t RING_BYTES =
        (size_t)SA * B_BYTES + (size_t)S8 * W8_BYTES + (ROWS8 ? (size_t)SR * R8_BYTES : 0) + PART_BYTES;
    static constexpr size_t SMEM_BYTES = RING_BYTES + 1024 + kBarrierBytes + 2 * (kMaxExperts + 1) * sizeof(int32_t);
    static_assert(TB == 64 || (TB == 128 && !ROWS8), "tile heights");
    // each issuer adds BK / ISSUERS products per k-block; fp32 holds every integer sum of
    // at most 1024 int8 products exactly
    static_assert(CHUNK_KB * (BK / ISSUERS) <= 1024, "exact chunk");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
    static_assert(A_COL0 + SA * A_STAGE_COLS <= TMEM_COLS, "TMEM budget");
    static_assert((2 * S8 + 2 * SR + 2 * SA + 2 * NBUF + 1 + 2 * EPI_WARPS) * 8 + 16 <= (int)kBarrierBytes, "barriers");
};

struct TilesDev {
    const int32_t *offsets;
    int E, n_wblocks, num_kb, Nout, splits;
    int64_t cap_rows;
    const float *w_scales, *row_scales, *bias;
    __nv_bfloat16 *y16;
    float *y32;
    int32_t *status;
    int early;           // everything but the codes and their scales was final before the kernel before this one began
};

struct Tile {
    int e, row0, rows, wb;
};
template <int TB>
__device__ __forceinline__ Tile decode_tile(int64_t tile, int n_wblocks, int E, const int32_t *s_blk, const int32_t *s_off) {
    Tile t;
    const int blk = (int)(tile / n_wblocks);
    t.wb = (int)(tile % n_wblocks);
    int lo = 0, hi = E - 1;
    while (lo < hi) {   // last group whose first block is <= blk
        const int mid = (lo + hi + 1) >> 1;
        if (s_blk[mid] <= blk) lo = mid; else hi = mid - 1;
    }
    t.e = lo;
    t.row0 = s_off[lo] + (blk - s_blk[lo]) * TB;
    t.rows = min(TB, s_off[lo + 1] - t.row0);
    return t;
}

// Waits for arrivals from the cluster's other CTAs, and sees what they wrote before.
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kWaitSliceNs)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int32_t *status) {
    const uint64_t t0 = globaltimer();
    for (;;) {
        if (try_wait_cluster(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer() - t0 > kTimeoutNs) {
            *abort_flag = 1;
            atomicOr(status, MOE_DEV_TIMEOUT);
            return false;
        }
    }
}
// 16 bytes into a cluster CTA's shared memory, counted by the barrier there.  Only in
// launches with a cluster: without one it is an illegal instruction.
__device__ __forceinline__ void store_part(uint32_t addr, int32_t a, int32_t b, int32_t c, int32_t d, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.s32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int TB, bool ROWS8>
__global__ void __launch_bounds__(THREADS, 1)
k_int8_tiles(const __grid_constant__ CUtensorMap tmRows, const __grid_constant__ CUtensorMap tmW, TilesDev p) {
    using C = Cfg<TB, ROWS8>;
    constexpr int NBUF = C::NBUF, CHUNK_KB = C::CHUNK_KB, EPI_COLS = C::EPI_COLS, S8 = C::S8, SR = C::SR, SA = C::SA;
    constexpr int B_HALF_BYTES = C::B_HALF_BYTES, B_BYTES = C::B_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *ringB = smem;
    uint8_t *ring8 = smem + (size_t)SA * B_BYTES;
    uint8_t *ringR = ring8 + (size_t)S8 * W8_BYTES;
    uint8_t *part_mem = ringR + (ROWS8 ? (size_t)SR * C::R8_BYTES : 0);
    uint64_t *w8_full = reinterpret_cast<uint64_t *>(smem + C::RING_BYTES);
    uint64_t *w8_empty = w8_full + S8;
    uint64_t *r8_full = w8_empty + S8;
    uint64_t *r8_empty = r8_full + SR;
    uint64_t *ab_full = r8_empty + SR;
    uint64_t *ab_empty = ab_full + SA;
    uint64_t *acc_full = ab_empty + SA;
    uint64_t *acc_empty = acc_full + NBUF;
    uint64_t *drain = acc_empty + NBUF;
    uint64_t *parts = drain + 1;               // [EPI_WARPS] the parts for this CTA's warp are there
    uint64_t *parts_read = parts + EPI_WARPS;  // [EPI_WARPS] the same warps of the cluster have read theirs
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(parts_read + EPI_WARPS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int32_t *s_blk = reinterpret_cast<int32_t *>(smem + C::RING_BYTES + kBarrierBytes);
    int32_t *s_off = s_blk + (kMaxExperts + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = p.splits, rank = splits > 1 ? (int)cluster_ctarank() : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S8; ++s) {
            mbar_init(&w8_full[s], 1);
            mbar_init(&w8_empty[s], 4);
        }
        for (int s = 0; s < SR; ++s) {
            mbar_init(&r8_full[s], 1);
            mbar_init(&r8_empty[s], 4);
        }
        for (int s = 0; s < SA; ++s) {
            mbar_init(&ab_full[s], ROWS8 ? 4 : 5);
            mbar_init(&ab_empty[s], ISSUERS);
        }
        for (int b = 0; b < NBUF; ++b) {
            mbar_init(&acc_full[b], ISSUERS);
            mbar_init(&acc_empty[b], EPI_WARPS);
        }
        mbar_init(drain, ISSUERS);
        for (int w = 0; w < EPI_WARPS; ++w) {
            mbar_init(&parts[w], 1);
            mbar_init(&parts_read[w], (uint32_t)splits);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmRows) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmW) : "memory");
    }
    if (splits > 1) {
        __syncwarp();
        cluster_arrive();   // the others may arrive at this CTA's barriers once all have come so far
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    if (!p.early) pdl_wait();
    const int64_t first = blockIdx.x / splits, step = gridDim.x / splits;
    const int kb0 = p.num_kb * rank / splits, kb1 = p.num_kb * (rank + 1) / splits;   // this CTA's k-blocks
    // With one group the first tile's weights need no offsets (int8, 17 rows of 4096 x 7168
    // 12.7 -> 11.9 us, 32 of 7168 x 2048 9.9 -> 9.4, with the cluster that need not end together, below).
    // The offsets are asked for first: behind the weights they would come later.
    const int ahead = p.E == 1 ? min(S8, kb1 - kb0) : 0;
    int32_t off = 0;
    if (warp == 0 && lane <= p.E) off = p.offsets[lane];
    if (threadIdx.x == 0)
        for (int s = 0; s < ahead; ++s) {
            mbar_arrive_expect_tx(&w8_full[s], W8_BYTES);
            tma_load_3d(ring8 + (size_t)s * W8_BYTES, &tmW, &w8_full[s], (kb0 + s) * BK, (int)(first % p.n_wblocks) * BW, 0);
        }
    __syncwarp();
    if (warp == 0) {
        if (lane <= p.E) s_off[lane] = off;
        for (int i = lane + 32; i <= p.E; i += 32) s_off[i] = p.offsets[i];
        __syncwarp();
        bound_offsets(s_off, p.E, p.cap_rows);
        count_blocks(s_off, s_blk, p.E, TB);
    }
    tc_fence_before();
    __syncthreads();
    if (splits > 1) cluster_wait();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int64_t tiles = (int64_t)s_blk[p.E] * p.n_wblocks;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ weight producer
            int stage = 0;
            uint32_t phase = 0;
            int issued_phase[S8];
#pragma unroll
            for (int s = 0; s < S8; ++s) issued_phase[s] = s < ahead ? 0 : -1;
            if (ahead == S8) phase = 1;
            else stage = ahead;
            bool ok = true;
            for (int64_t tile = first; ok && tile < tiles; tile += step) {
                const Tile t = decode_tile<TB>(tile, p.n_wblocks, p.E, s_blk, s_off);
                for (int kb = tile == first ? kb0 + ahead : kb0; kb < kb1; ++kb) {
                    if (!wait_bounded(&w8_empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    mbar_arrive_expect_tx(&w8_full[stage], W8_BYTES);
                    tma_load_3d(ring8 + (size_t)stage * W8_BYTES, &tmW, &w8_full[stage], kb * BK, t.wb * BW, t.e);
                    issued_phase[stage] = (int)phase;
                    if (++stage == S8) { stage = 0; phase ^= 1u; }
                }
            }
            for (int s = 0; s < S8; ++s)   // copies in flight land before the CTA's memory goes
                if (issued_phase[s] >= 0)
                    wait_bounded(&w8_full[s], (uint32_t)issued_phase[s], abort_flag, p.status, false);
        }
    } else if (warp == 2) {
        if (lane == 0) {
            // ------------------------------------------------ row producer: bytes, or images straight into
            // the operand stages
            constexpr int S = ROWS8 ? SR : SA;
            uint64_t *full = ROWS8 ? r8_full : ab_full, *empty = ROWS8 ? r8_empty : ab_empty;
            if (p.early) pdl_wait();
            int stage = 0;
            uint32_t phase = 0;
            int issued_phase[S];
#pragma unroll
            for (int s = 0; s < S; ++s) issued_phase[s] = -1;
            bool ok = true;
            for (int64_t tile = first; ok && tile < tiles; tile += step) {
                const Tile t = decode_tile<TB>(tile, p.n_wblocks, p.E, s_blk, s_off);
                for (int kb = kb0; ok && kb < kb1; ++kb) {
                    ok = wait_bounded(&empty[stage], phase ^ 1u, abort_flag, p.status);
                    if (!ok) break;
                    if (ROWS8) {
                        mbar_arrive_expect_tx(&full[stage], (uint32_t)C::R8_BYTES);
                        tma_load_2d(ringR + (size_t)stage * C::R8_BYTES, &tmRows, &full[stage], kb * BK, t.row0);
                    } else {
                        uint8_t *dst = ringB + (size_t)stage * B_BYTES;
                        mbar_arrive_expect_tx(&full[stage], (uint32_t)B_BYTES);
                        tma_load_2d(dst, &tmRows, &full[stage], kb * BK, t.row0);
                        tma_load_2d(dst + B_HALF_BYTES, &tmRows, &full[stage], kb * BK + BKH, t.row0);
                    }
                    issued_phase[stage] = (int)phase;
                    if (++stage == S) { stage = 0; phase ^= 1u; }
                }
            }
            // copies in flight land before the CTA's memory goes; an operand stage that waits for
            // converters which gave up would never fill, so that there the time limit is the wait
            for (int s = 0; s < S; ++s)
                if (issued_phase[s] >= 0)
                    wait_bounded(&full[s], (uint32_t)issued_phase[s], abort_flag, p.status, false);
        }
    } else if (warp == 1 || warp == 3) {
        // ---------------------------------------------------- MMA issuers
        const int is = __shfl_sync(kFull, warp >> 1, 0);   // 0 or 1: K [64 is, 64 is + 64) of every k-block
        const uint32_t tm = __shfl_sync(kFull, tmem_base, 0);
        int stage = 0, accb = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int64_t tile = first; ok && tile < tiles; tile += step) {
            const Tile t = decode_tile<TB>(tile, p.n_wblocks, p.E, s_blk, s_off);
            const uint32_t idesc = __shfl_sync(kFull, idesc_f16(BW, (t.rows + 15) / 16 * 16), 0);
            for (int c0 = kb0; ok && c0 < kb1; c0 += CHUNK_KB) {
                ok = __all_sync(kFull, wait_bounded(&acc_empty[accb], acc_phase ^ 1u, abort_flag, p.status));
                if (!ok) break;
                tc_fence_after();
                const uint32_t d_tmem = tm + (uint32_t)(is * ACC_COLS + accb * TB);
                const int c1 = min(c0 + CHUNK_KB, kb1);
                for (int kb = c0; kb < c1; ++kb) {
                    ok = __all_sync(kFull, wait_bounded(&ab_full[stage], phase, abort_flag, p.status));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a_tmem = tm + A_COL0 + (uint32_t)stage * A_STAGE_COLS;
                    const uint32_t b_addr = smem_u32(ringB + (size_t)stage * B_BYTES);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // K = 16: 8 TMEM columns, 32 bytes of a row
                            mma_f16_ta(d_tmem, a_tmem + 32 * is + 8 * k, desc_sw128(b_addr + is * B_HALF_BYTES + 32 * k),
                                       idesc, (kb > c0 || k > 0) ? 1u : 0u);
                        mma_commit(&ab_empty[stage]);
                    }
                    __syncwarp();
                    if (++stage == SA) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                if (elect_one()) mma_commit(&acc_full[accb]);
                __syncwarp();
                if (++accb == NBUF) { accb = 0; acc_phase ^= 1u; }
            }
        }
        if (elect_one()) mma_commit(drain);
        __syncwarp();
        wait_bounded(drain, 0, abort_flag, p.status, false);
    } else if (warp >= CONV_WARP0) {
        // ---------------------------------------------------- converters
        if (p.early) pdl_wait();
        if (ROWS8 && blockIdx.x == 0 && threadIdx.x == 32 * CONV_WARP0) *p.status = 0;   // else cleared already
        const int q = warp & 3, set = (warp - CONV_WARP0) >> 2;
        const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
        const int nk = kb1 - kb0;
        int s8 = set, sr = set, sa = set;        // this set's next block's stages
        uint32_t ph8 = 0, phr = 0, pha = 0;
        int next = set;                          // and its number in the tile
        // Widens this set's blocks before number `to` of a tile with rows16 rows.
        auto widen = [&](int to, int rows16) -> bool {
            for (; next < to; next += kSets) {
                // ab_empty first: the slot's block before is another set's, and until it has been multiplied its
                // own rows may still be on their way (copies land in any order), one phase behind, where this
                // block's parity passes at once.  ab_empty itself cannot be two phases behind: MMAs complete in
                // order, and this set has seen the block after that one multiplied.
                bool w = wait_bounded_inline(&ab_empty[sa], pha ^ 1u, abort_flag, p.status) &&
                         (!ROWS8 || wait_bounded_inline(&r8_full[sr], phr, abort_flag, p.status));
                if (!__all_sync(kFull, w)) return false;
                if (ROWS8) {
                    // rows: bytes in ringR -> fp16 in ringB, 128-byte rows of 64 values.  Values 16 u .. go to
                    // units 2 (u % 4) and the next of half u / 4; the halves store theirs in opposite orders, so
                    // that no bank is met twice.
                    const uint32_t rows8 = smem_u32(ringR + (size_t)sr * C::R8_BYTES);
                    const uint32_t rowsB = smem_u32(ringB + (size_t)sa * B_BYTES);
#pragma unroll 4
                    for (int it = 0; it < TB / 16; ++it) {
                        const int r = it * 16 + q * 4 + (lane >> 3), u = lane & 7;
                        if (r < rows16) {
                            const uint4 v = si8::lds16(rows8 + (uint32_t)(r * 128) + si8::unit_at(r, u));
                            const uint32_t x[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
                            const uint32_t row = rowsB + (uint32_t)((u >> 2) * B_HALF_BYTES + r * 128);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int half = j ^ (u >> 2);
                                const uint32_t a = half ? x[2] : x[0], b = half ? x[3] : x[1];
                                sts16(row + si8::unit_at(r, 2 * (u & 3) + half), widen_lo(a), widen_hi(a), widen_lo(b), widen_hi(b));
                            }
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                w = wait_bounded_inline(&w8_full[s8], ph8, abort_flag, p.status);
                if (!__all_sync(kFull, w)) return false;
                if (ROWS8 && lane == 0) mbar_arrive(&r8_empty[sr]);
                // weights: this thread's channel, 128 bytes -> its TMEM lane
                const int row = q * 32 + lane;
                const uint32_t src = smem_u32(ring8 + (size_t)s8 * W8_BYTES) + (uint32_t)row * 128u;
                const uint32_t dst = tmem_base + lane_addr + A_COL0 + (uint32_t)sa * A_STAGE_COLS;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t words[16];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 x = si8::lds16(src + si8::unit_at(row, 2 * h + i));
                        const uint32_t b4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            words[8 * i + 2 * j] = widen_lo(b4[j]);
                            words[8 * i + 2 * j + 1] = widen_hi(b4[j]);
                        }
                    }
                    tmem_st16(dst + 16 * h, words);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&w8_empty[s8]);
                    mbar_arrive(&ab_full[sa]);
                }
                s8 += kSets;
                if (s8 >= S8) { s8 -= S8; ph8 ^= 1u; }
                sr += kSets;
                if (sr >= SR) { sr -= SR; phr ^= 1u; }
                sa += kSets;
                if (sa >= SA) { sa -= SA; pha ^= 1u; }
            }
            return true;
        };
        const int ew = warp - EPI_WARP0;         // below 0: no part in the epilogue
        const int c0 = (ew >> 2) * EPI_COLS;     // first tile row of this warp
        int accb = 0;
        uint32_t acc_phase = 0, part_phase = 0, read_phase = 1;
        // columns per TMEM load: 16 when a warp holds 64 rows' sums, so the load
        // buffer and the sums fit the registers together
        constexpr int LDW = EPI_COLS > 32 ? 16 : 32;
        bool ok = true;
        for (int64_t tile = first; ok && tile < tiles; tile += step, next -= nk) {
            const Tile t = decode_tile<TB>(tile, p.n_wblocks, p.E, s_blk, s_off);
            const int rows16 = (t.rows + 15) / 16 * 16;
            const int n = ew < 0 ? 0 : max(0, min(t.rows - c0, EPI_COLS));   // this warp's rows
            // behind the sums a lane takes row lane / 8 of a row group, channels ch .. ch + 3 (N is a multiple of 8)
            const int ch = t.wb * BW + q * 32 + (lane & 7) * 4;
            const bool in = ch < p.Nout && n > 0;
            const int64_t wn = (int64_t)t.e * p.Nout + ch;
            if (in) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.w_scales + wn));
            int32_t acc[EPI_COLS];
#pragma unroll
            for (int i = 0; i < EPI_COLS; ++i) acc[i] = 0;
            for (int c = 0; c < nk; c += CHUNK_KB) {
                ok = widen(min(nk, c + CHUNK_KB + C::kAhead), rows16);
                if (!ok) break;
                if (ew < 0) continue;
                ok = __all_sync(kFull, wait_bounded_inline(&acc_full[accb], acc_phase, abort_flag, p.status));
                if (!ok) break;
                tc_fence_after();
                const uint32_t taddr = tmem_base + lane_addr + (uint32_t)(accb * TB + c0);
#pragma unroll
                for (int j = 0; j < EPI_COLS / LDW; ++j) {
                    if (LDW * j < n) {
#pragma unroll
                        for (int is = 0; is < ISSUERS; ++is) {
                            uint32_t r[LDW];
                            if constexpr (LDW == 32)
                                tmem_ld32(taddr + is * ACC_COLS + LDW * j, r);
                            else
                                tmem_ld16(taddr + is * ACC_COLS + LDW * j, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < LDW; ++i) acc[LDW * j + i] += __float2int_rn(__uint_as_float(r[i]));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[accb]);
                if (++accb == NBUF) { accb = 0; acc_phase ^= 1u; }
            }
            if (!ok) break;
            if (n == 0) continue;
            const float *s2 = p.row_scales + t.row0 + c0;
            float s_lane[EPI_COLS / 32];         // the rows' scales, one a lane
#pragma unroll
            for (int h = 0; h < EPI_COLS / 32; ++h) s_lane[h] = 32 * h + lane < n ? __ldcg(s2 + 32 * h + lane) : 0.0f;
            float4 sc = make_float4(0.0f, 0.0f, 0.0f, 0.0f), bias = sc;
            if (in) sc = __ldg(reinterpret_cast<const float4 *>(p.w_scales + wn));
            if (in && p.bias) bias = __ldg(reinterpret_cast<const float4 *>(p.bias + wn));
            // The sums go through shared memory, split or not: a loop over it is short code, where
            // registers would be stored in straight code that is fetched line by line.  Row group g
            // (four rows) goes to CTA g % splits, place (its rank, g / splits) of this warp's slots there.
            const int groups = (n + 3) / 4, mine = (groups - rank + splits - 1) / splits;   // rank < splits: not negative
            // channel `lane` at a place from where eight lanes read every fourth without a bank twice
            const uint32_t slots = smem_u32(part_mem) + (uint32_t)(ew * (EPI_COLS / 4) * 512 + (lane ^ (lane >> 3)) * 16);
            const uint32_t per = (uint32_t)(EPI_COLS / 4 / splits) * 512u;
            if (splits > 1) {
                ok = __all_sync(kFull, wait_cluster(&parts_read[ew], read_phase, abort_flag, p.status));
                if (!ok) break;
                read_phase ^= 1u;
            }
            if (splits > 1 && lane == 0 && mine > 0) mbar_arrive_expect_tx(&parts[ew], (uint32_t)(mine * splits * 512));
            uint32_t at = slots + (uint32_t)rank * per;
            int to = 0;
#pragma unroll
            for (int g = 0; g < EPI_COLS / 4; ++g) {
                asm volatile("" : "+r"(at));
                if (4 * g < n && splits == 1) sts16(at, acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
                if (4 * g < n && splits > 1)
                    store_part(map_rank(at, to), acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3],
                               map_rank(smem_u32(&parts[ew]), to));
                if (++to == splits) { to = 0; at += 512; }
            }
            if (splits > 1 && mine > 0) {
                ok = __all_sync(kFull, wait_cluster(&parts[ew], part_phase, abort_flag, p.status));
                if (!ok) break;
                part_phase ^= 1u;
            }
            __syncwarp();
            const int c4 = (lane & 7) * 4, r4 = lane >> 3;
            const int32_t *part = reinterpret_cast<const int32_t *>(part_mem) + ew * (EPI_COLS / 4) * 128 + r4;
            const int per4 = (int)(per / 4);
            const bool with_bias = p.bias != nullptr;
#pragma unroll 1
            for (int g = rank; g < groups; g += splits, part += 128) {
                int32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 2
                for (int s = 0; s < splits; ++s)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] += part[s * per4 + ((c4 + j) ^ (c4 >> 3)) * 4];
                const float s = __shfl_sync(kFull, EPI_COLS == 32 || g < 8 ? s_lane[0] : s_lane[EPI_COLS / 32 - 1],
                                            (4 * g + r4) & 31);
                const float w[4] = {sc.x, sc.y, sc.z, sc.w}, b[4] = {bias.x, bias.y, bias.z, bias.w};
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = __fmul_rn(__fmul_rn(__int2float_rn(sum[j]), w[j]), s);
                    const float vb = __fadd_rn(v[j], b[j]);
                    v[j] = with_bias ? vb : v[j];
                }
                const int64_t o = (int64_t)(t.row0 + c0 + 4 * g + r4) * p.Nout + ch;
                if (in && 4 * g + r4 < n) {
                    if (p.y32) {
                        *reinterpret_cast<float4 *>(p.y32 + o) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
                        *reinterpret_cast<uint2 *>(p.y16 + o) =
                            make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                    }
                }
            }
            __syncwarp();
            // (not behind the last tile: nobody waits for it)
            if (splits > 1 && lane < splits && tile + step < tiles) mbar_arrive_remote(&parts_read[ew], lane);
        }
    }

    tc_fence_before();
    __syncthreads();
    // With one tile a CTA has waited for all that is written to it.  With more, arrivals may still be on
    // their way; and where a wait gave up, parts, which get time to land.
    if (splits > 1 && (*abort_flag || first + step < tiles)) {
        if (*abort_flag) {
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 100000ull) __nanosleep(2000);
        }
        __syncwarp();
        cluster_sync();
    }
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
}

// Clusters of `splits` CTAs that the GPU holds at once.
template <int TB, bool ROWS8>
int clusters_at_once(int splits) {
    static int known[kMaxDevices][kMaxSplits + 1];   // clusters + 1, 0 where not asked yet
    int &cached = known[current_device()][splits];
    if (cached == 0) {
        if (!set_smem_limit((const void *)(k_int8_tiles<TB, ROWS8>), (Cfg<TB, ROWS8>::SMEM_BYTES))) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms() / splits * splits));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = (Cfg<TB, ROWS8>::SMEM_BYTES);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)splits;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, (const void *)(k_int8_tiles<TB, ROWS8>), &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        cached = n + 1;
    }
    return cached - 1;
}

// One group's rows are known, those of several spread (rows dealt to groups at random, us, tiles of 64
// rows against 128: 48 a group, 7 of 1000 x 1456 10.6 / 12.0, 32 of 2048 x 2048 38.8 / 39.6; 60 a group
// 12.3 / 12.2, 44.5 / 41.1).
bool wide_tiles(int64_t rows, int64_t E) { return rows > (E == 1 ? 64 : 48 * E); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int TB, bool ROWS8>
moe_status launch_tb(const Int8TilesArgs &a, int splits, cudaStream_t stream) {
    CUtensorMap mr, mw;
    const uint64_t rdims[2] = {(uint64_t)a.Kd, (uint64_t)a.cap_rows};
    const uint64_t rstr[1] = {(uint64_t)a.Kd * (ROWS8 ? 1 : 2)};
    const uint32_t rbox[2] = {(uint32_t)(ROWS8 ? BK : BKH), TB};
    const uint64_t wdims[3] = {(uint64_t)a.Kd, (uint64_t)a.N, (uint64_t)a.E};
    const uint64_t wstr[2] = {(uint64_t)a.Kd, (uint64_t)a.Kd * a.N};
    const uint32_t wbox[3] = {BK, BW, 1};
    if (!make_tensor_map(&mr, ROWS8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                         CU_TENSOR_MAP_SWIZZLE_128B, a.rows, 2, rdims, rstr, rbox) ||
        !make_tensor_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, a.w, 3, wdims, wstr, wbox))
        return MOE_ERR_CUDA;
    TilesDev d;
    d.offsets = a.offsets;
    d.E = (int)a.E;
    d.n_wblocks = (int)ceil_div(a.N, BW);
    d.num_kb = (int)ceil_div(a.Kd, BK);
    d.Nout = (int)a.N;
    d.splits = splits;
    d.cap_rows = a.cap_rows;
    d.w_scales = a.w_scales;
    d.row_scales = a.row_scales;
    d.bias = a.bias;
    d.y16 = a.out_bf16 ? static_cast<__nv_bfloat16 *>(a.c) : nullptr;
    d.y32 = a.out_bf16 ? nullptr : static_cast<float *>(a.c);
    d.status = a.status;
    d.early = a.early;
    constexpr size_t smem = (Cfg<TB, ROWS8>::SMEM_BYTES);
    if (!set_smem_limit((const void *)(k_int8_tiles<TB, ROWS8>), smem)) return MOE_ERR_CUDA;
    const int64_t tiles = (a.cap_rows / TB + std::min(a.E, a.cap_rows)) * d.n_wblocks;   // at most
    if (splits > 1) {
        const int64_t clusters = std::min<int64_t>(tiles, (clusters_at_once<TB, ROWS8>(splits)));
        MOE_LAUNCH_CLUSTER("int8_tiles", (k_int8_tiles<TB, ROWS8>), (unsigned)(clusters * splits), THREADS, smem, stream,
                           (unsigned)splits, mr, mw, d);
    } else {
        MOE_LAUNCH("int8_tiles", (k_int8_tiles<TB, ROWS8>), (unsigned)std::min<int64_t>(tiles, num_sms()), THREADS, smem, stream,
                   mr, mw, d);
    }
    return MOE_OK;
}

}  // namespace

// Measured (us), in brackets the small-batch kernel with whole tiles:
//   one group, 64 rows: 4096 x 7168 in four 16.3 (39), 7168 x 2048 in two 12.2 (17)
//   128 rows: 4096 x 7168 in four 19.3 (33), 1536 x 2048 in four 11.4 (13.5), 7168 x 2048 in two 15.3 (13.4)
//   32 groups of 20 rows, 2048 x 2048, 512 tiles: 42 (39)
// Tiles of 128 rows are bound by their copies, so that a split has to save more than the exchange takes;
// where there are more tiles than SMs, the small-batch kernel, whose epilogue does not widen, goes on with the next.
Int8TilesPlan int8_tiles_plan(int64_t rows, bool bytes, int64_t E, int64_t N, int64_t Kd) {
    Int8TilesPlan t;
    t.wide = wide_tiles(rows, E);
    const int64_t tb = t.wide ? 128 : 64, groups = std::max<int64_t>(1, std::min(E, rows));
    const int64_t tiles = groups * ceil_div(ceil_div(rows, groups), tb) * ceil_div(N, BW);   // with the rows spread evenly
    const int64_t waves = ceil_div(tiles, num_sms());
    t.splits = (int)std::max<int64_t>(1, std::min<int64_t>({num_sms() / std::max<int64_t>(1, tiles), Kd / 512, kMaxSplits}));
    auto fit = [&](int splits) {
        return t.wide ? clusters_at_once<128, false>(splits)
                      : bytes ? clusters_at_once<64, true>(splits) : clusters_at_once<64, false>(splits);
    };
    while (t.splits > 1 && ((t.splits & (t.splits - 1)) != 0 || fit(t.splits) < tiles)) --t.splits;
    // estimates (us) by the blocks of K that a CTA goes through
    const double kb = (double)ceil_div(Kd, BK);
    const double whole = 3.5 + (double)waves * (2.0 + kb * (t.wide ? 0.5 : 0.35));
    const double swapped = t.wide ? 8.0 + 0.85 * kb / t.splits : 7.0 + 0.4 * kb / t.splits;
    t.whole = waves > 1 || (t.wide && (t.splits == 1 || whole <= swapped));
    t.bytes = bytes && !t.whole && !t.wide;
    t.us = t.whole ? whole : swapped;
    return t;
}

moe_status launch_int8_tiles(const Int8TilesArgs &a, const Int8TilesPlan &t, cudaStream_t stream) {
    if (t.wide) return launch_tb<128, false>(a, t.splits, stream);
    return t.bytes ? launch_tb<64, true>(a, t.splits, stream) : launch_tb<64, false>(a, t.splits, stream);
}

}  // namespace moe
