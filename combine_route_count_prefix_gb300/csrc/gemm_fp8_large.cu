// gemm_fp8_large.cu -- grouped products of block-scaled e4m3 operands for many
// rows per expert, on pairs of SMs.
//
//   C[r, n] = sum_b a_scales[r, b] * w_scales[e, n / 128, b]
//                   * sum_{k in block b} A[r, k] * W[e, n, k]
//
// The tensor cores sum the 128 products of one block b in fp32; the scales
// differ from block to block, so every block gets an accumulator of its own,
// which the epilogue warps read back, multiply by the row's and the channel
// block's scale and add to fp32 sums in registers, while the tensor cores work
// on the next block in the other accumulator.
//
// Kernel shape (a cluster of two CTAs per 256-row x 256-channel tile, as many
// clusters as fit, 320 threads):
//   warp 0      TMA producer: the CTA's 128 rows and its 128 of the 256
//               channels, 128 bytes of K each (16 + 16 KB), six-stage ring;
//               both CTAs' loads complete on CTA 0's barrier
//   warp 1      TMEM (two 256-column accumulators) and, in CTA 0, the MMA
//               issuer: 4 x tcgen05.mma cta_group::2 M=256 N=256 K=32 a block
//   warps 2..9  epilogue: TMEM lane quadrant q (32 rows) x column half
// The pair's tile halves the weight bytes each SM stages, which a one-SM tile
// of the same height would read twice.
// SwiGLU form: CTA 0 stages 128 SiLU-half channels and CTA 1 the multiplier
// channels of the same numbers, so a tile holds 128 complete channels of g and
// the epilogue quantises them as one block; h never leaves the SM.
// Every wait is bounded (about two seconds) and sets MOE_DEV_TIMEOUT.
#include "common.cuh"
#include "fp8.cuh"
#include "tcgen05.cuh"

#include <cuda.h>

namespace moe {
namespace {

using namespace tc;

constexpr int BM = 128;                 // rows per CTA (256 per pair)
constexpr int BN = 256;                 // channels per tile
constexpr int BK = 128;                 // bytes of K per block: one scale
constexpr int STAGES = 6;
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = (BN / 2) * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr size_t RING_BYTES = (size_t)STAGES * STAGE_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 512;
constexpr size_t kBarrierBytes = 512;
constexpr size_t kAmaxBytes = 2 * 2 * BM * sizeof(float);
constexpr size_t SMEM_BYTES =
    RING_BYTES + 1024 + kBarrierBytes + kAmaxBytes + 2 * (kMaxExperts + 1) * sizeof(int32_t);
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert((2 * STAGES + 9) * 8 + 16 <= (int)kBarrierBytes, "barriers");

enum { EPI_F32 = 0, EPI_BF16 = 1, EPI_SWIGLU = 2 };

struct LargeDev {
    const int32_t *offsets;
    int E;
    int n_blocks;        // column blocks: 256 channels (128 channels of g for SwiGLU)
    int num_kb;
    int N;               // channels of W (both halves for SwiGLU)
    int w_blocks;        // ceil(N / 128)
    int64_t cap_rows;
    const float *a_scales;
    const float *w_scales;
    void *c;             // F32, BF16: [cap_rows, N]
    uint8_t *q2;         // SwiGLU: [cap_rows, N/2]
    float *s2;           //         [cap_rows, N/256]
    int32_t *status;
};

// The pair's tile: expert, this CTA's first row, its rows there (may be <= 0
// or more than BM) and the column block.
struct Tile {
    int e, row0, rows, nb;
};

// Column-block-major within an expert: the clusters in flight share few weight
// tiles, each read by all of the expert's row blocks while it is in L2.
__device__ __forceinline__ Tile decode(int64_t tile, const LargeDev &p, const int32_t *s_blk,
                                       const int32_t *s_off, int rank) {
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {   // last expert whose first tile is <= tile
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)s_blk[mid] * p.n_blocks <= tile) lo = mid; else hi = mid - 1;
    }
    const int nm = s_blk[lo + 1] - s_blk[lo];   // >= 1: an expert with no rows owns no tile
    const int64_t local = tile - (int64_t)s_blk[lo] * p.n_blocks;
    Tile t;
    t.e = lo;
    t.nb = (int)(local / nm);
    t.row0 = s_off[lo] + (int)(local % nm) * (2 * BM) + rank * BM;
    t.rows = s_off[lo + 1] - t.row0;
    return t;
}

// acc.xy += s.xy * d.xy, each lane one fp32 fused multiply-add.
__device__ __forceinline__ void fma2(float2 &acc, float s, uint32_t d0, uint32_t d1) {
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %4};\n\t"
        "mov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\t"
        "mov.b64 {%0, %1}, c;\n\t}"
        : "+f"(acc.x), "+f"(acc.y)
        : "r"(d0), "r"(d1), "f"(s));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Columns of accumulator half `hf` that the epilogue warp's sums 64 j .. 64 j + 63
// (j = 0, 1) come from: neighbours, or a SiLU quarter and its multipliers.
template <int EPI>
__device__ __forceinline__ int half_col(int hf, int j) {
    return EPI == EPI_SWIGLU ? 128 * j + 64 * hf : 128 * hf + 64 * j;
}

template <int EPI>
__global__ void __launch_bounds__(THREADS, 1)
k_gemm_fp8_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                LargeDev p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + RING_BYTES);   // used in CTA 0
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;
    uint64_t *acc_empty = acc_full + 2;                                 // used in CTA 0
    uint64_t *drain = acc_empty + 2;
    uint64_t *amax_bar = drain + 1;                                     // [4], one per quadrant
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(amax_bar + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *s_amax = reinterpret_cast<float *>(smem + RING_BYTES + kBarrierBytes);   // [2][2][BM]
    int32_t *s_off = reinterpret_cast<int32_t *>(smem + RING_BYTES + kBarrierBytes + kAmaxBytes);
    int32_t *s_blk = s_off + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);        // CTA 0's producer arms it with both halves' bytes
            mbar_init(&empty[s], 1);       // one commit per stage use
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * EPI_WARPS);   // both CTAs' epilogue warps
        }
        mbar_init(drain, 1);
        for (int q = 0; q < 4; ++q) mbar_init(&amax_bar[q], 2);   // the quadrant's two warps
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmB) : "memory");
    }
    pdl_wait();   // everything below may read what earlier kernels wrote
    for (int i = threadIdx.x; i <= p.E; i += blockDim.x) s_off[i] = p.offsets[i];
    __syncthreads();
    if (warp == 0) {
        // s_blk[e] = 256-row blocks of the experts before e (warp scan)
        int carry = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            const int c = e < p.E ? (s_off[e + 1] - s_off[e] + 2 * BM - 1) / (2 * BM) : 0;
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
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers and TMEM exist before any cross-CTA use
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int64_t total_tiles = (int64_t)s_blk[p.E] * p.n_blocks;
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;   // cluster index and count

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer (both CTAs)
            const uint32_t full0 = cluster_addr(full, 0);   // CTA 0's full[0]
            int stage = 0;
            uint32_t phase = 0;
            int armed_phase[STAGES];
#pragma unroll
            for (int s = 0; s < STAGES; ++s) armed_phase[s] = -1;
            bool ok = true;
            for (int64_t tile = first; ok && tile < total_tiles; tile += step) {
                const Tile t = decode(tile, p, s_blk, s_off, (int)rank);
                const int ch0 = EPI == EPI_SWIGLU ? (int)rank * (p.N / 2) + t.nb * 128
                                                  : t.nb * BN + (int)rank * (BN / 2);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    // freed by CTA 0's commit once the MMAs have read both halves
                    if (!wait_bounded(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    uint8_t *sa = smem + (size_t)stage * STAGE_BYTES;
                    if (leader) {
                        mbar_arrive_expect_tx(&full[stage], 2 * STAGE_BYTES);
                        armed_phase[stage] = (int)phase;
                    }
                    // rows past this CTA's half (or past the buffer) only reach
                    // accumulator rows that are never stored; bytes past K are 0
                    const uint32_t fb = full0 + (uint32_t)(stage * sizeof(uint64_t));
                    tma_load_2d_pair(sa, &tmA, fb, kb * BK, t.row0);
                    tma_load_3d_pair(sa + A_BYTES, &tmB, fb, kb * BK, ch0, t.e);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (leader) {
                // every armed stage must have landed (both CTAs' halves) before exit
                for (int s = 0; s < STAGES; ++s)
                    if (armed_phase[s] >= 0)
                        wait_bounded(&full[s], (uint32_t)armed_phase[s], abort_flag, p.status, false);
            } else if (!ok) {
                // the peer's loads complete on CTA 0's barriers; after a give-up,
                // leave the copies still in flight time to land before exit
                const uint64_t t0 = globaltimer();
                while (globaltimer() - t0 < 100000ull) __nanosleep(2000);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ------------------------------------------------ MMA issuer (CTA 0)
            constexpr uint32_t idesc = idesc_e4m3(2 * BM, BN);
            int stage = 0;
            uint32_t phase = 0;
            int accb = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int64_t tile = first; ok && tile < total_tiles; tile += step) {
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_bounded(&acc_empty[accb], acc_phase ^ 1u, abort_flag, p.status) ||
                        !wait_bounded(&full[stage], phase, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(accb * BN);
                    const uint32_t a_addr = smem_u32(smem + (size_t)stage * STAGE_BYTES);
                    const uint32_t b_addr = a_addr + A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_f8_pair(d_tmem, desc_sw128(a_addr + 32 * k), desc_sw128(b_addr + 32 * k),
                                    idesc, k > 0 ? 1u : 0u);
                    mma_commit_pair(&empty[stage], 0x3);
                    mma_commit_pair(&acc_full[accb], 0x3);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (++accb == 2) { accb = 0; acc_phase ^= 1u; }
                }
            }
            // no MMA may still be running when either CTA frees TMEM or exits
            mma_commit_pair(drain, 0x1);
            wait_bounded(drain, 0, abort_flag, p.status, false);
        }
    } else {
        // ---------------------------------------------------- epilogue warps (both CTAs)
        const int q = warp & 3;
        const int hf = (warp - 2) >> 2;
        const int rloc = q * 32 + lane;
        int accb = 0;
        uint32_t acc_phase = 0;
        uint32_t tile_par = 0;
        for (int64_t tile = first; tile < total_tiles; tile += step) {
            const Tile t = decode(tile, p, s_blk, s_off, (int)rank);
            const bool rows_here = q * 32 < t.rows;   // warp-uniform
            // a row that exists, so that every lane may read its scales
            const int64_t row = min((int64_t)t.row0 + (rloc < t.rows ? rloc : 0), p.cap_rows - 1);
            const float *sa = p.a_scales + row * p.num_kb;
            // scale rows of the two 64-column groups' channel blocks
            const int wb0 = EPI == EPI_SWIGLU ? t.nb : min(2 * t.nb + hf, p.w_blocks - 1);
            const float *sw0 = p.w_scales + ((int64_t)t.e * p.w_blocks + wb0) * p.num_kb;
            const float *sw1 = EPI == EPI_SWIGLU ? sw0 + (int64_t)(p.w_blocks / 2) * p.num_kb : sw0;
            float2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
            float sa_n = 0.0f, sw0_n = 0.0f, sw1_n = 0.0f;
            if (rows_here) {
                sa_n = __ldg(sa);
                sw0_n = __ldg(sw0);
                sw1_n = __ldg(sw1);
            }
            bool ok = true;
            for (int kb = 0; kb < p.num_kb; ++kb) {
                const float s0 = sa_n * sw0_n, s1 = sa_n * sw1_n;
                if (rows_here && kb + 1 < p.num_kb) {   // the next block's, while this one is awaited
                    sa_n = __ldg(sa + kb + 1);
                    sw0_n = __ldg(sw0 + kb + 1);
                    if (EPI == EPI_SWIGLU) sw1_n = __ldg(sw1 + kb + 1);
                    else sw1_n = sw0_n;
                }
                const bool w = wait_bounded(&acc_full[accb], acc_phase, abort_flag, p.status);
                if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                tc_fence_after();
                if (rows_here) {
                    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(accb * BN);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t r[32];
                        tmem_ld32(taddr + half_col<EPI>(hf, j >> 1) + 32 * (j & 1), r);
                        tmem_ld_wait();
                        const float s = j < 2 ? s0 : s1;
#pragma unroll
                        for (int i = 0; i < 16; ++i) fma2(acc[16 * j + i], s, r[2 * i], r[2 * i + 1]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(&acc_empty[accb], 0);
                if (++accb == 2) { accb = 0; acc_phase ^= 1u; }
            }
            if (!ok) break;
            const bool store = rloc < t.rows && (int64_t)t.row0 + rloc < p.cap_rows;
            if (EPI == EPI_SWIGLU) {
                if (rows_here) {
                    // sums 0..31 (pairs) are SiLU-half channels, 32..63 their multipliers
                    float amax = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        acc[i].x = silu_f32(acc[i].x) * acc[32 + i].x;
                        acc[i].y = silu_f32(acc[i].y) * acc[32 + i].y;
                        amax = fmaxf(amax, fmaxf(fabsf(acc[i].x), fabsf(acc[i].y)));
                    }
                    // the block's other 64 channels are the other warp's
                    float *mine = s_amax + ((tile_par * 2 + hf) * BM) + rloc;
                    const float *other = s_amax + ((tile_par * 2 + (hf ^ 1)) * BM) + rloc;
                    *mine = amax;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&amax_bar[q]);
                    const bool w = wait_bounded(&amax_bar[q], tile_par, abort_flag, p.status);
                    if (!__all_sync(0xffffffffu, w)) break;
                    amax = fmaxf(amax, *reinterpret_cast<const volatile float *>(other));
                    float s, inv;
                    block_scale(amax, s, inv);
                    if (store) {
                        const int Nh = p.N / 2;
                        const int64_t r = (int64_t)t.row0 + rloc;
                        uint4 *dst = reinterpret_cast<uint4 *>(p.q2 + r * Nh + t.nb * 128 + hf * 64);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w4[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const float2 a = acc[8 * i + 2 * u], b = acc[8 * i + 2 * u + 1];
                                w4[u] = e4m3x4(a.x * inv, a.y * inv, b.x * inv, b.y * inv);
                            }
                            dst[i] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                        }
                        if (hf == 0) p.s2[r * (Nh / kFp8Block) + t.nb] = s;
                    }
                    tile_par ^= 1u;
                }
            } else if (store) {
                const int64_t r = (int64_t)t.row0 + rloc;
                const int c0 = t.nb * BN + hf * 128;
                if (EPI == EPI_BF16) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.c) + r * p.N + c0);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + 8 * i < p.N)
                            dst[i] = make_uint4(pack_bf16(acc[4 * i].x, acc[4 * i].y),
                                                pack_bf16(acc[4 * i + 1].x, acc[4 * i + 1].y),
                                                pack_bf16(acc[4 * i + 2].x, acc[4 * i + 2].y),
                                                pack_bf16(acc[4 * i + 3].x, acc[4 * i + 3].y));
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.c) + r * p.N + c0);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c0 + 4 * i < p.N)
                            dst[i] = make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x,
                                                 acc[2 * i + 1].y);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// Clusters that fit on the GPU at once (0 if the kernel cannot run).
template <int EPI>
int clusters_that_fit() {
    static const int n = [] {
        if (!set_smem_limit((const void *)k_gemm_fp8_pair<EPI>, SMEM_BYTES)) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms() & ~1));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = SMEM_BYTES;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int c = 0;
        if (cudaOccupancyMaxActiveClusters(&c, (const void *)k_gemm_fp8_pair<EPI>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            c = 0;
        }
        return c;
    }();
    return n;
}

template <int EPI>
moe_status launch(const Fp8GemmArgs &a, const LargeDev &d, cudaStream_t stream) {
    const int clusters = clusters_that_fit<EPI>();
    if (clusters <= 0) return MOE_ERR_UNSUPPORTED;
    CUtensorMap ma, mb;
    const uint64_t adims[2] = {(uint64_t)a.Kd, (uint64_t)a.cap_rows};
    const uint64_t astr[1] = {(uint64_t)a.Kd};
    const uint32_t abox[2] = {BK, BM};
    const uint64_t bdims[3] = {(uint64_t)a.Kd, (uint64_t)a.N, (uint64_t)a.E};
    const uint64_t bstr[2] = {(uint64_t)a.Kd, (uint64_t)a.Kd * a.N};
    const uint32_t bbox[3] = {BK, BN / 2, 1};
    if (!make_tensor_map(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, a.a, 2, adims,
                         astr, abox) ||
        !make_tensor_map(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, a.w, 3, bdims,
                         bstr, bbox))
        return MOE_ERR_CUDA;
    const char *names[3] = {"gemm_fp8_f32", "gemm_fp8_bf16", "gemm_fp8_swiglu"};
    MOE_LAUNCH_CLUSTER(names[EPI], k_gemm_fp8_pair<EPI>, 2 * clusters, THREADS, SMEM_BYTES, stream, 2u,
                       ma, mb, d);
    return MOE_OK;
}

}  // namespace

moe_status launch_gemm_fp8_large(const Fp8GemmArgs &a, cudaStream_t stream) {
    LargeDev d;
    d.offsets = a.offsets;
    d.E = (int)a.E;
    d.num_kb = (int)((a.Kd + BK - 1) / BK);
    d.N = (int)a.N;
    d.w_blocks = (int)((a.N + kFp8Block - 1) / kFp8Block);
    d.n_blocks = (int)((a.N + BN - 1) / BN);
    d.cap_rows = a.cap_rows;
    d.a_scales = a.a_scales;
    d.w_scales = a.w_scales;
    d.c = a.c;
    d.q2 = static_cast<uint8_t *>(a.q2);
    d.s2 = a.s2;
    d.status = a.status;
    if (a.q2) return launch<EPI_SWIGLU>(a, d, stream);
    return a.out_bf16 ? launch<EPI_BF16>(a, d, stream) : launch<EPI_F32>(a, d, stream);
}

}  // namespace moe
