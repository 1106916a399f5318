// gemm_fp8_large.cu -- grouped products of block-scaled e4m3 operands for many
// rows per expert.
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
// Kernel shape (one persistent CTA per SM, 12 warps; tiles of 128 rows x 256
// channels, every CTA fetching all of its tile's operands):
//   warp 0      TMA producer, four-stage ring of 128 bytes of K
//   warps 1, 3  MMA issuers: 4 x tcgen05.mma M=128 N=256 K=32 a block, even
//               blocks into one 256-column accumulator and odd ones into the
//               other (one thread spends about 450 cycles on the issue of a
//               block, which the tensor cores finish in 512); warp 1 owns TMEM
//   warp 2      scales: four blocks at a time, the products of the rows'
//               scales and the two channel blocks' scales, for the epilogue in
//               a shared-memory ring (one 16-byte load a row and four blocks;
//               loads by the epilogue itself, a row a lane, stalled it)
//   warps 4..11 epilogue: TMEM lane quadrant q (32 rows) x 128 columns, 128
//               sums a thread
// Two SMs on one tile (cta_group::2) would move a third less, but the release
// of an accumulator then has to travel between them, about 1000 cycles from the
// end of a block's MMAs to the start of those that reuse its accumulator, and
// with two accumulators that, not the tensor cores, set the pace (630 ns a
// block; this form takes about 415, the MMAs alone 270).
// What bounds the block loop: 48 KB of operands come in from L2 (61 bytes a
// cycle, as measured) and are written to shared memory and read once by the MMAs
// (96 KB, 768 cycles at 128 bytes a cycle); and the round of an accumulator:
// issue to the end of its MMAs 900 cycles, the last epilogue warp's start 115
// (SwiGLU form 340), drain 450 (500), release to the next issue 230 (310), for
// every second block.  A block takes about 785 (905) cycles, and a tile about
// 4900 more for its start and its stores.  Measured, bf16 output: 8192 rows,
// 7168 x 7168, 309 us (2.7 PFLOP/s); 8192 rows, 7168 x 2048, 111 us (2.2).
// SwiGLU form: a tile is 128 SiLU-half channels and the multiplier channels of
// the same numbers, so it holds 128 complete channels of g and the epilogue
// quantises them as one block; h never leaves the SM.
// Every wait is bounded (about two seconds) and sets MOE_DEV_TIMEOUT.
#include "common.cuh"
#include "fp8.cuh"
#include "tcgen05.cuh"

#include <cuda.h>

namespace moe {
namespace {

using namespace tc;

constexpr int BM = 128;                 // rows per tile
constexpr int BN = 256;                 // channels per tile
constexpr int BK = 128;                 // bytes of K per block: one scale
constexpr int STAGES = 4;
// The two issuers take turns on the blocks.  With an even number of stages each
// always waits on its own ones; with an odd number a stage would pass from one
// to the other, and a wait could take the other's phase for its own.
static_assert(STAGES % 2 == 0, "stages belong to one issuer");
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = BN * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr size_t RING_BYTES = (size_t)STAGES * STAGE_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int CG = EPI_WARPS / 4;        // column groups
constexpr int CPT = BN / CG;             // sums per epilogue thread
constexpr int HC = CPT / 2;
constexpr int EPI_WARP0 = 4;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
// Registers: the block is launched with 168 a thread (65536 / 384, in steps of
// 8); the first warpgroup gives up what the two epilogue warpgroups take.  With
// 168 the epilogue's 128 sums and what it loads did not fit, and a few spilled
// words a block cost a tenth of the time.
constexpr int REGS_LAUNCH = 168, REGS_ISSUE = 72, REGS_EPI = 216;
static_assert(REGS_ISSUE + 2 * REGS_EPI <= 3 * REGS_LAUNCH, "register split");
constexpr uint32_t TMEM_COLS = 512;
constexpr size_t kBarrierBytes = 512;
constexpr size_t kAmaxBytes = 2 * CG * BM * sizeof(float);
constexpr int SB = 4;                   // blocks of K per batch of scales
constexpr int SC_STAGES = 3;
constexpr int SC_FLOATS = SB * 2 * BM;  // [block][channel block][row]
constexpr size_t kScaleBytes = SC_STAGES * SC_FLOATS * sizeof(float);
constexpr size_t SMEM_BYTES = RING_BYTES + 1024 + kBarrierBytes + kAmaxBytes + kScaleBytes +
                              2 * (kMaxExperts + 1) * sizeof(int32_t);
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert((2 * STAGES + 9 + 2 * SC_STAGES) * 8 + 16 <= (int)kBarrierBytes, "barriers");

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
    int reset_status;    // first kernel of its call
    int c_vec32;         // rows of C start on 32-byte boundaries
    int vec_scales;      // rows of a_scales can be read 16 bytes at a time
};

// Expert, first row, rows from there to the expert's end (may be more than BM),
// column block.
struct Tile {
    int e, row0, rows, nb;
};

// Tiles of an expert with `rows` rows.
__device__ __forceinline__ int tiles_of(int rows, int n_blocks) { return (rows + BM - 1) / BM * n_blocks; }

// Column-block-major within an expert: the CTAs in flight share few weight
// tiles, each read by all of the expert's row blocks while it is in L2.
__device__ __forceinline__ Tile decode(int tile, const LargeDev &p, const int32_t *s_tile,
                                       const int32_t *s_off) {
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {   // last expert whose first tile is <= tile
        const int mid = (lo + hi + 1) >> 1;
        if (s_tile[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    const int blocks = (s_off[lo + 1] - s_off[lo] + BM - 1) / BM;
    const int local = tile - s_tile[lo];
    Tile t;
    t.e = lo;
    t.nb = local / blocks;
    t.row0 = s_off[lo] + local % blocks * BM;
    t.rows = s_off[lo + 1] - t.row0;
    return t;
}

// acc += s * d on both numbers, each one an fp32 fused multiply-add.  Volatile,
// to stay behind the wait that makes the loaded d valid.
__device__ __forceinline__ void fma2(float2 &acc, float s, uint32_t d0, uint32_t d1) {
    asm volatile("{\n\t.reg .b64 a, b, c;\n\t"
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

// One 32-byte store to a 32-byte aligned global address: a whole sector.
__device__ __forceinline__ void st_global_v8(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Four neighbouring lanes hold 32-byte pieces 0..3 of a row each, c[piece];
// afterwards lane i of the four holds piece i of their rows, c[row].
__device__ __forceinline__ void transpose4(uint32_t (&c)[4][8], int lane) {
    const bool b0 = lane & 1, b1 = lane & 2;
    auto swap = [](uint32_t &x, uint32_t &y, bool up, int d) {   // the lower lane's y for the upper's x
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x : y, d);
        if (up) x = got; else y = got;
    };
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        swap(c[0][u], c[1][u], b0, 1);
        swap(c[2][u], c[3][u], b0, 1);
        swap(c[0][u], c[2][u], b1, 2);
        swap(c[1][u], c[3][u], b1, 2);
    }
}

// First accumulator column of the epilogue warp's sums HC j .. HC j + HC - 1 (j =
// 0, 1) in column group cg: neighbours, or SiLU channels and their multipliers.
template <int EPI>
__device__ __forceinline__ int group_col(int cg, int j) {
    return EPI == EPI_SWIGLU ? 128 * j + HC * cg : CPT * cg + HC * j;
}

template <int EPI>
__global__ void __launch_bounds__(THREADS, 1)
k_gemm_fp8_large(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 LargeDev p) {
    // aligned by its declaration, so that every address in it is a constant
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + RING_BYTES);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *drain = acc_empty + 2;
    uint64_t *amax_bar = drain + 1;                                     // [4], one per quadrant
    uint64_t *sc_full = amax_bar + 4;
    uint64_t *sc_empty = sc_full + SC_STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sc_empty + SC_STAGES);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *s_amax = reinterpret_cast<float *>(smem + RING_BYTES + kBarrierBytes);   // [2][CG][BM]
    float *s_scale = s_amax + kAmaxBytes / sizeof(float);
    int32_t *s_off = reinterpret_cast<int32_t *>(s_scale + kScaleBytes / sizeof(float));
    int32_t *s_tile = s_off + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], EPI_WARPS);
        }
        mbar_init(drain, 2);               // both issuers
        for (int s = 0; s < SC_STAGES; ++s) {
            mbar_init(&sc_full[s], 1);
            mbar_init(&sc_empty[s], EPI_WARPS);
        }
        for (int q = 0; q < 4; ++q) mbar_init(&amax_bar[q], CG);   // the quadrant's warps
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmB) : "memory");
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    pdl_wait();   // everything below may read what earlier kernels wrote
    // Block 0 starts no later than any other, and no wait gives up before two
    // seconds have passed, so no bit set by this call is lost.
    if (p.reset_status && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    for (int i = threadIdx.x; i <= p.E; i += blockDim.x) s_off[i] = p.offsets[i];
    __syncthreads();
    if (warp == 0) {
        // s_tile[e] = tiles of the experts before e (warp scan)
        int carry = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            const int c = e < p.E ? tiles_of(s_off[e + 1] - s_off[e], p.n_blocks) : 0;
            int x = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            if (e < p.E) s_tile[e] = carry + x - c;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) s_tile[p.E] = carry;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int total_tiles = s_tile[p.E];   // C fits memory, so they are far below 2^31
    const int my_tiles = (int)blockIdx.x < total_tiles ? (total_tiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;

    if (warp < EPI_WARP0) {
      regs_dec<REGS_ISSUE>();
      if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0;
            int64_t armed = 0;   // stage uses
            bool ok = true;
            for (int i = 0; ok && i < my_tiles; ++i) {
                const Tile t = decode((int)(blockIdx.x + i * gridDim.x), p, s_tile, s_off);
                // the tile's two 128-channel halves
                const int ch0 = EPI == EPI_SWIGLU ? t.nb * 128 : t.nb * BN;
                const int ch1 = EPI == EPI_SWIGLU ? ch0 + p.N / 2 : ch0 + BN / 2;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!wait_bounded_inline(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
                    uint8_t *sa = smem + (size_t)stage * STAGE_BYTES;
                    mbar_arrive_expect_tx(&full[stage], STAGE_BYTES);
                    ++armed;
                    // rows past the tile's (or past the buffer) only reach accumulator
                    // rows that are never stored; bytes past K are 0
                    tma_load_2d(sa, &tmA, &full[stage], kb * BK, t.row0);
                    tma_load_3d(sa + A_BYTES, &tmB, &full[stage], kb * BK, ch0, t.e);
                    tma_load_3d(sa + A_BYTES + B_BYTES / 2, &tmB, &full[stage], kb * BK, ch1, t.e);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            // every armed stage must have landed before exit
            for (int64_t u = armed > STAGES ? armed - STAGES : 0; u < armed; ++u)
                wait_bounded_inline(&full[u % STAGES], (uint32_t)(u / STAGES) & 1u, abort_flag, p.status, false);
        }
      } else if (warp == 2) {
        // ---------------------------------------------------- scales
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = 0; ok && i < my_tiles; ++i) {
            const Tile t = decode((int)(blockIdx.x + i * gridDim.x), p, s_tile, s_off);
            // lane's rows lane + 32 u, clamped to rows that exist
            const int64_t row0 = min((int64_t)t.row0, p.cap_rows - 1);
            const int last = (int)min((int64_t)max(t.rows, 1), p.cap_rows - row0) - 1;
            const float *sa = p.a_scales + row0 * p.num_kb;
            int at[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) at[u] = min(lane + 32 * u, last) * p.num_kb;
            const int wb0 = EPI == EPI_SWIGLU ? t.nb : 2 * t.nb;
            // (clamped: the last tile may have only one block of 128 channels)
            const int wb1 = min(EPI == EPI_SWIGLU ? t.nb + p.w_blocks / 2 : 2 * t.nb + 1, p.w_blocks - 1);
            const float *sw0 = p.w_scales + ((int64_t)t.e * p.w_blocks + wb0) * p.num_kb;
            const float *sw1 = p.w_scales + ((int64_t)t.e * p.w_blocks + wb1) * p.num_kb;
            for (int kb = 0; kb < p.num_kb; kb += SB) {
                float v[4][SB], w0[SB], w1[SB];
                if (p.vec_scales) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float4 x = __ldg(reinterpret_cast<const float4 *>(sa + at[u] + kb));
                        v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int b = 0; b < SB; ++b) v[u][b] = __ldg(sa + at[u] + min(kb + b, p.num_kb - 1));
                }
#pragma unroll
                for (int b = 0; b < SB; ++b) {
                    w0[b] = __ldg(sw0 + min(kb + b, p.num_kb - 1));
                    w1[b] = __ldg(sw1 + min(kb + b, p.num_kb - 1));
                }
                if (!__all_sync(0xffffffffu, wait_bounded_inline(&sc_empty[stage], phase ^ 1u, abort_flag, p.status))) {
                    ok = false;
                    break;
                }
                float *dst = s_scale + stage * SC_FLOATS + lane;
#pragma unroll
                for (int b = 0; b < SB; ++b)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        dst[(2 * b) * BM + 32 * u] = v[u][b] * w0[b];
                        dst[(2 * b + 1) * BM + 32 * u] = v[u][b] * w1[b];
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[stage]);
                if (++stage == SC_STAGES) { stage = 0; phase ^= 1u; }
            }
        }
      } else if (lane == 0) {
        // ---------------------------------------------------- MMA issuers
        constexpr uint32_t idesc = idesc_e4m3(BM, BN);
        const int accb = warp >> 1;          // this issuer's accumulator: every second block
        int stage = 0;
        uint32_t phase = 0, acc_phase = 0;
        int turn = 0;                        // accumulator of the block at hand
        bool ok = true;
        const uint32_t d_tmem = tmem_base + (uint32_t)(accb * BN);
        for (int i = 0; ok && i < my_tiles; ++i) {
            for (int kb = 0; kb < p.num_kb; ++kb) {
                if (turn == accb) {
                    if (!wait_bounded_inline(&full[stage], phase, abort_flag, p.status) ||
                        !wait_bounded_inline(&acc_empty[accb], acc_phase ^ 1u, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem + (size_t)stage * STAGE_BYTES);
                    const uint32_t b_addr = a_addr + A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_f8(d_tmem, desc_sw128(a_addr + 32 * k), desc_sw128(b_addr + 32 * k), idesc,
                               k > 0 ? 1u : 0u);
                    mma_commit(&acc_full[accb]);
                    mma_commit(&empty[stage]);
                    acc_phase ^= 1u;
                }
                turn ^= 1;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
        }
        // no MMA may still be running when TMEM is freed
        mma_commit(drain);
        wait_bounded_inline(drain, 0, abort_flag, p.status, false);
      }
    } else {
        // ---------------------------------------------------- epilogue warps
        regs_inc<REGS_EPI>();
        const int q = warp & 3;
        const int cg = (warp - EPI_WARP0) >> 2;   // column group
        const int rloc = q * 32 + lane;
        int accb = 0;
        uint32_t acc_phase = 0;
        uint32_t tile_par = 0;
        int sc_stage = 0;
        uint32_t sc_phase = 0;
        for (int tile = (int)blockIdx.x; tile < total_tiles; tile += gridDim.x) {
            const Tile t = decode(tile, p, s_tile, s_off);
            const bool rows_here = q * 32 < t.rows;   // warp-uniform
            float2 acc[CPT / 2];
#pragma unroll
            for (int i = 0; i < CPT / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
            bool ok = true;
            for (int kb = 0; kb < p.num_kb; ++kb) {
                if ((kb & (SB - 1)) == 0) {
                    // (not in line: nothing spills with the call, 28 bytes without)
                    const bool w = wait_bounded(&sc_full[sc_stage], sc_phase, abort_flag, p.status);
                    if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                }
                const float *sc = s_scale + sc_stage * SC_FLOATS + (kb & (SB - 1)) * 2 * BM + rloc;
                const float s0 = EPI == EPI_SWIGLU ? sc[0] : sc[cg * BM];
                const float s1 = EPI == EPI_SWIGLU ? sc[BM] : s0;
                const bool w = wait_bounded_inline(&acc_full[accb], acc_phase, abort_flag, p.status);
                if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                tc_fence_after();
                uint32_t r[16];
                const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(accb * BN);
                if (rows_here) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        tmem_ld16(taddr + group_col<EPI>(cg, j >> 2) + 16 * (j & 3), r);
                        tmem_ld_wait();
                        if (j == 7) break;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            fma2(acc[8 * j + i], j < 4 ? s0 : s1, r[2 * i], r[2 * i + 1]);
                    }
                }
                // the accumulator is read: the next block but one may use it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[accb]);
                if (rows_here) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) fma2(acc[56 + i], s1, r[2 * i], r[2 * i + 1]);
                }
                if (++accb == 2) { accb = 0; acc_phase ^= 1u; }
                if ((kb & (SB - 1)) == SB - 1 || kb + 1 == p.num_kb) {
                    if (lane == 0) mbar_arrive(&sc_empty[sc_stage]);   // read before the __syncwarp above
                    if (++sc_stage == SC_STAGES) { sc_stage = 0; sc_phase ^= 1u; }
                }
            }
            if (!ok) break;
            const bool store = rloc < t.rows && (int64_t)t.row0 + rloc < p.cap_rows;
            if (EPI == EPI_SWIGLU) {
                if (rows_here) {
                    // the first half of the pairs are SiLU channels, the others their multipliers
                    float amax = 0.0f;
#pragma unroll
                    for (int i = 0; i < HC / 2; ++i) {
                        acc[i].x = swiglu(acc[i].x, acc[HC / 2 + i].x);
                        acc[i].y = swiglu(acc[i].y, acc[HC / 2 + i].y);
                        amax = fmaxf(amax, fmaxf(fabsf(acc[i].x), fabsf(acc[i].y)));
                    }
                    // the block's other channels are with the quadrant's other warps
                    float *all = s_amax + tile_par * CG * BM + rloc;
                    all[cg * BM] = amax;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&amax_bar[q]);
                    const bool w = wait_bounded_inline(&amax_bar[q], tile_par, abort_flag, p.status);
                    if (!__all_sync(0xffffffffu, w)) break;
                    const volatile float *m = all;
                    float s, inv;
                    amax = m[0];
#pragma unroll
                    for (int g = 1; g < CG; ++g) amax = fmaxf(amax, m[g * BM]);
                    block_scale(amax, s, inv);
                    if (store) {
                        const int Nh = p.N / 2;
                        const int64_t r = (int64_t)t.row0 + rloc;
                        uint4 *dst = reinterpret_cast<uint4 *>(p.q2 + r * Nh + t.nb * 128 + cg * HC);
#pragma unroll
                        for (int i = 0; i < HC / 16; ++i) {
                            uint32_t w4[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const float2 a = acc[8 * i + 2 * u], b = acc[8 * i + 2 * u + 1];
                                w4[u] = e4m3x4(a.x * inv, a.y * inv, b.x * inv, b.y * inv);
                            }
                            dst[i] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                        }
                        if (cg == 0) p.s2[r * (Nh / kFp8Block) + t.nb] = s;
                    }
                    tile_par ^= 1u;
                }
            } else if (EPI == EPI_BF16) {
                if (store) {
                    const int c0 = t.nb * BN + cg * CPT;
                    __nv_bfloat16 *row = static_cast<__nv_bfloat16 *>(p.c) + ((int64_t)t.row0 + rloc) * p.N + c0;
                    if (p.c_vec32 && c0 + CPT <= p.N) {
#pragma unroll
                        for (int i = 0; i < CPT / 16; ++i) {
                            uint32_t w[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) w[u] = pack_bf16(acc[8 * i + u].x, acc[8 * i + u].y);
                            st_global_v8(row + 16 * i, w);
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(row);
#pragma unroll
                        for (int i = 0; i < CPT / 8; ++i)
                            if (c0 + 8 * i < p.N)
                                dst[i] = make_uint4(pack_bf16(acc[4 * i].x, acc[4 * i].y),
                                                    pack_bf16(acc[4 * i + 1].x, acc[4 * i + 1].y),
                                                    pack_bf16(acc[4 * i + 2].x, acc[4 * i + 2].y),
                                                    pack_bf16(acc[4 * i + 3].x, acc[4 * i + 3].y));
                    }
                }
            } else if (rows_here) {
                // A row's 512 bytes a lane: in pieces of 32 bytes, four lanes store
                // 128 bytes of one row at a time, so that whole lines go to L2 (1533
                // rows, 1000 x 1456: 14.6 -> 12.3 us in a graph).  The bf16 form, of
                // half the bytes, keeps a lane's own row: the exchange cost its block
                // loop more (8192 rows, 7168 x 7168: 320 -> 337 us).
                const int c0 = t.nb * BN + cg * CPT + (lane & 3) * 8;
                const int r4 = rloc & ~3;
                float *row = static_cast<float *>(p.c) + ((int64_t)t.row0 + r4) * p.N + c0;
                const int64_t left = min((int64_t)t.rows, p.cap_rows - t.row0) - r4;
#pragma unroll
                for (int h = 0; h < CPT / 32; ++h) {
                    uint32_t c[4][8];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float2 v = acc[16 * h + 4 * j + u / 2];
                            c[j][u] = __float_as_uint(u & 1 ? v.y : v.x);
                        }
                    transpose4(c, lane);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float *dst = row + (int64_t)k * p.N + 32 * h;
                        if (k >= left || c0 + 32 * h >= p.N) continue;
                        if (p.c_vec32) {
                            st_global_v8(dst, c[k]);
                        } else {
                            reinterpret_cast<uint4 *>(dst)[0] = make_uint4(c[k][0], c[k][1], c[k][2], c[k][3]);
                            reinterpret_cast<uint4 *>(dst)[1] = make_uint4(c[k][4], c[k][5], c[k][6], c[k][7]);
                        }
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
}

template <int EPI>
moe_status launch(const Fp8GemmArgs &a, const LargeDev &d, cudaStream_t stream) {
    if (!set_smem_limit((const void *)k_gemm_fp8_large<EPI>, SMEM_BYTES)) return MOE_ERR_CUDA;
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
    MOE_LAUNCH(names[EPI], k_gemm_fp8_large<EPI>, (unsigned)num_sms(), THREADS, SMEM_BYTES, stream, ma, mb, d);
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
    d.reset_status = a.reset_status;
    d.c_vec32 = (uintptr_t)a.c % 32 == 0 && a.N * (a.out_bf16 ? 2 : 4) % 32 == 0;
    d.vec_scales = d.num_kb % SB == 0 && (uintptr_t)a.a_scales % 16 == 0;
    if (a.q2) return launch<EPI_SWIGLU>(a, d, stream);
    return a.out_bf16 ? launch<EPI_BF16>(a, d, stream) : launch<EPI_F32>(a, d, stream);
}

}  // namespace moe
