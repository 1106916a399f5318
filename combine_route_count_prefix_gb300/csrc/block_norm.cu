// block_norm.cu -- the boundary between two blocks: norm of a block's output, its
// gate, the scaled residual addition, and the next block's norm.
//
//   a = x * rsqrt(sum(x^2) / H + eps) * post_weight          (x without one)
//   h = residual_scale * residual + branch_scale * act(gate) * a
//   v = h * rsqrt(sum(h^2) / H + eps) * weight
// h to bf16, v to bf16 and / or block-scaled e4m3.
//
// Memory bounds it: every input is read once and every output written once (11
// bytes an element with a gate per token and all outputs).  Persistent CTAs walk the
// tokens; a token's rows of x, residual and gate come by bulk copies into a
// shared-memory ring, the next tokens' on their way meanwhile, and stay in
// registers from there to the stores, through both sums.  Thread i holds the
// 16-byte vectors i, i + threads, ... (eight channels each); a block of 128 channels
// is 16 neighbouring vectors, half a warp: its maximum is four shuffles.
// 16384 tokens of 7168 channels, a gate per token, all outputs: 204 us, 6.3 TB/s, 0.94
// of a plain copy's rate; without gate and outer norm 172 us, 6.1 TB/s; one
// token 3.3 us in a graph, the latency of two sums over the row.  Rows of a few KB are
// bounded by the sums' barriers instead (16384 x 2048 63 us, 4.8 TB/s).
#include "common.cuh"
#include "fp8.cuh"
#include "norm.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kMaxStages = 3;

struct BlockNormDev {
    const uint4 *x, *residual, *gate;
    const void *post, *weight;
    uint4 *residual_out, *y;
    uint2 *q;
    float *scales;
    int64_t T, gate_tokens, gate_stride8;   // tokens that share a gate row; vectors from one to the next
    int H8, nb, stages, gate_act;
    float eps, inv_h, residual_scale, branch_scale;
};

template <bool W_BF16>
__device__ __forceinline__ void load_weight(const void *w, int i, float (&f)[8]) {
    if (W_BF16) {
        unpack8(__ldg(static_cast<const uint4 *>(w) + i), f);
    } else {
        const float4 a = __ldg(static_cast<const float4 *>(w) + 2 * i), b = __ldg(static_cast<const float4 *>(w) + 2 * i + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}

// 1 / (1 + exp(-g)), the hardware's exponential and reciprocal.  Relative error at most
// 2^-22 of the exponential, 2^-24 of the sum and 2^-23 of the reciprocal, and |g| (2^-24 +
// 2^-25) of the exponential's argument, rounded once from a rounded factor: 4.2e-7 + 0.9e-7
// |g|, beside bf16 gates that stand for 4e-3 of themselves.
__device__ __forceinline__ float sigmoid(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

template <int V, bool W_BF16, bool KEEP>
__global__ void __launch_bounds__(kNormMaxThreads)
k_block_norm(BlockNormDev p) {
    extern __shared__ __align__(128) uint8_t smem[];   // [stages][x, residual, gate][H]
    __shared__ __align__(16) float part[2][kNormMaxThreads / 32];
    __shared__ uint64_t full[kMaxStages];
    __shared__ volatile int abort_flag;
    const int tid = threadIdx.x, lane = tid & 31, nt = blockDim.x;
    const uint32_t row_bytes = (uint32_t)p.H8 * 16u;
    const bool gate_rows = p.gate && p.gate_tokens < p.T;   // else one row for all, read from L1
    const uint32_t in_bytes = (gate_rows ? 3u : 2u) * row_bytes;
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        abort_flag = 0;
        for (int w = nt >> 5; w < kNormMaxThreads / 32; ++w) part[0][w] = part[1][w] = 0.0f;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    auto load = [&](int64_t t, int s) {
        uint8_t *dst = smem + (size_t)s * in_bytes;
        mbar_arrive_expect_tx(&full[s], in_bytes);
        bulk_load(dst, p.x + t * p.H8, row_bytes, &full[s]);
        bulk_load(dst + row_bytes, p.residual + t * p.H8, row_bytes, &full[s]);
        if (gate_rows) bulk_load(dst + 2 * row_bytes, p.gate + t / p.gate_tokens * p.gate_stride8, row_bytes, &full[s]);
    };
    if (tid == 0)
        for (int s = 0; s < p.stages; ++s)
            if (blockIdx.x + (int64_t)s * gridDim.x < p.T) load(blockIdx.x + (int64_t)s * gridDim.x, s);

    // KEEP: the weights come into registers before the first wait (a token alone would wait for L2 twice)
    uint4 kept[KEEP ? 2 : 1][V];
    if (KEEP) {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = u * nt + tid;
            if (i < p.H8) {
                if (p.post) kept[0][u] = __ldg(static_cast<const uint4 *>(p.post) + i);
                if (p.weight) kept[KEEP ? 1 : 0][u] = __ldg(static_cast<const uint4 *>(p.weight) + i);
            }
        }
    }
    int s = 0, turn = 0;
    uint32_t phase = 0;
    bool failed = false;
    // rsqrt(sum(v^2) / H + eps) over the row; where squares pass fp32's range (|v|
    // above about 1e17) the same with v * 2^-80, beside which eps is nothing.  An infinite
    // or NaN v leaves it at 0 or NaN, as the formula does.
    auto inverse_rms = [&](float (&v)[V][8], bool fail) {
        float ss = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int c = 0; c < 8; ++c) ss = fmaf(v[u][c], v[u][c], ss);
        ss = block_sum(ss, part[turn], fail, failed);
        turn ^= 1;
        if (ss <= kF32Max || failed) return __frsqrt_rn(fmaf(ss, p.inv_h, p.eps));
        ss = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                v[u][c] *= 0x1p-80f;
                ss = fmaf(v[u][c], v[u][c], ss);
            }
        ss = block_sum(ss, part[turn], false, failed);
        turn ^= 1;
        return __frsqrt_rn(ss * p.inv_h);
    };
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const bool ok = wait_bounded(&full[s], phase, &abort_flag, nullptr);
        const uint4 *sx = reinterpret_cast<const uint4 *>(smem + (size_t)s * in_bytes);
        float h[V][8];
        uint4 res[V], gt[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = u * nt + tid;
#pragma unroll
            for (int c = 0; c < 8; ++c) h[u][c] = 0.0f;
            res[u] = gt[u] = make_uint4(0, 0, 0, 0);
            if (i < p.H8) {
                unpack8(sx[i], h[u]);
                res[u] = sx[p.H8 + i];
                if (p.gate) gt[u] = gate_rows ? sx[2 * p.H8 + i] : __ldg(p.gate + i);
            }
        }
        float r = 1.0f;
        if (p.post) {
            r = inverse_rms(h, !ok);
            if (failed) break;
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = u * nt + tid;
            if (i < p.H8) {
                float f[8];
                if (p.post) {
                    if (KEEP) unpack8(kept[0][u], f);
                    else load_weight<W_BF16>(p.post, i, f);
#pragma unroll
                    for (int c = 0; c < 8; ++c) h[u][c] *= r * f[c];
                }
                if (p.gate) {
                    unpack8(gt[u], f);
#pragma unroll
                    for (int c = 0; c < 8; ++c) h[u][c] *= p.gate_act ? sigmoid(f[c]) : f[c];
                }
                unpack8(res[u], f);
#pragma unroll
                for (int c = 0; c < 8; ++c) h[u][c] = fmaf(p.branch_scale, h[u][c], p.residual_scale * f[c]);
                if (ok) p.residual_out[t * p.H8 + i] = pack8(h[u]);
            }
        }
        r = inverse_rms(h, !ok);
        if (failed) break;
        // everyone has read the stage: the token `stages` ahead may land in it
        if (tid == 0 && t + (int64_t)p.stages * gridDim.x < p.T) load(t + (int64_t)p.stages * gridDim.x, s);
        if (++s == p.stages) { s = 0; phase ^= 1u; }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = u * nt + tid;
            const bool in = i < p.H8;
            float amax = 0.0f;
            if (in && p.weight) {
                float w[8];
                if (KEEP) unpack8(kept[KEEP ? 1 : 0][u], w);
                else load_weight<W_BF16>(p.weight, i, w);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    h[u][c] *= w[c];
                    amax = fmaxf(amax, fabsf(h[u][c]));
                }
                if (p.y) {
                    float v[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = h[u][c] * r;
                    p.y[t * p.H8 + i] = pack8(v);
                }
            }
            if (p.q) {
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
                if (in) {
                    // v = r * (h w), and r is the same all over the block: the codes
                    // are (h w) * 448 / max|h w|, one rounding fewer, unless the floor
                    // or the range of h w says otherwise
                    const float a = fmaxf(amax * r, kAmaxFloor);
                    const float sc = a * (1.0f / kE4m3Max);
                    const float inv = amax >= kAmaxFloor && amax * r >= kAmaxFloor
                                          ? inverse_scale(amax) : inverse_scale(a) * r;
                    p.q[t * p.H8 + i] =
                        make_uint2(e4m3x4(h[u][0] * inv, h[u][1] * inv, h[u][2] * inv, h[u][3] * inv),
                                   e4m3x4(h[u][4] * inv, h[u][5] * inv, h[u][6] * inv, h[u][7] * inv));
                    if ((lane & 15) == 0) p.scales[t * p.nb + (i >> 4)] = sc;
                }
            }
        }
    }
    if (failed) {   // copies still in flight get time to land before the block's memory goes
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 100000ull) __nanosleep(2000);
    }
}

template <int V, bool W_BF16, bool KEEP>
moe_status launch(BlockNormDev p, cudaStream_t stream) {
    auto kernel = k_block_norm<V, W_BF16, KEEP>;
    const bool gate_rows = p.gate && p.gate_tokens < p.T;
    const size_t stage = (size_t)(gate_rows ? 3 : 2) * p.H8 * 16;
    const size_t room = 224 * 1024;
    const int threads = ((p.H8 + V - 1) / V + 31) / 32 * 32;
    // as many CTAs as registers (64 a thread, 128 with four vectors) and rings let stand beside each
    // other on an SM, with three stages where two CTAs fit so, else two: 16384 x 7168
    // with gates, one CTA of three stages 291 us, two of two 204 us
    const int64_t by_regs = std::max<int64_t>(1, (V > 2 ? 512 : 1024) / threads);
    auto beside = [&](int stages) { return std::min<int64_t>(by_regs, room / (stages * stage + 1024)); };
    p.stages = beside(kMaxStages) >= std::min<int64_t>(2, by_regs) ? kMaxStages : 2;
    const size_t smem = p.stages * stage;
    if (!set_smem_limit((const void *)kernel, smem)) return MOE_ERR_CUDA;
    const int64_t cap = num_sms() * std::max<int64_t>(1, beside(p.stages));
    const unsigned grid = (unsigned)(p.T < cap ? p.T : cap);
    MOE_LAUNCH("block_norm", kernel, grid, threads, smem, stream, p);
    return MOE_OK;
}

template <int V>
moe_status launch_v(const BlockNormDev &p, bool w_bf16, cudaStream_t stream) {
    if constexpr (V <= 2) {
        // a token a CTA: 128 x 7168 with gates 4.46 -> 3.78 us; for many tokens the registers cost
        // CTAs (16384 x 7168, one gate, 195 -> 209 us)
        if (w_bf16 && p.T <= num_sms()) return launch<V, true, true>(p, stream);
    }
    return w_bf16 ? launch<V, true, false>(p, stream) : launch<V, false, false>(p, stream);
}

}  // namespace

moe_status launch_block_norm(const moe_block_norm_desc &d, const void *x, const void *residual,
                             const void *post_weight, const void *gate, const void *weight,
                             void *residual_out, void *y, void *q, float *scales, cudaStream_t stream) {
    BlockNormDev p;
    p.x = static_cast<const uint4 *>(x);
    p.residual = static_cast<const uint4 *>(residual);
    p.gate = static_cast<const uint4 *>(gate);
    p.post = post_weight;
    p.weight = weight;
    p.residual_out = static_cast<uint4 *>(residual_out);
    p.y = static_cast<uint4 *>(y);
    p.q = static_cast<uint2 *>(q);
    p.scales = scales;
    p.T = d.num_tokens;
    p.gate_tokens = gate ? d.num_tokens / d.gate_rows : 0;
    p.gate_stride8 = d.gate_stride / 8;
    p.H8 = (int)(d.hidden / 8);
    p.nb = (int)((d.hidden + kFp8Block - 1) / kFp8Block);
    p.gate_act = d.gate_act;
    p.eps = d.eps;
    p.inv_h = 1.0f / (float)d.hidden;
    p.residual_scale = d.residual_scale;
    p.branch_scale = d.branch_scale;
    const bool w_bf16 = d.weight_dtype == MOE_DTYPE_BF16;
    // Vectors a thread: few enough for registers, many enough for at most 512 threads.
    // Two rather than one also for short rows, whose CTAs are many then (16384 x 2048: 63
    // against 69 us), unless one token a CTA is all there is (1023 x 1000: 4.0 against 3.6 us).
    const int64_t threads1 = (p.H8 + 31) / 32 * 32;
    if (p.H8 <= 256 && p.T <= num_sms() * (1024 / threads1)) return launch_v<1>(p, w_bf16, stream);
    if (p.H8 <= 1024) return launch_v<2>(p, w_bf16, stream);
    return launch_v<4>(p, w_bf16, stream);
}

}  // namespace moe
