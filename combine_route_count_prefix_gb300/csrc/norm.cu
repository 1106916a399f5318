// norm.cu -- residual addition, root-mean-square norm and block-scaled e4m3.
//
// Memory bounds it: every input is read once and every output written once
// (9 bytes an element with a residual and all outputs).  16384 tokens of 7168
// channels, all outputs: 180 us, 5.9 TB/s, 0.88 of a plain copy's rate; one
// token is 2.5 us in a graph, the latency of its few dependent steps.
// Persistent CTAs walk
// the tokens; a token's rows of x and residual come by bulk copies into a
// shared-memory ring, the next tokens' on their way while this one is summed
// and written, and stay in registers from the sum to the stores.  Thread i
// holds the 16-byte vectors i, i + threads, ... (eight channels each), with as
// many threads as make the row come out even.  A block of 128 channels is 16
// neighbouring vectors, half a warp: its maximum is four shuffles.
#include "common.cuh"
#include "fp8.cuh"
#include "norm.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kStages = 3;

struct NormDev {
    const uint4 *x, *residual;
    const void *weight;
    uint4 *residual_out, *y;
    uint2 *q;
    float *scales;
    int64_t T;
    int H8, nb;
    float eps, inv_h;
};

template <int V, bool W_BF16, bool RES>
__global__ void __launch_bounds__(kNormMaxThreads)
k_add_rms_norm(NormDev p) {
    extern __shared__ __align__(128) uint8_t smem[];   // [kStages][x, residual][H]
    __shared__ __align__(16) float part[2][kNormMaxThreads / 32];
    __shared__ uint64_t full[kStages];
    __shared__ volatile int abort_flag;
    const int tid = threadIdx.x, lane = tid & 31, nt = blockDim.x;
    const uint32_t row_bytes = (uint32_t)p.H8 * 16u;
    constexpr int IN = RES ? 2 : 1;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
        abort_flag = 0;
        for (int w = nt >> 5; w < kNormMaxThreads / 32; ++w) part[0][w] = part[1][w] = 0.0f;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    auto load = [&](int64_t t, int s) {
        uint8_t *dst = smem + (size_t)s * IN * row_bytes;
        mbar_arrive_expect_tx(&full[s], IN * row_bytes);
        bulk_load(dst, p.x + t * p.H8, row_bytes, &full[s]);
        if (RES) bulk_load(dst + row_bytes, p.residual + t * p.H8, row_bytes, &full[s]);
    };
    if (tid == 0)
        for (int s = 0; s < kStages; ++s)
            if (blockIdx.x + (int64_t)s * gridDim.x < p.T) load(blockIdx.x + (int64_t)s * gridDim.x, s);
    // the thread's weights, for every token
    constexpr int WN = W_BF16 ? 1 : 2;
    uint4 wv[V][WN];
#pragma unroll
    for (int u = 0; u < V; ++u)
        if (u * nt + tid < p.H8)
#pragma unroll
            for (int k = 0; k < WN; ++k)
                wv[u][k] = __ldg(static_cast<const uint4 *>(p.weight) + WN * (u * nt + tid) + k);

    int s = 0, turn = 0;
    uint32_t phase = 0;
    bool failed = false;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const bool ok = wait_bounded(&full[s], phase, &abort_flag, nullptr);
        const uint4 *sx = reinterpret_cast<const uint4 *>(smem + (size_t)s * IN * row_bytes);
        float h[V][8];
        float ss = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = u * nt + tid;
#pragma unroll
            for (int c = 0; c < 8; ++c) h[u][c] = 0.0f;
            if (i < p.H8) {
                unpack8(sx[i], h[u]);
                if (RES) {
                    float r[8];
                    unpack8(sx[p.H8 + i], r);
#pragma unroll
                    for (int c = 0; c < 8; ++c) h[u][c] += r[c];
                    if (p.residual_out && ok) p.residual_out[t * p.H8 + i] = pack8(h[u]);
                }
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) ss = fmaf(h[u][c], h[u][c], ss);
        }
        ss = block_sum(ss, part[turn], !ok, failed);
        if (failed) break;
        turn ^= 1;
        // everyone has read the stage: the token kStages ahead may land in it
        if (tid == 0 && t + (int64_t)kStages * gridDim.x < p.T) load(t + (int64_t)kStages * gridDim.x, s);
        if (++s == kStages) { s = 0; phase ^= 1u; }
        float r = __frsqrt_rn(fmaf(ss, p.inv_h, p.eps));
        if (!(ss <= kF32Max)) {
            // squares past fp32's range (|h| above about 1e17): the same with
            // h * 2^-80, beside which eps is nothing.  An infinite or NaN h
            // leaves r at 0 or NaN, as the formula does.
            ss = 0.0f;
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    h[u][c] *= 0x1p-80f;
                    ss = fmaf(h[u][c], h[u][c], ss);
                }
            r = __frsqrt_rn(block_sum(ss, part[turn], false, failed) * p.inv_h);
            turn ^= 1;
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = u * nt + tid;
            const bool in = i < p.H8;
            float amax = 0.0f;
            if (in) {
                float w[8];
                if (W_BF16) {
                    unpack8(wv[u][0], w);
                } else {
                    const uint4 a = wv[u][0], b = wv[u][WN - 1];
                    w[0] = __uint_as_float(a.x); w[1] = __uint_as_float(a.y);
                    w[2] = __uint_as_float(a.z); w[3] = __uint_as_float(a.w);
                    w[4] = __uint_as_float(b.x); w[5] = __uint_as_float(b.y);
                    w[6] = __uint_as_float(b.z); w[7] = __uint_as_float(b.w);
                }
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

template <int V, bool W_BF16, bool RES>
moe_status launch(const NormDev &p, cudaStream_t stream) {
    auto kernel = k_add_rms_norm<V, W_BF16, RES>;
    const size_t smem = (size_t)kStages * (RES ? 2 : 1) * p.H8 * 16;
    if (!set_smem_limit((const void *)kernel, smem)) return MOE_ERR_CUDA;
    const int threads = ((p.H8 + V - 1) / V + 31) / 32 * 32;
    // as many blocks as fit beside each other on every SM
    const size_t room = 224 * 1024;
    const int64_t per_sm = std::max<int64_t>(1, std::min<int64_t>(room / (smem + 1024), 2048 / 3 * 2 / threads));
    const int64_t cap = num_sms() * per_sm;
    const unsigned grid = (unsigned)(p.T < cap ? p.T : cap);
    MOE_LAUNCH("add_rms_norm", kernel, grid, threads, smem, stream, p);
    return MOE_OK;
}

template <int V>
moe_status launch_v(const NormDev &p, bool w_bf16, cudaStream_t stream) {
    if (p.residual) return w_bf16 ? launch<V, true, true>(p, stream) : launch<V, false, true>(p, stream);
    return w_bf16 ? launch<V, true, false>(p, stream) : launch<V, false, false>(p, stream);
}

}  // namespace

moe_status launch_add_rms_norm(int64_t T, int64_t H, const void *x, const void *residual,
                               const void *weight, bool w_bf16, float eps, void *residual_out,
                               void *y, void *q, float *scales, cudaStream_t stream) {
    NormDev p;
    p.x = static_cast<const uint4 *>(x);
    p.residual = static_cast<const uint4 *>(residual);
    p.weight = weight;
    p.residual_out = static_cast<uint4 *>(residual_out);
    p.y = static_cast<uint4 *>(y);
    p.q = static_cast<uint2 *>(q);
    p.scales = scales;
    p.T = T;
    p.H8 = (int)(H / 8);
    p.nb = (int)((H + kFp8Block - 1) / kFp8Block);
    p.eps = eps;
    p.inv_h = 1.0f / (float)H;
    // vectors a thread: few enough for registers, many enough for at most 512 threads
    if (p.H8 <= 256) return launch_v<1>(p, w_bf16, stream);
    if (p.H8 <= 1024) return launch_v<2>(p, w_bf16, stream);
    return launch_v<4>(p, w_bf16, stream);
}

}  // namespace moe
