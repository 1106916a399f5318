// norm.cu -- residual addition, root-mean-square norm and block-scaled e4m3.
//
// One CTA per token.  Thread i holds the 16-byte vectors i, i + 256, ... of the
// row (eight channels each) in registers from the load to the stores, so every
// input is read once.  A block of 128 channels is 16 neighbouring vectors, half
// a warp: its maximum is four shuffles.
#include "common.cuh"
#include "fp8.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kNormThreads = 256;
constexpr float kF32Max = 3.402823466e38f;

struct NormDev {
    const uint4 *x, *residual;
    const void *weight;
    uint4 *residual_out, *y;
    uint2 *q;
    float *scales;
    int64_t T;
    int H, H8, nb;
    float eps, inv_h;
};

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
}

// Sum over the CTA, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kNormThreads / 32; ++w) v += part[w];
    return v;
}

template <int V, bool W_BF16>
__global__ void __launch_bounds__(kNormThreads)
k_add_rms_norm(NormDev p) {
    __shared__ float part[kNormThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        float h[V][8];
        float ss = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = u * kNormThreads + tid;
#pragma unroll
            for (int c = 0; c < 8; ++c) h[u][c] = 0.0f;
            if (i < p.H8) {
                unpack8(p.x[t * p.H8 + i], h[u]);
                if (p.residual) {
                    float r[8];
                    unpack8(p.residual[t * p.H8 + i], r);
#pragma unroll
                    for (int c = 0; c < 8; ++c) h[u][c] += r[c];
                    if (p.residual_out) p.residual_out[t * p.H8 + i] = pack8(h[u]);
                }
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) ss = fmaf(h[u][c], h[u][c], ss);
        }
        ss = block_sum(ss, part);
        float r = __frsqrt_rn(fmaf(ss, p.inv_h, p.eps));
        if (!(ss <= kF32Max)) {
            // squares past fp32's range (|h| above about 1e17): the same sum of
            // (h * 2^-80)^2, beside which eps is nothing.  An infinite or NaN
            // h leaves r at 0 or NaN, as the formula does.
            ss = 0.0f;
#pragma unroll
            for (int u = 0; u < V; ++u)
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float d = h[u][c] * 0x1p-80f;
                    ss = fmaf(d, d, ss);
                }
            r = __frsqrt_rn(block_sum(ss, part) * p.inv_h) * 0x1p-80f;
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int i = u * kNormThreads + tid;
            const bool in = i < p.H8;
            float amax = 0.0f;
            if (in) {
                float w[8];
                if (W_BF16) {
                    unpack8(static_cast<const uint4 *>(p.weight)[i], w);
                } else {
                    const float4 a = static_cast<const float4 *>(p.weight)[2 * i];
                    const float4 b = static_cast<const float4 *>(p.weight)[2 * i + 1];
                    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
                    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    h[u][c] = h[u][c] * r * w[c];
                    amax = fmaxf(amax, fabsf(h[u][c]));
                }
                if (p.y) p.y[t * p.H8 + i] = pack8(h[u]);
            }
            if (p.q) {
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
                if (in) {
                    float s, inv;
                    block_scale(amax, s, inv);
                    p.q[t * p.H8 + i] =
                        make_uint2(e4m3x4(h[u][0] * inv, h[u][1] * inv, h[u][2] * inv, h[u][3] * inv),
                                   e4m3x4(h[u][4] * inv, h[u][5] * inv, h[u][6] * inv, h[u][7] * inv));
                    if ((lane & 15) == 0) p.scales[t * p.nb + (i >> 4)] = s;
                }
            }
        }
    }
}

template <int V>
moe_status launch_v(const NormDev &p, bool w_bf16, cudaStream_t stream) {
    const int64_t cap = (int64_t)num_sms() * 8;
    const unsigned grid = (unsigned)(p.T < cap ? p.T : cap);
    if (w_bf16) MOE_LAUNCH("add_rms_norm", (k_add_rms_norm<V, true>), grid, kNormThreads, 0, stream, p);
    else MOE_LAUNCH("add_rms_norm", (k_add_rms_norm<V, false>), grid, kNormThreads, 0, stream, p);
    return MOE_OK;
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
    p.H = (int)H;
    p.H8 = (int)(H / 8);
    p.nb = (int)((H + kFp8Block - 1) / kFp8Block);
    p.eps = eps;
    p.inv_h = 1.0f / (float)H;
    const int v = (p.H8 + kNormThreads - 1) / kNormThreads;
    if (v <= 1) return launch_v<1>(p, w_bf16, stream);
    if (v <= 2) return launch_v<2>(p, w_bf16, stream);
    if (v <= 4) return launch_v<4>(p, w_bf16, stream);
    return launch_v<8>(p, w_bf16, stream);
}

}  // namespace moe
