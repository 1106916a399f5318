// gate.cu -- router: scores, balance bias, expert groups, top-k, weights.
//
// One warp per token.  Lane l holds the logits of experts l, l + 32, ... in
// registers, so every load of the warp is one contiguous run whatever the row
// stride.  The choice is K rounds of a warp-wide arg-max over (key, lower
// index first); groups are valued from a copy of the keys in shared memory.
#include "common.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kGateWarps = 4;
constexpr float kClosed = -1e30f;          // a logit at or below this closes the expert
constexpr float kF32Max = 3.402823466e38f;

struct GateDev {
    const void *logits;
    const float *bias;
    const uint8_t *mask;
    int32_t *ids;
    float *scales;
    uint8_t *route_mask;
    int64_t T, stride;
    int E, K, G, KG, per;     // per = E / G
    int bf16, sigmoid, top2, renorm;
    float scale;
};

__device__ __forceinline__ float ninf() { return __uint_as_float(0xff800000u); }

// Larger key first, lower index first among equal keys.
__device__ __forceinline__ void warp_argmax(float &v, int &i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float ov = __shfl_xor_sync(kFull, v, o);
        const int oi = __shfl_xor_sync(kFull, i, o);
        if (ov > v || (ov == v && oi < i)) { v = ov; i = oi; }
    }
}

template <int VPL>
__global__ void __launch_bounds__(32 * kGateWarps)
k_gate(GateDev p) {
    extern __shared__ float sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *skey = sm + warp * (p.E + p.G);    // keys, then group values
    float *sgrp = skey + p.E;
    pdl_wait();
    for (int64_t t = (int64_t)blockIdx.x * kGateWarps + warp; t < p.T;
         t += (int64_t)gridDim.x * kGateWarps) {
        const bool active = p.mask == nullptr || p.mask[t] != 0;
        float l[VPL], score[VPL], key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int i = j * 32 + lane;
            float v = ninf();
            if (active && i < p.E) {
                const int64_t at = t * p.stride + i;
                v = p.bf16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p.logits)[at])
                           : static_cast<const float *>(p.logits)[at];
            }
            l[j] = v > kClosed ? fminf(v, kF32Max) : ninf();   // NaN compares false: closed
        }
        if (p.sigmoid) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) score[j] = __fdiv_rn(1.0f, 1.0f + expf(-l[j]));
        } else {
            float m = -kF32Max;
#pragma unroll
            for (int j = 0; j < VPL; ++j) m = fmaxf(m, l[j]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                score[j] = expf(l[j] - m);
                s += score[j];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            s = fmaxf(s, 1e-30f);
#pragma unroll
            for (int j = 0; j < VPL; ++j) score[j] = __fdiv_rn(score[j], s);
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int i = j * 32 + lane;
            const float b = (p.bias && i < p.E) ? p.bias[i] : 0.0f;
            key[j] = l[j] == ninf() ? ninf() : score[j] + b;
        }
        if (p.G > 1) {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (j * 32 + lane < p.E) skey[j * 32 + lane] = key[j];
            __syncwarp();
            for (int g = lane; g < p.G; g += 32) {
                float a = ninf(), b = ninf();
                for (int i = 0; i < p.per; ++i) {
                    const float v = skey[g * p.per + i];
                    b = fmaxf(b, fminf(a, v));
                    a = fmaxf(a, v);
                }
                sgrp[g] = (p.top2 && b != ninf()) ? a + b : a;
            }
            __syncwarp();
            // the KG best groups: mark each winner in place by NaN
            for (int r = 0; r < p.KG; ++r) {
                float bv = ninf();
                int bi = INT32_MAX;
                for (int g = lane; g < p.G; g += 32)
                    if (sgrp[g] > bv) { bv = sgrp[g]; bi = g; }
                warp_argmax(bv, bi);
                if (bi == INT32_MAX) break;     // the groups left are closed
                if (lane == 0) sgrp[bi] = __uint_as_float(0x7fc00000u);
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int i = j * 32 + lane;
                if (i < p.E && sgrp[i / p.per] == sgrp[i / p.per]) key[j] = ninf();
            }
            __syncwarp();
        }
        int my_id = -1;                 // lane k keeps the k-th choice
        float my_w = 0.0f;
        for (int k = 0; k < p.K; ++k) {
            float bv = ninf();
            int bi = INT32_MAX;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (key[j] > bv) { bv = key[j]; bi = j * 32 + lane; }
            warp_argmax(bv, bi);
            if (bi == INT32_MAX) break;         // nothing open is left
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (bi == j * 32 + lane) { s = score[j]; key[j] = ninf(); }
            s = __shfl_sync(kFull, s, bi & 31);
            if (lane == k) { my_id = bi; my_w = s; }
        }
        float sum = my_w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (p.renorm) my_w = __fdiv_rn(my_w, sum + 1e-20f);
        if (lane < p.K) {
            const int64_t at = t * p.K + lane;
            p.ids[at] = my_id;
            p.scales[at] = my_w * p.scale;
            if (p.route_mask) p.route_mask[at] = my_id >= 0;
        }
    }
}

}  // namespace

moe_status launch_gate(const moe_gate_desc &d, const void *logits, const float *bias,
                       const uint8_t *mask, int32_t *ids, float *scales, uint8_t *route_mask,
                       cudaStream_t stream) {
    GateDev p;
    p.logits = logits;
    p.bias = bias;
    p.mask = mask;
    p.ids = ids;
    p.scales = scales;
    p.route_mask = route_mask;
    p.T = d.num_tokens;
    p.stride = d.logits_stride;
    p.E = (int)d.num_experts;
    p.K = (int)d.topk;
    p.G = (int)d.num_groups;
    p.KG = (int)d.topk_groups;
    p.per = p.E / p.G;
    p.bf16 = d.logits_dtype == MOE_DTYPE_BF16;
    p.sigmoid = d.score == MOE_GATE_SIGMOID;
    p.top2 = d.group_score == MOE_GATE_GROUP_TOP2;
    p.renorm = d.renormalize;
    p.scale = d.scale;
    const int64_t want = (p.T + kGateWarps - 1) / kGateWarps;
    const int64_t cap = (int64_t)num_sms() * 16;
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    const size_t smem = (size_t)kGateWarps * (p.E + p.G) * sizeof(float);
    const int vpl = (p.E + 31) / 32;
    if (vpl <= 1) MOE_LAUNCH("gate", k_gate<1>, grid, 32 * kGateWarps, smem, stream, p);
    else if (vpl <= 2) MOE_LAUNCH("gate", k_gate<2>, grid, 32 * kGateWarps, smem, stream, p);
    else if (vpl <= 4) MOE_LAUNCH("gate", k_gate<4>, grid, 32 * kGateWarps, smem, stream, p);
    else if (vpl <= 8) MOE_LAUNCH("gate", k_gate<8>, grid, 32 * kGateWarps, smem, stream, p);
    else if (vpl <= 16) MOE_LAUNCH("gate", k_gate<16>, grid, 32 * kGateWarps, smem, stream, p);
    else MOE_LAUNCH("gate", k_gate<32>, grid, 32 * kGateWarps, smem, stream, p);
    return MOE_OK;
}

}  // namespace moe
