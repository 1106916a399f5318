// gate.cu -- router: scores, balance bias, expert groups, top-k, weights.
//
// One warp per token.  Lane l holds the keys of the VPL experts l * VPL ... in
// registers.  The choice:
//   1. K or a few more rounds over the lanes' largest keys (a warp-wide maximum
//      by redux; the lanes that have it step out) give a lower bound of the
//      K-th largest key.  Only keys at or above it can be chosen: about 9 of
//      256 for K = 8, 22 of 1000 for K = 16.
//   2. Those candidates are collected in the order of their experts, one a lane.
//   3. A candidate's place is the number of candidates before it (larger key,
//      or equal key and lower expert).
// More than 32 candidates (many equal keys) are chosen one by one instead.
// K rounds of a full arg-max, each lane looking through its registers after a
// win, measured 26 us against 11 for this (32768 tokens, 256 experts, K = 8).
//
// A warp's instructions bound it, not memory: so nothing is computed for
// experts that is not needed for the choice.  Without a bias the keys are the
// logits themselves (scores order as they do); with one, the scores behind the
// keys use the hardware's approximate exponential and reciprocal (a few units
// in the last place); the K scores that become weights are computed again from
// their logits with expf.
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
    int vec;                  // a lane's logits load as 16-byte vectors (or whole, if shorter)
    int lanes_per_group;      // lanes a group fills exactly (a power of two), 0 if it does not
    float scale;
};

__device__ __forceinline__ float ninf() { return __uint_as_float(0xff800000u); }

// Largest of the warp's values (no NaN among them).
__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm("redux.sync.max.f32 %0, %1, %2;" : "=f"(m) : "f"(v), "r"(kFull));
    return m;
}

// A logit as the keys see it: closed experts (NaN included) at -inf.
__device__ __forceinline__ float open_logit(float v) { return v > kClosed ? v : ninf(); }

__device__ __forceinline__ float load_logit(const GateDev &p, int64_t at) {
    return p.bf16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p.logits)[at])
                  : static_cast<const float *>(p.logits)[at];
}

// kSmemStride: floats between two lanes' registers in shared memory, odd so
// that the lanes' reads fall into different banks.
template <int VPL>
constexpr int kSmemStride = VPL + (VPL > 1);

template <int VPL>
__device__ __forceinline__ float lane_max(const float (&key)[VPL]) {
    float m = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) m = fmaxf(m, key[j]);
    return m;
}

template <int VPL>
__global__ void __launch_bounds__(32 * kGateWarps)
k_gate(GateDev p) {
    __shared__ float s_keys[kGateWarps][32 * kSmemStride<VPL>];
    __shared__ __align__(16) float s_key[kGateWarps][32];   // candidates
    __shared__ int s_cand[kGateWarps][32];
    __shared__ int s_ids[kGateWarps][kMaxTopK];
    extern __shared__ float s_groups[];         // [warps][G], groups that straddle lanes only
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *sk = s_keys[warp];
    const int e0 = lane * VPL;                  // the lane's first expert
    pdl_wait();
    for (int64_t t = (int64_t)blockIdx.x * kGateWarps + warp; t < p.T;
         t += (int64_t)gridDim.x * kGateWarps) {
        const bool active = p.mask == nullptr || p.mask[t] != 0;
        const int64_t row = t * p.stride;
        float key[VPL];
        // ---- logits
        if (!active) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = ninf();
        } else if (VPL <= 8 && p.vec) {
            const bool in = e0 < p.E;
            if (p.bf16) {
                const uint16_t *src = static_cast<const uint16_t *>(p.logits) + row + e0;
                uint32_t w[VPL > 1 ? VPL / 2 : 1];
#pragma unroll
                for (int j = 0; j < (VPL > 1 ? VPL / 2 : 1); ++j) w[j] = 0;
                if (in) {
                    if constexpr (VPL == 8) *reinterpret_cast<uint4 *>(w) = __ldg(reinterpret_cast<const uint4 *>(src));
                    else if constexpr (VPL == 4) *reinterpret_cast<uint2 *>(w) = __ldg(reinterpret_cast<const uint2 *>(src));
                    else if constexpr (VPL == 2) w[0] = __ldg(reinterpret_cast<const uint32_t *>(src));
                    else w[0] = __ldg(src);
                }
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    key[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
            } else {
                const float *src = static_cast<const float *>(p.logits) + row + e0;
                if (in) {
                    if constexpr (VPL >= 4) {
#pragma unroll
                        for (int j = 0; j < VPL; j += 4)
                            *reinterpret_cast<float4 *>(key + j) = __ldg(reinterpret_cast<const float4 *>(src + j));
                    } else if constexpr (VPL == 2) {
                        *reinterpret_cast<float2 *>(key) = __ldg(reinterpret_cast<const float2 *>(src));
                    } else {
                        key[0] = __ldg(src);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = in ? open_logit(key[j]) : ninf();
        } else {
            // neighbours on neighbouring lanes (whole sectors whatever the
            // alignment), then through shared memory to the lanes that hold them
            __syncwarp();
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = 32 * j + lane < p.E ? load_logit(p, row + 32 * j + lane) : ninf();
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int i = 32 * j + lane;
                sk[i / VPL * kSmemStride<VPL> + i % VPL] = open_logit(key[j]);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = sk[lane * kSmemStride<VPL> + j];
        }
        // ---- scores and keys
        float top = 0.0f, sum = 1.0f;           // softmax: the largest logit, the exponentials' sum
        if (!p.sigmoid) {
            top = fminf(fmaxf(warp_max(lane_max<VPL>(key)), -kF32Max), kF32Max);
            if (!p.renorm || p.bias) {          // renormalised weights do not need the sum
                sum = 0.0f;
#pragma unroll
                for (int j = 0; j < VPL; ++j) sum += __expf(fminf(key[j], kF32Max) - top);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
                sum = fmaxf(sum, 1e-30f);
            }
        }
        if (p.bias) {
            const float inv = __fdividef(1.0f, sum);
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const float s = p.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-key[j]))
                                          : __expf(fminf(key[j], kF32Max) - top) * inv;
                const float b = e0 + j < p.E ? __ldg(p.bias + e0 + j) : 0.0f;
                key[j] = key[j] == ninf() ? ninf() : s + b;
            }
        }
        // ---- groups
        if (p.G > 1) {
            // Without a bias the keys are logits; a group's value is of scores.
            const bool logit_keys = p.top2 && !p.bias;
            auto value = [&](float k) {
                if (!logit_keys || k == ninf()) return k;
                return p.sigmoid ? __fdividef(1.0f, 1.0f + expf(-k)) : expf(fminf(k, kF32Max) - top);
            };
            auto group_value = [&](float a, float b) {
                return p.top2 && b != ninf() ? value(a) + value(b) : value(a);
            };
            if (p.lanes_per_group) {
                float a = ninf(), b = ninf();   // the group's two largest keys
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    b = fmaxf(b, fminf(a, key[j]));
                    a = fmaxf(a, key[j]);
                }
                for (int o = 1; o < p.lanes_per_group; o <<= 1) {
                    const float oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
                    b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                    a = fmaxf(a, oa);
                }
                const float gv = group_value(a, b);
                const int mine = lane / p.lanes_per_group;
                int rank = 0;                   // groups that come before the lane's
                for (int g = 0; g < p.G; ++g) {
                    const float v = __shfl_sync(kFull, gv, g * p.lanes_per_group);
                    rank += v > gv || (v == gv && g < mine);
                }
                if (rank >= p.KG || mine >= p.G) {
#pragma unroll
                    for (int j = 0; j < VPL; ++j) key[j] = ninf();
                }
            } else {
                float *sg = s_groups + warp * p.G;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < VPL; ++j) sk[lane * kSmemStride<VPL> + j] = key[j];
                __syncwarp();
                for (int g = lane; g < p.G; g += 32) {
                    float a = ninf(), b = ninf();
                    for (int i = g * p.per; i < (g + 1) * p.per; ++i) {
                        const float v = sk[i / VPL * kSmemStride<VPL> + i % VPL];
                        b = fmaxf(b, fminf(a, v));
                        a = fmaxf(a, v);
                    }
                    sg[g] = group_value(a, b);
                }
                __syncwarp();
                // a group stays if fewer than KG come before it
                for (int g0 = 0; g0 < p.G; g0 += 32) {
                    const int g = g0 + lane;
                    const float gv = g < p.G ? sg[g] : ninf();
                    int rank = 0;
                    for (int o = 0; o < p.G; ++o) {
                        const float v = sg[o];
                        rank += v > gv || (v == gv && o < g);
                    }
                    __syncwarp();
                    const uint32_t stay = __ballot_sync(kFull, g < p.G && rank < p.KG);
                    if (lane == 0) sk[g0 / 32] = __uint_as_float(stay);
                }
                __syncwarp();
                const uint32_t *stay = reinterpret_cast<const uint32_t *>(sk);
                int g = e0 / p.per, left = (g + 1) * p.per - e0;   // experts to the group's end
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    if (e0 + j < p.E && !((stay[g >> 5] >> (g & 31)) & 1u)) key[j] = ninf();
                    if (--left == 0) { left = p.per; ++g; }
                }
                __syncwarp();
            }
        }
        // ---- the K best
        float bound = ninf(), cur = lane_max<VPL>(key);
        for (int k = 0; k < p.K; k += 4)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                bound = warp_max(cur);
                cur = cur == bound ? ninf() : cur;
            }
        // candidates of the lower lanes come first
        int own = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) own += key[j] >= bound && key[j] > ninf();
        int upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += v;
        }
        const int count = __shfl_sync(kFull, upto, 31);
        const int n = min(count, p.K);          // experts that are chosen
        if (count <= 32) {
            s_key[warp][lane] = ninf();
            __syncwarp();
            int at = upto - own;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (key[j] >= bound && key[j] > ninf()) {
                    s_key[warp][at] = key[j];
                    s_cand[warp][at] = e0 + j;
                    ++at;
                }
            __syncwarp();
            const float mine = s_key[warp][lane];
            int place = 0;
            for (int i = 0; i < count; i += 4) {
                const float4 o = *reinterpret_cast<const float4 *>(&s_key[warp][i]);
                place += (o.x > mine || (o.x == mine && i < lane)) + (o.y > mine || (o.y == mine && i + 1 < lane)) +
                         (o.z > mine || (o.z == mine && i + 2 < lane)) + (o.w > mine || (o.w == mine && i + 3 < lane));
            }
            if (lane < count && place < p.K) s_ids[warp][place] = s_cand[warp][lane];
        } else {
            uint32_t used = 0;
            for (int k = 0; k < n; ++k) {
                float m = ninf();
                int j1 = 0;
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    if (!((used >> j) & 1u) && key[j] > m) { m = key[j]; j1 = j; }
                const float best = warp_max(m);
                const uint32_t have = __ballot_sync(kFull, m == best);
                if (m == best && (have & lanemask_lt()) == 0) {
                    s_ids[warp][k] = e0 + j1;
                    used |= 1u << j1;
                }
            }
        }
        __syncwarp();
        // ---- weights: lane k has the k-th choice
        int id = -1;
        float w = 0.0f;
        if (lane < n) {
            id = s_ids[warp][lane];
            const float l = fminf(load_logit(p, row + id), kF32Max);
            w = __fdividef(p.sigmoid ? 1.0f : expf(l - top), p.sigmoid ? 1.0f + expf(-l) : sum);
        }
        __syncwarp();
        if (p.renorm) {
            float s = w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            w = __fdividef(w, s + 1e-20f);
        }
        if (lane < p.K) {
            const int64_t at = t * p.K + lane;
            p.ids[at] = id;
            p.scales[at] = w * p.scale;
            if (p.route_mask) p.route_mask[at] = id >= 0;
        }
    }
}

template <int VPL>
moe_status launch_vpl(GateDev &p, const moe_gate_desc &d, cudaStream_t stream) {
    const size_t esize = p.bf16 ? 2 : 4;
    const size_t lane_bytes = VPL * esize;
    const size_t align = lane_bytes < 16 ? lane_bytes : 16;
    // up to eight experts a lane a vector load of the lane's own logits uses
    // whole sectors; with more, or unaligned rows, they go through shared memory
    p.vec = VPL <= 8 && p.E % VPL == 0 && (uintptr_t)p.logits % align == 0 &&
            (size_t)d.logits_stride * esize % align == 0;
    const int lanes = p.per % VPL == 0 ? p.per / VPL : 0;
    p.lanes_per_group = lanes > 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    const int64_t want = (p.T + kGateWarps - 1) / kGateWarps;
    const int64_t cap = (int64_t)num_sms() * 16;
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    const size_t smem = p.G > 1 && !p.lanes_per_group ? (size_t)kGateWarps * p.G * sizeof(float) : 0;
    MOE_LAUNCH("gate", k_gate<VPL>, grid, 32 * kGateWarps, smem, stream, p);
    return MOE_OK;
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
    const int vpl = (p.E + 31) / 32;
    if (vpl <= 1) return launch_vpl<1>(p, d, stream);
    if (vpl <= 2) return launch_vpl<2>(p, d, stream);
    if (vpl <= 4) return launch_vpl<4>(p, d, stream);
    if (vpl <= 8) return launch_vpl<8>(p, d, stream);
    if (vpl <= 16) return launch_vpl<16>(p, d, stream);
    return launch_vpl<32>(p, d, stream);
}

}  // namespace moe
