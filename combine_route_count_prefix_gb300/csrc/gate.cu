// gate.cu -- router: scores, balance bias, expert groups, top-k, weights.
//
// One warp per token.  A lane holds the keys of a run of up to VPL neighbouring
// experts in registers; the runs are in the lanes' order, and with groups a
// whole power of two of lanes holds a group, so that its value is a few
// shuffles (where that would take runs of more than 32, the keys go through
// shared memory instead).  The choice:
//   1. K or a few more rounds over the lanes' largest keys (a warp-wide maximum
//      by redux; the lanes that have it step out) give a lower bound of the
//      K-th largest key; over quarters of the lanes' keys where few lanes
//      have any.  Only keys at or above it can be chosen: about 9 of
//      256 for K = 8, 22 of 1000 for K = 16.
//   2. Those candidates are collected in the order of their experts, one a lane.
//   3. A candidate's place is the number of candidates before it (larger key,
//      or equal key and lower expert).
// More than 32 candidates (many equal keys) are chosen one by one instead.
// K rounds of a full arg-max, each lane looking through its registers after a
// win, measured 26 us against 11 for this (32768 tokens, 256 experts, K = 8).
//
// A warp's instructions bound it, not memory (32768 tokens, 256 experts of
// bf16 logits, K = 8: 11 us with the logits in L2, where their bytes would take
// 2.9 us from HBM): so nothing is computed for
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
    int sigmoid, top2, renorm;
    int run;                  // experts a lane holds at most
    int padded;               // runs of VPL: in shared memory a float is left out after each
    int group_lanes;          // lanes that hold a group, 0 if runs do not end with the groups
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

template <bool BF16>
__device__ __forceinline__ float load_logit(const GateDev &p, int64_t at) {
    return BF16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p.logits)[at])
                  : static_cast<const float *>(p.logits)[at];
}

template <int VPL>
__device__ __forceinline__ float lane_max(const float (&key)[VPL]) {
    float m = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) m = fmaxf(m, key[j]);
    return m;
}

// VEC: runs load as vectors.
template <int VPL, bool BF16, bool VEC>
__global__ void __launch_bounds__(32 * kGateWarps, 8)
k_gate(GateDev p) {
    __shared__ float s_keys[kGateWarps][32 * VPL + 32];
    __shared__ float s_bias[32 * VPL + 32];
    __shared__ __align__(16) float2 s_cand[kGateWarps][32];   // candidates: key, expert
    __shared__ int s_ids[kGateWarps][kMaxTopK];
    extern __shared__ float s_groups[];         // [warps][G], where group_lanes is 0
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *sk = s_keys[warp];
    // Shared memory holds the experts in order; runs of VPL, a power of two,
    // with a float left out after each, so that the lanes' reads of their runs
    // fall into different banks.
    const int pad = p.padded ? 1 : 0;
    const int store0 = lane + pad * (lane / VPL), store_step = 32 + pad * (32 / VPL);
    // the lane's first expert, and how many it has
    int e0 = lane * p.run, have = min(p.run, p.E - e0);
    if (p.group_lanes) {
        const int g = lane / p.group_lanes, l = lane % p.group_lanes;
        e0 = g * p.per + l * p.run;
        have = g < p.G ? min(p.run, p.per - l * p.run) : 0;
    }
    const int run0 = e0 + pad * lane;           // the run's place in shared memory
    pdl_wait();
    if (p.bias) {
        for (int i = threadIdx.x; i < p.E; i += 32 * kGateWarps) s_bias[i + pad * (i / VPL)] = p.bias[i];
        __syncthreads();
    }
    for (int64_t t = (int64_t)blockIdx.x * kGateWarps + warp; t < p.T;
         t += (int64_t)gridDim.x * kGateWarps) {
        const bool active = p.mask == nullptr || p.mask[t] != 0;
        const int64_t row = t * p.stride;
        float key[VPL];
        // ---- logits: what is not loaded stays NaN, which closes it
        if constexpr (VEC) {
            const bool in = active && have > 0;
            if constexpr (BF16) {
                const uint16_t *src = static_cast<const uint16_t *>(p.logits) + row + e0;
                uint32_t w[VPL > 1 ? VPL / 2 : 1];
#pragma unroll
                for (int j = 0; j < (VPL > 1 ? VPL / 2 : 1); ++j) w[j] = 0xffffffffu;
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
#pragma unroll
                for (int j = 0; j < VPL; ++j) key[j] = __uint_as_float(0xffffffffu);
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
        } else {
            // neighbours on neighbouring lanes (whole sectors whatever the
            // alignment), then through shared memory to the lanes that hold them
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                key[j] = __uint_as_float(0xffffffffu);
                if (active && 32 * j + lane < p.E) key[j] = load_logit<BF16>(p, row + 32 * j + lane);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                sk[store0 + j * store_step] = key[j];
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                key[j] = j < have ? sk[run0 + j] : __uint_as_float(0xffffffffu);
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) key[j] = open_logit(key[j]);
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
                if (key[j] != ninf()) key[j] = s + s_bias[run0 + j];
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
            if (p.group_lanes) {
                float a = ninf(), b = ninf();   // the group's two largest keys
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    b = fmaxf(b, fminf(a, key[j]));
                    a = fmaxf(a, key[j]);
                }
                for (int o = 1; o < p.group_lanes; o <<= 1) {
                    const float oa = __shfl_xor_sync(kFull, a, o), ob = __shfl_xor_sync(kFull, b, o);
                    b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                    a = fmaxf(a, oa);
                }
                const float gv = group_value(a, b);
                const int mine = lane / p.group_lanes;
                int rank = 0;                   // groups that come before the lane's
                for (int g = 0; g < p.G; ++g) {
                    const float v = __shfl_sync(kFull, gv, g * p.group_lanes);
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
                for (int j = 0; j < VPL; ++j)
                    if (j < have) sk[run0 + j] = key[j];
                __syncwarp();
                for (int g = lane; g < p.G; g += 32) {
                    float a = ninf(), b = ninf();
#pragma unroll 8
                    for (int i = g * p.per; i < (g + 1) * p.per; ++i) {
                        const float v = sk[i + pad * (i / VPL)];
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
                int g = have > 0 ? e0 / p.per : 0, left = (g + 1) * p.per - e0;   // experts to the group's end
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    if (j < have && !((stay[g >> 5] >> (g & 31)) & 1u)) key[j] = ninf();
                    if (--left == 0) { left = p.per; ++g; }
                }
                __syncwarp();
            }
        }
        // ---- the K best
        float bound = ninf(), cur = lane_max<VPL>(key);
        if (VPL == 1 || __popc(__ballot_sync(kFull, cur > ninf())) >= 2 * p.K) {
            for (int k = 0; k < p.K; k += 4)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    bound = warp_max(cur);
                    cur = cur == bound ? ninf() : cur;
                }
        } else {
            // with few open lanes (the others' groups fell out) that bound would be
            // low and the candidates many: the same over the largest keys of each
            // lane's quarters
            constexpr int Q = VPL < 4 ? VPL : 4;
            float part[Q];
#pragma unroll
            for (int u = 0; u < Q; ++u) {
                part[u] = key[u];
#pragma unroll
                for (int j = u + Q; j < VPL; j += Q) part[u] = fmaxf(part[u], key[j]);
            }
            for (int k = 0; k < p.K; ++k) {
                bound = warp_max(lane_max<Q>(part));
#pragma unroll
                for (int u = 0; u < Q; ++u) part[u] = part[u] == bound ? ninf() : part[u];
            }
        }
        bound = fmaxf(bound, -kF32Max);         // closed experts are no candidates
        // candidates of the lower lanes come first
        int own = 0;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (key[j] >= bound) ++own;
        int upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += v;
        }
        const int count = __shfl_sync(kFull, upto, 31);
        const int n = min(count, p.K);          // experts that are chosen
        if (count <= 32) {
            float2 *cand = s_cand[warp];
            cand[lane] = make_float2(ninf(), 0.0f);
            __syncwarp();
            float2 *to = cand + (upto - own);
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (key[j] >= bound) *to++ = make_float2(key[j], __int_as_float(e0 + j));
            __syncwarp();
            const float2 own_cand = cand[lane];
            const float mine = own_cand.x;
            int place = 0;
            for (int i = 0; i < count; i += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(cand + i);
                const float4 b = *reinterpret_cast<const float4 *>(cand + i + 2);
                const float4 o = make_float4(a.x, a.z, b.x, b.z);
                // an equal key before the lane's own comes before it
                if (i < lane ? o.x >= mine : o.x > mine) ++place;
                if (i + 1 < lane ? o.y >= mine : o.y > mine) ++place;
                if (i + 2 < lane ? o.z >= mine : o.z > mine) ++place;
                if (i + 3 < lane ? o.w >= mine : o.w > mine) ++place;
            }
            if (lane < count && place < p.K) s_ids[warp][place] = __float_as_int(own_cand.y);
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
            const float l = fminf(load_logit<BF16>(p, row + id), kF32Max);
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

template <int VPL, bool BF16>
moe_status launch_vpl(const GateDev &p, cudaStream_t stream) {
    const size_t lane_bytes = VPL * (BF16 ? 2 : 4);
    const size_t align = lane_bytes < 16 ? lane_bytes : 16;
    // up to eight experts a lane a vector load of the lane's own logits uses
    // whole sectors; with more, or unaligned rows, they go through shared memory
    const bool vec = VPL <= 8 && (VPL == 1 || (p.padded && p.E % VPL == 0)) &&
                     (uintptr_t)p.logits % align == 0 &&
                     (size_t)p.stride * (BF16 ? 2 : 4) % align == 0;
    const int64_t want = (p.T + kGateWarps - 1) / kGateWarps;
    const int64_t cap = (int64_t)num_sms() * 16;
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    const size_t smem = p.G > 1 && !p.group_lanes ? (size_t)kGateWarps * p.G * sizeof(float) : 0;
    auto kernel = vec ? k_gate<VPL, BF16, VPL <= 8> : k_gate<VPL, BF16, false>;
    MOE_LAUNCH("gate", kernel, grid, 32 * kGateWarps, smem, stream, p);
    return MOE_OK;
}

template <bool BF16>
moe_status launch_type(const GateDev &p, int vpl, cudaStream_t stream) {
    switch (vpl) {
        case 1: return launch_vpl<1, BF16>(p, stream);
        case 2: return launch_vpl<2, BF16>(p, stream);
        case 4: return launch_vpl<4, BF16>(p, stream);
        case 8: return launch_vpl<8, BF16>(p, stream);
        case 16: return launch_vpl<16, BF16>(p, stream);
    }
    return launch_vpl<32, BF16>(p, stream);
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
    p.sigmoid = d.score == MOE_GATE_SIGMOID;
    p.top2 = d.group_score == MOE_GATE_GROUP_TOP2;
    p.renorm = d.renormalize;
    p.scale = d.scale;
    // Lanes for a group: the most that 32 lanes give each, in powers of two.
    p.group_lanes = 0;
    p.run = (p.E + 31) / 32;
    if (p.G > 1 && p.G <= 32) {
        int lanes = 32;
        while (lanes * p.G > 32) lanes /= 2;
        const int run = (p.per + lanes - 1) / lanes;
        if (run <= 32) {
            p.group_lanes = lanes;
            p.run = run;
        }
    }
    int vpl = 1;
    while (vpl < p.run) vpl *= 2;
    if (!p.group_lanes) p.run = vpl;   // whole vectors
    p.padded = p.run == vpl && vpl > 1 && (!p.group_lanes || p.per == p.group_lanes * p.run);
    return d.logits_dtype == MOE_DTYPE_BF16 ? launch_type<true>(p, vpl, stream)
                                            : launch_type<false>(p, vpl, stream);
}

}  // namespace moe
