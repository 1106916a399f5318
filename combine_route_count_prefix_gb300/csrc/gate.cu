// gate.cu -- router: scores, balance bias, expert groups, top-k, weights.
//
// One warp per token.  A lane holds the keys of a run of up to VPL neighbouring
// experts; the runs are in the lanes' order, and with groups a whole power of
// two of lanes holds a group where that leaves runs of at most 32, so that its
// value is a few shuffles.  Otherwise a group no shorter than a run is joined
// from its lanes' parts, and shorter ones are looked through in shared memory.
// The choice:
//   1. K or a few more rounds over the lanes' largest keys (a warp-wide maximum
//      by redux; the lanes that have it step out) give a lower bound of the
//      K-th largest key; over quarters of the lanes' keys where few lanes
//      have any.  Only keys at or above it can be chosen: about 9 of
//      256 for K = 8, 22 of 1000 for K = 16.
//   2. Those candidates are collected in the order of their experts, one a lane,
//      which computes its expert's score from the logit with expf.
//   3. A candidate's place is the number of larger candidates and of equal ones
//      in lower lanes; its lane computes its weight and writes it there.
// More than 32 candidates (many equal keys) are chosen one by one instead.
// K rounds of a full arg-max, each lane looking through its keys after a win,
// took 2.4 times as long.
//
// A warp's instructions bound it, not memory, and of those the comparisons,
// maxima and selections, which run at half the rate of the others (32768
// tokens, 256 experts of bf16 logits, K = 8: 16.9 us a call, where the bytes
// take 2.9 us; 4097 tokens, 1000 experts, 20 groups, K = 16: 14.5 us, 2.5).  So
// nothing is computed for experts that is not needed for the choice, and counts
// are kept in floats, so that they are not added on that pipe too (18.6 -> 16.2 us
// together with the next token's logits on their way).  Without a bias the keys
// are the logits until the candidates are known, whose scores then decide (16.3
// -> 16.9 us against the logits alone, whose order is another where scores are
// equal).  With a bias, and for the groups' values, the scores behind the keys use the
// hardware's approximate exponential and reciprocal (a few units in the last
// place); the scores that become weights are always those with expf.
#include "common.cuh"

#include <type_traits>

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kGateWarps = 4;
// Blocks on an SM: 72 registers a thread.  With 8 blocks of 64 some forms spill
// (4097 tokens of 1000 experts 24.8 us against 24.1, 32768 of 512 38.5 against 35.8).
constexpr int kGateBlocks = 7;
constexpr float kClosed = -1e30f;          // a logit at or below this closes the expert
constexpr float kLeastOpen = -0x1.93e592p+99f;   // the next float above it
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
    int padded;               // runs of VPL, one after the other
    int wide;                 // rows can be loaded 16 bytes at a time
    int group_lanes;          // lanes that hold a group, 0 if runs do not end with the groups
    int scratch;              // floats a warp joins the groups' values in
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

// N floats of a lane's run from shared memory: 16 bytes at a time where the runs
// are whole (and so aligned), else the first `have`, the rest closed.
template <int N>
__device__ __forceinline__ void read_run(float (&v)[N], const float *from, bool whole, int have) {
    if (N >= 4 && whole) {
#pragma unroll
        for (int j = 0; j + 3 < N; j += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(from + j);
            v[j] = a.x; v[j + 1] = a.y; v[j + 2] = a.z; v[j + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = whole || j < have ? from[j] : ninf();
    }
}

template <int N>
__device__ __forceinline__ void write_run(const float (&v)[N], float *to, bool whole, int have) {
    if (N >= 4 && whole) {
#pragma unroll
        for (int j = 0; j + 3 < N; j += 4)
            *reinterpret_cast<float4 *>(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (whole || j < have) to[j] = v[j];
    }
}

// 1 / (1 + exp(-x)) with the hardware's approximate exponential and reciprocal,
// whose results at the ends of their ranges (0, infinity) are what is wanted here.
__device__ __forceinline__ float sigmoid_approx(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// The keys without a bias are logits until the candidates are known.  Different
// logits may have the same score in fp32 (1 above 16.6, 0 far below the largest
// one), and then the lower index comes first, whichever logit is larger.  So
// `b`, a lower bound of the K-th largest logit, goes down to where the scores
// are smaller for certain: to where 1 + exp(-l), or exp(l - top), is off by
// 2^-20 of itself and more, eight units in the last place.
__device__ __forceinline__ float sigmoid_floor(float b) {
    const float c = fminf(b, 12.0f);            // 1 - score(12) is 100 units in the last place
    return c < -80.0f ? ninf() : c - fmaf(__expf(c), 0x1p-20f, 0x1p-20f);
}
__device__ __forceinline__ float softmax_floor(float b, float top) {
    b = fminf(b, kF32Max);
    const float d = top - b;                    // rounded to 2^-24 of itself in a score
    return d > 80.0f ? ninf() : b - fmaf(d, 0x1p-21f, 0x1p-20f);
}

// VEC: runs load as vectors.  Runs of up to 16 keys stay in registers, longer
// ones in shared memory, from where eight at a time are looked at (32 keys in
// registers spill: 24 us against 20 for 4097 tokens of 1000 experts, flushed L2).
template <int VPL, bool BF16, bool VEC>
__global__ void __launch_bounds__(32 * kGateWarps, kGateBlocks)
k_gate(GateDev p) {
    __shared__ __align__(16) float s_keys[kGateWarps][32 * VPL + 128];
    __shared__ __align__(16) float s_bias[32 * VPL + 128];
    __shared__ __align__(16) float2 s_cand[kGateWarps][36];   // candidates: key, expert
    extern __shared__ __align__(16) float s_groups[];   // [warps][scratch], where group_lanes is 0
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *sk = s_keys[warp];
    // Shared memory holds the experts in order; whole runs of 8 and more, which
    // are read 16 bytes at a time, with four floats left out after each, so that
    // eight lanes' reads fall into different banks.
    const int pad = p.padded && VPL >= 8 ? 4 : 0;
    // the lane's first expert, and how many it has
    int e0 = lane * p.run, have = min(p.run, p.E - e0);
    if (p.group_lanes) {
        const int g = lane / p.group_lanes, l = lane % p.group_lanes;
        e0 = g * p.per + l * p.run;
        have = g < p.G ? min(p.run, p.per - l * p.run) : 0;
    }
    const int run0 = e0 + pad * lane;           // the run's place in shared memory
    pdl_wait();
    if (p.padded && !VEC)                       // whole runs are read past the last expert
        for (int i = p.E + lane; i < 32 * VPL; i += 32) sk[i + pad * (i / VPL)] = ninf();
    if (p.bias) {
        for (int i = threadIdx.x; i < p.E; i += 32 * kGateWarps) s_bias[i + pad * (i / VPL)] = p.bias[i];
        __syncthreads();
    }
    // without a bias and groups the keys are the logits as they come: the bound
    // keeps closed ones out
    const bool raw_keys = !p.bias && p.G == 1 && (p.sigmoid || p.renorm);
    // Where the runs do not end with the groups and a group is no shorter than
    // a run: the group that the lane's run begins in, and how much of it
    const bool two_groups = p.G > 1 && !p.group_lanes && p.per >= VPL;
    const int first_group = two_groups ? e0 / p.per : 0;
    const int in_first = two_groups ? (first_group + 1) * p.per - e0 : 0;
    const int64_t step = (int64_t)gridDim.x * kGateWarps;
    // a token's run, as it is stored; what is not loaded stays NaN, which closes it
    constexpr int RAW = BF16 ? (VPL > 1 ? VPL / 2 : 1) : VPL;
    uint32_t raw[VEC ? RAW : 1];
    auto fetch = [&](int64_t t) {
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < RAW; ++j) raw[j] = 0xffffffffu;
            if (t >= p.T || have <= 0 || (p.mask && p.mask[t] == 0)) return;
            const uint8_t *src = static_cast<const uint8_t *>(p.logits) +
                                 (t * p.stride + e0) * (BF16 ? 2 : 4);
            if constexpr (BF16 && VPL == 1) raw[0] = __ldg(reinterpret_cast<const uint16_t *>(src));
            else if constexpr (RAW == 1) raw[0] = __ldg(reinterpret_cast<const uint32_t *>(src));
            else if constexpr (RAW == 2) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src));
                raw[0] = v.x; raw[1] = v.y;
            } else {
#pragma unroll
                for (int j = 0; j < RAW; j += 4) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + j / 4);
                    raw[j] = v.x; raw[j + 1] = v.y; raw[j + 2] = v.z; raw[j + 3] = v.w;
                }
            }
        }
    };
    constexpr bool MEM = VPL > 16;
    constexpr int C = MEM ? 8 : VPL;            // keys looked at together
    float key[MEM ? 1 : VPL];
    // f(keys, number of the first) over the lane's run; STORE: f changes them
    auto each = [&](auto store, auto f) {
        if constexpr (MEM) {
#pragma unroll 2
            for (int j0 = 0; j0 < VPL; j0 += C) {
                float k[C];
                read_run<C>(k, sk + run0 + j0, p.padded, have - j0);
                f(k, j0);
                if constexpr (decltype(store)::value) write_run<C>(k, sk + run0 + j0, p.padded, have - j0);
            }
        } else {
            f(key, 0);
        }
    };
    constexpr std::true_type change{};
    constexpr std::false_type look{};
    auto largest = [&]() {                      // of the lane's keys, NaN aside
        float m = ninf();
        each(look, [&](auto &k, int) {
#pragma unroll
            for (int j = 0; j < C; ++j) m = fmaxf(m, k[j]);
        });
        return m;
    };
    int64_t t = (int64_t)blockIdx.x * kGateWarps + warp;
    fetch(t);
    for (; t < p.T; t += step) {
        const int64_t row = t * p.stride;
        // ---- logits
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                key[j] = __uint_as_float(!BF16 ? raw[j] : j & 1 ? raw[j / 2] & 0xffff0000u : raw[j / 2] << 16);
            fetch(t + step);
        } else if (p.mask && p.mask[t] == 0) {
            each(change, [&](auto &k, int) {
#pragma unroll
                for (int j = 0; j < C; ++j) k[j] = ninf();
            });
        } else {
            // neighbours on neighbouring lanes (whole sectors whatever the
            // alignment), then through shared memory to the lanes that hold them
            constexpr int EV = BF16 ? 8 : 4;
            if (VPL >= 16 && p.wide) {
                constexpr int U = VPL / EV < 4 ? (VPL / EV > 0 ? VPL / EV : 1) : 4;
#pragma unroll 1
                for (int j0 = 0; j0 < VPL / EV; j0 += U) {
                    uint4 v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int i = (32 * (j0 + u) + lane) * EV;
                        if (i < p.E)
                            v[u] = __ldg(reinterpret_cast<const uint4 *>(
                                static_cast<const uint8_t *>(p.logits) + (row + i) * (BF16 ? 2 : 4)));
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int i = (32 * (j0 + u) + lane) * EV;
                        if (i >= p.E) continue;
                        uint4 *to = reinterpret_cast<uint4 *>(sk + i + pad * (i / VPL));
                        if constexpr (BF16) {
                            to[0] = make_uint4(v[u].x << 16, v[u].x & 0xffff0000u, v[u].y << 16, v[u].y & 0xffff0000u);
                            to[1] = make_uint4(v[u].z << 16, v[u].z & 0xffff0000u, v[u].w << 16, v[u].w & 0xffff0000u);
                        } else {
                            to[0] = v[u];
                        }
                    }
                }
            } else {
                constexpr int U = VPL < 8 ? VPL : 8;
#pragma unroll 1
                for (int j0 = 0; j0 < VPL; j0 += U) {
                    float v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (32 * (j0 + u) + lane < p.E) v[u] = load_logit<BF16>(p, row + 32 * (j0 + u) + lane);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int i = 32 * (j0 + u) + lane;
                        if (i < p.E) sk[i + pad * (i / VPL)] = v[u];
                    }
                }
            }
            __syncwarp();
            if constexpr (!MEM) {
                read_run<VPL>(key, sk + run0, p.padded, have);
                __syncwarp();
            }
        }
        if (!raw_keys && !(p.bias && p.sigmoid))
            each(change, [&](auto &k, int) {
#pragma unroll
                for (int j = 0; j < C; ++j) k[j] = open_logit(k[j]);
            });
        // ---- scores and keys
        float top = 0.0f, sum = 1.0f;           // softmax: the largest logit, the exponentials' sum
        if (!p.sigmoid) {
            top = fminf(fmaxf(warp_max(largest()), -kF32Max), kF32Max);
            if (!p.renorm || p.bias) {          // renormalised weights do not need the sum
                sum = 0.0f;
                each(look, [&](auto &k, int) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (k[j] > kClosed) sum += __expf(fminf(k[j], kF32Max) - top);
                });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
                sum = fmaxf(sum, 1e-30f);
            }
        }
        if (p.bias) {
            const float inv = __fdividef(1.0f, sum);
            each(change, [&](auto &k, int j0) {
                constexpr int D = C < 4 ? C : 4;
#pragma unroll
                for (int d = 0; d < C; d += D) {
                    float bias[D];
                    read_run<D>(bias, s_bias + run0 + j0 + d, p.padded, have - j0 - d);
#pragma unroll
                    for (int j = 0; j < D; ++j) {
                        const float l = k[d + j];
                        const float score = p.sigmoid ? sigmoid_approx(l) : __expf(fminf(l, kF32Max) - top) * inv;
                        k[d + j] = l > kClosed ? score + bias[j] : ninf();
                    }
                }
            });
        }
        // ---- groups
        if (p.G > 1) {
            // Without a bias the keys are logits; a group's value is of scores.
            auto value = [&](float k) {
                if (p.bias || k == ninf()) return k;
                return p.sigmoid ? sigmoid_approx(k) : __expf(fminf(k, kF32Max) - top);
            };
            auto group_value = [&](float a, float b) {
                return p.top2 && b != ninf() ? value(a) + value(b) : value(a);
            };
            float *scratch = s_groups + warp * p.scratch;
            if (p.group_lanes) {
                float a = ninf(), b = ninf();   // the group's two largest keys
                if (p.top2)
                    each(look, [&](auto &k, int) {
#pragma unroll
                        for (int j = 0; j < C; ++j) {
                            b = fmaxf(b, fminf(a, k[j]));
                            a = fmaxf(a, k[j]);
                        }
                    });
                else
                    a = largest();
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
                if (rank >= p.KG || mine >= p.G)
                    each(change, [&](auto &k, int) {
#pragma unroll
                        for (int j = 0; j < C; ++j) k[j] = ninf();
                    });
            } else if (two_groups) {
                // the two largest keys of the run's part in either group
                float a0 = ninf(), b0 = ninf(), a1 = ninf(), b1 = ninf();
                auto parts = [&](auto two) {
                    each(look, [&](auto &k, int j0) {
#pragma unroll
                        for (int j = 0; j < C; ++j) {
                            const bool first = j0 + j < in_first;
                            const float k0 = first ? k[j] : ninf(), k1 = first ? ninf() : k[j];
                            if constexpr (decltype(two)::value) {
                                b0 = fmaxf(b0, fminf(a0, k0));
                                b1 = fmaxf(b1, fminf(a1, k1));
                            }
                            a0 = fmaxf(a0, k0);
                            a1 = fmaxf(a1, k1);
                        }
                    });
                };
                if (p.top2) parts(std::true_type{}); else parts(std::false_type{});
                float4 *part = reinterpret_cast<float4 *>(scratch);
                part[lane] = make_float4(a0, b0, a1, b1);
                __syncwarp();
                // lane g joins group g's parts: all but the first of its lanes
                // begin in it
                float a = ninf(), b = ninf();
                const int begin = lane * p.per;
                if (lane < p.G)
                    for (int l = begin / VPL; l * VPL < begin + p.per; ++l) {
                        const float4 v = part[l];
                        const float oa = l * VPL < begin ? v.z : v.x, ob = l * VPL < begin ? v.w : v.y;
                        b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                        a = fmaxf(a, oa);
                    }
                const float gv = group_value(a, b);
                int rank = 0;                   // groups that come before the lane's
                for (int g = 0; g < p.G; ++g) {
                    const float v = __shfl_sync(kFull, gv, g);
                    rank += v > gv || (v == gv && g < lane);
                }
                const uint32_t stay = __ballot_sync(kFull, lane < p.G && rank < p.KG);
                const bool stay0 = (stay >> first_group) & 1u;
                const bool stay1 = first_group < 31 && ((stay >> (first_group + 1)) & 1u);
                if (!stay0 || !stay1)
                    each(change, [&](auto &k, int j0) {
#pragma unroll
                        for (int j = 0; j < C; ++j)
                            if (!(j0 + j < in_first ? stay0 : stay1)) k[j] = ninf();
                    });
            } else {
                if constexpr (!MEM) {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < VPL; ++j)
                        if (j < have) sk[run0 + j] = key[j];
                }
                __syncwarp();
                for (int g = lane; g < p.G; g += 32) {
                    float a = ninf(), b = ninf();
#pragma unroll 8
                    for (int i = g * p.per; i < (g + 1) * p.per; ++i) {
                        const float v = sk[i + pad * (i / VPL)];
                        b = fmaxf(b, fminf(a, v));
                        a = fmaxf(a, v);
                    }
                    scratch[g] = group_value(a, b);
                }
                __syncwarp();
                // a group stays if fewer than KG come before it
                uint32_t *stay = reinterpret_cast<uint32_t *>(scratch + p.G);
                for (int g0 = 0; g0 < p.G; g0 += 32) {
                    const int g = g0 + lane;
                    const float gv = g < p.G ? scratch[g] : ninf();
                    int rank = 0;
                    for (int o = 0; o < p.G; ++o) {
                        const float v = scratch[o];
                        rank += v > gv || (v == gv && o < g);
                    }
                    const uint32_t word = __ballot_sync(kFull, g < p.G && rank < p.KG);
                    if (lane == 0) stay[g0 / 32] = word;
                }
                __syncwarp();
                int g = have > 0 ? e0 / p.per : 0, left = (g + 1) * p.per - e0;   // experts to the group's end
                each(change, [&](auto &k, int j0) {
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        if (j0 + j < have && !((stay[g >> 5] >> (g & 31)) & 1u)) k[j] = ninf();
                        if (--left == 0) { left = p.per; ++g; }
                    }
                });
            }
        }
        // ---- the K best
        float bound = ninf(), cur = largest();
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
            for (int u = 0; u < Q; ++u) part[u] = ninf();
            each(look, [&](auto &k, int) {
#pragma unroll
                for (int j = 0; j < C; ++j) part[j % Q] = fmaxf(part[j % Q], k[j]);
            });
            for (int k = 0; k < p.K; ++k) {
                float m = part[0];
#pragma unroll
                for (int u = 1; u < Q; ++u) m = fmaxf(m, part[u]);
                bound = warp_max(m);
#pragma unroll
                for (int u = 0; u < Q; ++u) part[u] = part[u] == bound ? ninf() : part[u];
            }
        }
        if (!p.bias) bound = p.sigmoid ? sigmoid_floor(bound) : softmax_floor(bound, top);
        bound = fmaxf(bound, raw_keys ? kLeastOpen : -kF32Max);   // closed experts are no candidates
        // candidates of the lower lanes come first
        float in_run = 0.0f;                    // counted where the comparisons do not run
        each(look, [&](auto &k, int) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (k[j] >= bound) in_run += 1.0f;
        });
        const int own = (int)in_run;
        int upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += v;
        }
        const int count = __shfl_sync(kFull, upto, 31);
        const int n = min(count, p.K);          // experts that are chosen
        // the lane's choice, if it has one: expert, key, score (SOFTMAX: before the
        // division by the sum) and place in the order
        int id = 0, place = p.K;
        float mine = 0.0f, score = 0.0f;
        auto score_of = [&](float l) {
            return p.sigmoid ? __frcp_rn(1.0f + expf(-l)) : expf(fminf(l, kF32Max) - top);
        };
        if (count <= 32) {
            float2 *cand = s_cand[warp];
            if (lane < 3) cand[count + lane].x = ninf();
            float2 *to = cand + (upto - own);
            if (!MEM || own)
                each(look, [&](auto &k, int j0) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (k[j] >= bound) *to++ = make_float2(k[j], __int_as_float(e0 + j0 + j));
                });
            __syncwarp();
            if (lane < count) {
                const float2 own_cand = cand[lane];
                mine = own_cand.x;
                id = __float_as_int(own_cand.y);
                score = score_of(p.bias ? load_logit<BF16>(p, row + id) : mine);
                if (!p.bias) cand[lane].x = mine = score;   // logits so far: the scores decide
            }
            __syncwarp();
            if (lane < count) {
                float before = 0.0f;            // counted where the comparisons do not run
                for (int i = 0; i < count; i += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(cand + i);
                    const float4 b = *reinterpret_cast<const float4 *>(cand + i + 2);
                    if (a.x > mine) before += 1.0f;
                    if (a.z > mine) before += 1.0f;
                    if (b.x > mine) before += 1.0f;
                    if (b.z > mine) before += 1.0f;
                }
                place = (int)before;
                // equal keys (0 and -0 among them): those of lower lanes come before
                place += __popc(__match_any_sync(count < 32 ? (1u << count) - 1u : kFull, __float_as_uint(mine + 0.0f)) & lanemask_lt());
            }
        } else {
            if (!p.bias) {                      // scores in the logits' places, in shared memory: rare
                if constexpr (!MEM) write_run(key, sk + run0, p.padded, have);
                const int keys = p.padded ? VPL : have;
#pragma unroll 1
                for (int j = 0; j < keys; ++j) {
                    const float l = sk[run0 + j];
                    sk[run0 + j] = l >= bound ? score_of(l) : ninf();
                }
                if constexpr (!MEM) read_run(key, sk + run0, p.padded, have);
            }
            uint32_t used = 0;
            for (int k = 0; k < n; ++k) {
                float m = ninf();
                int j1 = 0;
                each(look, [&](auto &k, int j0) {
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        if (!((used >> (j0 + j)) & 1u) && k[j] > m) { m = k[j]; j1 = j0 + j; }
                });
                const float best = warp_max(m);
                const uint32_t first = __ballot_sync(kFull, m == best);
                const int expert = __shfl_sync(kFull, e0 + j1, __ffs(first) - 1);
                if (m == best && (first & lanemask_lt()) == 0) used |= 1u << j1;
                if (lane == k) { id = expert; place = k; mine = best; }
            }
            if (place < p.K) score = p.bias ? score_of(load_logit<BF16>(p, row + id)) : mine;
        }
        // ---- weights
        const bool chosen = place < p.K;
        float w = 0.0f;
        if (chosen) w = p.sigmoid ? score : __fdividef(score, sum);
        if (p.renorm) {
            float s = w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            w = __fdividef(w, s + 1e-20f);
        }
        const int64_t at = t * p.K;
        if (chosen) {
            p.ids[at + place] = id;
            p.scales[at + place] = w * p.scale;
            if (p.route_mask) p.route_mask[at + place] = 1;
        }
        if (n < p.K && lane >= n && lane < p.K) {
            p.ids[at + lane] = -1;
            p.scales[at + lane] = 0.0f;
            if (p.route_mask) p.route_mask[at + lane] = 0;
        }
        __syncwarp();                           // the candidates' places are free again
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
    const int64_t cap = (int64_t)num_sms() * kGateBlocks;
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    const size_t smem = p.G > 1 && !p.group_lanes ? (size_t)kGateWarps * p.scratch * sizeof(float) : 0;
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
    p.scratch = (p.G + 3) / 4 * 4 + 128;
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
    p.padded = p.run == vpl && (!p.group_lanes || p.per == p.group_lanes * p.run);
    const size_t size = d.logits_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    p.wide = (uintptr_t)p.logits % 16 == 0 && p.stride * size % 16 == 0 && p.E * size % 16 == 0;
    return d.logits_dtype == MOE_DTYPE_BF16 ? launch_type<true>(p, vpl, stream)
                                            : launch_type<false>(p, vpl, stream);
}

}  // namespace moe
