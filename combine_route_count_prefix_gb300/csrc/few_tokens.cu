// few_tokens.cu -- the whole int8 MoE layer for a few tokens.
//
// out[t] = bf16(sum_k p[t,k] * y(t,k) + shared[t]) with the stages of the
// layer's other kernels, in the same arithmetic, so that the outputs are the
// same bit for bit (y's rounding to bf16 among them):
//   q1, s1 = quantised x[t];  h = (float(q1 . W1[e]) * scale1) * s1
//   g = silu(h_a) * h_b;      q2, s2 = quantised g
//   y = bf16((float(q2 . W2[e]) * scale2) * s2), or, where the caller chose it, the
//   fp32 value itself, so that the output is rounded once
// ("PTO MegaMoE Dispatch + Combine Fusion Example": GMM1, SwiGLU, GMM2, Unpermute;
// "aclnnMoeDistributeCombineV4": masks, shared, zero and copy experts.)
//
// Reading the chosen experts' weights bounds it (stream_i8.cuh), and for one
// token of small experts the steps between the reads.  So there are two
// kernels, and neither an expert-major copy of the rows nor a routing kernel:
//   k_few_gate_up  deals the (expert, 8 rows, 8 + 8 channels) units to its CTAs in
//                  turn, so that every CTA meets the crowded experts too (dealt in
//                  runs, 32 tokens took 780 us, in turn 755); the warps share out the
//                  stages of a batch of units.  The integer sums are exact, so they may be
//                  added in any order.
//   k_few_down     is launched while the first runs and fetches its first
//                  weights meanwhile; a CTA owns 16 output channels for every
//                  expert and route, so the weighted sum needs no other CTA.
// Every CTA finds the experts' rows from expert_ids by itself: up to 32 routes by
// one warp's votes, up to 512 by counts and sums.
// With few and short rows the CTAs also quantise by themselves (LOCAL): the tokens, each
// in the registers of its share of the eight warps (one token of any width, two up to 7168,
// four to 3584, eight to 1792), loaded before the routes are known; g, of 16384 values at
// most, a row to a warp.  Otherwise a small kernel before each product quantises the rows
// once, and the codes travel through the rings with the weights.
//
// Measured, 128 experts, top-8, in a graph (us, moe_layer's small-batch path, the
// weights at the HBM rate), slower and faster boxes 5 % apart:
//   tokens            1    2    4    8   16   32   64
//   H 7168, N 4096   62  110  200  343  540  754  880
//     moe_layer     143  171  250  404  622  838  934
//     weights        52  101  189  335  535  725  817
//   H 2048, N 1536   13   20   31   47   71   96  116
//     moe_layer      37   46   56   75   97  123  136
//     weights         6   11   20   36   57   78   88
// Time goes by what a kernel executes once, too: its instructions come from L2 line by
// line, so the parts outside the loops are kept short (scales loaded for 16 slots in
// straight code cost 4 us a batch of the second kernel).
#include "common.cuh"
#include "quant.cuh"
#include "stream_i8.cuh"
#include "tcgen05.cuh"

#include <algorithm>

namespace moe {
namespace {

using namespace si8;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMaxRoutes = MOE_FEW_TOKENS_MAX_ROUTES;

// LOCAL: every CTA quantises what it multiplies.  Eight warps and rings of 80 KB, so
// that a CTA of either kernel fits an SM beside one of the other.  Else the codes
// come through the rings, of twelve warps: 8 tokens of 7168 x 4096 took 584 us with 8
// warps of four stages, 407 with 16 of three (each before other changes), 8, 12 and 16
// warps of equal bytes then 356, 347 and 356.
// Rows of an expert that share a reading of its weights: 8 NB.
template <bool LOCAL, int D = 5, int NB = 1>
struct Cfg {
    static constexpr int kWarps = LOCAL ? 8 : 12;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kD = D;                                 // stages of a warp's ring
    static constexpr int kBytes = kWeightBytes + (LOCAL ? 0 : NB * kRowBytes);
    static constexpr int kRing = kWarps * kD * kBytes;
    static constexpr int kBlock = NB * kRows;
    static constexpr int kUnits = LOCAL || NB > 1 ? 8 : 16;     // of the first kernel, between two block barriers
};
// Routes up to which the rings are five stages deep, else four (the sums of more
// routes also need the room).  7168 x 4096, top-8, 128 experts (us, five against four): 2
// tokens 112 / 115, 8 tokens 347 / 355, 16 tokens 566 / 568, 32 tokens 784 / 768, 64 tokens 917 / 901.
constexpr int kDeepRoutes = 128;
// Routes an expert, on average, above which 16 rows share a reading of its weights instead of
// 8 (H 2048, N 1536, us, 16 against 8: 8 an expert 29.6 / 30.7, 16 an expert 69.3 / 77.9, 4 an
// expert 23.8 either way; H 3280, N 1792, 14 an expert 38.9 / 46.3).
constexpr int kCrowded = 4;
constexpr int kXVecs = 7, kGVecs = 8;           // vectors of eight values that a LOCAL thread holds
constexpr int kQuantThreads = 256;

struct FewDev {
    const uint4 *x;            // bf16 [T, H]
    const int32_t *ids;
    const float *probs;
    const uint8_t *mask;
    const __nv_bfloat16 *shared;
    const uint8_t *w1, *w2;    // biased bytes
    const float *scale1, *scale2;
    __nv_bfloat16 *out;
    float *g;                  // [T*K, Nh]
    const int8_t *q;           // codes of the rows (not LOCAL): [T, H] or [T*K, Nh]
    const float *qs;           // and their scales
    int32_t *status;
    int T, K, R, E, Z, C, H, Nh, mask_kind, y_f32;
    Divisor by_k, by_units, by_stages1, by_stages2;   // K, Nh / 8, stages of H and of Nh
};

// What a CTA knows of the routes, in shared memory.
struct Routes {
    int32_t code[kMaxRoutes];      // expert, -1 none, -2 zero expert, -3 copy expert
    uint16_t list[kMaxRoutes];     // the routes of each expert, expert after expert
    uint16_t place[kMaxRoutes];    // a route's place in that list
    uint16_t blk_e[kMaxRoutes];    // blocks of up to kBlock routes of one expert
    uint16_t blk_first[kMaxRoutes];
    uint8_t blk_n[kMaxRoutes];
    uint32_t count[kMaxExperts];
    uint32_t part[32];
    int32_t blocks, rows, bad;
};

// Before the inputs may be read.
template <int kThreads>
__device__ __forceinline__ void clear_routes(const FewDev &p, Routes &r) {
    if (p.R > 32)
        for (int e = threadIdx.x; e < p.E; e += kThreads) r.count[e] = 0;
    if (threadIdx.x == 0) r.bad = 0;
    __syncthreads();
}

__device__ __forceinline__ int route_code(const FewDev &p, int i) {
    const int e = p.ids[i];
    bool on = true;
    if (p.mask_kind == 1) on = p.mask[p.by_k(i)] != 0;
    if (p.mask_kind == 2) on = p.mask[i] != 0;
    if (!on) return -1;
    if (e >= 0 && e < p.E) return e;
    if (e >= p.E && e < p.E + p.Z) return -2;
    if (e >= p.E + p.Z && e < p.E + p.Z + p.C) return -3;
    return -4;
}

// Up to 32 routes: one warp's votes, no counts per expert.
template <int kBlock>
__device__ __forceinline__ void find_routes_warp(const FewDev &p, Routes &r) {
    const int lane = threadIdx.x & 31;
    const int code = lane < p.R ? route_code(p, lane) : -1;
    if (lane < p.R) r.code[lane] = code == -4 ? -1 : code;
    if (code == -4) r.bad = 1;
    const uint32_t same = __match_any_sync(kFull, code);
    const int head = __ffs(same) - 1, n = __popc(same), nb = (n + kBlock - 1) / kBlock;
    const bool heads = code >= 0 && head == lane;
    const uint32_t own = heads ? (uint32_t)(n << 16 | nb) : 0u;
    uint32_t sum = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(kFull, sum, d);
        if (lane >= d) sum += v;
    }
    const int first = (int)((sum - own) >> 16), b0 = (int)((sum - own) & 0xffffu);
    if (heads)
        for (int b = 0; b < nb; ++b) {
            r.blk_e[b0 + b] = (uint16_t)code;
            r.blk_first[b0 + b] = (uint16_t)(first + b * kBlock);
            r.blk_n[b0 + b] = (uint8_t)min(kBlock, n - b * kBlock);
        }
    const int at = __shfl_sync(kFull, first, head) + __popc(same & lanemask_lt());
    if (code >= 0) {
        r.list[at] = (uint16_t)lane;
        r.place[lane] = (uint16_t)at;
    }
    if (lane == 31) {
        r.rows = (int)(sum >> 16);
        r.blocks = (int)(sum & 0xffffu);
    }
}

template <int kThreads, int kBlock>
__device__ __forceinline__ void find_routes(const FewDev &p, Routes &r) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.R <= 32) {
        if (warp == 0) find_routes_warp<kBlock>(p, r);
        __syncthreads();
        return;
    }
    constexpr int kOwn = (kMaxRoutes + kThreads - 1) / kThreads;
    uint32_t pos[kOwn];
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
        const int i = o * kThreads + tid;
        if (i >= p.R) break;
        const int code = route_code(p, i);
        if (code == -4) r.bad = 1;
        r.code[i] = code == -4 ? -1 : code;
        if (code >= 0) pos[o] = atomicAdd(&r.count[code], 1u);
    }
    __syncthreads();
    // exclusive sums over the experts of routes (upper half) and blocks (lower half)
    const int per = (p.E + kThreads - 1) / kThreads;
    const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
    uint32_t own = 0;
    for (int e = e0; e < e1; ++e) own += (r.count[e] << 16) | ((r.count[e] + kBlock - 1) / kBlock);
    uint32_t sum = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(kFull, sum, d);
        if (lane >= d) sum += v;
    }
    if (lane == 31) r.part[warp] = sum;
    __syncthreads();
    uint32_t at = sum - own;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
        if (w < warp) at += r.part[w];
    for (int e = e0; e < e1; ++e) {
        const int n = (int)r.count[e], first = (int)(at >> 16), b0 = (int)(at & 0xffffu);
        const int nb = (n + kBlock - 1) / kBlock;
        for (int b = 0; b < nb; ++b) {
            r.blk_e[b0 + b] = (uint16_t)e;
            r.blk_first[b0 + b] = (uint16_t)(first + b * kBlock);
            r.blk_n[b0 + b] = (uint8_t)min(kBlock, n - b * kBlock);
        }
        r.count[e] = (uint32_t)(first | n << 16);
        at += ((uint32_t)n << 16) | (uint32_t)nb;
    }
    if (tid == kThreads - 1) {
        r.rows = (int)(at >> 16);
        r.blocks = (int)(at & 0xffffu);
    }
    __syncthreads();
    int several = 0;
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
        const int i = o * kThreads + tid;
        if (i >= p.R) break;
        const int code = r.code[i];
        if (code >= 0) {
            pos[o] += r.count[code] & 0xffffu;
            several |= (r.count[code] >> 16) > kBlock;
            r.list[pos[o]] = (uint16_t)i;
            r.place[i] = (uint16_t)pos[o];
        }
    }
    // The order within an expert is that of the atomics, each CTA's own.  Where
    // an expert has several blocks the CTAs have to agree on who is in which:
    // ascending routes.
    if (__syncthreads_or(several)) {
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int i = o * kThreads + tid;
            if (i >= p.R) break;
            const int code = r.code[i];
            if (code < 0) continue;
            const int first = (int)(r.count[code] & 0xffffu), n = (int)(r.count[code] >> 16);
            pos[o] = first;
            for (int j = 0; j < n; ++j) pos[o] += r.list[first + j] < i;
        }
        __syncthreads();
#pragma unroll
        for (int o = 0; o < kOwn; ++o) {
            const int i = o * kThreads + tid;
            if (i >= p.R || r.code[i] < 0) continue;
            r.list[pos[o]] = (uint16_t)i;
            r.place[i] = (uint16_t)pos[o];
        }
        __syncthreads();
    }
}

__device__ __forceinline__ float max8(const float (&f)[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
    return m;
}
// Eight codes at column 8 i of row r of a CTA's own codes (rows of `pitch`
// bytes, in 128-byte pieces swizzled as a stage's rows are).
__device__ __forceinline__ void put_codes(uint8_t *codes, int r, int pitch, int i, uint2 v) {
    uint8_t *at = codes + (size_t)r * pitch + (i >> 4) * kDepth + unit_at(r, (i >> 1) & 7) + (i & 1) * 8;
    *reinterpret_cast<uint2 *>(at) = v;
}

__host__ __device__ inline int padded(int k) { return (k + kDepth - 1) / kDepth * kDepth; }

// ---------------------------------------------------------------- h = q1 . W1, g = silu(h_a) h_b
// Unit u of block u / (Nh / 8): SiLU channels 8 j .. 8 j + 7 and their
// multipliers (16 rows of the packed W1, two runs of eight).
template <bool LOCAL, int D, int NB>
__global__ void __launch_bounds__(Cfg<LOCAL>::kThreads, LOCAL ? 2 : 1)
k_few_gate_up(FewDev p) {
    using C = Cfg<LOCAL, D, NB>;
    constexpr int kThreads = C::kThreads, kWarps = C::kWarps, kBatchUnits = C::kUnits;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Routes r;
    __shared__ int32_t acc[2][kBatchUnits][C::kBlock][kChannels];
    __shared__ uint32_t amax[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5;
    uint8_t *codes = smem + C::kRing;
    const int H = p.H, KS = (H + kDepth - 1) / kDepth, pitch = KS * kDepth, NU = p.Nh / 8;
    const Lane l;

    for (int i = tid; i < 2 * kBatchUnits * C::kBlock * kChannels; i += kThreads) (&acc[0][0][0][0])[i] = 0;
    if (LOCAL)
        for (int i = tid; i < p.T; i += kThreads) amax[i] = 0;
    clear_routes<kThreads>(p, r);
    // with LOCAL unset, the kernel before this one has waited for the inputs
    // LOCAL: a token's row is shared by `group` warps, this one's part starts at vector x0
    const int H8 = H / 8, group = kWarps / min(p.T, kWarps), xt = warp / group;
    const int x0 = (warp - xt * group) * 32 + (tid & 31);
    uint4 xv[LOCAL ? kXVecs : 1];
    if (LOCAL) {
        pdl_wait();
        if (xt < p.T)
#pragma unroll
            for (int u = 0; u < kXVecs; ++u)
                if (x0 + 32 * group * u < H8) xv[u] = p.x[xt * H8 + x0 + 32 * group * u];
    }
    find_routes<kThreads, C::kBlock>(p, r);
    // this CTA's units are blockIdx.x, blockIdx.x + gridDim.x, ...: every CTA meets every expert, the
    // crowded ones, whose rows take more arithmetic, too
    const int units = r.blocks * NU, u_end = (units - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    const int u_begin = 0;
    auto unit_of = [&](int i) { return (int)blockIdx.x + i * (int)gridDim.x; };

    // this warp's share of a batch of units: first unit, its first stage, stages
    auto share = [&](int first, int &unit, int &ks, int &n) {
        const int total = min(kBatchUnits, u_end - first) * KS;
        const int a = total * warp / kWarps, b = total * (warp + 1) / kWarps, q = p.by_stages1(a);
        unit = first + q;
        ks = a - q * KS;
        n = b - a;
    };
    // the stages to fetch, batch by batch
    const uint64_t once = l2_policy_evict_first();
    auto copy_weights = [&](uint32_t dst, const void *src, bool in) { copy16_once(dst, src, in, once); };
    struct Next {
        int batch, unit, ks, left;
        const uint8_t *src;          // the lane's bytes of the next stage
        const int8_t *row[2 * NB];   // and of the rows, where they are
    } f = {u_begin, 0, 0, 0, nullptr, {}};
    auto enter = [&]() {
        const int unit = unit_of(f.unit), blk = p.by_units(unit), j = (unit - blk * NU) * 8;
        const int64_t prow = (int64_t)r.blk_e[blk] * (2 * p.Nh) + (j >> 6) * 128 + ((j >> 4) & 3) * 32 + (j & 15);
        f.src = p.w1 + (prow + l.cr) * H + f.ks * kDepth + l.cu * 16;
        if (!LOCAL) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                const int row = 4 * i + l.cr;
                f.row[i] = nullptr;
                if (row < r.blk_n[blk])
                    f.row[i] = p.q + (int64_t)p.by_k(r.list[r.blk_first[blk] + row]) * H + f.ks * kDepth + l.cu * 16;
            }
        }
    };
    if (u_begin < u_end) share(u_begin, f.unit, f.ks, f.left);
    if (f.left > 0) enter();
    auto fetch = [&](uint32_t slot, bool weights, bool rows) {
        if (f.left == 0) {
            while (f.left == 0 && f.batch + kBatchUnits < u_end) {
                f.batch += kBatchUnits;
                share(f.batch, f.unit, f.ks, f.left);
            }
            if (f.left == 0) return;
            enter();
        }
        const bool in = f.ks * kDepth + l.cu * 16 < H;
        if (weights) {
            copy_weights(slot + l.to0, f.src, in);
            copy_weights(slot + l.to1, f.src + (int64_t)4 * H, in);
            copy_weights(slot + l.to0 + 8 * kDepth, f.src + (int64_t)16 * H, in);
            copy_weights(slot + l.to1 + 8 * kDepth, f.src + (int64_t)20 * H, in);
        }
        f.src += kDepth;
        if (!LOCAL && rows) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
                if (f.row[i]) {
                    copy16(slot + (i & 1 ? l.to1 : l.to0) + kWeightBytes + (i >> 1) * kRowBytes, f.row[i], in);
                    f.row[i] += kDepth;
                }
        }
        --f.left;
        if (++f.ks == KS) {
            f.ks = 0;
            ++f.unit;
            if (f.left > 0) enter();
        }
    };
    Walk<C::kD, C::kBytes, LOCAL> walk(smem_u32(smem) + (uint32_t)(warp * C::kD * C::kBytes));
    if (LOCAL) {
        walk.first(fetch, true, true);
        // the tokens' codes, in every CTA
        if (xt < p.T) {
            float m = 0.0f;
#pragma unroll
            for (int u = 0; u < kXVecs; ++u)
                if (x0 + 32 * group * u < H8) {
                    float v[8];
                    unpack8(xv[u], v);
                    m = max8(v, m);
                }
            const uint32_t w = __reduce_max_sync(kFull, __float_as_uint(m));
            if ((tid & 31) == 0) atomicMax(&amax[xt], w);
        }
        __syncthreads();
        if (xt < p.T) {
            const float s = __fdiv_rn(__uint_as_float(amax[xt]), 127.0f), rs = __frcp_rn(s);
#pragma unroll
            for (int u = 0; u < kXVecs; ++u)
                if (x0 + 32 * group * u < H8) {
                    float v[8];
                    unpack8(xv[u], v);
                    put_codes(codes, xt, pitch, x0 + 32 * group * u, quant8(v, s, rs));
                }
        }
        if (H % kDepth) {   // zeros behind the rows' ends
            const int pad = pitch / 8 - H8;
            for (int i = tid; i < p.T * pad; i += kThreads)
                put_codes(codes, i / pad, pitch, H8 + i % pad, make_uint2(0, 0));
        }
        __syncthreads();
    } else {
        // the weights before the wait, the rows that the kernel before this one makes after it
        const Next start = f;
        walk.first(fetch, true, false);
        f = start;
        pdl_wait();
        walk.first(fetch, false, true);
    }

    int buf = 0;
    for (int first = u_begin; first < u_end; first += kBatchUnits, buf ^= 1) {
        const int nu = min(kBatchUnits, u_end - first);
        // this thread's unit of the batch, for the epilogue: its scales come meanwhile
        constexpr int kUnitThreads = kThreads / kBatchUnits;
        const int eu = tid / kUnitThreads, ej = tid & 7, er = (tid % kUnitThreads) >> 3;
        int eblk = 0, ech = 0;
        float sa = 0.0f, sb = 0.0f;
        if (eu < nu) {
            const int unit = unit_of(first + eu);
            eblk = p.by_units(unit);
            ech = (unit - eblk * NU) * 8 + ej;
            const float *sc = p.scale1 + (int64_t)r.blk_e[eblk] * (2 * p.Nh) + ech;
            sa = __ldg(sc);
            sb = __ldg(sc + p.Nh);
        }
        int unit, ks, n;
        share(first, unit, ks, n);
        while (n > 0) {
            const int blk = p.by_units(unit_of(unit)), m = min(n, KS - ks);
            int32_t (*a)[kChannels] = acc[buf][unit - first];
            auto row = [&](int i) -> uint32_t {
                if (!LOCAL) return kWeightBytes + i * kDepth + l.of_row(i);
                const int t = p.by_k(r.list[r.blk_first[blk] + i]);
                return smem_u32(codes) + (uint32_t)(t * pitch + ks * kDepth) + l.of_row(t);
            };
            auto add = [&](int i, int c, int32_t v) { atomicAdd(&a[i][c], v); };
            walk.template run<NB>(l, m, r.blk_n[blk], fetch, row, add);
            n -= m;
            ks = 0;
            ++unit;
        }
        __syncthreads();
        if (eu < nu) {
            const int nr = r.blk_n[eblk];
            for (int row = er; row < nr; row += kUnitThreads / 8) {
                const int route = r.list[r.blk_first[eblk] + row], t = p.by_k(route);
                int32_t *a = acc[buf][eu][row];
                const float s1 = LOCAL ? __fdiv_rn(__uint_as_float(amax[t]), 127.0f) : p.qs[t];
                const float ha = __fmul_rn(__fmul_rn(__int2float_rn(a[ej]), sa), s1);
                const float hb = __fmul_rn(__fmul_rn(__int2float_rn(a[ej + 8]), sb), s1);
                a[ej] = 0;
                a[ej + 8] = 0;
                p.g[(int64_t)route * p.Nh + ech] = __fmul_rn(tc::silu_f32(ha), hb);
            }
        }
    }
    if (blockIdx.x == 0 && tid == 0) *p.status = r.bad ? MOE_DEV_BAD_EXPERT_ID : 0;
}

// ---------------------------------------------------------------- y = q2 . W2, out
template <bool LOCAL, int D, int NB>
__global__ void __launch_bounds__(Cfg<LOCAL>::kThreads, LOCAL ? 2 : 1)
k_few_down(FewDev p) {
    using C = Cfg<LOCAL, D, NB>;
    constexpr int kThreads = C::kThreads, kWarps = C::kWarps;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Routes r;
    __shared__ float scale[kMaxRoutes];      // of g, by place in the list
    __shared__ float probs[kMaxRoutes];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int Nh = p.Nh, KS = (Nh + kDepth - 1) / kDepth, pitch = KS * kDepth;
    const Lane l;
    uint8_t *codes = smem + C::kRing;
    int32_t *acc = reinterpret_cast<int32_t *>(codes + (LOCAL ? (size_t)p.R * pitch : 0));   // [2][R][16]

    for (int i = tid; i < 2 * p.R * kChannels; i += kThreads) acc[i] = 0;
    clear_routes<kThreads>(p, r);
    // ids, mask, weights and probs were there before the kernel before this one began
    for (int i = tid; i < p.R; i += kThreads) probs[i] = p.probs[i];
    find_routes<kThreads, C::kBlock>(p, r);
    const int per_batch = r.blocks * KS;      // stages of 16 channels
    const int mine_a = per_batch * warp / kWarps, mine_n = per_batch * (warp + 1) / kWarps - mine_a;
    const int mine_blk = p.by_stages2(mine_a), mine_ks = mine_a - mine_blk * KS;
    const int batches = p.H / kChannels;

    const uint64_t once = l2_policy_evict_first();
    auto copy_weights = [&](uint32_t dst, const void *src, bool in) { copy16_once(dst, src, in, once); };
    struct Next {
        int batch, blk, ks, left;
        const uint8_t *src;
        const int8_t *row[2 * NB];
    } f = {(int)blockIdx.x, 0, 0, 0, nullptr, {}};
    auto enter = [&]() {
        f.src = p.w2 + ((int64_t)r.blk_e[f.blk] * p.H + f.batch * kChannels + l.cr) * Nh + f.ks * kDepth + l.cu * 16;
        if (!LOCAL) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                const int row = 4 * i + l.cr;
                f.row[i] = nullptr;
                if (row < r.blk_n[f.blk])
                    f.row[i] = p.q + (int64_t)r.list[r.blk_first[f.blk] + row] * Nh + f.ks * kDepth + l.cu * 16;
            }
        }
    };
    auto begin = [&]() {
        f.left = mine_n;
        f.blk = mine_blk;
        f.ks = mine_ks;
        if (f.left > 0) enter();
    };
    if (f.batch < batches) begin();
    auto fetch = [&](uint32_t slot, bool weights, bool rows) {
        if (f.left == 0) {
            if (mine_n == 0 || f.batch + (int)gridDim.x >= batches) return;
            f.batch += gridDim.x;
            begin();
        }
        const bool in = f.ks * kDepth + l.cu * 16 < Nh;
        if (weights) {
            copy_weights(slot + l.to0, f.src, in);
            copy_weights(slot + l.to1, f.src + (int64_t)4 * Nh, in);
            copy_weights(slot + l.to0 + 8 * kDepth, f.src + (int64_t)8 * Nh, in);
            copy_weights(slot + l.to1 + 8 * kDepth, f.src + (int64_t)12 * Nh, in);
        }
        f.src += kDepth;
        if (!LOCAL && rows) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i)
                if (f.row[i]) {
                    copy16(slot + (i & 1 ? l.to1 : l.to0) + kWeightBytes + (i >> 1) * kRowBytes, f.row[i], in);
                    f.row[i] += kDepth;
                }
        }
        --f.left;
        if (++f.ks == KS) {
            f.ks = 0;
            ++f.blk;
            if (f.left > 0) enter();
        }
    };
    Walk<C::kD, C::kBytes, LOCAL> walk(smem_u32(smem) + (uint32_t)(warp * C::kD * C::kBytes));
    if (LOCAL) {
        walk.first(fetch, true, true);
        pdl_wait();
        // the routes' codes, a row to a warp
        const int n8 = Nh / 8;
        for (int at = warp; at < r.rows; at += kWarps) {
            const float4 *src = reinterpret_cast<const float4 *>(p.g + (int64_t)r.list[at] * Nh);
            const int lane = tid & 31;
            float4 v[kGVecs][2];
            float m = 0.0f;
            for (int i0 = 0; i0 < n8; i0 += 32 * kGVecs) {
#pragma unroll
                for (int u = 0; u < kGVecs; ++u) {
                    const int i = i0 + 32 * u + lane;
                    v[u][0] = v[u][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i < n8) {
                        v[u][0] = src[2 * i];
                        v[u][1] = src[2 * i + 1];
                    }
                }
#pragma unroll
                for (int u = 0; u < kGVecs; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        m = fmaxf(fmaxf(m, fmaxf(fabsf(v[u][h].x), fabsf(v[u][h].y))),
                                  fmaxf(fabsf(v[u][h].z), fabsf(v[u][h].w)));
            }
            m = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(m)));
            const float s = __fdiv_rn(m, 127.0f), rs = __frcp_rn(s);
            if (lane == 0) scale[at] = s;
#pragma unroll 1
            for (int i = lane; i < n8; i += 64) {
                const int j = i + 32 < n8 ? i + 32 : i;
                const float4 a = src[2 * i], b = src[2 * i + 1], c = src[2 * j], d = src[2 * j + 1];
                const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                const float h[8] = {c.x, c.y, c.z, c.w, d.x, d.y, d.z, d.w};
                const uint2 q0 = quant8(f, s, rs), q1 = quant8(h, s, rs);
                put_codes(codes, at, pitch, i, q0);
                if (j != i) put_codes(codes, at, pitch, j, q1);
            }
        }
    } else {
        // the weights before the wait, the rows that the kernel before this one makes after it
        const Next start = f;
        walk.first(fetch, true, false);
        f = start;
        pdl_wait();
        walk.first(fetch, false, true);
        for (int i = tid; i < r.rows; i += kThreads) scale[i] = __ldcg(p.qs + r.list[i]);
    }
    __syncthreads();

    // what place `at` of the list multiplies its sums with
    auto scale2_of = [&](int i, int batch) {
        return __ldg(p.scale2 + (int64_t)r.code[r.list[i / kChannels]] * p.H + batch * kChannels + i % kChannels);
    };
    int buf = 0;
    const int outs = p.T * kChannels, sums = r.rows * kChannels;
    for (int batch = blockIdx.x; batch < batches; batch += gridDim.x, buf ^= 1) {
        int32_t *a = acc + (size_t)buf * p.R * kChannels;
        const float sc = tid < sums ? scale2_of(tid, batch) : 0.0f;   // on its way meanwhile
        const float shared = p.shared && tid < outs
                                 ? __bfloat162float(p.shared[(int64_t)(tid / kChannels) * p.H + batch * kChannels + tid % kChannels])
                                 : 0.0f;
        int blk = mine_blk, ks = mine_ks, n = mine_n;
        while (n > 0) {
            const int base = r.blk_first[blk], m = min(n, KS - ks);
            auto row = [&](int i) -> uint32_t {
                if (!LOCAL) return kWeightBytes + i * kDepth + l.of_row(i);
                return smem_u32(codes) + (uint32_t)((base + i) * pitch + ks * kDepth) + l.of_row(base + i);
            };
            auto add = [&](int i, int c, int32_t v) { atomicAdd(&a[(base + i) * kChannels + c], v); };
            walk.template run<NB>(l, m, r.blk_n[blk], fetch, row, add);
            n -= m;
            ks = 0;
            ++blk;
        }
        __syncthreads();
        // p * y of every route in the place of its sum, then the sum over a token's
        // routes in slot order from +0, as the combine kernel forms it
#pragma unroll 1
        for (int i = tid; i < sums; i += kThreads) {
            const int at = i / kChannels;
            const float w2s = i == tid ? sc : scale2_of(i, batch);
            float y = __fmul_rn(__fmul_rn(__int2float_rn(a[i]), w2s), scale[at]);
            // the layer's other kernels hand y over in memory, as bf16: rounded here too unless told
            // otherwise, so that prefill and decoding agree (against 64 bits 2.4e-3 off, without 1.65e-3)
            if (!p.y_f32) y = __bfloat162float(__float2bfloat16_rn(y));
            a[i] = __float_as_int(__fmul_rn(probs[r.list[at]], y));
        }
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < outs; i += kThreads) {
            const int t = i / kChannels, c = i % kChannels;
            const int64_t o = (int64_t)t * p.H + batch * kChannels + c;
            float v = 0.0f;
            for (int route = t * p.K; route < (t + 1) * p.K; ++route) {
                const int code = r.code[route];
                if (code >= 0) {
                    int32_t *s = a + r.place[route] * kChannels + c;
                    v = __fadd_rn(v, __int_as_float(*s));
                    *s = 0;
                } else if (code != -1) {
                    const float x = code == -3 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.x)[o]) : 0.0f;
                    v = __fadd_rn(v, __fmul_rn(probs[route], x));
                }
            }
            if (p.shared) v = __fadd_rn(v, i == tid ? shared : __bfloat162float(p.shared[o]));
            p.out[o] = __float2bfloat16_rn(v);
        }
    }
}

// ---------------------------------------------------------------- codes of rows, once for all CTAs
// bf16 or fp32 rows -> int8 codes and scales, a CTA a row.  A NaN stays out of its
// row's maximum, as in the layer's other kernels, or (NAN_SCALE) it and an infinity make
// the scale NaN.
template <typename T, bool NAN_SCALE>
__global__ void __launch_bounds__(kQuantThreads)
k_quant_rows_i8(const T *__restrict__ src, int64_t n, int8_t *__restrict__ q, float *__restrict__ s_out) {
    __shared__ float part[kQuantThreads / 32];
    pdl_wait();
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const int n8 = (int)(n / 8);
    auto load = [&](int i, float (&v)[8]) {
        if constexpr (sizeof(T) == 2) {
            unpack8(__ldcg(reinterpret_cast<const uint4 *>(src + row * n) + i), v);
        } else {
            const float4 *p = reinterpret_cast<const float4 *>(src + row * n);
            const float4 a = __ldcg(p + 2 * i), b = __ldcg(p + 2 * i + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    };
    auto add = [&](const float (&v)[8], float m) {
        if constexpr (NAN_SCALE) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                m = __uint_as_float(max(__float_as_uint(m), __float_as_uint(v[c]) & 0x7fffffffu));
            return m;
        } else {
            return max8(v, m);
        }
    };
    // the row's first kOwn * kQuantThreads vectors (up to 8192 values) stay in registers
    constexpr int kOwn = 4;
    float own[kOwn][8], m = 0.0f;
#pragma unroll
    for (int u = 0; u < kOwn; ++u) {
        const int i = u * kQuantThreads + tid;
        if (i < n8) {
            load(i, own[u]);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) own[u][c] = 0.0f;
        }
    }
#pragma unroll
    for (int u = 0; u < kOwn; ++u) m = add(own[u], m);
    for (int i = kOwn * kQuantThreads + tid; i < n8; i += kQuantThreads) {
        float v[8];
        load(i, v);
        m = add(v, m);
    }
    m = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(m)));
    if ((tid & 31) == 0) part[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w)
        m = __uint_as_float(max(__float_as_uint(m), __float_as_uint(part[w])));
    const float s = NAN_SCALE ? strict_scale(__float_as_uint(m)) : __fdiv_rn(m, 127.0f), rs = __frcp_rn(s);
    uint2 *out = reinterpret_cast<uint2 *>(q + row * n);
#pragma unroll
    for (int u = 0; u < kOwn; ++u) {
        const int i = u * kQuantThreads + tid;
        if (i < n8) out[i] = quant8(own[u], s, rs);
    }
    for (int i = kOwn * kQuantThreads + tid; i < n8; i += kQuantThreads) {
        float v[8];
        load(i, v);
        out[i] = quant8(v, s, rs);
    }
    if (tid == 0) s_out[row] = s;
}

}  // namespace

moe_status launch_quant_rows_i8(const void *src, bool bf16, bool nan_scale, int64_t rows, int64_t n,
                                int8_t *q, float *scales, cudaStream_t stream) {
    const auto *b = static_cast<const __nv_bfloat16 *>(src);
    if (bf16 && nan_scale) {
        MOE_LAUNCH("quant_rows_i8", (k_quant_rows_i8<__nv_bfloat16, true>), (unsigned)rows, kQuantThreads, 0,
                   stream, b, n, q, scales);
    } else if (bf16) {
        MOE_LAUNCH("quant_rows_i8", (k_quant_rows_i8<__nv_bfloat16, false>), (unsigned)rows, kQuantThreads, 0,
                   stream, b, n, q, scales);
    } else {
        MOE_LAUNCH("quant_rows_i8", (k_quant_rows_i8<float, false>), (unsigned)rows, kQuantThreads, 0, stream,
                   static_cast<const float *>(src), n, q, scales);
    }
    return MOE_OK;
}

// Whether each kernel's CTAs quantise for themselves: a row's part fits a warp's
// registers, and g is at most 16384 values.  Measured (us, so against with the two kernels
// before the products): 1 token, H 2048, N 1536 13.1 / 15.3; H 7168, N 4096 62.3 / 62.0; 2
// tokens, H 2048, N 1536 20.4 / 20.7.
static bool few_tokens_local(int64_t T, int64_t K, int64_t H, int64_t Nh) {
    constexpr int kWarps = Cfg<true>::kWarps;
    return T <= kWarps && (H / 8 + 31) / 32 <= kXVecs * (kWarps / T) && T * K * Nh <= 16384;
}

// extra1, extra2: shared memory of the two kernels beside their rings.
template <bool LOCAL, int D, int NB>
static moe_status launch_both(FewDev p, unsigned grid1, unsigned grid2, size_t extra1, size_t extra2,
                              const FewTokensArgs &a, cudaStream_t stream) {
    using C = Cfg<LOCAL, D, NB>;
    auto up = k_few_gate_up<LOCAL, D, NB>;
    auto down = k_few_down<LOCAL, D, NB>;
    if (!set_smem_limit((const void *)up, C::kRing + extra1) ||
        !set_smem_limit((const void *)down, C::kRing + extra2))
        return MOE_ERR_CUDA;
    if (!LOCAL) {
        MOE_TRY(launch_quant_rows_i8(a.x, true, false, p.T, p.H, a.q, a.qs, stream));
        p.q = a.q;
        p.qs = a.qs;
    }
    MOE_LAUNCH("few_gate_up", up, grid1, C::kThreads, C::kRing + extra1, stream, p);
    if (!LOCAL) {
        int8_t *q2 = a.q + align_up((size_t)p.T * p.H, kAlign);
        MOE_TRY(launch_quant_rows_i8(a.g, false, false, p.R, p.Nh, q2, a.qs + p.T, stream));
        p.q = q2;
        p.qs = a.qs + p.T;
    }
    MOE_LAUNCH("few_down", down, grid2, C::kThreads, C::kRing + extra2, stream, p);
    return MOE_OK;
}

moe_status launch_layer_few_tokens(const moe_shape &s, const FewTokensArgs &a, cudaStream_t stream) {
    const int64_t T = s.num_tokens, K = s.topk, H = s.hidden, Nh = s.ffn / 2, R = T * K;
    FewDev p;
    p.x = static_cast<const uint4 *>(a.x);
    p.ids = a.ids;
    p.probs = a.probs;
    p.mask = a.mask;
    p.shared = static_cast<const __nv_bfloat16 *>(a.shared);
    p.w1 = static_cast<const uint8_t *>(a.w1);
    p.w2 = static_cast<const uint8_t *>(a.w2);
    p.scale1 = a.scale1;
    p.scale2 = a.scale2;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.g = a.g;
    p.q = nullptr;
    p.qs = nullptr;
    p.status = a.status;
    p.T = (int)T;
    p.K = (int)K;
    p.R = (int)R;
    p.E = (int)s.num_experts;
    p.Z = (int)s.zero_experts;
    p.C = (int)s.copy_experts;
    p.H = (int)H;
    p.Nh = (int)Nh;
    p.mask_kind = s.mask_kind;
    p.y_f32 = a.y_f32;
    p.by_k = Divisor((uint32_t)K);
    p.by_units = Divisor((uint32_t)(Nh / 8));
    p.by_stages1 = Divisor((uint32_t)(padded((int)H) / kDepth));
    p.by_stages2 = Divisor((uint32_t)(padded((int)Nh) / kDepth));
    const unsigned sms = (unsigned)num_sms();
    const unsigned grid1 = (unsigned)std::min<int64_t>(sms, R * (Nh / 8));
    const unsigned grid2 = (unsigned)std::min<int64_t>(sms, H / kChannels);
    const size_t acc2 = (size_t)2 * R * kChannels * sizeof(int32_t);
    if (few_tokens_local(T, K, H, Nh))
        return launch_both<true, 5, 1>(p, grid1, grid2, (size_t)T * padded((int)H),
                                       (size_t)R * padded((int)Nh) + acc2, a, stream);
    if (R > kCrowded * s.num_experts) return launch_both<false, 3, 2>(p, grid1, grid2, 0, acc2, a, stream);
    return R <= kDeepRoutes ? launch_both<false, 5, 1>(p, grid1, grid2, 0, acc2, a, stream)
                            : launch_both<false, 4, 1>(p, grid1, grid2, 0, acc2, a, stream);
}

}  // namespace moe
