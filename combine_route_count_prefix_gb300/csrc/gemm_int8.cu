// gemm_int8.cu -- int8 products with one scale per row and one per output
// channel: the kernel for few rows a group, and the rows' images for the tile
// kernels.
//
//   C[r, n] = (float(sum_k q[r, k] * W[e, n, k]) * w_scale[e, n]) * row_scale[r] + bias[e, n]
//
// k_int8_few streams the weights (stream_i8.cuh): its CTAs share out the (group,
// 8 NB rows, 16 channels) units evenly in the weights' order, its warps a batch of
// units.  Reading the weights bounds it up to about 8 rows a group, and beyond that the
// widening of the rows and the mma (products) and the rows' stores.
// Rows come with the weights through the rings, or, LOCAL, are quantised from
// bf16 by every CTA into its own memory: up to 8 rows of one group, each of which fits the
// registers of its share of the twelve warps (one row up to a depth of 15360, two to
// 7680, four to 3840, eight to 1280).  The others take a kernel before (4096 x 7168, 8 rows,
// 22 us in every CTA, 10.5 with it).
// One bf16 row (us, of which the weights at the HBM rate): 4096 x 7168 7.0 (4.3), 7168 x
// 2048 4.8 (2.2), 1536 x 2048 4.0 (0.5); one int8 row 6.8, 4.6, 3.0; 16 bf16 rows 12.0, 8.0, 5.9.
#include "common.cuh"
#include "groups.cuh"
#include "quant.cuh"
#include "stream_i8.cuh"

#include <algorithm>

namespace moe {
namespace {

using namespace si8;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kXVecs = 5;        // vectors of eight values of a row that a LOCAL thread holds

struct Int8FewDev {
    const uint4 *x;            // bf16 rows (LOCAL)
    const int8_t *q;           // codes
    const float *qs;
    const int32_t *offsets;
    const uint8_t *w;
    const float *w_scales, *bias;
    void *c;
    int32_t *status;
    int64_t cap_rows;
    int E, N, Kd, out_bf16, early;
    Divisor by_units, by_stages;
};

template <bool LOCAL, int NB>
struct Cfg {
    static constexpr int kWarps = NB == 1 ? 12 : NB == 2 ? 12 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kD = NB == 1 ? 5 : 4;
    static constexpr int kBytes = kWeightBytes + (LOCAL ? 0 : NB * kRowBytes);
    static constexpr int kRing = kWarps * kD * kBytes;
    static constexpr int kUnits = NB == 1 ? 16 : NB == 2 ? 8 : 4;      // between two block barriers
    static constexpr int kMaxRows = NB * kRows;
};

// The largest magnitude as bits; a NaN counts above all (strict_scale).
__device__ __forceinline__ uint32_t max8(const float (&f)[8], uint32_t m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    return m;
}

template <bool LOCAL, int NB>
__global__ void __launch_bounds__(Cfg<LOCAL, NB>::kThreads, 1)
k_int8_few(Int8FewDev p) {
    using C = Cfg<LOCAL, NB>;
    constexpr int kThreads = C::kThreads, kWarps = C::kWarps, kUnits = C::kUnits, kMaxRows = C::kMaxRows;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int32_t acc[2][kUnits][kMaxRows][kChannels];
    __shared__ int32_t s_off[kMaxExperts + 1], s_blk[kMaxExperts + 1];
    __shared__ uint32_t amax[kRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t *codes = smem + C::kRing;
    const int Kd = p.Kd, KS = (Kd + kDepth - 1) / kDepth, pitch = KS * kDepth, NU = (p.N + kChannels - 1) / kChannels;
    const Lane l;

    for (int i = tid; i < 2 * kUnits * kMaxRows * kChannels; i += kThreads) (&acc[0][0][0][0])[i] = 0;
    if (LOCAL && tid < kRows) amax[tid] = 0;
    // early: the kernel before this one (the rows' codes) has waited for everything else
    if (!p.early) pdl_wait();
    // LOCAL: one group of a few rows, each shared by `group` warps; this one's part of
    // row xt starts at vector x0
    const int k8 = Kd / 8, group = kWarps / (int)min(p.cap_rows, (int64_t)kWarps), xt = warp / group;
    const int x0 = (warp - xt * group) * 32 + lane;
    uint4 xv[LOCAL ? kXVecs : 1];
    if (LOCAL && xt < p.cap_rows) {
#pragma unroll
        for (int u = 0; u < kXVecs; ++u)
            if (x0 + 32 * group * u < k8) xv[u] = p.x[(int64_t)xt * k8 + x0 + 32 * group * u];
    }
    // One group of at most one block of rows: no search, and LOCAL fetches weights before the offsets are
    // here (one row of 4096 x 7168 8.1 -> 7.0 us, of 1536 x 2048 4.9 -> 4.0).  They are asked for first:
    // behind the weights they take a microsecond more.
    const bool one = LOCAL || (p.E == 1 && p.cap_rows <= kMaxRows);
    const int one_first = one ? p.offsets[0] : 0, one_last = one ? p.offsets[1] : 0;
    int one_row0 = 0, one_rows = 0;
    auto see_offsets = [&]() {
        const int last = (int)max((int64_t)0, min((int64_t)one_last, p.cap_rows));
        one_row0 = min(max(one_first, 0), last);
        one_rows = last - one_row0;
    };
    if (one && !LOCAL) see_offsets();
    if (!one) {
        for (int i = tid; i <= p.E; i += kThreads) s_off[i] = p.offsets[i];
        __syncthreads();
        if (warp == 0) {
            bound_offsets(s_off, p.E, p.cap_rows);
            count_blocks(s_off, s_blk, p.E, kMaxRows);
        }
        __syncthreads();
    }
    const int64_t units = one ? NU : (int64_t)s_blk[p.E] * NU;
    const int64_t u_begin = units * blockIdx.x / gridDim.x, u_end = units * (blockIdx.x + 1) / gridDim.x;

    // unit -> group, first row, rows, first channel
    struct At {
        int e, row0, rows, ch;
    };
    auto find = [&](int64_t unit) {
        At a;
        if (one) {
            a.e = 0;
            a.row0 = one_row0;
            a.rows = one_rows;
            a.ch = (int)unit * kChannels;
            return a;
        }
        const int blk = units * NU <= UINT32_MAX ? p.by_units((int)unit) : (int)(unit / NU);
        int lo = 0, hi = p.E - 1;
        while (lo < hi) {   // last group whose first block is <= blk
            const int mid = (lo + hi + 1) >> 1;
            if (s_blk[mid] <= blk) lo = mid; else hi = mid - 1;
        }
        a.e = lo;
        a.row0 = s_off[lo] + (blk - s_blk[lo]) * kMaxRows;
        a.rows = min(kMaxRows, s_off[lo + 1] - a.row0);
        a.ch = (int)(unit - (int64_t)blk * NU) * kChannels;
        return a;
    };
    auto share = [&](int64_t first, int64_t &unit, int &ks, int &n) {
        const int total = (int)min((int64_t)kUnits, u_end - first) * KS;
        const int a = total * warp / kWarps, b = total * (warp + 1) / kWarps, q = p.by_stages(a);
        unit = first + q;
        ks = a - q * KS;
        n = b - a;
    };
    const uint64_t once = l2_policy_evict_first();
    struct Next {
        int64_t batch, unit;
        int ks, left, rows, ch;
        const uint8_t *src;          // the lane's bytes of the next stage
        const int8_t *row;           // and of the rows
    } f = {u_begin, 0, 0, 0, 0, 0, nullptr, nullptr};
    auto enter = [&]() {
        const At a = find(f.unit);
        f.ch = a.ch;
        f.src = p.w + ((int64_t)a.e * p.N + a.ch + l.cr) * Kd + f.ks * kDepth + l.cu * 16;
        if (!LOCAL) {
            f.rows = a.rows;
            f.row = p.q + (int64_t)(a.row0 + l.cr) * Kd + f.ks * kDepth + l.cu * 16;
        }
    };
    if (u_begin < u_end) share(u_begin, f.unit, f.ks, f.left);
    if (f.left > 0) enter();
    auto fetch = [&](uint32_t slot, bool weights, bool rows) {
        if (f.left == 0) {
            while (f.left == 0 && f.batch + kUnits < u_end) {
                f.batch += kUnits;
                share(f.batch, f.unit, f.ks, f.left);
            }
            if (f.left == 0) return;
            enter();
        }
        const bool in = f.ks * kDepth + l.cu * 16 < Kd;
        const bool in8 = in && f.ch + 8 < p.N;    // N is a multiple of 8
        if (weights) {
            copy16_once(slot + l.to0, f.src, in, once);
            copy16_once(slot + l.to1, f.src + (int64_t)4 * Kd, in, once);
            copy16_once(slot + l.to0 + 8 * kDepth, f.src + (int64_t)8 * Kd, in8, once);
            copy16_once(slot + l.to1 + 8 * kDepth, f.src + (int64_t)12 * Kd, in8, once);
        }
        f.src += kDepth;
        if (!LOCAL && rows) {
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                if (n * kRows + l.cr < f.rows)
                    copy16(slot + l.to0 + kWeightBytes + n * kRowBytes, f.row + (int64_t)(n * kRows) * Kd, in);
                if (n * kRows + 4 + l.cr < f.rows)
                    copy16(slot + l.to1 + kWeightBytes + n * kRowBytes, f.row + (int64_t)(n * kRows + 4) * Kd, in);
            }
        }
        if (!LOCAL) f.row += kDepth;
        --f.left;
        if (++f.ks == KS) {
            f.ks = 0;
            ++f.unit;
            if (f.left > 0) enter();
        }
    };
    Walk<C::kD, C::kBytes, LOCAL> walk(smem_u32(smem) + (uint32_t)(warp * C::kD * C::kBytes));
    if (!p.early) {
        walk.first(fetch, true, true);
    } else {
        // the weights before the wait, the rows after it
        const Next start = f;
        walk.first(fetch, true, false);
        f = start;
        pdl_wait();
        walk.first(fetch, false, true);
    }
    if (blockIdx.x == 0 && tid == 0) *p.status = 0;
    if (LOCAL) see_offsets();
    if (one && one_rows == 0) {   // the same for all threads
        copy_commit();
        copy_wait<0>();
        return;
    }
    if (one) __syncthreads();   // acc and amax are cleared
    if (LOCAL) {
        // the rows' codes, in every CTA
        if (xt < p.cap_rows) {
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < kXVecs; ++u)
                if (x0 + 32 * group * u < k8) {
                    float v[8];
                    unpack8(xv[u], v);
                    m = max8(v, m);
                }
            const uint32_t w = __reduce_max_sync(kFull, m);
            if (lane == 0) atomicMax(&amax[xt], w);
        }
        __syncthreads();
        if (xt < p.cap_rows) {
            const float s = strict_scale(amax[xt]), rs = __frcp_rn(s);
            auto put = [&](int i, uint2 q) {
                *reinterpret_cast<uint2 *>(codes + (size_t)xt * pitch + (i >> 4) * kDepth +
                                           unit_at(xt, (i >> 1) & 7) + (i & 1) * 8) = q;
            };
#pragma unroll
            for (int u = 0; u < kXVecs; ++u) {
                const int i = x0 + 32 * group * u;
                if (i < k8) {
                    float v[8];
                    unpack8(xv[u], v);
                    put(i, quant8(v, s, rs));
                }
            }
            for (int i = k8 + x0; i < pitch / 8; i += 32 * group) put(i, make_uint2(0, 0));
        }
        __syncthreads();
    }

    int buf = 0;
    for (int64_t first = u_begin; first < u_end; first += kUnits, buf ^= 1) {
        const int nu = (int)min((int64_t)kUnits, u_end - first);
        int64_t unit;
        int ks, n;
        share(first, unit, ks, n);
        while (n > 0) {
            const At at = find(unit);
            const int m = min(n, KS - ks);
            int32_t (*a)[kChannels] = acc[buf][unit - first];
            auto row = [&](int i) -> uint32_t {
                if (!LOCAL) return kWeightBytes + i * kDepth + l.of_row(i);
                const int r = at.row0 + i;      // LOCAL rows are those of the whole call
                return smem_u32(codes) + (uint32_t)(r * pitch + ks * kDepth) + l.of_row(r);
            };
            auto add = [&](int i, int c, int32_t v) { atomicAdd(&a[i][c], v); };
            walk.template run<NB>(l, m, at.rows, fetch, row, add);
            n -= m;
            ks = 0;
            ++unit;
        }
        __syncthreads();
        constexpr int kEach = kThreads / kChannels;     // units x rows that are written at once
#pragma unroll 1
        for (int i = tid / kChannels; i < nu * kMaxRows; i += kEach) {
            const At at = find(first + i / kMaxRows);
            const int row = i % kMaxRows, ch = at.ch + tid % kChannels;
            if (row >= at.rows) continue;
            int32_t *a = &acc[buf][i / kMaxRows][row][tid % kChannels];
            const int32_t sum = *a;
            *a = 0;
            if (ch >= p.N) continue;
            const int64_t r = at.row0 + row, wn = (int64_t)at.e * p.N + ch;
            // (with early, written while this kernel was running already: not for the read-only path)
            const float s = LOCAL ? strict_scale(amax[r]) : __ldcg(p.qs + r);
            float v = __fmul_rn(__fmul_rn(__int2float_rn(sum), __ldg(p.w_scales + wn)), s);
            if (p.bias) v = __fadd_rn(v, __ldg(p.bias + wn));
            if (p.out_bf16) static_cast<__nv_bfloat16 *>(p.c)[r * p.N + ch] = __float2bfloat16_rn(v);
            else static_cast<float *>(p.c)[r * p.N + ch] = v;
        }
    }
}

// ---------------------------------------------------------------- rows for the tile kernels
// A CTA a row: fp16 images of int8 codes, and their scale.
constexpr int kImgThreads = 256;
template <bool BF16>
__global__ void __launch_bounds__(kImgThreads)
k_rows_to_f16(const void *__restrict__ rows, const float *__restrict__ scales,
              const int32_t *__restrict__ offsets, int64_t E, int64_t cap_rows, int64_t Kd,
              uint4 *__restrict__ img, float *__restrict__ img_scales, int32_t *__restrict__ status) {
    __shared__ uint32_t part[kImgThreads / 32];
    const int tid = threadIdx.x;
    pdl_wait();
    if (blockIdx.x == 0 && tid == 0) *status = 0;
    const int64_t R = min((int64_t)offsets[E], cap_rows);
    const int k8 = (int)(Kd / 8);
    constexpr int kOwn = 4;      // vectors that stay in registers: rows of up to 8192
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        uint4 *out = img + r * k8;
        if constexpr (BF16) {
            const uint4 *src = static_cast<const uint4 *>(rows) + r * k8;
            uint4 raw[kOwn];
            uint32_t m = 0;
#pragma unroll
            for (int u = 0; u < kOwn; ++u) {
                const int i = u * kImgThreads + tid;
                raw[u] = i < k8 ? __ldcs(src + i) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kOwn; ++u) {
                float v[8];
                unpack8(raw[u], v);
                m = max8(v, m);
            }
            for (int i = kOwn * kImgThreads + tid; i < k8; i += kImgThreads) {
                float v[8];
                unpack8(src[i], v);
                m = max8(v, m);
            }
            m = __reduce_max_sync(kFull, m);
            __syncthreads();      // the row before has read part
            if ((tid & 31) == 0) part[tid >> 5] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kImgThreads / 32; ++w) m = max(m, part[w]);
            const float s = strict_scale(m), rs = __frcp_rn(s);
            auto put = [&](int i, const uint4 &x) {
                float v[8], c[8];
                unpack8(x, v);
                quant_codes<8>(v, s, rs, c);
                out[i] = make_uint4(pack_half2(c[0], c[1]), pack_half2(c[2], c[3]), pack_half2(c[4], c[5]),
                                    pack_half2(c[6], c[7]));
            };
#pragma unroll
            for (int u = 0; u < kOwn; ++u)
                if (u * kImgThreads + tid < k8) put(u * kImgThreads + tid, raw[u]);
            for (int i = kOwn * kImgThreads + tid; i < k8; i += kImgThreads) put(i, src[i]);
            if (tid == 0) img_scales[r] = s;
        } else {
            const uint2 *src = static_cast<const uint2 *>(rows) + r * k8;
            for (int i = tid; i < k8; i += kImgThreads) {
                const uint2 b = __ldcs(src + i);
                const uint32_t lo = b.x ^ 0x80808080u, hi = b.y ^ 0x80808080u;
                out[i] = make_uint4(widen_lo(lo), widen_hi(lo), widen_lo(hi), widen_hi(hi));
            }
            if (tid == 0) img_scales[r] = scales[r];
        }
    }
}

template <bool LOCAL, int NB>
moe_status launch(const Int8FewDev &p, size_t extra, cudaStream_t stream) {
    using C = Cfg<LOCAL, NB>;
    auto kernel = k_int8_few<LOCAL, NB>;
    if (!set_smem_limit((const void *)kernel, C::kRing + extra)) return MOE_ERR_CUDA;
    const int64_t units = p.cap_rows * ((p.N + kChannels - 1) / kChannels);
    const unsigned grid = (unsigned)std::min<int64_t>(num_sms(), units);
    MOE_LAUNCH("int8_few", kernel, grid, C::kThreads, C::kRing + extra, stream, p);
    return MOE_OK;
}

int64_t padded(int64_t k) { return (k + kDepth - 1) / kDepth * kDepth; }

}  // namespace

bool int8_few_local(int64_t rows, int64_t E, int64_t Kd) {
    constexpr int kWarps = Cfg<true, 1>::kWarps;
    return E == 1 && rows <= kRows && Kd / 8 <= kXVecs * 32 * (kWarps / rows);
}

moe_status launch_int8_few(const Int8FewArgs &a, cudaStream_t stream) {
    Int8FewDev p;
    p.x = static_cast<const uint4 *>(a.rows);
    p.q = static_cast<const int8_t *>(a.rows);
    p.qs = a.row_scales;
    p.offsets = a.offsets;
    p.w = static_cast<const uint8_t *>(a.w);
    p.w_scales = a.w_scales;
    p.bias = a.bias;
    p.c = a.c;
    p.status = a.status;
    p.cap_rows = a.cap_rows;
    p.E = (int)a.E;
    p.N = (int)a.N;
    p.Kd = (int)a.Kd;
    p.out_bf16 = a.out_bf16;
    p.early = a.early;
    p.by_units = Divisor((uint32_t)((a.N + kChannels - 1) / kChannels));
    p.by_stages = Divisor((uint32_t)(padded(a.Kd) / kDepth));
    if (a.rows_bf16) return launch<true, 1>(p, (size_t)(a.cap_rows * padded(a.Kd)), stream);
    if (a.cap_rows <= kRows * a.E) return launch<false, 1>(p, 0, stream);
    return a.cap_rows <= 2 * kRows * a.E ? launch<false, 2>(p, 0, stream) : launch<false, 4>(p, 0, stream);
}

moe_status launch_rows_to_f16(const void *rows, bool bf16, const float *scales, const int32_t *offsets,
                              int64_t E, int64_t cap_rows, int64_t Kd, void *img, float *img_scales,
                              int32_t *status, cudaStream_t stream) {
    const unsigned grid = (unsigned)std::min<int64_t>(cap_rows, (int64_t)num_sms() * 8);
    if (bf16) {
        MOE_LAUNCH("rows_to_f16", k_rows_to_f16<true>, grid, kImgThreads, 0, stream, rows, scales, offsets, E,
                   cap_rows, Kd, static_cast<uint4 *>(img), img_scales, status);
    } else {
        MOE_LAUNCH("rows_to_f16", k_rows_to_f16<false>, grid, kImgThreads, 0, stream, rows, scales, offsets, E,
                   cap_rows, Kd, static_cast<uint4 *>(img), img_scales, status);
    }
    return MOE_OK;
}

}  // namespace moe
