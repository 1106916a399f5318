// gather_fp8.cu -- expert-major copies of block-scaled e4m3 tokens.
//
// Row r of the gathered rows and their scales = token assist[r].  A warp per
// row, eight 16-byte loads a lane in flight.  HBM bounds it: every copy is
// written once (evict-first: they are larger than L2 before the first of them
// is read), and a token should be read once for its K copies.  In the rows' own
// order it is not: the experts follow each other and each goes through all the
// tokens, which fit L2 only with nothing else there (16384 tokens of 7168
// bytes, 8 copies: 668 MB read, 257 us).  So where the tokens
// are many, every expert's rows are cut into as many segments, and all experts'
// first segments come first: an expert's rows are in token order, so those
// are about the same tokens (290 MB read, 214 us).
#include "common.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kWarps = 8;
// Tokens up to these bytes are copied in the rows' order, without the
// segments' set-up (the largest expert is looked for, divisions per segment).
// In order against segments, 8 copies of 7168 bytes (us): 1024 tokens 15.3 /
// 17.1, 2048 23.9 / 26.1, 4096 48.0 / 47.6, 8192 112 / 101, 16384 257 / 214.
constexpr int64_t kInOrderBytes = 32 << 20;

struct GatherDev {
    const uint4 *x;
    const float *xs;
    const int32_t *assist, *offsets;
    int64_t T, M;
    uint4 *rows;
    float *rs;
    int64_t cap_rows;
    int E, H16, nb;
    int32_t *status;
};

__device__ __forceinline__ void copy_row(const GatherDev &p, int64_t r, int lane) {
    const int64_t t = (int64_t)p.assist[3 * r] * p.M + p.assist[3 * r + 1];
    if (t < 0 || t >= p.T) return;
    const uint4 *src = p.x + t * p.H16;
    uint4 *dst = p.rows + r * p.H16;
    for (int i0 = lane; i0 < p.H16; i0 += 256) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i0 + 32 * u < p.H16) v[u] = __ldg(src + i0 + 32 * u);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i0 + 32 * u < p.H16) __stcs(dst + i0 + 32 * u, v[u]);
    }
    for (int i = lane; i < p.nb; i += 32) p.rs[r * p.nb + i] = __ldg(p.xs + t * p.nb + i);
}

template <bool SEGMENTS>
__global__ void __launch_bounds__(32 * kWarps)
k_gather_fp8(GatherDev p) {
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if constexpr (!SEGMENTS) {
        const int64_t R = min((int64_t)p.offsets[p.E], p.cap_rows);
        for (int64_t r = (int64_t)blockIdx.x * kWarps + warp; r < R; r += (int64_t)gridDim.x * kWarps)
            copy_row(p, r, lane);
    } else {
        __shared__ int64_t s_off[kMaxExperts + 1];
        __shared__ int s_most;
        if (threadIdx.x == 0) s_most = 1;
        for (int e = threadIdx.x; e <= p.E; e += 32 * kWarps)
            s_off[e] = min(max((int64_t)p.offsets[e], (int64_t)0), p.cap_rows);
        __syncthreads();
        int most = 1;
        for (int e = threadIdx.x; e < p.E; e += 32 * kWarps)
            most = max(most, (int)(s_off[e + 1] - s_off[e]));
        atomicMax(&s_most, most);
        __syncthreads();
        // a row a warp in the largest expert's segments, but not more segments
        // than rows
        const int64_t n = max((int64_t)1, min((int64_t)(s_most + kWarps - 1) / kWarps, p.cap_rows / p.E));
        for (int64_t s = blockIdx.x; s < n * p.E; s += gridDim.x) {
            const int64_t i = s / p.E, e = s - i * p.E;
            const int64_t first = s_off[e], len = s_off[e + 1] - first;
            const int64_t end = first + len * (i + 1) / n;
            for (int64_t r = first + len * i / n + warp; r < end; r += kWarps) copy_row(p, r, lane);
        }
    }
}

}  // namespace

moe_status launch_gather_fp8(const void *x, const float *xs, const int32_t *assist,
                             const int32_t *offsets, int64_t E, int64_t T, int64_t M, void *rows,
                             float *rs, int64_t cap_rows, int64_t H, int32_t *status,
                             cudaStream_t stream) {
    const GatherDev p = {static_cast<const uint4 *>(x), xs, assist, offsets, T, M,
                         static_cast<uint4 *>(rows), rs, cap_rows, (int)E, (int)(H / 16),
                         (int)((H + 127) / 128), status};
    const unsigned grid = (unsigned)std::min<int64_t>((int64_t)num_sms() * 8, (cap_rows + kWarps - 1) / kWarps);
    auto kernel = T * H > kInOrderBytes ? k_gather_fp8<true> : k_gather_fp8<false>;
    MOE_LAUNCH("gather_fp8", kernel, grid, 32 * kWarps, 0, stream, p);
    return MOE_OK;
}

}  // namespace moe
