// gather_fp8.cu -- expert-major copies of block-scaled e4m3 tokens.
#include "common.cuh"

namespace moe {
namespace {

// Row r of the gathered rows and their scales = token assist[r].  A warp per
// row, eight 16-byte loads a lane in flight.
__global__ void __launch_bounds__(256)
k_gather_fp8(const uint4 *x, const float *xs, const int32_t *assist, const int32_t *offsets,
             int64_t E, int64_t T, int64_t M, uint4 *rows, float *rs, int64_t cap_rows, int H16,
             int nb, int32_t *status) {
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    const int lane = threadIdx.x & 31;
    const int64_t R = min((int64_t)offsets[E], cap_rows);
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < R; r += (int64_t)gridDim.x * 8) {
        const int64_t t = (int64_t)assist[3 * r] * M + assist[3 * r + 1];
        if (t < 0 || t >= T) continue;
        const uint4 *src = x + t * H16;
        uint4 *dst = rows + r * H16;
        for (int i0 = lane; i0 < H16; i0 += 256) {
            uint4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i0 + 32 * u < H16) v[u] = __ldg(src + i0 + 32 * u);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i0 + 32 * u < H16) __stcs(dst + i0 + 32 * u, v[u]);
        }
        for (int i = lane; i < nb; i += 32) rs[r * nb + i] = __ldg(xs + t * nb + i);
    }
}

}  // namespace

moe_status launch_gather_fp8(const void *x, const float *xs, const int32_t *assist,
                             const int32_t *offsets, int64_t E, int64_t T, int64_t M, void *rows,
                             float *rs, int64_t cap_rows, int64_t H, int32_t *status,
                             cudaStream_t stream) {
    const int64_t cap = (int64_t)num_sms() * 8, want = (cap_rows + 7) / 8;
    MOE_LAUNCH("gather_fp8", k_gather_fp8, (unsigned)(want < cap ? want : cap), 256, 0, stream,
               static_cast<const uint4 *>(x), xs, assist, offsets, E, T, M,
               static_cast<uint4 *>(rows), rs, cap_rows, (int)(H / 16), (int)((H + 127) / 128), status);
    return MOE_OK;
}

}  // namespace moe
