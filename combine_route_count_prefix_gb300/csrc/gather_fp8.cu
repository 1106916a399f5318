// gather_fp8.cu -- expert-major copies of block-scaled e4m3 tokens.
#include "common.cuh"

namespace moe {
namespace {

// Row r of the gathered rows and their scales = token assist[r].
__global__ void __launch_bounds__(128)
k_gather_fp8(const uint4 *x, const float *xs, const int32_t *assist, const int32_t *offsets,
             int64_t E, int64_t T, int64_t M, uint4 *rows, float *rs, int64_t cap_rows, int64_t H16,
             int64_t nb, int32_t *status) {
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    const int64_t R = min((int64_t)offsets[E], cap_rows);
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const int64_t t = (int64_t)assist[3 * r] * M + assist[3 * r + 1];
        if (t < 0 || t >= T) continue;
        for (int64_t i = threadIdx.x; i < H16; i += blockDim.x) rows[r * H16 + i] = x[t * H16 + i];
        for (int64_t i = threadIdx.x; i < nb; i += blockDim.x) rs[r * nb + i] = xs[t * nb + i];
    }
}

}  // namespace

moe_status launch_gather_fp8(const void *x, const float *xs, const int32_t *assist,
                             const int32_t *offsets, int64_t E, int64_t T, int64_t M, void *rows,
                             float *rs, int64_t cap_rows, int64_t H, int32_t *status,
                             cudaStream_t stream) {
    const int64_t cap = (int64_t)num_sms() * 16;
    MOE_LAUNCH("gather_fp8", k_gather_fp8, (unsigned)(cap_rows < cap ? cap_rows : cap), 128, 0, stream,
               static_cast<const uint4 *>(x), xs, assist, offsets, E, T, M,
               static_cast<uint4 *>(rows), rs, cap_rows, H / 16, (H + 127) / 128, status);
    return MOE_OK;
}

}  // namespace moe
