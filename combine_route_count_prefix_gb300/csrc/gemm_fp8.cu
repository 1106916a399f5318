// gemm_fp8.cu -- grouped products of block-scaled e4m3 operands and the fp8
// expert FFN's row kernels.
//
// Simple form: 64 x 64 tiles of the output, 16 x 16 threads with 4 x 4 fp32
// sums each, codes widened to fp32 in shared memory; the block's two scales
// are applied to the sum of its 128 products.
#include "common.cuh"
#include "fp8.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int TM = 64, TN = 64, TK = 32;

__device__ __forceinline__ float e4m3_to_float(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3);
    return __half2float(__half(h));
}

__global__ void __launch_bounds__(256)
k_gemm_fp8_simple(Fp8GemmArgs p, int kb_count) {
    __shared__ float sa[TK][TM + 4], sw[TK][TN + 4];
    pdl_wait();
    const int e = blockIdx.z;
    const int n0 = blockIdx.x * TN;
    const int64_t row_end = min((int64_t)p.offsets[e + 1], p.cap_rows);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const uint8_t *w = static_cast<const uint8_t *>(p.w) + (int64_t)e * p.N * p.Kd;
    const float *wsc = p.w_scales + (int64_t)e * ((p.N + 127) / 128) * kb_count;
    for (int64_t m0 = p.offsets[e] + (int64_t)blockIdx.y * TM; m0 < row_end;
         m0 += (int64_t)gridDim.y * TM) {
        float acc[4][4] = {};
        for (int kb = 0; kb < kb_count; ++kb) {
            float part[4][4] = {};
            for (int k0 = kb * 128; k0 < min((int64_t)kb * 128 + 128, p.Kd); k0 += TK) {
                __syncthreads();
                for (int i = threadIdx.x; i < TM * TK; i += 256) {
                    const int r = i / TK, k = i % TK;
                    const int64_t m = m0 + r, n = n0 + r;
                    sa[k][r] = (m < row_end && k0 + k < p.Kd)
                                   ? e4m3_to_float(static_cast<const uint8_t *>(p.a)[m * p.Kd + k0 + k])
                                   : 0.0f;
                    sw[k][r] = (n < p.N && k0 + k < p.Kd) ? e4m3_to_float(w[n * p.Kd + k0 + k]) : 0.0f;
                }
                __syncthreads();
                for (int k = 0; k < TK; ++k) {
                    float av[4], wv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        av[i] = sa[k][ty * 4 + i];
                        wv[i] = sw[k][tx * 4 + i];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(av[i], wv[j], part[i][j]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + ty * 4 + i;
                const float s = m < row_end ? p.a_scales[m * kb_count + kb] : 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = n0 + tx * 4 + j;
                    const float ws = n < p.N ? wsc[(int64_t)(n / 128) * kb_count + kb] : 0.0f;
                    acc[i][j] = fmaf(s * ws, part[i][j], acc[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + ty * 4 + i;
            if (m >= row_end) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx * 4 + j;
                if (n >= p.N) break;
                if (p.out_bf16)
                    static_cast<__nv_bfloat16 *>(p.c)[m * p.N + n] = __float2bfloat16_rn(acc[i][j]);
                else
                    static_cast<float *>(p.c)[m * p.N + n] = acc[i][j];
            }
        }
    }
}

// q, s = quantised silu(h[:Nh]) * h[Nh:]; one warp per row and 128 columns.
__global__ void __launch_bounds__(256)
k_swiglu_quant(const float *h, const int32_t *offsets, int64_t E, uint8_t *q, float *s,
               int64_t cap_rows, int64_t Nh) {
    pdl_wait();
    const int64_t nb = Nh / kFp8Block;
    const int64_t rows = min((int64_t)offsets[E], cap_rows);
    const int lane = threadIdx.x & 31;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < rows * nb;
         u += (int64_t)gridDim.x * 8) {
        const int64_t r = u / nb, b = u % nb;
        const float4 a = reinterpret_cast<const float4 *>(h + r * 2 * Nh + b * kFp8Block)[lane];
        const float4 m = reinterpret_cast<const float4 *>(h + r * 2 * Nh + Nh + b * kFp8Block)[lane];
        const float g[4] = {tc::silu_f32(a.x) * m.x, tc::silu_f32(a.y) * m.y,
                            tc::silu_f32(a.z) * m.z, tc::silu_f32(a.w) * m.w};
        float amax = fmaxf(fmaxf(fabsf(g[0]), fabsf(g[1])), fmaxf(fabsf(g[2]), fabsf(g[3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float sc, inv;
        block_scale(amax, sc, inv);
        reinterpret_cast<uint32_t *>(q + r * Nh + b * kFp8Block)[lane] =
            e4m3x4(g[0] * inv, g[1] * inv, g[2] * inv, g[3] * inv);
        if (lane == 0) s[r * nb + b] = sc;
    }
}

// Row r of the gathered rows and their scales = token assist[r].
__global__ void __launch_bounds__(128)
k_gather_fp8(const uint4 *x, const float *xs, const int32_t *assist, const int32_t *offsets,
             int64_t E, int64_t T, int64_t M, uint4 *rows, float *rs, int64_t cap_rows, int64_t H16,
             int64_t nb) {
    pdl_wait();
    const int64_t R = min((int64_t)offsets[E], cap_rows);
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const int64_t t = (int64_t)assist[3 * r] * M + assist[3 * r + 1];
        if (t < 0 || t >= T) continue;
        for (int64_t i = threadIdx.x; i < H16; i += blockDim.x) rows[r * H16 + i] = x[t * H16 + i];
        for (int64_t i = threadIdx.x; i < nb; i += blockDim.x) rs[r * nb + i] = xs[t * nb + i];
    }
}

}  // namespace

moe_status launch_gemm_fp8(const Fp8GemmArgs &a, cudaStream_t stream) {
    if (a.cap_rows <= 0) return MOE_OK;
    const int kb = (int)((a.Kd + 127) / 128);
    const int64_t mb = (a.cap_rows + TM - 1) / TM;
    const dim3 grid((unsigned)((a.N + TN - 1) / TN), (unsigned)(mb < 64 ? mb : 64), (unsigned)a.E);
    MOE_LAUNCH("gemm_fp8", k_gemm_fp8_simple, grid, 256, 0, stream, a, kb);
    return MOE_OK;
}

moe_status launch_swiglu_quant(const float *h, const int32_t *offsets, int64_t E, void *q, float *s,
                               int64_t cap_rows, int64_t Nh, cudaStream_t stream) {
    MOE_LAUNCH("swiglu_quant", k_swiglu_quant, num_sms() * 8, 256, 0, stream, h, offsets, E,
               static_cast<uint8_t *>(q), s, cap_rows, Nh);
    return MOE_OK;
}

moe_status launch_gather_fp8(const void *x, const float *xs, const int32_t *assist,
                             const int32_t *offsets, int64_t E, int64_t T, int64_t M, void *rows,
                             float *rs, int64_t cap_rows, int64_t H, cudaStream_t stream) {
    const int64_t cap = (int64_t)num_sms() * 16;
    MOE_LAUNCH("gather_fp8", k_gather_fp8, (unsigned)(cap_rows < cap ? cap_rows : cap), 128, 0, stream,
               static_cast<const uint4 *>(x), xs, assist, offsets, E, T, M,
               static_cast<uint4 *>(rows), rs, cap_rows, H / 16, (H + 127) / 128);
    return MOE_OK;
}

}  // namespace moe
