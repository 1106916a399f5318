// norm.cuh -- what the two norm kernels share: packed bf16 vectors, a sum over the CTA.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {

constexpr uint32_t kFull = 0xffffffffu;
constexpr float kF32Max = 3.402823466e38f;
constexpr int kNormMaxThreads = 512;

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
}

// Sum over the CTA, the same in every thread.  `fail` from any thread makes
// `failed` true in all.  Every thread's earlier shared-memory reads are done
// when it returns.
__device__ __forceinline__ float block_sum(float v, float *part, bool fail, bool &failed) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    failed = __syncthreads_or(fail);
    // places of warps that the block does not have hold 0
    const float4 *p4 = reinterpret_cast<const float4 *>(part);
    float4 a = p4[0];
#pragma unroll
    for (int w = 1; w < kNormMaxThreads / 128; ++w) {
        const float4 b = p4[w];
        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
    }
    return (a.x + a.y) + (a.z + a.w);
}

}  // namespace moe
