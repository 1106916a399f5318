// groups.cuh -- the offsets of a grouped product's rows, as the caller gave them.
#pragma once
#include <stdint.h>

namespace moe {

// Offsets in shared memory, s_off[0 .. E], made ascending and at most min(s_off[E],
// rows), so that no group reaches outside the call's rows whatever they are.  One
// warp; the caller synchronises.
__device__ __forceinline__ void bound_offsets(int32_t *s_off, int E, int64_t rows) {
    const int lane = threadIdx.x & 31;
    const int32_t last = (int32_t)max((int64_t)0, min((int64_t)s_off[E], rows));
    __syncwarp();
    int32_t before = 0;
    for (int base = 0; base <= E; base += 32) {
        const int e = base + lane;
        int32_t x = e <= E ? min(max(s_off[e], before), last) : last;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) x = max(x, __shfl_up_sync(0xffffffffu, x, d));
        if (e <= E) s_off[e] = x;
        before = __shfl_sync(0xffffffffu, x, 31);
    }
    __syncwarp();
}

// s_blk[e]: the blocks of `block` rows of the groups before e; s_blk[E] all.  One warp;
// the caller synchronises.
__device__ __forceinline__ void count_blocks(const int32_t *s_off, int32_t *s_blk, int E, int block) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
        const int e = base + lane;
        const int c = e < E ? (s_off[e + 1] - s_off[e] + block - 1) / block : 0;
        int x = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (e < E) s_blk[e] = carry + x - c;
        carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_blk[E] = carry;
}

}  // namespace moe
