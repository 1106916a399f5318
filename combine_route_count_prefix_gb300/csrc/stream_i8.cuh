// stream_i8.cuh -- int8 products against a few rows, with the weights streamed
// through rings of shared memory that belong to one warp each.
//
// With a few rows an int8 product is a read of its weights.  A warp takes the
// weights in stages of 16 output channels x 128 of the inner dimension (2 KB:
// whole 128-byte lines), which its lanes fetch with 16-byte cp.async copies
// some stages ahead and read back themselves, so no barrier and no other
// warp is involved and a wait always ends.  sm_103a has no fast int8 matrix
// instruction (mma.sync s8: 158 Top/s, 0.08 of the fp16 rate of tcgen05), so
// the bytes are widened to fp16 in registers, exactly, and multiplied with
// mma.sync m16n8k16 (601 TFLOP/s measured; 16 channels by 8 rows, no
// tensor memory to fill and drain), whose fp32 sums are exact below 2^24, that is
// for 1024 products.
// 16 channels x 8 rows x 128 take 4 + 2 shared loads, 96 integer and half
// instructions for the widening and 8 mma per warp; one row takes 32 with dp4a. With
// the copies and the loop a stage of one row is 114 instructions of a warp, a quarter
// of the issue slots at the rate the stages arrive at from HBM.  A copy of 1 GB in
// this shape runs at 6.5 TB/s with about 96 KB in flight on an SM.
#pragma once
#include <stdint.h>

#include "ptx.cuh"

namespace moe {
namespace si8 {

constexpr int kChannels = 16;                      // output channels of a stage
constexpr int kDepth = 128;                        // its share of the inner dimension
constexpr int kWeightBytes = kChannels * kDepth;
constexpr int kRows = 8;                           // rows of one mma
constexpr int kRowBytes = kRows * kDepth;
constexpr int kExactStages = 1024 / kDepth;        // stages that an fp32 sum holds exactly

// 16 bytes global -> shared, zeros where `on` is false (src is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16u : 0u)
                 : "memory");
}
// The same for bytes that are read once: they leave L2 before anything else does, so
// that a call's stream of weights does not push out what every call needs again (the
// kernels' instructions, scales, the next call's inputs).
__device__ __forceinline__ void copy16_once(uint32_t dst, const void *src, bool on, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
                 "r"(on ? 16u : 0u), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Row r of a block of 128-byte rows keeps its 16-byte unit u at u ^ (r % 8):
// lanes that read the same unit of eight neighbouring rows meet no bank twice.
__device__ __forceinline__ uint32_t unit_at(int r, int u) { return (uint32_t)((u ^ (r & 7)) << 4); }

// Two biased bytes b + 128 of `word` (bytes 0, 1 or 2, 3) -> the fp16 pair of
// their b: the byte in the low mantissa bits of the fp16 number 1024 is 1024 +
// (b + 128) exactly, and 1152 less is b.
__device__ __forceinline__ uint32_t widen_lo(uint32_t word) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(__byte_perm(word, 0x64646464u, 0x4140)), "r"(0x64806480u));
    return d;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t word) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(__byte_perm(word, 0x64646464u, 0x4342)), "r"(0x64806480u));
    return d;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                 "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Lane (g, t) = (lane / 4, lane % 4) multiplies bytes [32 t, 32 t + 32) of
// channels g and g + 8 with the same bytes of row g: which of the 128 inner
// positions an mma calls k does not matter as long as both operands agree.
// c[n][p]: the sums of row block n (p splits them in two where there is one
// block, so that an mma need not wait for the one before it); c[][][0..1] are
// channel g of rows 2 t and 2 t + 1, [2..3] channel g + 8.
// at: the lane's first 16 bytes of channel g in the stage (biased bytes; the next
// 16 are at at ^ 16).  row[n]: the same of row g of block n (plain int8).
template <int NB>
struct Sums {
    static constexpr int kSplit = NB == 1 ? 2 : 1;
    float c[NB][kSplit][4];
    int32_t total[NB][4];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) total[n][i] = 0;
#pragma unroll
            for (int p = 0; p < kSplit; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) c[n][p][i] = 0.0f;
        }
    }
    // fp32 sums of at most 1024 products -> the int32 totals
    __device__ __forceinline__ void flush() {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int p = 0; p < kSplit; ++p)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    total[n][i] += __float2int_rn(c[n][p][i]);
                    c[n][p][i] = 0.0f;
                }
    }
    __device__ __forceinline__ void add_stage(uint32_t at, const uint32_t (&row)[NB]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 wa = lds16(at ^ (h << 4)), wb = lds16((at ^ (h << 4)) + 8 * kDepth);
            uint4 xr[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) xr[n] = lds16(row[n] ^ (h << 4));
            const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = widen_lo(a[i]), a1 = widen_lo(b[i]);
                const uint32_t a2 = widen_hi(a[i]), a3 = widen_hi(b[i]);
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const uint32_t x4[4] = {xr[n].x, xr[n].y, xr[n].z, xr[n].w};
                    const uint32_t x = x4[i] ^ 0x80808080u;
                    mma_f16(c[n][i % kSplit], a0, a1, a2, a3, widen_lo(x), widen_hi(x));
                }
            }
        }
    }
};

// The same products for NR <= 4 rows with dp4a, on the integer pipe (64 lanes a
// clock of an SM): 16 instructions a row and stage, against the 104 that the widening
// and the mma take whatever the rows (even at about five).  Lane (g, t) adds
// bytes [32 t, 32 t + 32) of channels g and g + 8.
template <int NR>
__device__ __forceinline__ void dot_stage(int32_t (&acc)[NR][2], uint32_t at, const uint32_t (&row)[NR]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 wa = lds16(at ^ (h << 4)), wb = lds16((at ^ (h << 4)) + 8 * kDepth);
        const uint32_t a[4] = {wa.x ^ 0x80808080u, wa.y ^ 0x80808080u, wa.z ^ 0x80808080u,
                               wa.w ^ 0x80808080u};
        const uint32_t b[4] = {wb.x ^ 0x80808080u, wb.y ^ 0x80808080u, wb.z ^ 0x80808080u,
                               wb.w ^ 0x80808080u};
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const uint4 x = lds16(row[n] ^ (h << 4));
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[n][0] = __dp4a((int)a[i], (int)xs[i], acc[n][0]);
                acc[n][1] = __dp4a((int)b[i], (int)xs[i], acc[n][1]);
            }
        }
    }
}

// Quotients by a divisor that is the same all over a launch, a * d < 2^32.
struct Divisor {
    uint32_t d, m;
    __host__ explicit Divisor(uint32_t by = 1) : d(by), m(by > 1 ? (uint32_t)(0x100000000ull / by) + 1 : 0) {}
    __device__ __forceinline__ int operator()(int a) const { return m ? (int)__umulhi((uint32_t)a, m) : a; }
};

// What the lanes of a warp need to fetch and find their parts of a stage.
struct Lane {
    int cu, cr;           // copies: 16-byte unit of a 128-byte row, row of a group of four
    uint32_t to0, to1;    // where rows cr and cr + 4 of a group of eight go
    int g, t;             // products: channel (row) of eight, quarter of the 128 bytes
    uint32_t from;        // its first 16 bytes of channel g
    __device__ __forceinline__ Lane() {
        const int lane = threadIdx.x & 31;
        cu = lane & 7;
        cr = lane >> 3;
        to0 = (uint32_t)(cr * kDepth) + unit_at(cr, cu);
        to1 = (uint32_t)((cr + 4) * kDepth) + unit_at(cr + 4, cu);
        g = lane >> 2;
        t = lane & 3;
        from = (uint32_t)(g * kDepth) + unit_at(g, 2 * t);
    }
    // row r of a block of 128-byte rows: this lane's first 16 bytes
    __device__ __forceinline__ uint32_t of_row(int r) const { return unit_at(r, 2 * t); }
};

// One warp's way through its stages.  The ring holds kD; stage i + kD - 1 is
// fetched once every lane has read stage i - 1, into its slot.
// LOCAL: the rows' codes lie elsewhere in shared memory, stage after stage;
// else they come with the weights, behind them in the slot.
template <int kD, int kBytes, bool LOCAL>
struct Walk {
    uint32_t base, cur, prev;
    __device__ __forceinline__ explicit Walk(uint32_t b)
        : base(b), cur(b), prev(b + (uint32_t)((kD - 1) * kBytes)) {}
    // The first kD - 1 stages.  fetch(slot, weights, rows) copies one or both and steps on.
    template <typename Fetch>
    __device__ __forceinline__ void first(Fetch &fetch, bool weights, bool rows) {
#pragma unroll 1
        for (int i = 0; i < kD - 1; ++i) {
            fetch(base + (uint32_t)(i * kBytes), weights, rows);
            if (rows) copy_commit();   // weights copied before belong to the first group then
        }
    }
    template <typename Fetch>
    __device__ __forceinline__ uint32_t next(Fetch &fetch) {
        copy_wait<kD - 2>();
        __syncwarp();
        fetch(prev, true, true);
        copy_commit();
        prev = cur;
        cur = cur + kBytes == base + kD * kBytes ? base : cur + kBytes;
        return prev;
    }
    template <int NR, typename Fetch, typename Row, typename Add>
    __device__ __forceinline__ void dots(const Lane &l, int stages, Fetch &fetch, Row &row, Add &add) {
        int32_t acc[NR][2];
        uint32_t r[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            acc[n][0] = acc[n][1] = 0;
            r[n] = row(n);
        }
#pragma unroll 1
        for (int i = 0; i < stages; ++i) {
            const uint32_t st = next(fetch);
            uint32_t at[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                at[n] = LOCAL ? r[n] : st + r[n];
                if (LOCAL) r[n] += kDepth;
            }
            dot_stage<NR>(acc, st + l.from, at);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                acc[n][c] += __shfl_xor_sync(0xffffffffu, acc[n][c], 1);
                acc[n][c] += __shfl_xor_sync(0xffffffffu, acc[n][c], 2);
            }
            if (n == l.t) {
                add(n, l.g, acc[n][0]);
                add(n, l.g + 8, acc[n][1]);
            }
        }
    }
    template <int NB, typename Fetch, typename Row, typename Add>
    __device__ __forceinline__ void blocks(const Lane &l, int stages, int nr, Fetch &fetch, Row &row, Add &add) {
        Sums<NB> s;
        s.clear();
        uint32_t r[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {   // lanes of rows that are not there read the last
            const int i = kRows * n + l.g;
            r[n] = row(i < nr ? i : nr - 1);
        }
#pragma unroll 1
        for (int i = 0; i < stages; ++i) {
            const uint32_t st = next(fetch);
            uint32_t at[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                at[n] = LOCAL ? r[n] : st + r[n];
                if (LOCAL) r[n] += kDepth;
            }
            s.add_stage(st + l.from, at);
            if (i % kExactStages == kExactStages - 1) s.flush();
        }
        s.flush();
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r0 = kRows * n + 2 * l.t + (i & 1);
                if (r0 < nr) add(r0, l.g + (i >> 1) * 8, s.total[n][i]);
            }
    }
    // `stages` stages of one unit with nr <= 8 NB rows.  row(n): the lane's first
    // bytes of row n (LOCAL: at the first stage; else in the slot); add(n, c, v) takes
    // the sum of row n and channel c (0 .. 15), from one lane each.
    // (One loop that branches on nr inside measured 4 to 8 % slower.)
    template <int NB, typename Fetch, typename Row, typename Add>
    __device__ __forceinline__ void run(const Lane &l, int stages, int nr, Fetch &fetch, Row &row, Add &add) {
        if (nr == 1) {
            dots<1>(l, stages, fetch, row, add);
        } else if (nr == 2) {
            dots<2>(l, stages, fetch, row, add);
        } else if (nr == 3) {
            dots<3>(l, stages, fetch, row, add);
        } else if (nr == 4) {
            dots<4>(l, stages, fetch, row, add);
        } else if (NB == 1 || nr <= kRows) {
            blocks<1>(l, stages, nr, fetch, row, add);
        } else if (NB == 2 || nr <= 2 * kRows) {
            blocks<2>(l, stages, nr, fetch, row, add);
        } else {
            blocks<NB>(l, stages, nr, fetch, row, add);
        }
    }
};

}  // namespace si8
}  // namespace moe
