// capi_fp8.cu -- the C ABI of the fp8 expert path (include/moe_gb300.h):
// argument checks, workspace layout and the order of kernels.
#include "common.cuh"

#include <algorithm>
#include <cmath>

namespace moe {
namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

template <typename T>
T *at(void *ws, size_t off) {
    return reinterpret_cast<T *>(reinterpret_cast<uint8_t *>(ws) + off);
}

struct Fp8Layout {
    size_t status = 0;   // int32 status word
    size_t rows = 0;     // e4m3 [cap, H] gathered tokens
    size_t row_s = 0;    // fp32 [cap, ceil(H/128)]
    size_t q2 = 0;       // e4m3 [cap, N/2]
    size_t s2 = 0;       // fp32 [cap, N/256]
    size_t total = 0;
};

struct Carve {
    size_t off = 0;
    size_t take(size_t bytes) {
        const size_t a = off;
        off = align_up(off + (bytes ? bytes : 1), kAlign);
        return a;
    }
};

Fp8Layout gemm_layout() {
    Fp8Layout L;
    Carve c;
    L.status = c.take(4);
    L.total = c.off;
    return L;
}

Fp8Layout ffn_layout(const moe_shape &s) {
    Fp8Layout L;
    Carve c;
    const size_t cap = (size_t)(s.num_tokens * s.topk);
    L.status = c.take(4);
    L.rows = c.take(cap * s.hidden);
    L.row_s = c.take(cap * ((s.hidden + 127) / 128) * sizeof(float));
    L.q2 = c.take(cap * (s.ffn / 2));
    L.s2 = c.take(cap * (s.ffn / 256) * sizeof(float));
    L.total = c.off;
    return L;
}

// AUTO's choice for a product, by an estimate of both kernels' time where the
// weights' bytes do not bound it: tiles a multiprocessor works through x
// blocks of K x the time a block takes it.  Measured times per block: a 128 x
// 256 tile 0.48 us; 128 channels against up to 64 rows 0.32 us; 128 channels
// of g against up to 32 rows 0.3 us and 64 rows 0.85 us (two accumulators to
// read back for each).  Rows are taken as spread evenly.
// What it chooses, measured (us, small against large): one product of 4096 x
// 7168 with 256 rows 27/33, with 512 rows 45/33; 128 experts, 7168 x 4096 FFN,
// 8 rows each 839/861, 32 rows each 1037/882.
bool small_is_faster(const Fp8GemmArgs &a) {
    const int64_t experts = std::min(a.E, a.cap_rows), rows = (a.cap_rows + experts - 1) / experts;
    const int64_t num_kb = (a.Kd + 127) / 128, wblocks = (a.N + 127) / 128 / (a.q2 ? 2 : 1);
    const int64_t blocks = (rows + 127) / 128, cols = (a.N + 255) / 256;
    const int64_t sms = num_sms();
    const double large = (double)((experts * blocks * cols + sms - 1) / sms * num_kb) * 0.48;
    const int64_t tb = gemm_fp8_small_tile_rows(a);
    const int64_t small_tiles = experts * ((rows + tb - 1) / tb) * wblocks;
    const double small = (double)((small_tiles + sms - 1) / sms * num_kb) / gemm_fp8_small_split(a) *
                         (a.q2 ? (tb > 32 ? 0.85 : 0.3) : 0.32);
    return small <= 1.2 * large;   // a tie goes to the one that also prefetches its weights
}

moe_status run_gemm(int path, const Fp8GemmArgs &a, cudaStream_t stream) {
    const bool small = path == MOE_FFN_PATH_SMALL || (path == MOE_FFN_PATH_AUTO && small_is_faster(a));
    return small ? launch_gemm_fp8_small(a, stream) : launch_gemm_fp8_large(a, stream);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_add_rms_norm(int64_t num_tokens, int64_t hidden, const void *x,
                            const void *residual, const void *weight, int weight_dtype, float eps,
                            void *residual_out, void *y, void *q, float *scales,
                            cudaStream_t stream) {
    if (num_tokens < 0 || num_tokens > INT32_MAX || hidden < 8 || hidden % 8 != 0 || hidden > 16384)
        return MOE_FAIL(MOE_ERR_SHAPE);
    if (weight_dtype != MOE_DTYPE_F32 && weight_dtype != MOE_DTYPE_BF16)
        return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (!(eps >= 1e-30f) || !std::isfinite(eps)) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (residual_out && !residual) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (!weight) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (num_tokens > 0) {
        if (!x || (!y && !q)) return MOE_FAIL(MOE_ERR_NULLPTR);
        if ((q == nullptr) != (scales == nullptr)) return MOE_FAIL(MOE_ERR_NULLPTR);
    }
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
        !aligned(residual_out, 16) || !aligned(y, 16) || !aligned(q, 16) || !aligned(scales, 4))
        return MOE_FAIL(MOE_ERR_ALIGNMENT);
    if (num_tokens == 0) return MOE_OK;
    return launch_add_rms_norm(num_tokens, hidden, x, residual, weight,
                               weight_dtype == MOE_DTYPE_BF16, eps, residual_out, y, q, scales,
                               stream);
}

moe_status moe_block_norm(const moe_block_norm_desc *desc, const void *x, const void *residual,
                          const void *post_weight, const void *gate, const void *weight,
                          void *residual_out, void *y, void *q, float *scales,
                          cudaStream_t stream) {
    if (!desc) return MOE_FAIL(MOE_ERR_NULLPTR);
    const moe_block_norm_desc &d = *desc;
    const int64_t T = d.num_tokens, H = d.hidden;
    if (T < 0 || T > INT32_MAX || H < 8 || H % 8 != 0 || H > 16384) return MOE_FAIL(MOE_ERR_SHAPE);
    if ((d.weight_dtype != MOE_DTYPE_F32 && d.weight_dtype != MOE_DTYPE_BF16) ||
        (d.gate_act != MOE_GATE_ACT_NONE && d.gate_act != MOE_GATE_ACT_SIGMOID) || d.reserved != 0)
        return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (!(d.eps >= 1e-30f) || !std::isfinite(d.eps) || !std::isfinite(d.residual_scale) ||
        !std::isfinite(d.branch_scale))
        return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (d.gate_rows < 0 || d.gate_stride < 0 || (d.gate_rows == 0) != (d.gate_stride == 0) ||
        (d.gate_rows > 0 && (T % d.gate_rows != 0 || d.gate_rows > std::max<int64_t>(T, 1) ||
                             d.gate_stride < H || d.gate_stride % 8 != 0 || d.gate_stride > INT32_MAX)))
        return MOE_FAIL(MOE_ERR_SHAPE);
    if (d.gate_rows == 0 && gate) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (!weight && (y || q)) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (T > 0) {
        if (!x || !residual || !residual_out || (d.gate_rows > 0 && !gate)) return MOE_FAIL(MOE_ERR_NULLPTR);
        if ((q == nullptr) != (scales == nullptr)) return MOE_FAIL(MOE_ERR_NULLPTR);
    }
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(post_weight, 16) || !aligned(gate, 16) ||
        !aligned(weight, 16) || !aligned(residual_out, 16) || !aligned(y, 16) || !aligned(q, 16) ||
        !aligned(scales, 4))
        return MOE_FAIL(MOE_ERR_ALIGNMENT);
    if (T == 0) return MOE_OK;
    return launch_block_norm(d, x, residual, post_weight, gate, weight, residual_out, y, q, scales, stream);
}

moe_status moe_gate(const moe_gate_desc *desc, const void *logits, const float *bias,
                    const uint8_t *x_active_mask, int32_t *expert_ids, float *expert_scales,
                    uint8_t *route_mask, cudaStream_t stream) {
    if (!desc) return MOE_FAIL(MOE_ERR_NULLPTR);
    const moe_gate_desc &d = *desc;
    if (d.num_experts < 1 || d.num_experts > kMaxExperts || d.topk < 1 || d.topk > kMaxTopK ||
        d.num_groups < 1 || d.num_groups > d.num_experts || d.num_experts % d.num_groups != 0 ||
        d.topk_groups < 1 || d.topk_groups > d.num_groups ||
        d.topk > d.topk_groups * (d.num_experts / d.num_groups))
        return MOE_FAIL(MOE_ERR_SHAPE);
    if (d.num_tokens < 0 || d.num_tokens * d.topk > INT32_MAX || d.num_tokens > INT32_MAX ||
        d.logits_stride < d.num_experts || d.logits_stride > INT32_MAX)
        return MOE_FAIL(MOE_ERR_SHAPE);
    if ((d.logits_dtype != MOE_DTYPE_F32 && d.logits_dtype != MOE_DTYPE_BF16) ||
        (d.score != MOE_GATE_SOFTMAX && d.score != MOE_GATE_SIGMOID) ||
        (d.group_score != MOE_GATE_GROUP_MAX && d.group_score != MOE_GATE_GROUP_TOP2) ||
        (d.renormalize != 0 && d.renormalize != 1) || d.reserved != 0 || !std::isfinite(d.scale))
        return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (d.num_tokens == 0) return MOE_OK;
    if (!logits || !expert_ids || !expert_scales) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!aligned(logits, d.logits_dtype == MOE_DTYPE_F32 ? 4 : 2) || !aligned(bias, 4) ||
        !aligned(expert_ids, 4) || !aligned(expert_scales, 4))
        return MOE_FAIL(MOE_ERR_ALIGNMENT);
    return launch_gate(d, logits, bias, x_active_mask, expert_ids, expert_scales, route_mask, stream);
}

moe_status moe_grouped_gemm_fp8_workspace_size(int64_t rows, int64_t E, int64_t N, int64_t Kd,
                                               size_t *bytes) {
    if (!bytes) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (rows < 0 || rows > INT32_MAX || E < 1 || E > kMaxExperts || N < 8 || N % 8 != 0 || Kd < 16 ||
        Kd % 16 != 0 || N > (1 << 20) || Kd > 131072)
        return MOE_FAIL(MOE_ERR_SHAPE);
    *bytes = gemm_layout().total;
    return MOE_OK;
}

moe_status moe_grouped_gemm_fp8(int64_t rows, int64_t E, int64_t N, int64_t Kd,
                                const int32_t *expert_offsets, const void *A,
                                const float *a_scales, const void *W, const float *w_scales,
                                void *C, int out_dtype, int path, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream) {
    size_t need = 0;
    MOE_TRY(moe_grouped_gemm_fp8_workspace_size(rows, E, N, Kd, &need));
    if (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16)
        return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (path < MOE_FFN_PATH_AUTO || path > MOE_FFN_PATH_LARGE_PAIR) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    const bool empty = rows == 0;
    if (!expert_offsets || !W || !w_scales || !workspace) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!empty && (!A || !a_scales || !C)) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!aligned(A, 16) || !aligned(W, 16) || !aligned(C, 16) || !aligned(a_scales, 4) ||
        !aligned(w_scales, 4) || !aligned(expert_offsets, 4) || !aligned(workspace, kAlign))
        return MOE_FAIL(MOE_ERR_ALIGNMENT);
    if (workspace_bytes < need) return MOE_FAIL(MOE_ERR_WORKSPACE);
    if (empty) return MOE_OK;
    const Fp8Layout L = gemm_layout();
    Fp8GemmArgs g{};
    g.a = A;
    g.a_scales = a_scales;
    g.w = W;
    g.w_scales = w_scales;
    g.offsets = expert_offsets;
    g.cap_rows = rows;
    g.E = E;
    g.N = N;
    g.Kd = Kd;
    g.c = C;
    g.out_bf16 = out_dtype == MOE_DTYPE_BF16;
    g.status = at<int32_t>(workspace, L.status);
    g.reset_status = true;
    return run_gemm(path, g, stream);
}

moe_status moe_grouped_ffn_fp8_workspace_size(const moe_shape *shape, size_t *bytes) {
    MOE_TRY(check_shape(shape, true));
    if (!bytes) return MOE_FAIL(MOE_ERR_NULLPTR);
    *bytes = ffn_layout(*shape).total;
    return MOE_OK;
}

moe_status moe_grouped_ffn_fp8(const moe_shape *shape, const void *x, const float *x_scales,
                               const int32_t *assist, const int32_t *expert_offsets,
                               const void *w1, const float *w1_scales, const void *w2,
                               const float *w2_scales, void *y, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
    MOE_TRY(check_shape(shape, true));
    const moe_shape &s = *shape;
    const bool empty = s.num_tokens == 0;   // the per-token and per-row arrays may then be NULL
    if (!expert_offsets || !w1 || !w1_scales || !w2 || !w2_scales || !workspace)
        return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!empty && (!x || !x_scales || !y)) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(w1, 16) || !aligned(w2, 16) ||
        !aligned(x_scales, 4) || !aligned(w1_scales, 4) || !aligned(w2_scales, 4) ||
        !aligned(assist, 4) || !aligned(expert_offsets, 4) || !aligned(workspace, kAlign))
        return MOE_FAIL(MOE_ERR_ALIGNMENT);
    const Fp8Layout L = ffn_layout(s);
    if (workspace_bytes < L.total) return MOE_FAIL(MOE_ERR_WORKSPACE);
    if (empty) return MOE_OK;
    const int64_t cap = s.num_tokens * s.topk, H = s.hidden, E = s.num_experts, Nh = s.ffn / 2;
    const void *rows = x;
    const float *row_s = x_scales;
    if (assist) {
        MOE_TRY(launch_gather_fp8(x, x_scales, assist, expert_offsets, E, s.num_tokens,
                                  s.num_tokens / s.num_partitions, at<void>(workspace, L.rows),
                                  at<float>(workspace, L.row_s), cap, H,
                                  at<int32_t>(workspace, L.status), stream));
        rows = at<void>(workspace, L.rows);
        row_s = at<float>(workspace, L.row_s);
    }
    Fp8GemmArgs g1{};
    g1.a = rows;
    g1.a_scales = row_s;
    g1.w = w1;
    g1.w_scales = w1_scales;
    g1.offsets = expert_offsets;
    g1.cap_rows = cap;
    g1.E = E;
    g1.N = s.ffn;
    g1.Kd = H;
    g1.q2 = at<void>(workspace, L.q2);
    g1.s2 = at<float>(workspace, L.s2);
    g1.status = at<int32_t>(workspace, L.status);
    g1.reset_status = assist == nullptr;   // the gather has done it
    g1.early = assist != nullptr;
    MOE_TRY(run_gemm(s.ffn_path, g1, stream));
    Fp8GemmArgs g2{};
    g2.a = at<void>(workspace, L.q2);
    g2.a_scales = at<float>(workspace, L.s2);
    g2.w = w2;
    g2.w_scales = w2_scales;
    g2.offsets = expert_offsets;
    g2.cap_rows = cap;
    g2.E = E;
    g2.N = H;
    g2.Kd = Nh;
    g2.c = y;
    g2.out_bf16 = true;
    g2.status = at<int32_t>(workspace, L.status);
    g2.early = true;
    return run_gemm(s.ffn_path, g2, stream);
}

}  // extern "C"
