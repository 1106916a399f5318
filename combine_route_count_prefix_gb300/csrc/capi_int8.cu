// capi_int8.cu -- the C ABI of the int8 calls around a decoding batch
// (include/moe_gb300.h): argument checks, workspace layout and the order of kernels.
#include "common.cuh"

namespace moe {
namespace {

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

template <typename T>
T *at(void *ws, size_t off) {
    return reinterpret_cast<T *>(reinterpret_cast<uint8_t *>(ws) + off);
}

struct Carve {
    size_t off = 0;
    size_t take(size_t bytes) {
        const size_t a = off;
        off = align_up(off + (bytes ? bytes : 1), kAlign);
        return a;
    }
};

struct FewLayout {
    size_t status, g, q, qs, total;
};

FewLayout few_layout(const moe_shape &s) {
    FewLayout L;
    Carve c;
    const size_t T = (size_t)s.num_tokens, R = T * (size_t)s.topk, H = (size_t)s.hidden, Nh = (size_t)s.ffn / 2;
    L.status = c.take(4);
    L.g = c.take(R * Nh * sizeof(float));
    L.q = c.take(align_up(T * H, kAlign) + R * Nh);
    L.qs = c.take((T + R) * sizeof(float));
    L.total = c.off;
    return L;
}

moe_status check_few(const moe_shape *shape) {
    MOE_TRY(check_shape(shape, true));
    if (shape->num_tokens * shape->topk > MOE_FEW_TOKENS_MAX_ROUTES) return MOE_FAIL(MOE_ERR_SHAPE);
    if (shape->ffn_path != MOE_FFN_PATH_SMALL && shape->ffn_path != MOE_FFN_PATH_AUTO)
        return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_layer_few_tokens_workspace_size(const moe_shape *shape, size_t *bytes) {
    MOE_TRY(check_few(shape));
    if (!bytes) return MOE_FAIL(MOE_ERR_NULLPTR);
    *bytes = few_layout(*shape).total;
    return MOE_OK;
}

moe_status moe_layer_few_tokens(const moe_shape *shape, const void *x, const int32_t *expert_ids,
                                const float *expert_scales, const uint8_t *x_active_mask,
                                const void *shared_expert_x, const void *w1_packed,
                                const float *scale1, const void *w2_packed, const float *scale2,
                                void *x_out, void *workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    MOE_TRY(check_few(shape));
    const moe_shape &s = *shape;
    const bool empty = s.num_tokens == 0;   // the per-token and per-route arrays may then be NULL
    if (!w1_packed || !scale1 || !w2_packed || !scale2 || !workspace) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!empty && (!x || !expert_ids || !expert_scales || !x_out)) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!empty && s.has_shared && !shared_expert_x) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!s.has_shared && shared_expert_x) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (!empty && s.mask_kind != 0 && !x_active_mask) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (s.mask_kind == 0 && x_active_mask) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (!aligned(x, 16) || !aligned(x_out, 16) || !aligned(scale1, 16) || !aligned(scale2, 16) ||
        !aligned(shared_expert_x, 16) || !aligned(w1_packed, kAlign) || !aligned(w2_packed, kAlign) ||
        !aligned(workspace, kAlign) || !aligned(expert_ids, 4) || !aligned(expert_scales, 4))
        return MOE_FAIL(MOE_ERR_ALIGNMENT);
    const FewLayout L = few_layout(s);
    if (workspace_bytes < L.total) return MOE_FAIL(MOE_ERR_WORKSPACE);
    if (empty) return MOE_OK;
    const int64_t E = s.num_experts, N = s.ffn, H = s.hidden;
    FewTokensArgs a{};
    a.x = x;
    a.ids = expert_ids;
    a.probs = expert_scales;
    a.mask = x_active_mask;
    a.shared = shared_expert_x;
    a.w1 = packed_i8(w1_packed, s.ffn_path, E, N, H);
    a.w2 = packed_i8(w2_packed, s.ffn_path, E, H, N / 2);
    a.scale1 = scale1;
    a.scale2 = scale2;
    a.out = x_out;
    a.g = at<float>(workspace, L.g);
    a.q = at<int8_t>(workspace, L.q);
    a.qs = at<float>(workspace, L.qs);
    a.status = at<int32_t>(workspace, L.status);
    return launch_layer_few_tokens(s, a, stream);
}

}  // extern "C"
