// capi_int8.cu -- the C ABI of the int8 calls around a decoding batch
// (include/moe_gb300.h): argument checks, workspace layout and the order of kernels.
#include "common.cuh"

#include <algorithm>

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

// ---------------------------------------------------------------- product with token and channel scales
bool valid_path(int path) { return path >= MOE_FFN_PATH_AUTO && path <= MOE_FFN_PATH_LARGE_PAIR; }
bool has_images(int path) { return path != MOE_FFN_PATH_SMALL; }
bool has_bytes(int path) { return path == MOE_FFN_PATH_SMALL || path == MOE_FFN_PATH_AUTO; }
size_t image_bytes(int64_t E, int64_t N, int64_t Kd) { return align_up((size_t)E * N * Kd * 2, kAlign); }

constexpr int64_t kMaxDepth = 131056;     // products of 2^14 at most: sums below 2^31
constexpr int64_t kMaxRows = INT32_MAX - 255;   // the end of a tile of 256 rows is a 32-bit number too
moe_status check_int8(int64_t E, int64_t N, int64_t Kd) {
    if (E < 1 || E > kMaxExperts || N < 8 || N % 8 != 0 || N > (1 << 20) || Kd < 16 || Kd % 16 != 0 ||
        Kd > kMaxDepth)
        return MOE_FAIL(MOE_ERR_SHAPE);
    return MOE_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a call multiplies, measured (us, bf16 rows, in brackets int8):
//   N x Kd, one group, rows      stream         tiles          large
//     4096 x 7168       16     12.4 (10.8)    13.3 (12.2)
//                       32     17.1 (15.4)    15.0 (12.8)
//                       64     28.8 (26.5)    16.3 (13.9)
//                      256     90.7           26.0           47.0
//                      512                    32.6           49.5
//                     1024                    59.0           53.3
//     7168 x 2048       16      8.5  (7.1)    10.8  (9.2)
//                       32     11.8 (10.3)    10.9  (9.8)
//                       64     18.9 (17.3)    11.8 (10.6)
//                      512                    21.4           23.5
//     1536 x 2048       32      7.7  (5.6)     8.2  (7.3)
//                     1024                    15.0           23.6
//   32 groups, 2048 x 2048, rows a group
//                        4     26.4           32.0           62.8
//                       16     45.4           33.7           65.2
//                      200                    72.6           88.5
//   64 groups, 2048 x 1024
//                        4     37.3           31.7
//                       64                    45.8           90.1
// So the ways go by estimates (us): of the stream by its readings of the weights, for 8, 16 or
// 32 rows each, of the tiles by int8_tiles_plan, of the SM-pair tiles by their waves and blocks
// of K (0.74 us of 256 x 256 on a pair, under the power cap) and their images of the weights.
enum class How { Stream, Tiles, Large };
How how(int path, int64_t rows, int64_t E, int64_t N, int64_t Kd, const Int8TilesPlan &plan) {
    if (path == MOE_FFN_PATH_LARGE || path == MOE_FFN_PATH_LARGE_PAIR) return How::Large;
    const int64_t groups = std::min(E, rows), per = ceil_div(rows, groups);
    const double w = (double)(groups * N), k = (double)Kd;
    const double stream = rows <= 8 * E    ? 4.0 + w * (0.155e-6 * k + 1.0e-4)
                          : rows <= 16 * E ? 4.0 + w * (0.25e-6 * k + 1.5e-4)
                                           : 5.0 + w * (double)ceil_div(per, 32) * (0.38e-6 * k + 2.0e-4);
    const int64_t waves = ceil_div(groups * ceil_div(per, 256) * ceil_div(N, 256), num_sms() / 2);
    const double large = 10.0 + (double)waves * (2.0 + (double)ceil_div(Kd, 128) * 0.74) + (double)(E * N) * k * 0.24e-6;
    if (stream <= plan.us && (path == MOE_FFN_PATH_SMALL || stream <= large)) return How::Stream;
    return path == MOE_FFN_PATH_SMALL || plan.us <= large ? How::Tiles : How::Large;
}

struct Int8Layout {
    size_t status, rows, scales, total;
};
Int8Layout int8_layout(int64_t rows, int64_t Kd) {
    Int8Layout L;
    Carve c;
    L.status = c.take(4);
    L.rows = c.take((size_t)rows * Kd * 2);      // codes or fp16 images
    L.scales = c.take((size_t)rows * sizeof(float));
    L.total = c.off;
    return L;
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
    return moe_layer_few_tokens_y(shape, MOE_DTYPE_BF16, x, expert_ids, expert_scales, x_active_mask,
                                  shared_expert_x, w1_packed, scale1, w2_packed, scale2, x_out, workspace,
                                  workspace_bytes, stream);
}

moe_status moe_layer_few_tokens_y(const moe_shape *shape, int y_dtype, const void *x,
                                  const int32_t *expert_ids, const float *expert_scales,
                                  const uint8_t *x_active_mask, const void *shared_expert_x,
                                  const void *w1_packed, const float *scale1, const void *w2_packed,
                                  const float *scale2, void *x_out, void *workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
    MOE_TRY(check_few(shape));
    if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
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
    a.y_f32 = y_dtype == MOE_DTYPE_F32;
    return launch_layer_few_tokens(s, a, stream);
}

moe_status moe_int8_packed_bytes(int64_t E, int64_t N, int64_t Kd, int path, size_t *bytes) {
    if (!bytes) return MOE_FAIL(MOE_ERR_NULLPTR);
    MOE_TRY(check_int8(E, N, Kd));
    if (!valid_path(path)) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    *bytes = (has_images(path) ? image_bytes(E, N, Kd) : 0) + (has_bytes(path) ? (size_t)E * N * Kd : 0);
    return MOE_OK;
}

moe_status moe_pack_int8(int64_t E, int64_t N, int64_t Kd, int path, const int8_t *w, void *w_packed,
                         cudaStream_t stream) {
    MOE_TRY(check_int8(E, N, Kd));
    if (!valid_path(path)) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (!w || !w_packed) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!aligned(w, 16) || !aligned(w_packed, kAlign)) return MOE_FAIL(MOE_ERR_ALIGNMENT);
    if (has_images(path)) MOE_TRY(launch_i8_to_f16(w, w_packed, E * N * Kd, stream));
    if (has_bytes(path))
        MOE_TRY(launch_bias_i8(w, static_cast<uint8_t *>(w_packed) + (has_images(path) ? image_bytes(E, N, Kd) : 0),
                               E * N * Kd, stream));
    return MOE_OK;
}

moe_status moe_grouped_gemm_int8_workspace_size(int64_t rows, int64_t E, int64_t N, int64_t Kd,
                                                size_t *bytes) {
    if (!bytes) return MOE_FAIL(MOE_ERR_NULLPTR);
    MOE_TRY(check_int8(E, N, Kd));
    if (rows < 0 || rows > kMaxRows || rows * Kd >= (int64_t)1 << 40) return MOE_FAIL(MOE_ERR_SHAPE);
    *bytes = int8_layout(rows, Kd).total;
    return MOE_OK;
}

moe_status moe_grouped_gemm_int8(int64_t rows, int64_t E, int64_t N, int64_t Kd,
                                 const int32_t *expert_offsets, const void *A, int a_dtype,
                                 const float *a_scales, const void *w_packed,
                                 const float *w_scales, const float *bias, void *C, int out_dtype,
                                 int path, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream) {
    size_t need = 0;
    MOE_TRY(moe_grouped_gemm_int8_workspace_size(rows, E, N, Kd, &need));
    if ((a_dtype != MOE_DTYPE_BF16 && a_dtype != MOE_DTYPE_I8) ||
        (out_dtype != MOE_DTYPE_F32 && out_dtype != MOE_DTYPE_BF16) || !valid_path(path))
        return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    const bool bf16 = a_dtype == MOE_DTYPE_BF16, empty = rows == 0;
    if (bf16 && a_scales) return MOE_FAIL(MOE_ERR_PARAM_INVALID);
    if (!expert_offsets || !w_packed || !w_scales || !workspace) return MOE_FAIL(MOE_ERR_NULLPTR);
    if (!empty && (!A || !C || (!bf16 && !a_scales))) return MOE_FAIL(MOE_ERR_NULLPTR);
    // fp32 rows of C are stored 32 bytes at a time, the scales read 16
    if (!aligned(A, 16) || !aligned(C, out_dtype == MOE_DTYPE_F32 ? 32 : 16) || !aligned(a_scales, 4) ||
        !aligned(w_scales, 16) || !aligned(bias, 16) || !aligned(expert_offsets, 4) ||
        !aligned(w_packed, kAlign) || !aligned(workspace, kAlign))
        return MOE_FAIL(MOE_ERR_ALIGNMENT);
    if (workspace_bytes < need) return MOE_FAIL(MOE_ERR_WORKSPACE);
    if (empty) return MOE_OK;
    const Int8Layout L = int8_layout(rows, Kd);
    const Int8TilesPlan plan = int8_tiles_plan(rows, !bf16, E, N, Kd);
    int32_t *status = at<int32_t>(workspace, L.status);
    const How way = how(path, rows, E, N, Kd, plan);
    const uint8_t *bytes = static_cast<const uint8_t *>(w_packed) + (has_images(path) ? image_bytes(E, N, Kd) : 0);
    if (way == How::Stream) {
        Int8FewArgs f{};
        f.rows = A;
        f.rows_bf16 = bf16;
        f.row_scales = a_scales;
        f.offsets = expert_offsets;
        f.cap_rows = rows;
        f.E = E;
        f.N = N;
        f.Kd = Kd;
        f.w = bytes;
        f.w_scales = w_scales;
        f.bias = bias;
        f.c = C;
        f.out_bf16 = out_dtype == MOE_DTYPE_BF16;
        f.status = status;
        if (bf16 && !int8_few_local(rows, E, Kd)) {
            MOE_TRY(launch_quant_rows_i8(A, true, true, rows, Kd, at<int8_t>(workspace, L.rows),
                                         at<float>(workspace, L.scales), stream));
            f.rows = at<void>(workspace, L.rows);
            f.row_scales = at<float>(workspace, L.scales);
            f.rows_bf16 = false;
            f.early = true;
        }
        return launch_int8_few(f, stream);
    }
    const bool images = way == How::Large || !plan.bytes;
    if (images)
        MOE_TRY(launch_rows_to_f16(A, bf16, a_scales, expert_offsets, E, rows, Kd, at<void>(workspace, L.rows),
                                   at<float>(workspace, L.scales), status, stream));
    if (way == How::Tiles && !plan.whole) {
        Int8TilesArgs t{};
        t.rows = images ? at<void>(workspace, L.rows) : A;
        t.row_scales = images ? at<float>(workspace, L.scales) : a_scales;
        t.offsets = expert_offsets;
        t.cap_rows = rows;
        t.E = E;
        t.N = N;
        t.Kd = Kd;
        t.w = bytes;
        t.w_scales = w_scales;
        t.bias = bias;
        t.c = C;
        t.out_bf16 = out_dtype == MOE_DTYPE_BF16;
        t.status = status;
        t.early = images;
        return launch_int8_tiles(t, plan, stream);
    }
    GemmArgs g{};
    g.a_img = at<void>(workspace, L.rows);
    g.cap_rows = rows;
    g.b_img = way == How::Large ? w_packed : bytes;
    g.E = E;
    g.Nout = N;
    g.Kd = Kd;
    g.offsets = expert_offsets;
    g.y = C;
    g.y_f32 = out_dtype == MOE_DTYPE_F32;
    g.scale2 = w_scales;
    g.s2 = at<float>(workspace, L.scales);
    g.bias = bias;
    g.status = status;
    g.wide = plan.wide;
    if (way == How::Tiles) return launch_grouped_gemm_small(Epi::Linear, g, stream);
    return launch_grouped_gemm(Epi::Linear, g, stream, path != MOE_FFN_PATH_LARGE);
}

}  // extern "C"
