// mx4_api.hip -- the C ABI declared in include/mx4.h and include/mx4_route.h:
// host-side argument checks and launches on the caller's stream.  Nothing here
// allocates, synchronises or keeps state.
#include <stdint.h>

#include "../../include/mx4_route.h"
#include "mx4_checks.hpp"

using namespace mx4;

namespace {

// Slots times tiles of the expert layer's outputs, for the same reason as kMaxMN.
constexpr int64_t kMaxMoeBlocks = (int64_t)1 << 24;

int gemm(const uint16_t* x, int64_t ldx, mx4::Mat xm, int64_t M, mx4::Mat w, int64_t N, int64_t K,
         void* y, int64_t ldy, int y_type, void* ws, size_t ws_bytes, void* stream) {
    if (int rc = check_y(y, N, ldy, y_type)) return rc;
    if (!aligned(w.codes, 16) || !aligned(w.scales, 16)) return W12_ERR_ALIGN;
    const size_t need = mx4::gemm_workspace_bytes(M, N, K, x == nullptr);
    if (int rc = check_ws(ws, ws_bytes, need)) return rc;
    if (M == 0) return W12_OK;
    mx4::GemmArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.xm = xm;
    a.w = w;
    a.M = (int)M;
    a.N = N;
    a.K = K;
    a.G = (int)mx4::groups(K);
    a.Q = (int)mx4::quads(K);
    a.y = y;
    a.ldy = ldy;
    a.y_f32 = y_type == W12_OUT_F32;
    return status_of(mx4::launch_gemm(a, ws, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

const char* mx4_status_string(int status) {
    switch (status) {
        case W12_OK: return "ok";
        case W12_ERR_NULL: return "a required pointer is NULL";
        case W12_ERR_SHAPE:
            return "bad shape (K and I are positive multiples of 32 below 2^24, N >= 1, row "
                   "strides cover their rows, an output's matrices lie apart, 1 <= top_k <= E)";
        case W12_ERR_ALIGN:
            return "misaligned pointer or stride (16-byte rows of x, containers and decoded rows)";
        case W12_ERR_DTYPE: return "unknown element type";
        case W12_ERR_UNSUPPORTED:
            return "more tokens, experts or experts a token than mx4_moe takes";
        case W12_ERR_HIP: return "HIP launch failed";
        case W12_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
        default: return "unknown status";
    }
}

size_t mx4_codes_bytes(int64_t B, int64_t R, int64_t K) {
    if (check_container(B, R, K) != W12_OK) return 0;
    return (size_t)(B * mx4::tiles(R) * mx4::groups(K) * mx4::kCodeBlock);
}

size_t mx4_scales_bytes(int64_t B, int64_t R, int64_t K) {
    if (check_container(B, R, K) != W12_OK) return 0;
    return (size_t)(B * mx4::tiles(R) * mx4::quads(K) * mx4::kScaleBlock);
}

int mx4_quantize(const void* x, int x_type, int64_t B, int64_t R, int64_t K, int64_t ldx,
                 int64_t ldb, void* codes, void* scales, void* stream) {
    if (int rc = check_container(B, R, K)) return rc;
    if (type_bytes(x_type) == 0) return W12_ERR_DTYPE;
    if (R > 0 && (!x || !codes || !scales)) return W12_ERR_NULL;
    if (int rc = check_rows(x, x_type, B, K, ldx, ldb)) return rc;
    if (!aligned(codes, 16) || !aligned(scales, 16)) return W12_ERR_ALIGN;
    if (R == 0) return W12_OK;
    return status_of(mx4::launch_quantize(x, x_type == W12_OUT_F32, B, R, K, ldx, ldb,
                                          static_cast<uint8_t*>(codes),
                                          static_cast<uint8_t*>(scales),
                                          static_cast<hipStream_t>(stream)));
}

int mx4_dequantize(const void* codes, const void* scales, int64_t B, int64_t R, int64_t K, void* y,
                   int y_type, int64_t ldy, int64_t ldb, void* stream) {
    if (int rc = check_container(B, R, K)) return rc;
    if (type_bytes(y_type) == 0) return W12_ERR_DTYPE;
    if (R > 0 && (!y || !codes || !scales)) return W12_ERR_NULL;
    if (int rc = check_rows(y, y_type, B, K, ldy, ldb)) return rc;
    if (!aligned(codes, 16) || !aligned(scales, 16)) return W12_ERR_ALIGN;
    if (R == 0) return W12_OK;
    if (B > 1 && !apart(B, R, K, ldy, ldb)) return W12_ERR_SHAPE;
    return status_of(mx4::launch_dequantize(mat(codes, scales), B, R, K, y, y_type == W12_OUT_F32,
                                            ldy, ldb, static_cast<hipStream_t>(stream)));
}

int mx4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_mx4, size_t* bytes) {
    if (bytes == nullptr) return W12_ERR_NULL;
    *bytes = 0;
    if (int rc = check_gemm_shape(M, N, K)) return rc;
    *bytes = mx4::gemm_workspace_bytes(M, N, K, x_mx4 != 0);
    return W12_OK;
}

int mx4_gemm(const uint16_t* x, int64_t M, int64_t ldx, const void* w_codes, const void* w_scales,
             int64_t N, int64_t K, void* y, int64_t ldy, int y_type, void* workspace,
             size_t workspace_bytes, void* stream) {
    if (!w_codes || !w_scales || (M > 0 && (!x || !y))) return W12_ERR_NULL;
    if (int rc = check_gemm_shape(M, N, K)) return rc;
    if (int rc = check_rows(x, W12_OUT_BF16, 1, K, ldx, 0)) return rc;
    if (ldx >= mx4::kFarRows && M > mx4::kMaxFarRows) return W12_ERR_SHAPE;
    return gemm(x, ldx, mx4::Mat{}, M, mat(w_codes, w_scales), N, K, y, ldy, y_type, workspace,
                workspace_bytes, stream);
}

int mx4_gemm_mx4(const void* x_codes, const void* x_scales, int64_t M, const void* w_codes,
                 const void* w_scales, int64_t N, int64_t K, void* y, int64_t ldy, int y_type,
                 void* workspace, size_t workspace_bytes, void* stream) {
    if (!w_codes || !w_scales || (M > 0 && (!x_codes || !x_scales || !y))) return W12_ERR_NULL;
    if (int rc = check_gemm_shape(M, N, K)) return rc;
    if (!aligned(x_codes, 16) || !aligned(x_scales, 16)) return W12_ERR_ALIGN;
    return gemm(nullptr, 0, mat(x_codes, x_scales), M, mat(w_codes, w_scales), N, K, y, ldy, y_type,
                workspace, workspace_bytes, stream);
}

static int check_moe_shape(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    if (T < 0 || E < 1 || top_k < 1 || top_k > E || H < 1) return W12_ERR_SHAPE;
    if (H % MX4_BLOCK != 0 || I < MX4_BLOCK || I % MX4_BLOCK != 0) return W12_ERR_SHAPE;
    if (T > MX4_MAX_T || E > MX4_MAX_E || top_k > MX4_MAX_TOP_K) return W12_ERR_UNSUPPORTED;
    if (int rc = check_container(E, H, I)) return rc;
    if (int rc = check_container(E, 2 * I, H)) return rc;
    const int64_t pairs = T * top_k, slots = (E < pairs ? E : pairs) + pairs / 16;
    if (slots * (H / 16) > kMaxMoeBlocks || slots * (I / 16) > kMaxMoeBlocks) return W12_ERR_SHAPE;
    return W12_OK;
}

int mx4_moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k, int y_type,
                            size_t* bytes) {
    if (bytes == nullptr) return W12_ERR_NULL;
    *bytes = 0;
    if (type_bytes(y_type) == 0) return W12_ERR_DTYPE;
    if (int rc = check_moe_shape(T, H, I, E, top_k)) return rc;
    if (T > 0) *bytes = mx4::moe_workspace_bytes(T, H, I, E, top_k, y_type == W12_OUT_F32);
    return W12_OK;
}

// The layer on logits, or (chosen) on a given choice.
static int moe(const uint16_t* x, int64_t T, int64_t ldx, const float* logits, int64_t ldl,
               const int32_t* chosen, const float* given, mx4::Mat w13, mx4::Mat w2, int64_t H,
               int64_t I, int64_t E, int64_t top_k, int renormalize, void* y, int64_t ldy,
               int y_type, void* workspace, size_t workspace_bytes, void* stream) {
    if (!w13.codes || !w13.scales || !w2.codes || !w2.scales) return W12_ERR_NULL;
    if (T > 0 && (!x || !y || !(logits || (chosen && given)))) return W12_ERR_NULL;
    if (int rc = check_moe_shape(T, H, I, E, top_k)) return rc;
    if (int rc = check_rows(x, W12_OUT_BF16, 1, H, ldx, 0)) return rc;
    if (int rc = check_y(y, H, ldy, y_type)) return rc;
    if (ldl < E || ldl >= kMaxElems) return W12_ERR_SHAPE;
    if (!aligned(logits, 4) || !aligned(chosen, 4) || !aligned(given, 4) ||
        !aligned(w13.codes, 16) || !aligned(w13.scales, 16) || !aligned(w2.codes, 16) ||
        !aligned(w2.scales, 16))
        return W12_ERR_ALIGN;
    size_t need = 0;
    if (T > 0) need = mx4::moe_workspace_bytes(T, H, I, E, top_k, y_type == W12_OUT_F32);
    if (int rc = check_ws(workspace, workspace_bytes, need)) return rc;
    if (T == 0) return W12_OK;
    mx4::MoeArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.logits = logits;
    a.ldl = ldl;
    a.chosen = chosen;
    a.given = given;
    a.w13 = w13;
    a.w2 = w2;
    a.T = (int)T;
    a.H = (int)H;
    a.I = (int)I;
    a.E = (int)E;
    a.top_k = (int)top_k;
    a.renormalize = renormalize != 0;
    a.y = y;
    a.ldy = ldy;
    a.y_f32 = y_type == W12_OUT_F32;
    return status_of(mx4::launch_moe(a, workspace, static_cast<hipStream_t>(stream)));
}

int mx4_moe(const uint16_t* x, int64_t T, int64_t ldx, const float* logits, int64_t ldl,
            const void* w13_codes, const void* w13_scales, const void* w2_codes,
            const void* w2_scales, int64_t H, int64_t I, int64_t E, int64_t top_k, int renormalize,
            void* y, int64_t ldy, int y_type, void* workspace, size_t workspace_bytes,
            void* stream) {
    return moe(x, T, ldx, logits, ldl, nullptr, nullptr, mat(w13_codes, w13_scales),
               mat(w2_codes, w2_scales), H, I, E, top_k, renormalize, y, ldy, y_type, workspace,
               workspace_bytes, stream);
}

int mx4_moe_routed(const uint16_t* x, int64_t T, int64_t ldx, const int32_t* experts,
                   const float* shares, const void* w13_codes, const void* w13_scales,
                   const void* w2_codes, const void* w2_scales, int64_t H, int64_t I, int64_t E,
                   int64_t top_k, void* y, int64_t ldy, int y_type, void* workspace,
                   size_t workspace_bytes, void* stream) {
    return moe(x, T, ldx, nullptr, E, experts, shares, mat(w13_codes, w13_scales),
               mat(w2_codes, w2_scales), H, I, E, top_k, 0, y, ldy, y_type, workspace,
               workspace_bytes, stream);
}

int mx4_route(const void* logits, int logits_type, int64_t T, int64_t E, int64_t ldl,
              const float* bias, int score, int64_t groups, int64_t kept_groups, int group_terms,
              int64_t top_k, int renormalize, float scale, int32_t* experts, float* shares,
              void* stream) {
    if (T < 0 || E < 1 || top_k < 1 || top_k > E || groups < 1 || E % groups != 0 ||
        kept_groups < 1 || kept_groups > groups || group_terms < 1 || group_terms > 2)
        return W12_ERR_SHAPE;
    if (T > MX4_MAX_ROUTE_T || E > MX4_MAX_E || top_k > MX4_MAX_TOP_K || groups > MX4_MAX_GROUPS)
        return W12_ERR_UNSUPPORTED;
    if (type_bytes(logits_type) == 0) return W12_ERR_DTYPE;
    if (score != MX4_SCORE_SOFTMAX && score != MX4_SCORE_SIGMOID) return W12_ERR_DTYPE;
    if (T > 0 && (!logits || !experts || !shares)) return W12_ERR_NULL;
    if (ldl < E || ldl >= kMaxElems) return W12_ERR_SHAPE;
    if (!aligned(logits, (uintptr_t)type_bytes(logits_type)) || !aligned(bias, 4) ||
        !aligned(experts, 4) || !aligned(shares, 4))
        return W12_ERR_ALIGN;
    if (T == 0) return W12_OK;
    mx4::RouteArgs a{};
    a.logits = logits;
    a.f32 = logits_type == W12_OUT_F32;
    a.T = T;
    a.ldl = ldl;
    a.E = (int)E;
    a.top_k = (int)top_k;
    a.bias = bias;
    a.sigmoid = score == MX4_SCORE_SIGMOID;
    a.groups = (int)groups;
    a.kept = (int)kept_groups;
    a.terms = group_terms;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    a.experts = experts;
    a.shares = shares;
    return status_of(mx4::launch_pick(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
