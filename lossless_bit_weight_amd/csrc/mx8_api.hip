// mx8_api.hip -- the C ABI declared in include/mx8.h and include/mx8_plan.h: host-side
// argument checks and launches on the caller's stream.  Nothing here allocates, synchronises or
// keeps state.
#include <stdint.h>

#include "../../include/mx8.h"
#include "../../include/mx8_plan.h"
#include "mx4_checks.hpp"
#include "mx8_internal.hpp"

using namespace mx4;

namespace {

// R rows of values and of scales
int check_mx8(const void* values, int64_t ldv, const void* scales, int64_t lds, int64_t K) {
    if (ldv < K || ldv >= kMaxElems || lds < mx8::scale_row(K) || lds >= kMaxElems)
        return W12_ERR_SHAPE;
    if (!aligned(values, 16) || !aligned(scales, 16) || ldv % 16 != 0 || lds % 16 != 0)
        return W12_ERR_ALIGN;
    return W12_OK;
}

int codec(const void* x, int x_type, int64_t R, int64_t K, int64_t ldx, const void* values,
          int64_t ldv, const void* scales, int64_t lds) {
    if (int rc = check_container(1, R, K)) return rc;
    if (type_bytes(x_type) == 0) return W12_ERR_DTYPE;
    if (R > 0 && (!x || !values || !scales)) return W12_ERR_NULL;
    if (int rc = check_rows(x, x_type, 1, K, ldx, 0)) return rc;
    return check_mx8(values, ldv, scales, lds, K);
}

}  // namespace

extern "C" {

const char* mx8_status_string(int status) {
    switch (status) {
        case W12_OK: return "ok";
        case W12_ERR_NULL: return "a required pointer is NULL";
        case W12_ERR_SHAPE:
            return "bad shape (K is a positive multiple of 32 below 2^24, N >= 1, strides cover "
                   "their rows)";
        case W12_ERR_ALIGN:
            return "misaligned pointer or stride (16-byte rows of x, values and scales)";
        case W12_ERR_DTYPE: return "unknown element type";
        case W12_ERR_UNSUPPORTED: return "more values a row than mx8_rms_norm takes";
        case W12_ERR_HIP: return "HIP launch failed";
        case W12_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
        default: return "unknown status";
    }
}

size_t mx8_scale_row_bytes(int64_t K) {
    return check_container(1, 0, K) == W12_OK ? (size_t)mx8::scale_row(K) : 0;
}

int mx8_quantize(const void* x, int x_type, int64_t R, int64_t K, int64_t ldx, void* values,
                 int64_t ldv, void* scales, int64_t lds, void* stream) {
    const bool fine = (x_type & MX8_FINE_STEPS) != 0;
    x_type &= ~MX8_FINE_STEPS;
    if (int rc = codec(x, x_type, R, K, ldx, values, ldv, scales, lds)) return rc;
    if (R == 0) return W12_OK;
    return status_of(mx8::launch_quantize(x, x_type == W12_OUT_F32, mx8::quarters_below(fine), R, K,
                                          ldx, static_cast<uint8_t*>(values), ldv,
                                          static_cast<uint8_t*>(scales), lds,
                                          static_cast<hipStream_t>(stream)));
}

int mx8_dequantize(const void* values, int64_t ldv, const void* scales, int64_t lds, int64_t R,
                   int64_t K, void* y, int y_type, int64_t ldy, void* stream) {
    if (int rc = codec(y, y_type, R, K, ldy, values, ldv, scales, lds)) return rc;
    if (R == 0) return W12_OK;
    return status_of(mx8::launch_dequantize(static_cast<const uint8_t*>(values), ldv,
                                            static_cast<const uint8_t*>(scales), lds, R, K, y,
                                            y_type == W12_OUT_F32, ldy,
                                            static_cast<hipStream_t>(stream)));
}

int mx8_rms_norm(const void* x, int x_type, int64_t ldx, const void* residual, void* residual_out,
                 int res_type, int64_t ldr, int64_t ldo, const void* weight, int w_type, float eps,
                 int64_t M, int64_t K, void* y, int y_type, int64_t ldy, void* y_scales,
                 int64_t lds, void* stream) {
    if (M < 0 || M > kMaxM) return W12_ERR_SHAPE;
    if (int rc = check_container(1, M, K)) return rc;
    if (K > MX8_MAX_NORM_K) return W12_ERR_UNSUPPORTED;
    const bool fine = y_type == (MX8_OUT | MX8_FINE_STEPS), out8 = fine || y_type == MX8_OUT;
    if (type_bytes(x_type) == 0 || type_bytes(w_type) == 0 || (!out8 && type_bytes(y_type) == 0))
        return W12_ERR_DTYPE;
    if (residual != nullptr && type_bytes(res_type) == 0) return W12_ERR_DTYPE;
    if (!weight || (M > 0 && (!x || !y || (out8 && !y_scales) || (residual && !residual_out))))
        return W12_ERR_NULL;
    if (int rc = check_rows(x, x_type, 1, K, ldx, 0)) return rc;
    if (residual != nullptr) {
        if (int rc = check_rows(residual, res_type, 1, K, ldr, 0)) return rc;
        if (int rc = check_rows(residual_out, res_type, 1, K, ldo, 0)) return rc;
    }
    if (out8) {
        if (int rc = check_mx8(y, ldy, y_scales, lds, K)) return rc;
    } else if (int rc = check_rows(y, y_type, 1, K, ldy, 0)) {
        return rc;
    }
    if (!aligned(weight, 16)) return W12_ERR_ALIGN;
    if (M == 0) return W12_OK;
    mx8::NormArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.res = residual;
    a.res_out = residual_out;
    a.ldr = ldr;
    a.ldo = ldo;
    a.w = weight;
    a.eps = eps;
    a.M = M;
    a.K = (int)K;
    a.y = y;
    a.ldy = ldy;
    a.ys = static_cast<uint8_t*>(y_scales);
    a.lds = lds;
    a.x_f32 = x_type == W12_OUT_F32;
    a.res_f32 = res_type == W12_OUT_F32;
    a.w_f32 = w_type == W12_OUT_F32;
    a.y_type = fine ? 3 : y_type;
    return status_of(mx8::launch_norm(a, static_cast<hipStream_t>(stream)));
}

int mx8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
    if (bytes == nullptr) return W12_ERR_NULL;
    *bytes = 0;
    if (int rc = check_gemm_shape(M, N, K)) return rc;
    if (M > 0) *bytes = mx8::plan_gemm(M, N, K).workspace;
    return W12_OK;
}

const char* mx8_gemm_plan(int64_t M, int64_t N, int64_t K, int* slices) {
    if (slices != nullptr) *slices = 0;
    if (M < 1 || check_gemm_shape(M, N, K) != W12_OK) return nullptr;
    const mx8::Plan plan = mx8::plan_gemm(M, N, K);
    if (slices != nullptr) *slices = plan.S;
    return mx8::kernel_name(plan);
}

int mx8_gemm(const void* x_values, int64_t ldv, const void* x_scales, int64_t lds, int64_t M,
             const void* w_codes, const void* w_scales, int64_t N, int64_t K, void* y, int64_t ldy,
             int y_type, void* workspace, size_t workspace_bytes, void* stream) {
    if (!w_codes || !w_scales || (M > 0 && (!x_values || !x_scales || !y))) return W12_ERR_NULL;
    if (int rc = check_gemm_shape(M, N, K)) return rc;
    if (int rc = check_mx8(x_values, ldv, x_scales, lds, K)) return rc;
    if (ldv >= (int64_t)1 << 31 || lds >= (int64_t)1 << 31) return W12_ERR_SHAPE;
    if (int rc = check_y(y, N, ldy, y_type)) return rc;
    if (!aligned(w_codes, 16) || !aligned(w_scales, 16)) return W12_ERR_ALIGN;
    if (M == 0) return W12_OK;
    const mx8::Plan plan = mx8::plan_gemm(M, N, K);
    if (int rc = check_ws(workspace, workspace_bytes, plan.workspace)) return rc;
    mx8::GemmArgs a{};
    a.x = static_cast<const uint8_t*>(x_values);
    a.xs = static_cast<const uint8_t*>(x_scales);
    a.ldv = ldv;
    a.lds = lds;
    a.w = mat(w_codes, w_scales);
    a.M = (int)M;
    a.N = N;
    a.K = K;
    a.G = (int)groups(K);
    a.Q = (int)quads(K);
    a.y = y;
    a.ldy = ldy;
    a.y_f32 = y_type == W12_OUT_F32;
    return status_of(mx8::launch_gemm(a, plan, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
