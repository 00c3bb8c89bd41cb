// mx4_api.hip -- the C ABI declared in include/mx4.h: host-side argument checks
// and launches on the caller's stream.  Nothing here allocates, synchronises or
// keeps state.
#include <stdint.h>

#include "../../include/mx4.h"
#include "mx4_internal.hpp"

namespace {

// Padded values of a container: keeps every grid far below 2^31 blocks and
// every byte offset inside int64.  K below 2^24 keeps group indices and the
// kernels' in-row offsets in 32 bits.
constexpr int64_t kMaxElems = (int64_t)1 << 40;
constexpr int64_t kMaxK = (int64_t)1 << 24;
constexpr int64_t kMaxM = (int64_t)1 << 24;
// A launch counts its work items along x in 32 bits: N and M * N up to these keep
// every product's grid within (2^27 / 32 workgroups of 512 in the few-row kernel).
constexpr int64_t kMaxN = (int64_t)1 << 27;
constexpr int64_t kMaxMN = (int64_t)1 << 37;
// The same for the expert layer: slots times tiles of its outputs.
constexpr int64_t kMaxMoeBlocks = (int64_t)1 << 24;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_container(int64_t B, int64_t R, int64_t K) {
    if (B < 1 || R < 0 || K < MX4_BLOCK || K % MX4_BLOCK != 0 || K >= kMaxK) return W12_ERR_SHAPE;
    if (R >= kMaxElems || B >= kMaxElems) return W12_ERR_SHAPE;
    const int64_t per = mx4::quads(K) * 8192;       // padded values of one tile
    if (mx4::tiles(R) > kMaxElems / per) return W12_ERR_SHAPE;
    if (mx4::tiles(R) > 0 && B > kMaxElems / per / mx4::tiles(R)) return W12_ERR_SHAPE;
    return W12_OK;
}

int type_bytes(int t) { return t == W12_OUT_F32 ? 4 : t == W12_OUT_BF16 ? 2 : 0; }

// rows of K values with strides ldx, ldb that start on 16 bytes
int check_rows(const void* p, int type, int64_t B, int64_t K, int64_t ld, int64_t ldb) {
    const int64_t n = 16 / type_bytes(type);
    if (ld < K || ld >= kMaxElems || (B > 1 && (ldb < 0 || ldb >= kMaxElems))) return W12_ERR_SHAPE;
    if (!aligned(p, 16) || ld % n != 0 || (B > 1 && ldb % n != 0)) return W12_ERR_ALIGN;
    return W12_OK;
}

// B matrices of R rows that share no value: one behind the other, or all of them
// between two rows of one (matrices that overlap would be written twice)
bool apart(int64_t B, int64_t R, int64_t K, int64_t ld, int64_t ldb) {
    if (ldb < K) return false;
    return (ldb - K) / ld >= R - 1 || (ld - K) / ldb >= B - 1;      // ld >= K >= 1
}

int check_y(const void* y, int64_t N, int64_t ldy, int y_type) {
    if (type_bytes(y_type) == 0) return W12_ERR_DTYPE;
    if (ldy < N || ldy >= kMaxElems) return W12_ERR_SHAPE;
    if (!aligned(y, (uintptr_t)type_bytes(y_type))) return W12_ERR_ALIGN;
    return W12_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
    if (need == 0) return W12_OK;
    return ws == nullptr || have < need || !aligned(ws, 256) ? W12_ERR_WORKSPACE : W12_OK;
}

int status_of(hipError_t e) { return e == hipSuccess ? W12_OK : W12_ERR_HIP; }

int check_gemm_shape(int64_t M, int64_t N, int64_t K) {
    if (N < 1 || M < 0 || M > kMaxM || N > kMaxN) return W12_ERR_SHAPE;
    if (M > 0 && N > kMaxMN / M) return W12_ERR_SHAPE;
    return check_container(1, N, K);
}

mx4::Mat mat(const void* codes, const void* scales) {
    return mx4::Mat{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales)};
}

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

int mx4_moe(const uint16_t* x, int64_t T, int64_t ldx, const float* logits, int64_t ldl,
            const void* w13_codes, const void* w13_scales, const void* w2_codes,
            const void* w2_scales, int64_t H, int64_t I, int64_t E, int64_t top_k, int renormalize,
            void* y, int64_t ldy, int y_type, void* workspace, size_t workspace_bytes,
            void* stream) {
    if (!w13_codes || !w13_scales || !w2_codes || !w2_scales) return W12_ERR_NULL;
    if (T > 0 && (!x || !logits || !y)) return W12_ERR_NULL;
    if (int rc = check_moe_shape(T, H, I, E, top_k)) return rc;
    if (int rc = check_rows(x, W12_OUT_BF16, 1, H, ldx, 0)) return rc;
    if (int rc = check_y(y, H, ldy, y_type)) return rc;
    if (ldl < E || ldl >= kMaxElems) return W12_ERR_SHAPE;
    if (!aligned(logits, 4) || !aligned(w13_codes, 16) || !aligned(w13_scales, 16) ||
        !aligned(w2_codes, 16) || !aligned(w2_scales, 16))
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
    a.w13 = mat(w13_codes, w13_scales);
    a.w2 = mat(w2_codes, w2_scales);
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

}  // extern "C"
