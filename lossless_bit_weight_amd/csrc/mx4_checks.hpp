// mx4_checks.hpp -- host-side argument checks that the C entry points of the MX4
// containers and of the calls beside them share.
#pragma once

#include <stdint.h>

#include "../../include/mx4.h"
#include "mx4_internal.hpp"

namespace mx4 {

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

inline bool aligned(const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

inline int check_container(int64_t B, int64_t R, int64_t K) {
    if (B < 1 || R < 0 || K < MX4_BLOCK || K % MX4_BLOCK != 0 || K >= kMaxK) return W12_ERR_SHAPE;
    if (R >= kMaxElems || B >= kMaxElems) return W12_ERR_SHAPE;
    const int64_t per = quads(K) * 8192;       // padded values of one tile
    if (tiles(R) > kMaxElems / per) return W12_ERR_SHAPE;
    if (tiles(R) > 0 && B > kMaxElems / per / tiles(R)) return W12_ERR_SHAPE;
    return W12_OK;
}

inline int check_gemm_shape(int64_t M, int64_t N, int64_t K) {
    if (N < 1 || M < 0 || M > kMaxM || N > kMaxN) return W12_ERR_SHAPE;
    if (M > 0 && N > kMaxMN / M) return W12_ERR_SHAPE;
    return check_container(1, N, K);
}

inline int type_bytes(int t) { return t == W12_OUT_F32 ? 4 : t == W12_OUT_BF16 ? 2 : 0; }

// rows of K values with strides ldx, ldb that start on 16 bytes
inline int check_rows(const void* p, int type, int64_t B, int64_t K, int64_t ld, int64_t ldb) {
    const int64_t n = 16 / type_bytes(type);
    if (ld < K || ld >= kMaxElems || (B > 1 && (ldb < 0 || ldb >= kMaxElems))) return W12_ERR_SHAPE;
    if (!aligned(p, 16) || ld % n != 0 || (B > 1 && ldb % n != 0)) return W12_ERR_ALIGN;
    return W12_OK;
}

// B matrices of R rows that share no value: one behind the other, or all of them
// between two rows of one (matrices that overlap would be written twice)
inline bool apart(int64_t B, int64_t R, int64_t K, int64_t ld, int64_t ldb) {
    if (ldb < K) return false;
    return (ldb - K) / ld >= R - 1 || (ld - K) / ldb >= B - 1;      // ld >= K >= 1
}

inline int check_y(const void* y, int64_t N, int64_t ldy, int y_type) {
    if (type_bytes(y_type) == 0) return W12_ERR_DTYPE;
    if (ldy < N || ldy >= kMaxElems) return W12_ERR_SHAPE;
    if (!aligned(y, (uintptr_t)type_bytes(y_type))) return W12_ERR_ALIGN;
    return W12_OK;
}

inline int check_ws(const void* ws, size_t have, size_t need) {
    if (need == 0) return W12_OK;
    return ws == nullptr || have < need || !aligned(ws, 256) ? W12_ERR_WORKSPACE : W12_OK;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? W12_OK : W12_ERR_HIP; }

inline Mat mat(const void* codes, const void* scales) {
    return Mat{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales)};
}

}  // namespace mx4
