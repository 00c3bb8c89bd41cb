// mx4_internal.hpp -- device helpers and launchers of the MX4 calls
// (../../include/mx4.h has the format).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx4 {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kBlock = 32;
constexpr int64_t kGroup = 128;        // K of one 1 KB code block
constexpr int kCodeBlock = 1024;       // bytes of codes a (tile, group)
constexpr int kScaleBlock = 256;       // bytes of scales a (tile, four groups)

__host__ __device__ inline int64_t groups(int64_t K) { return (K + kGroup - 1) / kGroup; }
__host__ __device__ inline int64_t quads(int64_t K) { return (K + 4 * kGroup - 1) / (4 * kGroup); }
__host__ __device__ inline int64_t tiles(int64_t R) { return (R + 15) / 16; }

// A container's codes and scales.
struct Mat {
    const uint8_t* codes;
    const uint8_t* scales;
};

// The conversions take the scale as the fp32 number 2^(e - 127); they read its
// exponent field alone, so e = 0 (2^-127) and e = 255 (NaN) need no case of
// their own.
__device__ __forceinline__ float scale_f32(uint32_t e) { return __uint_as_float(e << 23); }

// Eight codes (one dword of a piece) as BF16, exactly: the value's three
// significant bits and 2^-128 * 1 .. 2^128 fit BF16's normal and subnormal
// numbers (above, infinity).
__device__ __forceinline__ bf16x8_t expand8(uint32_t d, float s) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2);
    const bf16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3);
    return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// A piece as the 4-bit operand of the scaled matrix instructions, which read
// the first four of its eight registers.
__device__ __forceinline__ i32x8_t operand4(u32x4_t v) {
    return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

__device__ __forceinline__ f32x4_t mfma_bf16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 16x16x128 of two 4-bit operands (format 4) under the scales in byte J of sa
// and sb.
template <int J = 0>
__device__ __forceinline__ f32x4_t mfma_mx4(i32x8_t a, i32x8_t b, f32x4_t c, uint32_t sa,
                                            uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, J, (int)sa, J, (int)sb);
}

__device__ __forceinline__ u32x4_t load16_nt(const uint8_t* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
}

// A uniform pointer to global memory that the compiler keeps in scalar registers: folded
// with the lane's offset it would hold two vector registers through the loop.  (What is
// read through it must not look like a generic pointer: every wait for LDS would wait for
// flat loads too.)
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
    typedef const __attribute__((address_space(1))) uint8_t* global_t;
    global_t g = (global_t)p;
    asm volatile("" : "+s"(g));
    return (const uint8_t*)g;
}

template <bool NT>
__device__ __forceinline__ u32x4_t load16(const uint8_t* p) {
    if constexpr (NT) return load16_nt(p);
    return *reinterpret_cast<const u32x4_t*>(p);
}

// fp32 -> BF16 bits, to nearest even (NaN stays NaN).
__device__ __forceinline__ uint16_t bf16_bits(float f) {
    const __bf16 h = (__bf16)f;
    return __builtin_bit_cast(uint16_t, h);
}

// Odd rows of 16 lanes of a and even rows of b change places.
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// Place, of 16, of x's piece q, b (values 32 q + 8 b .. + 7 of a group) in LDS row
// `row`.  A read takes one b from 16 rows for each q; the LDS serves it 16 lanes
// at a time, rows 0-3 and 12-15 of one q with rows 4-11 of the next, whose places
// differ for this order of the pieces (with 4 q + b in front of the row's bits they
// coincide: a third of the LDS cycles of QKV M = 2048 were such conflicts).
__host__ __device__ constexpr int x_place(int q, int b, int row) {
    return (4 * b + q) ^ (row & 15);
}
// The same for piece p = 4 q + b.
__host__ __device__ constexpr int x_place(int p, int row) {
    return x_place((p >> 2) & 3, p & 3, row);
}

struct GemmArgs {
    const uint16_t* x;      // BF16 activations (or NULL: xm)
    int64_t ldx;
    Mat xm;
    Mat w;
    int M;
    int64_t N, K;
    int G, Q;               // groups of 128 and of 512 along K
    void* y;
    int64_t ldy;
    int y_f32;
    int S, gs;              // K slices over workgroups, groups a slice
    float* part;            // S > 1: partial sums [S][M][N]
};

hipError_t launch_quantize(const void* x, int x_f32, int64_t B, int64_t R, int64_t K, int64_t ldx,
                           int64_t ldb, uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_dequantize(Mat m, int64_t B, int64_t R, int64_t K, void* y, int y_f32,
                             int64_t ldy, int64_t ldb, hipStream_t s);
// Rows of x this far apart are past the tile kernel's row offsets, which are products of
// 24-bit numbers: the few-row kernel takes them, up to kMaxFarRows (its grid's y).
constexpr int64_t kFarRows = (int64_t)1 << 23;
constexpr int64_t kMaxFarRows = 65535 * 16;
size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, bool x_mx4);
hipError_t launch_gemm(GemmArgs a, void* ws, hipStream_t s);

// ---- expert layer --------------------------------------------------------------
constexpr int kMaxTokens = 128;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;

// Up to 16 of the pairs (token, chosen expert) of one expert: words [0] the
// expert, [1] their number (0: none, nothing to do), [2] the first pair's place
// among all, [16 + i] the i-th pair's token (past the last: the first's).  Where
// tokens go one by one a slot is a pair: words 0 and [3], the expert's share (fp32).
constexpr int kSlotWords = 32;

struct MoeArgs {
    const uint16_t* x;
    int64_t ldx;
    const float* logits;
    int64_t ldl;
    const int* chosen;      // or, without logits, each token's experts [T][top_k] and
    const float* given;     // their shares
    Mat w13, w2;
    int T, H, I, E, top_k, renormalize;
    void* y;
    int64_t ldy;
    int y_f32;
    int max_slots;          // min(E, pairs) + pairs / 16, or pairs
    // workspace: the pairs in the order of (expert, token), cut into slots (tokens one by
    // one: slots and h only)
    int* slots;             // [max_slots][kSlotWords]
    int* place;             // [T][top_k] place of token t's j-th pair, or -1
    float* share;           // [T][top_k]
    float* out;             // [pairs][H] an expert's output for a token
    void* h;                // hidden values: [pairs][I] fp32, or (y_f32) BF16 parts [3][pairs][I]
};

size_t moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k, bool y_f32);
// Point the workspace fields of `a` at `ws` (moe_workspace_bytes) and launch.
hipError_t launch_moe(MoeArgs a, void* ws, hipStream_t s);

// ---- routing (../../include/mx4_route.h) ----------------------------------------
struct RouteArgs {
    const void* logits;
    int f32;
    int64_t T, ldl;
    int E, top_k;
    const float* bias;
    int sigmoid, groups, kept, terms, renormalize;
    float scale;
    int* experts;
    float* shares;
};
hipError_t launch_pick(const RouteArgs& a, hipStream_t s);

}  // namespace mx4
