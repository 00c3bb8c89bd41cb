// mx8_internal.hpp -- device helpers and launchers of the MX8 calls
// (../../include/mx8.h has the format).
#pragma once

#include "mx4_internal.hpp"

namespace mx8 {

using mx4::f32x2_t;
using mx4::f32x4_t;
using mx4::i32x8_t;
using mx4::u32x2_t;
using mx4::u32x4_t;

// Bytes of a row's scales, and the place of the scale of the block that k lies in.
__host__ __device__ inline int64_t scale_row(int64_t K) { return 16 * mx4::quads(K); }
__host__ __device__ inline int scale_place(int k) {
    return (k >> 9) * 16 + ((k >> 5) & 3) * 4 + ((k >> 7) & 3);
}

// max over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);   // 1 0 3 2
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);            // 2 3 0 1
    return v > o ? v : o;
}

// Eight fp32 values of a row, and as many of BF16 or fp32 in memory.
struct Eight {
    float f[8];

    template <bool F32>
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        if constexpr (F32) {
            const float* s = static_cast<const float*>(p) + i;
            const f32x4_t a = *reinterpret_cast<const f32x4_t*>(s);
            const f32x4_t b = *reinterpret_cast<const f32x4_t*>(s + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j] = a[j];
                f[4 + j] = b[j];
            }
        } else {
            const u32x4_t v =
                *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = __uint_as_float(v[j] << 16);
                f[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
            }
        }
    }
    __device__ __forceinline__ u32x4_t bf16() const {
        u32x4_t v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = mx4::bf16_bits(f[2 * j]) | (uint32_t)mx4::bf16_bits(f[2 * j + 1]) << 16;
        return v;
    }
    template <bool F32>
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        if constexpr (F32) {
            float* d = static_cast<float*>(p) + i;
            *reinterpret_cast<f32x4_t*>(d) = f32x4_t{f[0], f[1], f[2], f[3]};
            *reinterpret_cast<f32x4_t*>(d + 4) = f32x4_t{f[4], f[5], f[6], f[7]};
        } else {
            *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i) = bf16();
        }
    }
    // As MX8: the four lanes of a quad hold one block between them.  The largest
    // magnitude lies in [256, 512) * 2^(e - 127); multiplying by the power of two is
    // exact (but for what rounds to zero anyway).  Below `quarters` (4, where E4M3 goes
    // finer; 0 for MX8_FINE_STEPS) values are rounded to multiples of 1/4 first (the header
    // says why); what is above 448 is brought there, as the conversion would make a NaN of it.
    __device__ __forceinline__ u32x2_t encode(uint32_t& e, float quarters) const {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(f[j]) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        }
        const uint32_t E = quad_max(top) >> 23;
        e = E > 8u ? E - 8u : 0u;
        const float s = __uint_as_float((254u - e) << 23);
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = f[j] * s;
            t[j] = __builtin_fabsf(v) < quarters ? __builtin_rintf(v * 4.f) * 0.25f
                                                 : __builtin_amdgcn_fmed3f(v, -448.f, 448.f);
        }
        u32x2_t v;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            int d = 0;
            d = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * j], t[4 * j + 1], d, false);
            d = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * j + 2], t[4 * j + 3], d, true);
            v[j] = E == 255u ? 0u : (uint32_t)d;
        }
        e = E == 255u ? 255u : e;
        return v;
    }
};

// Eight::encode's `quarters`, in units of the block.
__host__ __device__ constexpr float quarters_below(bool fine) { return fine ? 0.f : 4.f; }

struct NormArgs {
    const void* x;
    int64_t ldx;
    const void* res;
    void* res_out;
    int64_t ldr, ldo;
    const void* w;
    float eps;
    int64_t M;
    int K;
    void* y;
    int64_t ldy;
    uint8_t* ys;
    int64_t lds;
    int x_f32, res_f32, w_f32;
    int y_type;             // 0 BF16, 1 fp32, 2 MX8, 3 MX8 in fine steps
};

struct GemmArgs {
    const uint8_t* x;
    const uint8_t* xs;
    int64_t ldv, lds;
    mx4::Mat w;
    int M;
    int64_t N, K;
    int G, Q;               // groups of 128 and of 512 along K
    void* y;
    int64_t ldy;
    int y_f32;
    int S, gs;              // K slices over workgroups, groups a slice (a multiple of 4)
    float* part;            // S > 1: partial sums [S][M][N rounded up to 4]
};

hipError_t launch_quantize(const void* x, int x_f32, float quarters, int64_t R, int64_t K,
                           int64_t ldx, uint8_t* values, int64_t ldv, uint8_t* scales,
                           int64_t lds, hipStream_t s);
hipError_t launch_dequantize(const uint8_t* values, int64_t ldv, const uint8_t* scales,
                             int64_t lds, int64_t R, int64_t K, void* y, int y_f32, int64_t ldy,
                             hipStream_t s);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
// Kernel and split of a product.
struct Plan {
    int kernel, wn;         // one of mx8_gemm.hip's; its waves beside each other, if it chooses
    int S, gs;              // K slices, groups a slice (a multiple of 4)
    size_t workspace;       // bytes
};
Plan plan_gemm(int64_t M, int64_t N, int64_t K);
const char* kernel_name(const Plan& p);     // with its template arguments
hipError_t launch_gemm(GemmArgs a, const Plan& p, void* ws, hipStream_t s);

}  // namespace mx8
