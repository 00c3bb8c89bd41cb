// mx4_codec.hip -- BF16 or fp32 values to MX4 containers and back
// (../../include/mx4.h has the format).
//
// Per block of 32: e = max(0, E - 2) with E the largest biased exponent, codes
// the nearest of {0, .5, 1, 1.5, 2, 3, 4, 6} to |v| / 2^(e - 127), ties to even.
// The largest magnitude lies in [4, 8) * 2^(e - 127), so the top binade uses
// the codes 4 and 6 and what lies above 6 saturates.  v_cvt_scalef32_pk_fp4
// does the division, rounding and saturation of two values at once (checked
// here against the formula for every BF16 value).
//
// A wave takes 4 rows x 512 values: in step j lane 16 r + p holds the 8 values
// 128 j + 8 p .. of row r, so every load reads 256 (fp32 512) contiguous bytes
// a row, the four lanes of a block agree on its largest exponent in two
// quad permutes, and after four steps one lane of each block holds the scale
// dword.  The four waves of a workgroup fill one tile's 4 KB of codes and 256
// bytes of scales.  Bound by memory: 2 (4) + 0.53 bytes a value.
#include "mx4_internal.hpp"

namespace mx4 {
namespace {

constexpr int kThreads = 256;

// A grid's x holds fewer than 2^24 workgroups of 256 (work items are counted in 32
// bits); more go along y.
constexpr int64_t kGridX = (int64_t)1 << 22;
dim3 grid_of(int64_t blocks) {
    return blocks <= kGridX ? dim3((unsigned)blocks)
                            : dim3((unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t block_index() {
    return (int64_t)blockIdx.y * kGridX + blockIdx.x;
}

// max over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);   // 1 0 3 2
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);            // 2 3 0 1
    return v > o ? v : o;
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <bool F32>
struct Values;

template <>
struct Values<false> {
    u32x4_t v;
    __device__ void clear() { v = u32x4_t{0, 0, 0, 0}; }
    __device__ void load(const void* x, int64_t i) {
        v = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(x) + i);
    }
    // largest biased exponent of the eight
    __device__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = max_u32(m, max_u32(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
        return m >> 7;
    }
    __device__ uint32_t encode(float s) const {
        // by value: __builtin_bit_cast of a vector's element reads element 0
        const uint32_t v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
        uint32_t d = 0;
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf16x2_t, v0), s, 0);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf16x2_t, v1), s, 1);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf16x2_t, v2), s, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(d, __builtin_bit_cast(bf16x2_t, v3), s, 3);
        return d;
    }
};

template <>
struct Values<true> {
    f32x4_t a, b;
    __device__ void clear() { a = b = f32x4_t{0, 0, 0, 0}; }
    __device__ void load(const void* x, int64_t i) {
        const float* p = static_cast<const float*>(x) + i;
        a = *reinterpret_cast<const f32x4_t*>(p);
        b = *reinterpret_cast<const f32x4_t*>(p + 4);
    }
    __device__ uint32_t top() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = max_u32(m, max_u32(__float_as_uint(a[i]) & 0x7FFFFFFFu,
                                   __float_as_uint(b[i]) & 0x7FFFFFFFu));
        return m >> 23;
    }
    __device__ uint32_t encode(float s) const {
        uint32_t d = 0;
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, a[0], a[1], s, 0);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, a[2], a[3], s, 1);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, b[0], b[1], s, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, b[2], b[3], s, 3);
        return d;
    }
};

template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ x, int64_t R,
                                                            int64_t K, int64_t ldx, int64_t ldb,
                                                            int G, int Q, int64_t tiles_mat,
                                                            int64_t blocks,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
    const int64_t block = block_index();
    if (block >= blocks) return;
    const int64_t T = block / Q;                    // tile over all matrices
    const int Qi = (int)(block % Q);
    const int64_t mat = T / tiles_mat;
    const int lane = threadIdx.x & 63;
    const int c = (threadIdx.x >> 6) * 4 + (lane >> 4);   // row of the tile
    const int p = lane & 15;
    const int piece = 16 * (p >> 2) + c;
    const int64_t r = (T - mat * tiles_mat) * 16 + c;
    const int64_t k0 = (int64_t)Qi * 512 + 8 * p;
    const int64_t at = mat * ldb + r * ldx + k0;

    Values<F32> v[4];
    bool in[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        in[j] = r < R && k0 + 128 * j < K;          // a block lies inside or outside as a whole
        v[j].clear();
        if (in[j]) v[j].load(x, at + 128 * j);
    }
    uint32_t scale_word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t E = quad_max(v[j].top());
        const bool bad = E == 255u;                 // an infinity or a NaN in the block
        uint32_t e = E > 2u ? E - 2u : 0u;
        uint32_t d = v[j].encode(scale_f32(e));
        if (bad) {
            e = 255u;
            d = 0u;
        }
        if (!in[j]) e = 127u;
        scale_word |= e << (8 * j);
        const int g = 4 * Qi + j;
        if (g < G)
            *reinterpret_cast<uint32_t*>(codes + (T * G + g) * kCodeBlock + piece * 16 +
                                         4 * (p & 3)) = d;
    }
    if ((p & 3) == 0)
        *reinterpret_cast<uint32_t*>(scales + (T * Q + Qi) * kScaleBlock + piece * 4) = scale_word;
}

// The inverse.  A lane writes 16 contiguous bytes at a time, the 16 lanes of a row
// 256: eight BF16 from one dword of codes, or twice four fp32 from half a dword
// (as 32 bytes a lane, fp32 wrote half lines: 100 us for 5119 x 17408 values,
// now 77, and 66 past the caches, which the output would only flush).
__device__ __forceinline__ void store16(void* p, u32x4_t v) {
    __builtin_nontemporal_store(v, static_cast<u32x4_t*>(p));
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(Mat m, int64_t R, int64_t K, int G,
                                                              int Q, int64_t tiles_mat,
                                                              int64_t blocks,
                                                              void* __restrict__ y, int64_t ldy,
                                                              int64_t ldb) {
    const int64_t block = block_index();
    if (block >= blocks) return;
    const int64_t T = block / Q;
    const int Qi = (int)(block % Q);
    const int64_t mat = T / tiles_mat;
    const int lane = threadIdx.x & 63;
    const int c = (threadIdx.x >> 6) * 4 + (lane >> 4);
    const int p = lane & 15;
    const int64_t r = (T - mat * tiles_mat) * 16 + c;
    if (r >= R) return;
    const int64_t k0 = (int64_t)Qi * 512;
    const int64_t at = mat * ldb + r * ldy + k0;
    const uint8_t* codes = m.codes + (T * G + 4 * Qi) * kCodeBlock;
    const uint8_t* scales = m.scales + (T * Q + Qi) * kScaleBlock;

    if constexpr (F32) {
        // chunk h of a group: values 64 h + 4 p .. + 3, in piece (2 h + p / 8, c)
        uint32_t d[4][2], sw[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int piece = 16 * (2 * h + (p >> 3)) + c;
            sw[h] = *reinterpret_cast<const uint32_t*>(scales + piece * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j][h] = 0;
                if (k0 + 128 * j + 64 * h + 4 * p < K)
                    d[j][h] = *reinterpret_cast<const uint16_t*>(
                        codes + j * kCodeBlock + piece * 16 + 2 * (p & 7));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 128 * j + 64 * h + 4 * p;
                if (k0 + k >= K) continue;
                const float s = scale_f32((sw[h] >> (8 * j)) & 255u);
                const f32x2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d[j][h], s, 0);
                const f32x2_t v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d[j][h], s, 1);
                const f32x4_t v = {v0[0], v0[1], v1[0], v1[1]};
                store16(static_cast<float*>(y) + at + k, __builtin_bit_cast(u32x4_t, v));
            }
    } else {
        const int piece = 16 * (p >> 2) + c;
        uint32_t d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            d[j] = 0;
            if (k0 + 128 * j + 8 * p < K)
                d[j] = *reinterpret_cast<const uint32_t*>(codes + j * kCodeBlock + piece * 16 +
                                                          4 * (p & 3));
        }
        const uint32_t scale_word = *reinterpret_cast<const uint32_t*>(scales + piece * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = 128 * j + 8 * p;
            if (k0 + k >= K) continue;
            const bf16x8_t v = expand8(d[j], scale_f32((scale_word >> (8 * j)) & 255u));
            store16(static_cast<uint16_t*>(y) + at + k, __builtin_bit_cast(u32x4_t, v));
        }
    }
}

}  // namespace

hipError_t launch_quantize(const void* x, int x_f32, int64_t B, int64_t R, int64_t K, int64_t ldx,
                           int64_t ldb, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    const int G = (int)groups(K), Q = (int)quads(K);
    const int64_t tm = tiles(R);
    const int64_t blocks = B * tm * Q;
    const dim3 grid = grid_of(blocks);
    if (x_f32)
        hipLaunchKernelGGL(quantize_kernel<true>, grid, dim3(kThreads), 0, s, x, R, K, ldx, ldb, G,
                           Q, tm, blocks, codes, scales);
    else
        hipLaunchKernelGGL(quantize_kernel<false>, grid, dim3(kThreads), 0, s, x, R, K, ldx, ldb, G,
                           Q, tm, blocks, codes, scales);
    return hipGetLastError();
}

hipError_t launch_dequantize(Mat m, int64_t B, int64_t R, int64_t K, void* y, int y_f32,
                             int64_t ldy, int64_t ldb, hipStream_t s) {
    const int G = (int)groups(K), Q = (int)quads(K);
    const int64_t tm = tiles(R);
    const int64_t blocks = B * tm * Q;
    const dim3 grid = grid_of(blocks);
    if (y_f32)
        hipLaunchKernelGGL(dequantize_kernel<true>, grid, dim3(kThreads), 0, s, m, R, K, G, Q, tm,
                           blocks, y, ldy, ldb);
    else
        hipLaunchKernelGGL(dequantize_kernel<false>, grid, dim3(kThreads), 0, s, m, R, K, G, Q, tm,
                           blocks, y, ldy, ldb);
    return hipGetLastError();
}

}  // namespace mx4
