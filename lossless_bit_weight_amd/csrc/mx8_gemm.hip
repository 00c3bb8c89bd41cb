// mx8_gemm.hip -- y = x W^T with W in MX4 and x in MX8 (../../include/mx8.h).
//
// The matrix instruction takes 16 x 128 of 4-bit values against 128 x 16 of 8-bit
// ones, with a scale a lane on each side.  Lane 16 q + c holds weight row c's piece
// k = 32 q .. + 31 (as stored), and of x's row c the halves k = 16 q .. + 15 and
// 64 + 16 q .. + 15; its scale is that of row c's block q on either side.  The result has
// lane (c, q) holding weight rows 4 q .. 4 q + 3 for row c of x.
// Inside, products of eight neighbours in k meet first, without what lies more than 13
// bits below the largest one's exponent (1 + 2^-14 in one eight gives 1, across eights it
// holds to 2^-23).  What mx8_quantize writes never reaches that far: K = 17376 of normal
// values gives sums that are 0 off the exact ones' fp32 rounding; with all of E4M3's
// finest steps they were 4.5e-6 off.
#include <type_traits>

#include "mx8_internal.hpp"

namespace mx8 {
namespace {

using mx4::kCodeBlock;
using mx4::kScaleBlock;
using mx4::scalar;
using mx4::tiles;

__device__ __forceinline__ void store_y(const GemmArgs& a, int64_t m, int64_t n, float v) {
    if (a.y_f32)
        static_cast<float*>(a.y)[m * a.ldy + n] = v;
    else
        static_cast<uint16_t*>(a.y)[m * a.ldy + n] = mx4::bf16_bits(v);
}

template <int J>
__device__ __forceinline__ f32x4_t mfma(u32x4_t w, u32x4_t x0, u32x4_t x1, f32x4_t c, uint32_t sw,
                                        uint32_t sx) {
    const i32x8_t b = {(int)x0[0], (int)x0[1], (int)x0[2], (int)x0[3],
                       (int)x1[0], (int)x1[1], (int)x1[2], (int)x1[3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx4::operand4(w), b, c, 4, 0, J, (int)sw,
                                                            J, (int)sx);
}

// ---- a few rows of x, read by every wave ----------------------------------------
// Up to 16 rows of x a workgroup: its KW waves split K between them, by quads of
// groups, and each streams R tiles of 16 weight rows.  The waves' sums meet in LDS in
// wave order.  No load takes a branch: a group or row past the last is the last one
// again, with zeros for x.
template <int R, int KW>
__global__ __launch_bounds__(KW * 64) void small_kernel(GemmArgs a) {
    __shared__ f32x4_t red[KW][R][64];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int64_t last = tiles(a.N) - 1;
    const int64_t tile0 = (int64_t)blockIdx.x * R;
    const int m0 = blockIdx.y * 16;
    const int q0 = (int)((int64_t)a.Q * w / KW), q1 = (int)((int64_t)a.Q * (w + 1) / KW);

    const uint8_t* wp[R];
    const uint8_t* sp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t t = tile0 + r < last ? tile0 + r : last;
        wp[r] = a.w.codes + t * a.G * kCodeBlock + lane * 16;
        sp[r] = a.w.scales + t * a.Q * kScaleBlock + lane * 4;
    }
    const int64_t m = m0 + c < a.M ? m0 + c : a.M - 1;
    const uint8_t* xp = a.x + m * a.ldv;
    const uint8_t* xs = a.xs + m * a.lds + 4 * q;

    f32x4_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
    for (int Qi = q0; Qi < q1; ++Qi) {
        u32x4_t wb[4][R], xb[4][2];
        uint32_t ws[R];
        const uint32_t xsc = *reinterpret_cast<const uint32_t*>(xs + 16 * (int64_t)Qi);
#pragma unroll
        for (int r = 0; r < R; ++r)
            ws[r] = *reinterpret_cast<const uint32_t*>(sp[r] + (int64_t)Qi * kScaleBlock);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int g = 4 * Qi + j < a.G ? 4 * Qi + j : a.G - 1;
#pragma unroll
            for (int r = 0; r < R; ++r) wb[j][r] = mx4::load16_nt(wp[r] + (int64_t)g * kCodeBlock);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 512 * Qi + 128 * j + 64 * h + 16 * q;
                const bool in = k < a.K;
                xb[j][h] = *reinterpret_cast<const u32x4_t*>(xp + (in ? k : 0));
#pragma unroll
                for (int e = 0; e < 4; ++e) xb[j][h][e] = in ? xb[j][h][e] : 0u;
            }
        }
        auto group = [&](auto jc) {
            constexpr int J = decltype(jc)::value;
#pragma unroll
            for (int r = 0; r < R; ++r)
                acc[r] = mfma<J>(wb[J][r], xb[J][0], xb[J][1], acc[r], ws[r], xsc);
        };
        group(std::integral_constant<int, 0>{});
        group(std::integral_constant<int, 1>{});
        group(std::integral_constant<int, 2>{});
        group(std::integral_constant<int, 3>{});
    }

#pragma unroll
    for (int r = 0; r < R; ++r) red[w][r][lane] = acc[r];
    __syncthreads();
    const float* rf = reinterpret_cast<const float*>(red);
    for (int i = threadIdx.x; i < 256 * R; i += KW * 64) {
        const int row = i / (16 * R), col = i % (16 * R);
        const int r = col >> 4, wr = col & 15;
        const int64_t nn = tile0 * 16 + col;
        if (m0 + row >= a.M || nn >= a.N) continue;
        const int at = r * 256 + ((wr >> 2) * 16 + row) * 4 + (wr & 3);
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < KW; ++v) s += rf[v * R * 256 + at];
        store_y(a, m0 + row, nn, s);
    }
}

template <int R, int KW>
hipError_t launch_small(const GemmArgs& a, hipStream_t s) {
    const int64_t mb = tiles(a.M);
    const int64_t per = 65535;          // row blocks of a launch (its grid's y)
    for (int64_t b = 0; b < mb; b += per) {
        GemmArgs p = a;
        p.x += b * 16 * a.ldv;
        p.xs += b * 16 * a.lds;
        p.M = (int)(a.M - b * 16);
        p.y = static_cast<uint8_t*>(a.y) + b * 16 * a.ldy * (a.y_f32 ? 4 : 2);
        const dim3 grid((unsigned)((tiles(a.N) + R - 1) / R),
                        (unsigned)(mb - b < per ? mb - b : per));
        hipLaunchKernelGGL((small_kernel<R, KW>), grid, dim3(KW * 64), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace

size_t gemm_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm(GemmArgs a, void*, hipStream_t s) { return launch_small<2, 4>(a, s); }

}  // namespace mx8
