// mx4_gemm.hip -- y = x W^T with W in MX4 and x in BF16 or MX4
// (../../include/mx4.h has the format).
#include "mx4_internal.hpp"

namespace mx4 {
namespace {

__device__ __forceinline__ void store_y(const GemmArgs& a, int64_t m, int64_t n, float v) {
    if (a.y_f32)
        static_cast<float*>(a.y)[m * a.ldy + n] = v;
    else
        static_cast<uint16_t*>(a.y)[m * a.ldy + n] = bf16_bits(v);
}

// ---- a few rows of x ----------------------------------------------------------
// Up to 16 rows of x a workgroup: its KW waves split K between them and each
// streams R tiles of 16 weight rows, D groups in flight.  Lane 16 q + c holds
// piece (c, q) of the weight block and, of x, row c's values of the same 32 k:
// with W as the first operand a matrix instruction's lane needs 8 k of its row
// (BF16: four instructions a piece, k = 32 q + 8 b + e in instruction b -- any
// one-to-one assignment of k serves, as long as both operands share it) or the
// whole piece (MX4: one instruction a group).  The result has lane (c, q)
// holding weight rows 4 q .. 4 q + 3 for row c of x.  The waves' sums meet in
// LDS in wave order.
template <int R, int KW, int D, bool XM>
__global__ __launch_bounds__(KW * 64) void small_kernel(GemmArgs a) {
    __shared__ f32x4_t red[KW][R][64];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int64_t last = tiles(a.N) - 1;
    const int64_t tile0 = (int64_t)blockIdx.x * R;
    const int m0 = blockIdx.y * 16;
    const int g0 = (int)((int64_t)a.G * w / KW), g1 = (int)((int64_t)a.G * (w + 1) / KW);
    const int n = g1 - g0;

    const uint8_t* wp[R];
    const uint8_t* sp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t t = tile0 + r < last ? tile0 + r : last;
        wp[r] = a.w.codes + t * a.G * kCodeBlock + lane * 16;
        sp[r] = a.w.scales + t * a.Q * kScaleBlock + lane * 4;
    }
    const bool row = m0 + c < a.M;
    const uint16_t* xp = nullptr;
    const uint8_t* xcp = nullptr;
    const uint8_t* xsp = nullptr;
    if constexpr (XM) {
        xcp = a.xm.codes + (int64_t)blockIdx.y * a.G * kCodeBlock + lane * 16;
        xsp = a.xm.scales + (int64_t)blockIdx.y * a.Q * kScaleBlock + lane * 4;
    } else {
        xp = a.x + (int64_t)(row ? m0 + c : m0) * a.ldx + 32 * q;
    }

    constexpr int XV = XM ? 1 : 4;
    u32x4_t wb[D][R], xb[D][XV];
    uint32_t ws[D][R], xs[D];
#pragma unroll
    for (int d = 0; d < D; ++d) {
        xs[d] = 0;
#pragma unroll
        for (int b = 0; b < XV; ++b) xb[d][b] = u32x4_t{0, 0, 0, 0};
    }
    auto load = [&](int d, int g) {
        const int64_t so = (int64_t)(g >> 2) * kScaleBlock + (g & 3);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            wb[d][r] = load16_nt(wp[r] + (int64_t)g * kCodeBlock);
            ws[d][r] = sp[r][so];
        }
        if constexpr (XM) {
            xb[d][0] = *reinterpret_cast<const u32x4_t*>(xcp + (int64_t)g * kCodeBlock);
            xs[d] = xsp[so];
        } else {
            // rows past M load nothing: their results are not stored.  Blocks past K
            // (the last group of a ragged K) must be zero: their codes are, and
            // nothing times zero but a finite number is.
            const bool in = row && 128 * (int64_t)g + 32 * q < a.K;
            const u32x4_t zero = {0, 0, 0, 0};
            if (g == a.G - 1) {
#pragma unroll
                for (int b = 0; b < XV; ++b) xb[d][b] = zero;
            }
            if (in) {
#pragma unroll
                for (int b = 0; b < XV; ++b)
                    xb[d][b] = *reinterpret_cast<const u32x4_t*>(xp + 128 * (int64_t)g + 8 * b);
            }
        }
    };
    f32x4_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
    auto product = [&](int d) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if constexpr (XM) {
                acc[r] = mfma_mx4(operand4(wb[d][r]), operand4(xb[d][0]), acc[r], ws[d][r], xs[d]);
            } else {
                const float s = scale_f32(ws[d][r]);
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    acc[r] = mfma_bf16(expand8(wb[d][r][b], s),
                                       __builtin_bit_cast(bf16x8_t, xb[d][b]), acc[r]);
            }
        }
    };

    if (n > 0) {
#pragma unroll
        for (int d = 0; d < D; ++d) load(d, g0 + (d < n ? d : n - 1));
        int i = 0;
        for (; i + 2 * D <= n; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                product(d);
                load(d, g0 + i + D + d);
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i + d < n) product(d);
            if (i + D + d < n) load(d, g0 + i + D + d);
        }
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (i + D + d < n) product(d);
    }

#pragma unroll
    for (int r = 0; r < R; ++r) red[w][r][lane] = acc[r];
    __syncthreads();
    const float* rf = reinterpret_cast<const float*>(red);
    for (int i = threadIdx.x; i < 256 * R; i += KW * 64) {
        const int m = i / (16 * R), col = i % (16 * R);
        const int r = col >> 4, wr = col & 15;
        const int64_t nn = tile0 * 16 + col;
        if (m0 + m >= a.M || nn >= a.N) continue;
        const int at = r * 256 + ((wr >> 2) * 16 + m) * 4 + (wr & 3);
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < KW; ++v) s += rf[v * R * 256 + at];
        store_y(a, m0 + m, nn, s);
    }
}

template <int R, int KW, int D>
hipError_t launch_small(const GemmArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((tiles(a.N) + R - 1) / R), (unsigned)tiles(a.M));
    if (a.x == nullptr)
        hipLaunchKernelGGL((small_kernel<R, KW, D, true>), grid, dim3(KW * 64), 0, s, a);
    else
        hipLaunchKernelGGL((small_kernel<R, KW, D, false>), grid, dim3(KW * 64), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t gemm_workspace_bytes(int64_t, int64_t, int64_t, bool) { return 0; }

hipError_t launch_gemm(GemmArgs a, void*, hipStream_t s) {
    return launch_small<1, 8, 4>(a, s);
}

}  // namespace mx4
