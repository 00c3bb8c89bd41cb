// mx8_codec.hip -- BF16 or fp32 values to MX8 and back (../../include/mx8.h has
// the format).
//
// A wave takes 512 values of one row, a lane eight: the four lanes of a block
// agree on its largest exponent in two quad permutes, every load and store of a
// wave is contiguous, and the wave writes the 16 scale bytes of its 512 values,
// those past K too.  Bound by memory: 2 (4) + 1.03 bytes a value: 4096 x 5120 BF16 to MX8
// 13.6 us (4.7 TB/s), back 11.4 (5.6 TB/s).  Two pieces of a row a lane: 13.2, but 2.8
// instead of 2.3 for one row; of fp32 17.3 instead of 16.9.
#include "mx8_internal.hpp"

namespace mx8 {
namespace {

constexpr int kThreads = 256;

// A grid's x holds fewer than 2^24 workgroups of 256 (work items are counted in 32
// bits); more go along y.
constexpr int64_t kGridX = (int64_t)1 << 22;
dim3 grid_of(int64_t waves) {
    const int64_t blocks = (waves + 3) / 4;
    return blocks <= kGridX ? dim3((unsigned)blocks)
                            : dim3((unsigned)kGridX, (unsigned)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t wave_index() {
    return ((int64_t)blockIdx.y * kGridX + blockIdx.x) * 4 + (threadIdx.x >> 6);
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const void* __restrict__ x,
                                                            float quarters, int64_t R, int K,
                                                            int Q, int64_t ldx,
                                                            uint8_t* __restrict__ values,
                                                            int64_t ldv,
                                                            uint8_t* __restrict__ scales,
                                                            int64_t lds) {
    const int64_t wave = wave_index();
    if (wave >= R * Q) return;
    const int64_t r = wave / Q;
    const int lane = threadIdx.x & 63, k = (int)(wave % Q) * 512 + 8 * lane;
    const bool in = k < K;              // a block lies inside or outside as a whole
    Eight v;
    v.load<F32>(x, r * ldx + (in ? k : 0));
    uint32_t e;
    const u32x2_t d = v.encode(e, quarters);
    if (in) *reinterpret_cast<u32x2_t*>(values + r * ldv + k) = d;
    if ((lane & 3) == 0) scales[r * lds + scale_place(k)] = (uint8_t)(in ? e : 127u);
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ values,
                                                              int64_t ldv,
                                                              const uint8_t* __restrict__ scales,
                                                              int64_t lds, int64_t R, int K, int Q,
                                                              void* __restrict__ y, int64_t ldy) {
    const int64_t wave = wave_index();
    if (wave >= R * Q) return;
    const int64_t r = wave / Q;
    const int k = (int)(wave % Q) * 512 + 8 * (threadIdx.x & 63);
    if (k >= K) return;
    const u32x2_t d = *reinterpret_cast<const u32x2_t*>(values + r * ldv + k);
    const uint32_t e = scales[r * lds + scale_place(k)];
    // 2^(e - 127), subnormal for e = 0
    const float s = e == 0u     ? __uint_as_float(0x00400000u)
                    : e == 255u ? __builtin_nanf("")
                                : __uint_as_float(e << 23);
    Eight v;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)d[j], false);
        const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8((int)d[j], true);
        v.f[4 * j] = a[0] * s;
        v.f[4 * j + 1] = a[1] * s;
        v.f[4 * j + 2] = b[0] * s;
        v.f[4 * j + 3] = b[1] * s;
    }
    v.store<F32>(y, r * ldy + k);
}

}  // namespace

hipError_t launch_quantize(const void* x, int x_f32, float quarters, int64_t R, int64_t K,
                           int64_t ldx, uint8_t* values, int64_t ldv, uint8_t* scales,
                           int64_t lds, hipStream_t s) {
    const int Q = (int)mx4::quads(K);
    const dim3 grid = grid_of(R * Q);
    if (x_f32)
        hipLaunchKernelGGL(quantize_kernel<true>, grid, dim3(kThreads), 0, s, x, quarters, R,
                           (int)K, Q, ldx, values, ldv, scales, lds);
    else
        hipLaunchKernelGGL(quantize_kernel<false>, grid, dim3(kThreads), 0, s, x, quarters, R,
                           (int)K, Q, ldx, values, ldv, scales, lds);
    return hipGetLastError();
}

hipError_t launch_dequantize(const uint8_t* values, int64_t ldv, const uint8_t* scales,
                             int64_t lds, int64_t R, int64_t K, void* y, int y_f32, int64_t ldy,
                             hipStream_t s) {
    const int Q = (int)mx4::quads(K);
    const dim3 grid = grid_of(R * Q);
    if (y_f32)
        hipLaunchKernelGGL(dequantize_kernel<true>, grid, dim3(kThreads), 0, s, values, ldv, scales,
                           lds, R, (int)K, Q, y, ldy);
    else
        hipLaunchKernelGGL(dequantize_kernel<false>, grid, dim3(kThreads), 0, s, values, ldv,
                           scales, lds, R, (int)K, Q, y, ldy);
    return hipGetLastError();
}

}  // namespace mx8
