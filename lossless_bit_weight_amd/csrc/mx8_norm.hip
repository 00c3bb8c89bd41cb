// mx8_norm.hip -- residual addition, root-mean-square norm and its output in BF16,
// fp32 or MX8 (../../include/mx8.h states the operation).
//
// s = x + residual is read once and stays in registers: a row's threads hold C chunks of
// eight values each, thread t of T the chunks t + T i.  The sum of squares is held in 64
// bits (two instructions a value beside the memory's time), so that no square overflows
// that s itself does not, and so is y = s * r * weight, from the registers, to be rounded
// once (BF16: from fp32); in MX8 the four lanes of a quad hold one block.
// One pass over the data, bound by memory: 4096 x 5120, fp32 x, BF16 residual, MX8 out:
// 35.9 us (189 MB, 5.3 TB/s, part of it from the last-level cache); 20680 x 128, BF16 in
// and out, 4.9 us (10.6 MB, 2.2 TB/s with the launch's start and end).  One row of 5120,
// 3.6 us, is a launch's start and end and the way to memory and back.
#include "mx8_internal.hpp"

namespace mx8 {
namespace {

// Over the T threads of a row, or (T = 0) over the workgroup.
template <int T>
__device__ __forceinline__ double row_sum(double v, double* part) {
    constexpr int kLanes = T != 0 ? T : 64;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
    if constexpr (T == 0) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0;
        for (int i = 0; i < (int)blockDim.x / 64; ++i) v += part[i];
    }
    return v;
}

// y in fp32's 24 bits, cut off, the last of them set if anything was cut: rounding that to
// MX8 is the same as rounding y itself.  (Of values rounded to fp32 first, some in a million
// land on a border of MX8 and go the wrong way from there.)  With it and the products in 64
// bits 4096 x 5120 to MX8 takes 35.9 us; in fp32 throughout it took 33.7.
__device__ __forceinline__ float to_odd(double y) {
    const uint64_t u = __builtin_bit_cast(uint64_t, y);
    const uint32_t lo = (uint32_t)u, rest = lo & 0x1FFFFFFFu;
    const uint32_t odd = rest != 0 ? 0x20000000u : 0u;
    return (float)__builtin_bit_cast(double, (u & ~(uint64_t)0x1FFFFFFFu) | odd);
}

// A grid's x holds fewer than 2^32 work items: more blocks go along y.
constexpr int64_t kGridX = (int64_t)1 << 21;

constexpr int kMost = 1024;             // threads of a row

// T: threads of a row, of which a workgroup of 256 has several; 0: a row's are the workgroup.
// RES: 0 none, 1 BF16, 2 fp32
template <int T, int C, bool XF32, int RES>
__global__ __launch_bounds__(T != 0 ? 256 : kMost) void norm_kernel(NormArgs a) {
    __shared__ double part[T != 0 ? 1 : kMost / 64];
    constexpr int kRows = T != 0 ? 256 / T : 1;
    const int TPR = T != 0 ? T : (int)blockDim.x;
    const int t = T != 0 ? threadIdx.x % T : threadIdx.x;
    int64_t row = ((int64_t)blockIdx.y * kGridX + blockIdx.x) * kRows;
    if constexpr (T != 0) row += threadIdx.x / T;
    const bool live = row < a.M;
    if (!live) row = a.M - 1;           // (lanes or a workgroup of their own: nothing is stored)

    // (the weights of long rows are read behind the sum: there are no registers for them)
    constexpr bool kEarly = C <= 2;
    Eight v[C], w[kEarly ? C : 1];
    auto weights = [&](Eight& e, int at) {
        if (a.w_f32)
            e.load<true>(a.w, at);
        else
            e.load<false>(a.w, at);
    };
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int k = 8 * (t + TPR * i), at = k < a.K ? k : 0;
        v[i].template load<XF32>(a.x, row * a.ldx + at);
        if constexpr (RES != 0) {
            Eight r;
            r.load<RES == 2>(a.res, row * a.ldr + at);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i].f[j] += r.f[j];
        }
        if constexpr (kEarly) weights(w[i], at);
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int k = 8 * (t + TPR * i);
        if constexpr (RES == 1) {
            // the norm is of what the residual keeps
            const u32x4_t b = v[i].bf16();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i].f[2 * j] = __uint_as_float(b[j] << 16);
                v[i].f[2 * j + 1] = __uint_as_float(b[j] & 0xFFFF0000u);
            }
        }
        if constexpr (RES != 0) {
            if (live && k < a.K) v[i].template store<RES == 2>(a.res_out, row * a.ldo + k);
        }
        if (k < a.K) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double d = v[i].f[j];
                sum = __builtin_fma(d, d, sum);
            }
        }
    }
    sum = row_sum<T>(sum, part);
    const double r = 1.0 / __builtin_sqrt(sum / a.K + (double)a.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int k = 8 * (t + TPR * i);
        Eight& wi = w[kEarly ? i : 0];
        if constexpr (!kEarly) weights(wi, k < a.K ? k : 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double y = (double)v[i].f[j] * r * (double)wi.f[j];
            v[i].f[j] = a.y_type >= 2 ? to_odd(y) : (float)y;
        }
        const bool in = live && k < a.K;
        if (a.y_type >= 2) {
            uint32_t e;
            const u32x2_t d = v[i].encode(e, quarters_below(a.y_type == 3));
            uint8_t* y = static_cast<uint8_t*>(a.y);
            if (in) *reinterpret_cast<u32x2_t*>(y + row * a.ldy + k) = d;
            if ((t & 3) == 0 && live && k < a.K)
                a.ys[row * a.lds + scale_place(k)] = (uint8_t)e;
        } else if (in) {
            if (a.y_type == 1)
                v[i].template store<true>(a.y, row * a.ldy + k);
            else
                v[i].template store<false>(a.y, row * a.ldy + k);
        }
    }
    // the scales past K
    if (a.y_type >= 2 && live) {
        const int first = a.K / 32, n = (int)mx4::quads(a.K) * 16 - first;
        for (int i = t; i < n; i += TPR)
            a.ys[row * a.lds + scale_place((first + i) * 32)] = 127;
    }
}

template <int T, int C>
hipError_t launch(const NormArgs& a, hipStream_t s) {
    constexpr int kRows = T != 0 ? 256 / T : 1;
    const int64_t blocks = (a.M + kRows - 1) / kRows;
    const dim3 grid((unsigned)(blocks < kGridX ? blocks : kGridX),
                    (unsigned)((blocks + kGridX - 1) / kGridX));
    const dim3 block(T != 0 ? 256 : (a.K / 8 + 64 * C - 1) / (64 * C) * 64);
    const int res = a.res == nullptr ? 0 : a.res_f32 ? 2 : 1;
    switch (res * 2 + a.x_f32) {
        case 0: hipLaunchKernelGGL((norm_kernel<T, C, false, 0>), grid, block, 0, s, a); break;
        case 1: hipLaunchKernelGGL((norm_kernel<T, C, true, 0>), grid, block, 0, s, a); break;
        case 2: hipLaunchKernelGGL((norm_kernel<T, C, false, 1>), grid, block, 0, s, a); break;
        case 3: hipLaunchKernelGGL((norm_kernel<T, C, true, 1>), grid, block, 0, s, a); break;
        case 4: hipLaunchKernelGGL((norm_kernel<T, C, false, 2>), grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL((norm_kernel<T, C, true, 2>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace

// A chunk a thread keeps most loads on their way and the fewest behind each other; a row of
// up to 64 threads is a part of a wave or a wave (40000 x 128: 16 threads 10.8 us, 64 23.7;
// 40000 x 256: 32 threads 19.0, 64 30.1).  Beyond 512 chunks many rows go faster by two, as
// a CU has places for more workgroups at different points of their rows (4096 x 5120: two
// 35.9 us, one 41.2; 4096 x 7168: 48.7 and 61.6; 4096 x 4096: 27.2 and 26.7; 512 x 5120: 8.8
// and 8.6; 64 x 5120: 5.2 and 4.5).  More than two only where 1024 threads need them.
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    const int chunks = a.K / 8;
    if (chunks <= 16) return launch<16, 1>(a, s);
    if (chunks <= 32) return launch<32, 1>(a, s);
    if (chunks <= 64) return launch<64, 1>(a, s);
    if (chunks <= 512 || (chunks <= kMost && a.M <= 1024)) return launch<0, 1>(a, s);
    if (chunks <= 2 * kMost) return launch<0, 2>(a, s);
    return launch<0, 4>(a, s);
}

}  // namespace mx8
