// mx4_route.hip -- each token's experts and their shares (../../include/mx4_route.h
// states the operation).
//
// A wave takes one token: lane l holds the experts EV l .. EV l + EV - 1, so that the
// lowest lane of a tie has the lowest expert.  Scores and ranks are fp64 (a choice
// between two that differ in the last of fp32's bits is then the same for every way of
// computing them); a rank becomes a 64-bit number of the same order, and the chosen
// ones are taken by repeated maxima over the wave.
#include "exp64.hpp"
#include "mx4_internal.hpp"

namespace mx4 {
namespace {

// Order of ranks as unsigned numbers: NaN above all, -0 as +0; 0 is no rank's.
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | 1ull << 63;
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint64_t o = (uint64_t)__shfl_xor((long long)v, d);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

template <int EV, bool F32>
__global__ __launch_bounds__(256) void pick_kernel(RouteArgs a) {
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const int lane = threadIdx.x & 63;

    double score[EV];
    uint64_t key[EV];               // 0: not to be chosen
    float l[EV];
#pragma unroll
    for (int i = 0; i < EV; ++i) {
        const int e = EV * lane + i;
        l[i] = -__builtin_inff();
        if (e < a.E) {
            if constexpr (F32)
                l[i] = static_cast<const float*>(a.logits)[t * a.ldl + e];
            else
                l[i] = __uint_as_float(
                    (uint32_t)static_cast<const uint16_t*>(a.logits)[t * a.ldl + e] << 16);
        }
    }
    if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            const double d = l[i];
            score[i] = d != d ? d : 1.0 / (1.0 + exp2_64(-d * kLog2E));
        }
    } else {
        float top = -__builtin_inff();
        bool bad = false;
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            top = l[i] > top ? l[i] : top;
            bad = bad || l[i] != l[i] || l[i] == __builtin_inff();
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
        bad = __ballot(bad) != 0;
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            score[i] = l[i] == -__builtin_inff()
                           ? 0.0
                           : exp2_64(((double)l[i] - (double)top) * kLog2E);
            sum += score[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < EV; ++i) score[i] = bad ? __builtin_nan("") : score[i] / sum;
    }
    double biased[EV];
    bool any[EV];
#pragma unroll
    for (int i = 0; i < EV; ++i) {
        const int e = EV * lane + i;
        const float b = a.bias != nullptr && e < a.E ? a.bias[e] : 0.f;
        biased[i] = score[i] + (double)b;
        any[i] = e < a.E && l[i] != -__builtin_inff() && b != -__builtin_inff();
        key[i] = any[i] ? order_key(a.bias != nullptr ? biased[i] : (double)l[i]) : 0;
        if (a.bias != nullptr && l[i] != l[i] && any[i]) key[i] = ~0ull;
    }

    // the groups that count: lane g holds the value of group g
    if (a.kept < a.groups) {
        const int per = a.E / a.groups;
        uint64_t mine = 0;
        for (int g = 0; g < a.groups; ++g) {
            uint64_t v = 0;
#pragma unroll
            for (int i = 0; i < EV; ++i)
                if ((EV * lane + i) / per == g && key[i] > v) v = key[i];
            v = wave_max(v);
            if (a.terms == 2 && v != 0) {
                double one = -__builtin_inf(), two = -__builtin_inf();
                bool nan = false;
#pragma unroll
                for (int i = 0; i < EV; ++i) {
                    if ((EV * lane + i) / per != g || !any[i]) continue;
                    const double s = biased[i];
                    nan = nan || s != s;
                    two = fmax(two, s < one ? s : one);
                    one = fmax(one, s);
                }
#pragma unroll
                for (int d = 32; d > 0; d >>= 1) {
                    const double o1 = __shfl_xor(one, d), o2 = __shfl_xor(two, d);
                    two = fmax(fmax(two, o2), one < o1 ? one : o1);
                    one = fmax(one, o1);
                }
                v = __ballot(nan)                ? ~0ull
                    : two == -__builtin_inf() ? order_key(one)
                                              : order_key(one + two);
            }
            if (lane == g) mine = v;
        }
        // those above a group, and those equal before it
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const uint64_t o = (uint64_t)__shfl((long long)mine, g);
            before += o > mine || (o == mine && g < lane);
        }
        const uint64_t keep = __ballot(before < a.kept && lane < a.groups);
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            const int g = (EV * lane + i) / per;
            if (g > 63 || !(keep >> g & 1)) key[i] = 0;
        }
    }

    int found = -1;
    double share = 0.0;
    for (int j = 0; j < a.top_k; ++j) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        }
        const uint64_t m = wave_max(best);
        if (m == 0) break;
        const int src = __builtin_ctzll(__ballot(best == m));
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            if (i == at) s = score[i];
            if (lane == src && i == at) key[i] = 0;
        }
        const int e = EV * src + __shfl(at, src);
        s = __shfl(s, src);
        if (lane == j) {
            found = e;
            share = s;
        }
    }
    if (a.renormalize) {
        const double sum = wave_sum(share);
        share = sum == 0.0 ? 0.0 : share / sum;
    }
    if (lane < a.top_k) {
        a.experts[t * a.top_k + lane] = found;
        a.shares[t * a.top_k + lane] = (float)(found < 0 ? 0.0 : share * (double)a.scale);
    }
}

template <int EV>
void launch(const RouteArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
    if (a.f32)
        hipLaunchKernelGGL((pick_kernel<EV, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((pick_kernel<EV, false>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_pick(const RouteArgs& a, hipStream_t s) {
    if (a.E <= 64)
        launch<1>(a, s);
    else if (a.E <= 128)
        launch<2>(a, s);
    else if (a.E <= 256)
        launch<4>(a, s);
    else if (a.E <= 512)
        launch<8>(a, s);
    else
        launch<16>(a, s);
    return hipGetLastError();
}

}  // namespace mx4
