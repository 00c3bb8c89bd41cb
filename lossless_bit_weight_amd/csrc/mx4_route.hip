// mx4_route.hip -- each token's experts and their shares (../../include/mx4_route.h
// states the operation).
//
// A wave takes one token.  Where groups are limited a group has L neighbouring lanes, the
// largest power of two that 64 lanes have for each, else all 64 are one group; lane r of
// a group holds its experts r, r + L, r + 2 L ..: what a group is worth is then found for
// all groups at once, by exchanges between neighbours.
// A rank is a 64-bit number of the same order (fp64 scores plus bias: a choice between two
// that differ in the last of fp32's bits is then the same for every way of computing
// them; or the fp32 logit in the upper half).  The chosen ones are taken by maxima over
// the wave of the upper halves, and of the lower ones and the indices only where several
// share the largest: six lane moves a maximum, no LDS.  The scores of the chosen are
// computed again from their logits, a lane each, so that softmax with renormalised shares
// and no bias needs no exponential of the others.
// Bound by instructions, about 36 a wave for each chosen expert: 8191 tokens, 8 of 256
// experts in 4 of 8 groups, sigmoid and bias, 14.6 us (8.9 MB, which a copy moves in 1.8);
// 16 tokens, 6 of 64 experts 3.5, a launch's start and end.  The wave's maxima of whole
// 64-bit ranks, with the scores' exponentials behind branches, took 45.
#include <type_traits>

#include "exp64.hpp"
#include "mx4_internal.hpp"

namespace mx4 {
namespace {

// Order as unsigned numbers: NaN above all, -0 as +0; 0 is no rank's.
__device__ __forceinline__ uint32_t order32(float l) {
    if (l != l) return ~0u;
    const uint32_t u = __float_as_uint(l + 0.0f);
    return u >> 31 ? ~u : u | 1u << 31;
}
__device__ __forceinline__ uint64_t order64(double v) {
    if (v != v) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | 1ull << 63;
}

// Two copies of v between which the lanes D apart (in the order of mirrored rows below 16)
// have changed places: every lane finds its own value in one of them and the other lane's
// in the other.
template <int D>
__device__ __forceinline__ void exchange(uint32_t v, uint32_t& a, uint32_t& b) {
    a = b = v;
    if constexpr (D == 1) {
        b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);   // 1 0 3 2
    } else if constexpr (D == 2) {
        b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);   // 2 3 0 1
    } else if constexpr (D == 4) {
        b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);  // half mirror
    } else if constexpr (D == 8) {
        b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);  // mirror
    } else if constexpr (D == 16) {
        swap16(a, b);
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        a = r[0];
        b = r[1];
    }
}
template <int D, class T>
__device__ __forceinline__ void exchange64(T v, T& a, T& b) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t a0, a1, b0, b1;
    exchange<D>((uint32_t)u, a0, b0);
    exchange<D>((uint32_t)(u >> 32), a1, b1);
    a = __builtin_bit_cast(T, (uint64_t)a1 << 32 | a0);
    b = __builtin_bit_cast(T, (uint64_t)b1 << 32 | b0);
}
// f(D) for the distances within runs of L lanes, L a power of two that is the same in all.
template <class F>
__device__ __forceinline__ void within(int L, F f) {
    if (L > 1) f(std::integral_constant<int, 1>{});
    if (L > 2) f(std::integral_constant<int, 2>{});
    if (L > 4) f(std::integral_constant<int, 4>{});
    if (L > 8) f(std::integral_constant<int, 8>{});
    if (L > 16) f(std::integral_constant<int, 16>{});
    if (L > 32) f(std::integral_constant<int, 32>{});
}
__device__ __forceinline__ double wave_sum(double v) {
    within(64, [&](auto d) {
        double a, b;
        exchange64<decltype(d)::value>(v, a, b);
        v = a + b;
    });
    return v;
}
// The wave's largest: along the rows of 16 lanes, over the rows, then from the last lane (a
// lane without a source keeps its own).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    const auto step = [&](auto ctrl) {
        constexpr int C = decltype(ctrl)::value;
        const uint32_t o =
            (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, C, 0xF, 0xF, false);
        v = v > o ? v : o;
    };
    step(std::integral_constant<int, 0x111>{});     // row_shr:1
    step(std::integral_constant<int, 0x112>{});     // row_shr:2
    step(std::integral_constant<int, 0x114>{});     // row_shr:4
    step(std::integral_constant<int, 0x118>{});     // row_shr:8
    step(std::integral_constant<int, 0x142>{});     // row_bcast:15
    step(std::integral_constant<int, 0x143>{});     // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

template <bool F32>
__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int e) {
    if constexpr (F32) return static_cast<const float*>(a.logits)[t * a.ldl + e];
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[t * a.ldl + e] << 16);
}
// (results are selected, not branched to, so that the slots of a lane overlap)
constexpr double kLeast = -707.0;       // exp of less counts as 0
__device__ __forceinline__ double sigmoid(float l) {
    const double d = l, in = __builtin_fmin(__builtin_fmax(d, kLeast), -kLeast);
    const double x = 1.0 + exp2_64_within(-in, kLog2E);
    double s = __builtin_amdgcn_rcp(x);
    s = __builtin_fma(__builtin_fma(-x, s, 1.0), s, s);
    s = __builtin_fma(__builtin_fma(-x, s, 1.0), s, s);
    s = d < kLeast ? 0.0 : s;
    return d == d ? s : d;
}
// exp(l - top), whose sum is softmax's denominator
__device__ __forceinline__ double power(float l, float top) {
    const double d = (double)l - (double)top;
    const double p = exp2_64_within(__builtin_fmax(d, kLeast), kLog2E);
    return d < kLeast || l == -__builtin_inff() ? 0.0 : p;
}

template <int EV, bool F32>
__global__ __launch_bounds__(256) void pick_kernel(RouteArgs a, int groups, int log_lanes) {
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const int lane = threadIdx.x & 63;
    const int L = 1 << log_lanes, per = a.E / groups;
    const int g = lane >> log_lanes, r = lane & (L - 1);
    const int first = g * per + r;              // the expert of slot i is first + i L
    const bool any_bias = a.bias != nullptr, limited = groups > 1;

    float l[EV];
#pragma unroll
    for (int i = 0; i < EV; ++i) {
        const bool in = g < groups && i * L + r < per;
        l[i] = logit<F32>(a, t, in ? first + i * L : 0);
        l[i] = in ? l[i] : -__builtin_inff();
    }
    // softmax: the largest logit; without a distribution (a NaN, +inf) all scores are NaN
    float top = 0.f;
    bool bad = false;
    if (!a.sigmoid) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            const uint32_t o = order32(l[i]);
            m = o > m ? o : m;
        }
        m = wave_max(m);
        bad = m >= order32(__builtin_inff());
        top = __uint_as_float(m >> 31 ? m & 0x7FFFFFFFu : ~m);
    }
    double score[EV], sum = 1.0;
    // who needs the scores of all experts, and who their softmax's sum
    const bool all = any_bias || (limited && a.terms == 2);
    if (all || (!a.sigmoid && !a.renormalize)) {
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < EV; ++i) score[i] = sigmoid(l[i]);
        } else {
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < EV; ++i) {
                score[i] = power(l[i], top);
                sum += score[i];
            }
            sum = wave_sum(sum);
            if (all)
#pragma unroll
                for (int i = 0; i < EV; ++i) score[i] = bad ? __builtin_nan("") : score[i] / sum;
        }
    }
    uint32_t hi[EV], lo[EV];            // ranks; 0: not to be chosen
    double value[EV];                   // s + bias, -inf for those
    if (any_bias) {
        float b[EV];
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            const bool in = g < groups && i * L + r < per;
            b[i] = a.bias[in ? first + i * L : 0];
        }
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            const bool may = l[i] != -__builtin_inff() && b[i] != -__builtin_inff();
            const double v = score[i] + (double)b[i];
            const uint64_t o = order64(l[i] != l[i] ? (double)l[i] : v);
            hi[i] = may ? (uint32_t)(o >> 32) : 0u;
            lo[i] = may ? (uint32_t)o : 0u;
            value[i] = may ? v : -__builtin_inf();
        }
    } else {
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            const bool may = l[i] != -__builtin_inff();
            hi[i] = may ? order32(l[i]) : 0u;
            lo[i] = 0;
            value[i] = may && all ? score[i] : -__builtin_inf();
        }
    }

    if (limited) {
        uint64_t worth = 0;
        if (a.terms == 1) {
#pragma unroll
            for (int i = 0; i < EV; ++i) {
                const uint64_t k = (uint64_t)hi[i] << 32 | lo[i];
                worth = k > worth ? k : worth;
            }
            within(L, [&](auto d) {
                uint64_t x, y;
                exchange64<decltype(d)::value>(worth, x, y);
                worth = x > y ? x : y;
            });
        } else {
            // the two largest values; a NaN makes the sum one
            double one = -__builtin_inf(), two = one;
            bool nan = false;
#pragma unroll
            for (int i = 0; i < EV; ++i) {
                nan = nan || value[i] != value[i];
                two = fmax(two, fmin(one, value[i]));
                one = fmax(one, value[i]);
            }
            uint32_t nans = nan;
            within(L, [&](auto d) {
                constexpr int D = decltype(d)::value;
                double x1, y1, x2, y2;
                uint32_t xn, yn;
                exchange64<D>(one, x1, y1);
                exchange64<D>(two, x2, y2);
                exchange<D>(nans, xn, yn);
                two = fmax(fmax(x2, y2), fmin(x1, y1));
                one = fmax(x1, y1);
                nans = xn | yn;
            });
            if (nans)
                worth = ~0ull;
            else if (one != -__builtin_inf())
                worth = order64(two == -__builtin_inf() ? one : one + two);
        }
        // those worth more than this lane's group, and those equal before it
        int before = 0;
        for (int o = 0; o < groups; ++o) {
            const uint32_t o0 =
                (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)worth, o << log_lanes);
            const uint32_t o1 =
                (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(worth >> 32), o << log_lanes);
            const uint64_t other = (uint64_t)o1 << 32 | o0;
            before += other > worth || (other == worth && o < g);
        }
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            hi[i] = before < a.kept ? hi[i] : 0u;
            lo[i] = before < a.kept ? lo[i] : 0u;
        }
    }

    int found = -1;
    for (int j = 0; j < a.top_k; ++j) {
        // the lane's largest, of equal ones its lowest expert
        uint64_t top_key = (uint64_t)hi[0] << 32 | lo[0];
        int mine = first;
#pragma unroll
        for (int i = 1; i < EV; ++i) {
            const uint64_t k = (uint64_t)hi[i] << 32 | lo[i];
            mine = k > top_key ? first + i * L : mine;
            top_key = k > top_key ? k : top_key;
        }
        const uint32_t best = (uint32_t)(top_key >> 32), low = (uint32_t)top_key;
        const uint32_t most = wave_max(best);
        if (most == 0) break;
        uint64_t hits = __ballot(best == most);
        int e;
        if (__popcll(hits) == 1) {
            e = __builtin_amdgcn_readlane(mine, __builtin_ctzll(hits));
        } else {            // the largest lower half, and of its experts the lowest
            const uint32_t lower = wave_max(best == most ? low : 0u);
            e = (int)~wave_max(best == most && low == lower ? ~(uint32_t)mine : 0u);
        }
#pragma unroll
        for (int i = 0; i < EV; ++i) hi[i] = first + i * L == e ? 0u : hi[i];
        found = lane == j ? e : found;
    }

    double share = 0.0;
    if (found >= 0) {
        const float chosen = logit<F32>(a, t, found);
        if (a.sigmoid)
            share = sigmoid(chosen);
        else
            share = bad ? __builtin_nan("") : power(chosen, top);
    }
    if (a.renormalize) {
        const double whole = wave_sum(share);
        share = whole == 0.0 ? 0.0 : share / whole;
    } else if (!a.sigmoid) {
        share /= sum;
    }
    if (lane < a.top_k) {
        a.experts[t * a.top_k + lane] = found;
        a.shares[t * a.top_k + lane] = (float)(found < 0 ? 0.0 : share * (double)a.scale);
    }
}

template <int EV>
void launch(const RouteArgs& a, int groups, int log_lanes, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
    if (a.f32)
        hipLaunchKernelGGL((pick_kernel<EV, true>), grid, block, 0, s, a, groups, log_lanes);
    else
        hipLaunchKernelGGL((pick_kernel<EV, false>), grid, block, 0, s, a, groups, log_lanes);
}

}  // namespace

hipError_t launch_pick(const RouteArgs& a, hipStream_t s) {
    // groups that all count are as good as one
    const int groups = a.kept < a.groups ? a.groups : 1;
    int log_lanes = 6;
    while (groups > 64 >> log_lanes) --log_lanes;
    const int slots = (a.E / groups + (1 << log_lanes) - 1) >> log_lanes;
    if (slots <= 1)
        launch<1>(a, groups, log_lanes, s);
    else if (slots <= 2)
        launch<2>(a, groups, log_lanes, s);
    else if (slots <= 4)
        launch<4>(a, groups, log_lanes, s);
    else if (slots <= 8)
        launch<8>(a, groups, log_lanes, s);
    else if (slots <= 16)
        launch<16>(a, groups, log_lanes, s);
    else
        launch<32>(a, groups, log_lanes, s);
    return hipGetLastError();
}

}  // namespace mx4
