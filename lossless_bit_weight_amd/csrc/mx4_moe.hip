// mx4_moe.hip -- a mixture-of-experts layer for a few tokens on MX4 weights
// (../../include/mx4.h states the operation).
//
// Three launches.  route: each token's experts and their shares, and the pairs
// (token, expert) sorted by expert and cut into slots of at most 16.  up: per
// slot and 16 hidden values the products with the gate and the up rows and
// h = silu(g) * u.  down: per 16 R outputs all slots' products with h, weighted
// and added per token.  The chosen experts' weights are read once (an expert
// with more than 16 tokens: once a slot, the later reads from cache), which is
// what bounds the layer; everything else is smaller by T / 1000 or so.
#include "mx4_internal.hpp"

namespace mx4 {
namespace {

// ---- routing --------------------------------------------------------------------

constexpr int kRouteThreads = 1024;

// Order of the logits as unsigned numbers: NaN above all, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float l) {
    if (l != l) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(l + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;    // order_key(-inf)

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
        v = v > o ? v : o;
    }
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// One workgroup.  A wave takes a token: lane l holds the logits of the experts
// l, l + 64, ...; top_k rounds find the largest key (ties: the lowest expert)
// and strike it out.  Tokens per expert are kept as 128-bit sets, so the sorted
// place of a pair is a count of bits and depends on no order of execution.
template <int EV>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(MoeArgs a) {
    __shared__ uint32_t set[kMaxExperts][4];
    __shared__ int base[kMaxExperts];
    __shared__ int wave_tot[2][kRouteThreads / 64];
    __shared__ uint16_t chosen[kMaxTokens * kMaxTopK];
    __shared__ float share[kMaxTokens * kMaxTopK];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int i = tid; i < a.E * 4; i += kRouteThreads) (&set[0][0])[i] = 0;
    __syncthreads();

    for (int t = w; t < a.T; t += kRouteThreads / 64) {
        uint32_t key[EV];
        float l[EV];
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            const int e = lane + 64 * i;
            l[i] = e < a.E ? a.logits[t * a.ldl + e] : -__builtin_inff();
            key[i] = e < a.E ? order_key(l[i]) : 0u;
        }
        float top = 0.f, mine = 0.f;    // the largest logit; lane j: the j-th chosen one
        int mine_e = -1;
        for (int j = 0; j < a.top_k; ++j) {
            uint32_t best = 0;
            int be = 0;
#pragma unroll
            for (int i = 0; i < EV; ++i)
                if (key[i] > best) {
                    best = key[i];
                    be = lane + 64 * i;
                }
            const uint32_t m = wave_max(best);
            if (m <= kKeyNegInf) break;     // only -inf (or nothing) left
            // the lowest expert with that key
            const int e = (int)~wave_max(best == m ? ~(uint32_t)be : 0u);
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < EV; ++i)
                if (e == lane + 64 * i) {
                    key[i] = 0;
                    v = l[i];
                }
            v = __shfl(v, e & 63);
            if (j == 0) top = v;
            if (lane == j) {
                mine = v;
                mine_e = e;
            }
        }
        const float ex = mine_e >= 0 ? expf(mine - top) : 0.f;
        float sum;
        if (a.renormalize) {
            sum = wave_sum(ex);
        } else {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < EV; ++i)
                if (l[i] != -__builtin_inff()) s += expf(l[i] - top);
            sum = wave_sum(s);
        }
        if (lane < a.top_k) {
            chosen[t * a.top_k + lane] = (uint16_t)(mine_e < 0 ? 0xFFFF : mine_e);
            share[t * a.top_k + lane] = mine_e < 0 ? 0.f : ex / sum;
            if (mine_e >= 0) atomicOr(&set[mine_e][t >> 5], 1u << (t & 31));
        }
    }
    __syncthreads();

    // exclusive sums over the experts of their pairs and slots
    int cnt = 0;
    if (tid < a.E) {
#pragma unroll
        for (int i = 0; i < 4; ++i) cnt += __popc(set[tid][i]);
    }
    const int ns = (cnt + 15) >> 4;
    int ip = cnt, is = ns;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int op = __shfl_up(ip, d), os = __shfl_up(is, d);
        if (lane >= d) {
            ip += op;
            is += os;
        }
    }
    if (lane == 63) {
        wave_tot[0][w] = ip;
        wave_tot[1][w] = is;
    }
    __syncthreads();
    for (int i = 0; i < w; ++i) {
        ip += wave_tot[0][i];
        is += wave_tot[1][i];
    }
    if (tid < a.E) {
        base[tid] = ip - cnt;
        for (int i = 0; i < ns; ++i) {
            const int left = cnt - 16 * i;
            a.slots[is - ns + i] = MoeSlot{tid, ip - cnt + 16 * i, left < 16 ? left : 16, 0};
        }
    }
    if (tid == kRouteThreads - 1) a.n_slots[0] = is;
    __syncthreads();

    for (int i = tid; i < a.T * a.top_k; i += kRouteThreads) {
        const int e = chosen[i];
        if (e == 0xFFFF) continue;
        const int t = i / a.top_k;
        int p = base[e];
        for (int j = 0; j < (t >> 5); ++j) p += __popc(set[e][j]);
        p += __popc(set[e][t >> 5] & ((1u << (t & 31)) - 1u));
        a.pair_token[p] = t;
        a.pair_p[p] = share[i];
    }
}

// ---- gate and up ------------------------------------------------------------------
// A workgroup: one slot, 16 gate rows and the 16 up rows beside them; KW waves
// split H, D groups in flight, operands as in mx4_gemm.hip's few-row kernel.
template <int KW, int D, int PARTS>
__global__ __launch_bounds__(KW * 64) void up_kernel(MoeArgs a) {
    __shared__ f32x4_t red[KW][2][64];
    const int it = a.I / 16;
    const int slot = blockIdx.x / it, j = blockIdx.x % it;
    if (slot >= a.n_slots[0]) return;
    const MoeSlot sl = a.slots[slot];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int G = (int)groups(a.H), Q = (int)quads(a.H);
    const int g0 = G * w / KW, n = G * (w + 1) / KW - g0;

    const uint8_t* wp[2];
    const uint8_t* sp[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int64_t t = (int64_t)sl.e * 2 * it + r * it + j;
        wp[r] = a.w13.codes + t * G * kCodeBlock + lane * 16;
        sp[r] = a.w13.scales + t * Q * kScaleBlock + lane * 4;
    }
    const bool row = c < sl.count;
    const uint16_t* xp = a.x + (row ? a.pair_token[sl.p0 + c] : 0) * a.ldx + 32 * q;

    u32x4_t wb[D][2], xb[D][4];
    uint32_t ws[D][2];
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) xb[d][b] = u32x4_t{0, 0, 0, 0};
    auto load = [&](int d, int g) {
        const int64_t so = (int64_t)(g >> 2) * kScaleBlock + (g & 3);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            wb[d][r] = load16_nt(wp[r] + (int64_t)g * kCodeBlock);
            ws[d][r] = sp[r][so];
        }
        if (g == G - 1) {
#pragma unroll
            for (int b = 0; b < 4; ++b) xb[d][b] = u32x4_t{0, 0, 0, 0};
        }
        if (row && 128 * g + 32 * q < a.H) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
                xb[d][b] = *reinterpret_cast<const u32x4_t*>(xp + 128 * (int64_t)g + 8 * b);
        }
    };
    f32x4_t acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    auto product = [&](int d) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float s = scale_f32(ws[d][r]);
#pragma unroll
            for (int b = 0; b < 4; ++b)
                acc[r] = mfma_bf16(expand8(wb[d][r][b], s),
                                   __builtin_bit_cast(bf16x8_t, xb[d][b]), acc[r]);
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
    red[w][0][lane] = acc[0];
    red[w][1][lane] = acc[1];
    __syncthreads();
    const float* rf = reinterpret_cast<const float*>(red);
    const int64_t pairs = (int64_t)a.T * a.top_k;
    for (int i = threadIdx.x; i < 256; i += KW * 64) {
        const int m = i >> 4, wr = i & 15;
        if (m >= sl.count) continue;
        const int at = ((wr >> 2) * 16 + m) * 4 + (wr & 3);
        float g = 0.f, u = 0.f;
#pragma unroll
        for (int v = 0; v < KW; ++v) {
            g += rf[v * 512 + at];
            u += rf[v * 512 + 256 + at];
        }
        const float h = g / (1.f + expf(-g)) * u;
        uint16_t* o = a.h + (int64_t)(sl.p0 + m) * a.I + 16 * j + wr;
        // h = the sum of PARTS BF16 numbers, each the rounded rest of those before: two
        // hold 16 bits of its mantissa, three all 24
        float rest = h;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            const uint16_t b = bf16_bits(rest);
            o[(int64_t)p * pairs * a.I] = b;
            const float f = __uint_as_float((uint32_t)b << 16);
            rest = __builtin_isfinite(f) ? rest - f : 0.f;
        }
    }
}

// ---- down ---------------------------------------------------------------------------
// A workgroup: 16 R outputs for all tokens.  The work (slot, group of 128 hidden
// values) is one sequence, cut into KW equal runs, one a wave; a wave adds each
// slot's product, weighted, to its own sums in LDS [token][16 R], and the
// waves' sums are added in wave order.
template <int R, int KW, int D, int PARTS>
__global__ __launch_bounds__(KW * 64) void down_kernel(MoeArgs a) {
    extern __shared__ float sums[];         // [KW][T][16 R]
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int G = (int)groups(a.I), Q = (int)quads(a.I);
    const int ht = a.H / 16;
    const int tile0 = blockIdx.x * R;
    const int n_slots = __builtin_amdgcn_readfirstlane(a.n_slots[0]);
    const int items = n_slots * G;
    const int i0 = (int)((int64_t)items * w / KW), n = (int)((int64_t)items * (w + 1) / KW) - i0;
    const int64_t pairs = (int64_t)a.T * a.top_k;
    float* mine = sums + (int64_t)w * a.T * 16 * R;
    for (int i = lane; i < a.T * 16 * R; i += 64) mine[i] = 0.f;

    u32x4_t wb[D][R], hb[D][PARTS][4];
    uint32_t ws[D][R];
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int b = 0; b < 4; ++b) hb[d][p][b] = u32x4_t{0, 0, 0, 0};

    // the slot and group that is loaded next, and its pointers
    int ls = i0 / G, lg = i0 % G;
    const uint8_t* wp[R];
    const uint8_t* sp[R];
    const uint16_t* hp = nullptr;
    bool row = false;
    auto enter = [&]() {
        const MoeSlot sl = a.slots[ls];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int tt = tile0 + r < ht ? tile0 + r : ht - 1;
            const int64_t t = (int64_t)sl.e * ht + tt;
            wp[r] = a.w2.codes + t * G * kCodeBlock + lane * 16;
            sp[r] = a.w2.scales + t * Q * kScaleBlock + lane * 4;
        }
        row = c < sl.count;
        hp = a.h + (int64_t)(sl.p0 + (row ? c : 0)) * a.I + 32 * q;
    };
    auto load = [&](int d) {
        const int g = lg;
        const int so = (g >> 2) * kScaleBlock + (g & 3);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            wb[d][r] = load16_nt(wp[r] + (int64_t)g * kCodeBlock);
            ws[d][r] = sp[r][so];
        }
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                hb[d][p][b] = u32x4_t{0, 0, 0, 0};
                if (row && 128 * g + 32 * q < a.I)
                    hb[d][p][b] = *reinterpret_cast<const u32x4_t*>(hp + p * pairs * a.I +
                                                                   128 * g + 8 * b);
            }
        if (++lg == G) {
            lg = 0;
            if (++ls < n_slots) enter();
        }
    };
    f32x4_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
    int cs = ls, cg = lg;                    // the slot and group that is multiplied next
    auto flush = [&]() {
        const MoeSlot sl = a.slots[cs];
        if (c < sl.count) {
            const int t = a.pair_token[sl.p0 + c];
            const float p = a.pair_p[sl.p0 + c];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                f32x4_t* o = reinterpret_cast<f32x4_t*>(mine + (t * R + r) * 16 + 4 * q);
                f32x4_t v = *o;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += p * acc[r][i];
                *o = v;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
    };
    auto product = [&](int d, bool end) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float s = scale_f32(ws[d][r]);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const bf16x8_t wv = expand8(wb[d][r][b], s);
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    acc[r] = mfma_bf16(wv, __builtin_bit_cast(bf16x8_t, hb[d][p][b]), acc[r]);
            }
        }
        if (++cg == G || end) {
            flush();
            cg = 0;
            ++cs;
        }
    };
    if (n > 0) {
        enter();
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (d < n) load(d);
        for (int i = 0; i < n; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                if (i + d < n) product(d, i + d + 1 == n);
                if (i + D + d < n) load(d);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 16 * R; i += KW * 64) {
        const int t = i / (16 * R), col = i % (16 * R);
        const int64_t hcol = (int64_t)tile0 * 16 + col;
        if (hcol >= a.H) continue;
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < KW; ++v) s += sums[(int64_t)v * a.T * 16 * R + i];
        if (a.y_f32)
            static_cast<float*>(a.y)[t * a.ldy + hcol] = s;
        else
            static_cast<uint16_t*>(a.y)[t * a.ldy + hcol] = bf16_bits(s);
    }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

int64_t max_slots(int64_t T, int64_t E, int64_t top_k) {
    const int64_t pairs = T * top_k;
    return (E < pairs ? E : pairs) + pairs / 16;
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t I, int64_t E, int64_t top_k, bool y_f32) {
    const int64_t pairs = T * top_k;
    return 256 + up256((size_t)max_slots(T, E, top_k) * sizeof(MoeSlot)) +
           2 * up256((size_t)pairs * 4) + (size_t)(y_f32 ? 3 : 2) * pairs * I * 2;
}

hipError_t launch_moe(MoeArgs a, void* ws, hipStream_t s) {
    const int64_t pairs = (int64_t)a.T * a.top_k;
    a.max_slots = (int)max_slots(a.T, a.E, a.top_k);
    uint8_t* p = static_cast<uint8_t*>(ws);
    a.n_slots = reinterpret_cast<int*>(p);
    p += 256;
    a.slots = reinterpret_cast<MoeSlot*>(p);
    p += up256((size_t)a.max_slots * sizeof(MoeSlot));
    a.pair_token = reinterpret_cast<int*>(p);
    p += up256((size_t)pairs * 4);
    a.pair_p = reinterpret_cast<float*>(p);
    p += up256((size_t)pairs * 4);
    a.h = reinterpret_cast<uint16_t*>(p);

    const dim3 rt(kRouteThreads);
    if (a.E <= 64)
        hipLaunchKernelGGL(route_kernel<1>, dim3(1), rt, 0, s, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL(route_kernel<2>, dim3(1), rt, 0, s, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL(route_kernel<4>, dim3(1), rt, 0, s, a);
    else
        hipLaunchKernelGGL(route_kernel<16>, dim3(1), rt, 0, s, a);

    const dim3 ug((unsigned)((int64_t)a.max_slots * (a.I / 16)));
    const dim3 dg((unsigned)(a.H / 16));
    const unsigned lds = 8u * (unsigned)a.T * 16u * 4u;
    if (a.y_f32) {
        hipLaunchKernelGGL((up_kernel<8, 4, 3>), ug, dim3(512), 0, s, a);
        hipLaunchKernelGGL((down_kernel<1, 8, 2, 3>), dg, dim3(512), lds, s, a);
    } else {
        hipLaunchKernelGGL((up_kernel<8, 4, 2>), ug, dim3(512), 0, s, a);
        hipLaunchKernelGGL((down_kernel<1, 8, 2, 2>), dg, dim3(512), lds, s, a);
    }
    return hipGetLastError();
}

}  // namespace mx4
