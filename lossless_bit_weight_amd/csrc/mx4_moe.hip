// mx4_moe.hip -- a mixture-of-experts layer for a few tokens on MX4 weights
// (../../include/mx4.h states the operation).
//
// Up to 16 tokens four launches.  route: each token's experts and their shares, and
// the pairs (token, expert) sorted by expert and cut into slots of at most 16.  up:
// per slot the products with the gate and up rows and h = silu(g) * u.  down: per
// slot the products of h with the down rows.  join: each token's weighted sum.
// Above, a fifth before them (choose): the experts of each token.  One token, and few
// that would seldom share an expert, take two launches: up, where a token chooses
// for itself, and down over all its experts, which writes y.
// The chosen experts' weights are read once (an expert with more than 16 tokens:
// once a slot, the later reads from cache), which is what bounds the layer;
// activations and pair outputs are hundredths of them.
#include <type_traits>

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

// Largest value of the wave, in every lane: within rows of 16 lanes, across them,
// then read from the last lane (a lane without a source keeps its own value).
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
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// A token's logits over a wave: lane l holds the experts EV l .. EV l + EV - 1, so
// that the lowest lane of a tie has the lowest expert.
template <int EV>
struct Logits {
    float l[EV];
    uint32_t key[EV];

    __device__ __forceinline__ void load(const float* p, int E, int lane) {
#pragma unroll
        for (int i = 0; i < EV; ++i) {
            const int e = EV * lane + i;
            l[i] = e < E ? p[e] : -__builtin_inff();
        }
    }
    __device__ __forceinline__ void rank(int E, int lane) {
#pragma unroll
        for (int i = 0; i < EV; ++i) key[i] = EV * lane + i < E ? order_key(l[i]) : 0u;
    }
    // The expert with the largest key, struck out, and its logit; -1 when only -inf
    // is left.
    __device__ __forceinline__ int take(int lane, float& logit) {
        uint32_t best = key[0];
        int at = 0;
        float v = l[0];
#pragma unroll
        for (int i = 1; i < EV; ++i) {
            const bool more = key[i] > best;
            const uint32_t k = key[i];
            const float f = l[i];
            best = more ? k : best;
            at = more ? i : at;
            v = more ? f : v;
        }
        const uint32_t m = wave_max(best);
        if (m <= kKeyNegInf) return -1;
        const int src = __builtin_ctzll(__ballot(best == m));
        const int e = EV * src + __builtin_amdgcn_readlane(at, src);
        logit = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), src));
#pragma unroll
        for (int i = 0; i < EV; ++i) key[i] = lane == src && i == at ? 0u : key[i];
        return e;
    }
    // sum of exp(logit - top) over all experts
    __device__ __forceinline__ float total(float top) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EV; ++i)
            if (l[i] != -__builtin_inff()) s += expf(l[i] - top);
        return wave_sum(s);
    }
};

// The wave's token t: lane j gets its j-th expert (or -1) and that expert's share.
template <int EV>
__device__ __forceinline__ int choose(const MoeArgs& a, int t, int lane, float& p) {
    Logits<EV> g;
    g.load(a.logits + t * a.ldl, a.E, lane);
    g.rank(a.E, lane);
    float top = 0.f, mine = 0.f;
    int mine_e = -1;
    for (int j = 0; j < a.top_k; ++j) {
        float v = 0.f;
        const int e = g.take(lane, v);
        if (e < 0) break;
        if (j == 0) top = v;
        if (lane == j) {
            mine = v;
            mine_e = e;
        }
    }
    const float ex = mine_e >= 0 ? expf(mine - top) : 0.f;
    const float sum = a.renormalize ? wave_sum(ex) : g.total(top);
    p = mine_e < 0 ? 0.f : ex / sum;
    return mine_e;
}

// Above 16 tokens: the choice by itself, one token a wave (61 tokens, 8 of 127
// experts: with 16 waves taking them in turn route took 16 us, most of it
// issuing the reductions; now 4 + 6).
constexpr int kRouteTokens = kRouteThreads / 64;
template <int EV>
__global__ __launch_bounds__(256) void choose_kernel(MoeArgs a) {
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (t >= a.T) return;
    float p;
    const int e = choose<EV>(a, t, lane, p);
    if (lane < a.top_k) {
        a.place[t * a.top_k + lane] = e;
        a.share[t * a.top_k + lane] = p;
    }
}

// One workgroup.  Tokens per expert are kept as 128-bit sets, so the sorted place
// of a pair is a count of bits and depends on no order of execution.
template <int EV>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(MoeArgs a) {
    __shared__ uint32_t set[kMaxExperts][4];
    __shared__ int base[kMaxExperts];
    __shared__ int wave_tot[2][kRouteThreads / 64];
    __shared__ int16_t chosen[kMaxTokens * kMaxTopK];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    for (int i = tid; i < a.E * 4; i += kRouteThreads) (&set[0][0])[i] = 0;
    __syncthreads();

    if (a.T > kRouteTokens) {
        for (int i = tid; i < a.T * a.top_k; i += kRouteThreads) {
            const int e = a.place[i], t = i / a.top_k;
            chosen[i] = (int16_t)e;
            if (e >= 0) atomicOr(&set[e][t >> 5], 1u << (t & 31));
        }
    } else if (w < a.T) {
        float p;
        const int e = choose<EV>(a, w, lane, p);
        if (lane < a.top_k) {
            chosen[w * a.top_k + lane] = (int16_t)e;
            a.share[w * a.top_k + lane] = p;
            if (e >= 0) atomicOr(&set[e][w >> 5], 1u << (w & 31));
        }
    }
    __syncthreads();

    // exclusive sums over the experts of their pairs and slots
    uint32_t mask[4] = {0, 0, 0, 0};
    int cnt = 0;
    if (tid < a.E) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mask[i] = set[tid][i];
            cnt += __popc(mask[i]);
        }
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
    int total = 0;
    for (int i = 0; i < kRouteThreads / 64; ++i) {
        if (i < w) {
            ip += wave_tot[0][i];
            is += wave_tot[1][i];
        }
        total += wave_tot[1][i];
    }
    if (tid < a.E) {
        base[tid] = ip - cnt;
        int word = 0, first = 0;
        for (int i = 0; i < ns; ++i) {
            int* s = a.slots + (is - ns + i) * kSlotWords;
            const int n = cnt - 16 * i < 16 ? cnt - 16 * i : 16;
            s[0] = tid;
            s[1] = n;
            s[2] = ip - cnt + 16 * i;
            for (int j = 0; j < 16; ++j) {
                if (j < n) {
                    while (mask[word] == 0) ++word;
                    const int t = 32 * word + __builtin_ctz(mask[word]);
                    mask[word] &= mask[word] - 1;
                    if (j == 0) first = t;
                    s[16 + j] = t;
                } else {
                    s[16 + j] = first;
                }
            }
        }
    }
    for (int i = total + tid; i < a.max_slots; i += kRouteThreads) a.slots[i * kSlotWords + 1] = 0;
    __syncthreads();

    for (int i = tid; i < a.T * a.top_k; i += kRouteThreads) {
        const int e = chosen[i];
        int p = -1;
        if (e >= 0) {
            const int t = i / a.top_k;
            p = base[e];
            for (int j = 0; j < (t >> 5); ++j) p += __popc(set[e][j]);
            p += __popc(set[e][t >> 5] & ((1u << (t & 31)) - 1u));
        }
        a.place[i] = p;
    }
}

// ---- hidden values --------------------------------------------------------------------
// h goes to the matrix units as three BF16 numbers whose sum it is: all 24 bits of its
// mantissa, whatever the output's type (two of them would differ from an fp32 product
// by 2^-16 of h, which differences of hidden values do not hide).  Up stores it whole,
// 4 bytes that down splits (BF16 outputs, whose workspace stays as small), or as its
// parts, 6 bytes (fp32 outputs).  Neither is always the faster; whole layer, us, fp32
// output, whole / parts: 16 tokens, 6 of 64 experts, H = 5120, I = 1280 103.9 / 104.7;
// 61 tokens, 8 of 127, H = 2080, I = 736 86.2 / 89.2; 128 tokens, 2 of 8, H = 4096,
// I = 14336 337 / 328.
enum Hidden { kF32, kParts };

// V values of h (an infinity's rest is 0; a NaN that arithmetic made keeps its quiet bit
// in the upper half).
template <int V>
struct Values {
    typedef float f32_t __attribute__((ext_vector_type(V)));
    typedef uint32_t u32_t __attribute__((ext_vector_type(V / 2)));
    f32_t f;
    __device__ __forceinline__ void load(const float* p) {
        f = *reinterpret_cast<const f32_t*>(p);
    }
    // Part P of them, in order: the upper half of each number's bits, which are taken off.
    template <int P>
    __device__ __forceinline__ void take(uint8_t* to) {
        u32_t v;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            uint32_t b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = f[2 * j + i];
                b[i] = __float_as_uint(x);
                if (P < 2) f[2 * j + i] = x - __uint_as_float(b[i] & 0xFFFF0000u);
                if (P < 1 && __builtin_isinf(x)) f[2 * j + i] = 0.f;
            }
            v[j] = __builtin_amdgcn_perm(b[1], b[0], 0x07060302u);
        }
        *reinterpret_cast<u32_t*>(to) = v;
    }
    // Part p of them (zeros unless `in`) to place(p).
    template <class Place>
    __device__ __forceinline__ void split(bool in, Place place) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = in ? f[i] : 0.f;
        take<0>(place(0));
        take<1>(place(1));
        take<2>(place(2));
    }
};
// of a piece of eight that a thread takes where `pieces` of them are for `threads`
constexpr int values_each(int pieces, int threads) {
    return pieces >= threads ? 8 : pieces * 2 >= threads ? 4 : 2;
}

// ---- the experts' products -----------------------------------------------------------
// A workgroup: one slot by WN waves' weight tiles (up: a gate tile and the up tile
// beside it a wave; down: R tiles); KW groups of such waves take every KW-th unit
// of UG groups of K.  Weights come to registers a unit ahead of their products;
// the slot's rows (of x, gathered by token, or of h in PARTS parts) go through
// LDS, double-buffered, in the layout of mx4_gemm.hip's few-row kernel, ROWS of
// them: slots of up to four rows, the most by far, move a quarter of the bytes, and
// read weights that no other slot does (H = 5120, I = 1280: 16 tokens, 6 of 64 experts
// 105 us past the caches, 117 through them; 128 tokens, 8 of 64 the reverse, 209 and 199).
template <bool UP, int R, int WN, int KW, int UG4, int UG16>
struct Expert {
    static constexpr int PARTS = UP ? 1 : 3;
    // four groups of waves on h: one buffer, behind one more barrier a unit, so that two
    // workgroups fit a CU (12 tokens, 2 of 8 experts, H = 4096, I = 14336 169 -> 147 us)
    static constexpr int kBuffers = !UP && KW == 4 ? 1 : 2;
    static constexpr int kThreads = WN * KW * 64;
    static constexpr int ug(int rows) { return rows > 4 ? UG16 : UG4; }
    static constexpr int pieces(int rows) { return rows * 16 * ug(rows) * PARTS; }
    static constexpr int stage(int rows) {
        return (pieces(rows) + WN * 64 - 1) / (WN * 64) * (WN * 64) * 16;
    }
    static constexpr int lds(int rows) {
        const int x4 = kBuffers * KW * stage(4), x16 = rows > 4 ? kBuffers * KW * stage(16) : 0;
        const int x = x4 > x16 ? x4 : x16, red = KW * WN * R * 1024;
        return x > red ? x : red;
    }
};

template <int ROWS, bool UP, Hidden F, int R, int WN, int KW, int UG4, int UG16>
__device__ __forceinline__ void expert_body(const MoeArgs& a, const int* slot, int e, int count,
                                            int p0, int block, uint8_t* lds) {
    using X = Expert<UP, R, WN, KW, UG4, UG16>;
    constexpr bool kSplit = !UP && F == kF32;   // h comes whole and is split here
    constexpr int UG = X::ug(ROWS), PARTS = X::PARTS;
    constexpr int kStage = X::stage(ROWS);
    constexpr int kPart = ROWS * 16 * UG;       // pieces of one part of a unit
    constexpr int V = kSplit ? values_each(kPart, WN * 64) : 8;     // values a thread at a time
    constexpr int P = kSplit ? kPart * 8 / (V * WN * 64) : kStage / (WN * 64 * 16);
    static_assert(!kSplit || P * V * WN * 64 == kPart * 8, "every thread has as many");
    using Piece = std::conditional_t<kSplit, Values<V>, u32x4_t>;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = w / WN, wn = w % WN;
    const int c = lane & 15, q = lane >> 4;
    const int K = UP ? a.H : a.I;
    const int G = (int)groups(K), Q = (int)quads(K);
    const int U = (G + UG - 1) / UG, its = (U + KW - 1) / KW;
    const int nt = (UP ? a.I : a.H) / 16;       // tiles of this product's outputs
    const uint32_t lane16 = lane * 16, lane4 = lane * 4;
    const int64_t pairs = (int64_t)a.T * a.top_k;

    const uint8_t* wp[R];
    const uint8_t* sp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        int64_t t;
        if constexpr (UP) {
            const int j = block * WN + wn;
            t = (int64_t)e * 2 * nt + r * nt + (j < nt ? j : nt - 1);
        } else {
            const int j = (block * WN + wn) * R + r;
            t = (int64_t)e * nt + (j < nt ? j : nt - 1);
        }
        const Mat& m = UP ? a.w13 : a.w2;
        wp[r] = m.codes + t * G * kCodeBlock;
        sp[r] = m.scales + t * Q * kScaleBlock;
    }
    using Value = std::conditional_t<kSplit, float, uint16_t>;
    const Value* xp[P];
    int xk[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int value = ((i * WN + wn) * 64 + lane) * V, piece = value / 8;
        int part = piece / kPart;
        if (part > PARTS - 1) part = PARTS - 1;
        const int row = piece % kPart / (16 * UG);
        if constexpr (UP)
            xp[i] = a.x + (slot == nullptr ? 0 : slot[16 + row] * a.ldx);
        else if constexpr (kSplit)
            xp[i] = static_cast<const float*>(a.h) +
                    (p0 + (row < count ? row : 0)) * (int64_t)a.I;
        else
            xp[i] = static_cast<const uint16_t*>(a.h) +
                    (part * pairs + p0 + (row < count ? row : 0)) * (int64_t)a.I;
        xk[i] = value % (128 * UG);
    }
    uint8_t* mine = lds + kw * X::kBuffers * kStage;
    u32x4_t wb[2][UG][R];
    Piece xb[P];
    uint32_t ws[2][R];
    bool xin[P];
    // (no branch: a place past the last unit, group or K is a valid one whose x is
    // replaced by zeros)
    auto load = [&](int s, int it) {
        const int u = it * KW + kw;
        const int uc = u < U ? u : U - 1;
        const int64_t so = (int64_t)(uc * UG / 4) * kScaleBlock;
        const int shift = UG == 4 ? 0 : 8 * UG * (uc % (4 / UG));
#pragma unroll
        for (int r = 0; r < R; ++r)
            ws[s][r] = *reinterpret_cast<const uint32_t*>(scalar(sp[r] + so) + lane4) >> shift;
#pragma unroll
        for (int j = 0; j < UG; ++j) {
            const int g = uc * UG + j < G ? uc * UG + j : G - 1;
#pragma unroll
            for (int r = 0; r < R; ++r)
                wb[s][j][r] =
                    load16<ROWS == 4>(scalar(wp[r] + (int64_t)g * kCodeBlock) + lane16);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = u * UG * 128 + xk[i];
            xin[i] = u < U && k < K;
            if constexpr (kSplit)
                xb[i].load(xp[i] + (xin[i] ? k : 0));
            else
                xb[i] = *reinterpret_cast<const u32x4_t*>(xp[i] + (xin[i] ? k : 0));
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int value = ((i * WN + wn) * 64 + lane) * V;
            const auto place = [&](int p) {
                const int piece = value / 8 + p * kPart;
                const int at = (piece & ~15) + x_place(piece & 15, piece / (16 * UG));
                return mine + (X::kBuffers > 1 ? buf * kStage : 0) + at * 16 + value % 8 * 2;
            };
            if constexpr (kSplit) {
                xb[i].split(xin[i], place);
            } else {
                u32x4_t v;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = xin[i] ? xb[i][k] : 0u;
                *reinterpret_cast<u32x4_t*>(place(0)) = v;
            }
        }
    };
    f32x4_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
    // four rows leave columns of the operand for their parts: column 4 p + m is part p
    // of row m (the last four are the third part once more, unused), one matrix
    // instruction instead of three (16 tokens, 6 of 64 experts, H = 5120, I = 1280
    // 109.0 -> 104.4 us)
    constexpr bool kColumns = !UP && ROWS == 4;
    constexpr int kOperands = kColumns ? 1 : PARTS;
    const int row = kColumns ? (c < 12 ? c : c - 4) : c & (ROWS - 1);
    auto product = [&](auto sc) {
        constexpr int s = decltype(sc)::value;
        const uint8_t* xl = mine + (X::kBuffers > 1 ? s * kStage : 0);
#pragma unroll
        for (int j = 0; j < UG; ++j) {
            float f[R];
#pragma unroll
            for (int r = 0; r < R; ++r) f[r] = scale_f32((ws[s][r] >> (8 * j)) & 255u);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                bf16x8_t xv[kOperands];
#pragma unroll
                for (int p = 0; p < kOperands; ++p)
                    xv[p] = *reinterpret_cast<const bf16x8_t*>(
                        xl + (p * kPart + row * 16 * UG + 16 * j + x_place(q, b, row)) * 16);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const bf16x8_t wv = expand8(wb[s][j][r][b], f[r]);
#pragma unroll
                    for (int p = 0; p < kOperands; ++p) acc[r] = mfma_bf16(wv, xv[p], acc[r]);
                }
            }
        }
    };
    load(0, 0);
    stage(0);
    __syncthreads();
    auto step = [&](auto sc, int it) {
        constexpr int s = decltype(sc)::value;
        load(s ^ 1, it + 1);
        __builtin_amdgcn_sched_barrier(0);
        product(sc);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (X::kBuffers == 1) __syncthreads();
        stage(s ^ 1);
        __syncthreads();
    };
    for (int it = 0; it < its; it += 2) {
        step(std::integral_constant<int, 0>{}, it);
        if (it + 1 >= its) break;
        step(std::integral_constant<int, 1>{}, it + 1);
    }
    __syncthreads();

    float* red = reinterpret_cast<float*>(lds);         // [KW][WN][R][256]
#pragma unroll
    for (int r = 0; r < R; ++r)
        *reinterpret_cast<f32x4_t*>(red + (w * R + r) * 256 + lane * 4) = acc[r];
    __syncthreads();
    constexpr int kCols = UP ? 16 * WN : 16 * R * WN;
    for (int i = tid; i < ROWS * kCols; i += X::kThreads) {
        const int m = i / kCols, col = i % kCols;
        const int n = block * kCols + col, wr = col & 15;
        if (m >= count || n >= nt * 16) continue;
        const int in = ((wr >> 2) * 16 + m) * 4 + (wr & 3);
        if constexpr (UP) {
            const int at = col / 16 * R * 256 + in;
            float g = 0.f, u = 0.f;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                g += red[k * WN * R * 256 + at];
                u += red[k * WN * R * 256 + 256 + at];
            }
            const float h = g / (1.f + expf(-g)) * u;
            const int64_t at_h = (int64_t)(p0 + m) * a.I + n;
            if (!a.y_f32) {
                static_cast<float*>(a.h)[at_h] = h;
                continue;
            }
            // the parts as Values::take has them (rounded to nearest, the first of the
            // largest finite numbers would be infinite)
            uint16_t* o = static_cast<uint16_t*>(a.h) + at_h;
            float rest = h;
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const uint32_t b = __float_as_uint(rest);
                o[p * pairs * a.I] = (uint16_t)(b >> 16);
                rest = __builtin_isinf(rest) ? 0.f : rest - __uint_as_float(b & 0xFFFF0000u);
            }
        } else {
            const int at = col / 16 * 256 + in;
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const float* v = red + k * WN * R * 256 + at;
                s += kColumns ? v[0] + (v[16] + v[32]) : v[0];
            }
            a.out[(int64_t)(p0 + m) * a.H + n] = s;
        }
    }
}

template <bool MANY, bool UP, Hidden F, int R, int WN, int KW, int UG4, int UG16>
__global__ __launch_bounds__(WN* KW * 64) void expert_kernel(MoeArgs a, int blocks) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int* slot = a.slots + (blockIdx.x / blocks) * kSlotWords;
    const int e = slot[0], count = slot[1], p0 = slot[2], block = blockIdx.x % blocks;
    if (count == 0) return;
    if (MANY && count > 4)
        expert_body<16, UP, F, R, WN, KW, UG4, UG16>(a, slot, e, count, p0, block, lds);
    else
        expert_body<4, UP, F, R, WN, KW, UG4, UG16>(a, slot, e, count, p0, block, lds);
}

// up for few tokens, each by itself (blockIdx.y): the token chooses for itself, slot
// s is its expert with the s-th largest logit, found by every wave; the slot's first
// workgroup writes its words for down.
template <int EV, int WN, int KW, int UG>
__global__ __launch_bounds__(WN* KW * 64) void up_one_kernel(MoeArgs a, int blocks) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int s = blockIdx.x / blocks, block = blockIdx.x % blocks, lane = threadIdx.x & 63;
    const int t = blockIdx.y, pair = t * a.top_k + s;
    a.x += t * a.ldx;
    Logits<EV> g;
    g.load(a.logits + t * a.ldl, a.E, lane);
    g.rank(a.E, lane);
    float top = 0.f, mine = 0.f, sum = 0.f;
    int e = -1;
    const int rounds = block == 0 ? a.top_k : s + 1;
    for (int j = 0; j < rounds; ++j) {
        float v = 0.f;
        const int found = g.take(lane, v);
        if (found < 0) break;
        if (j == 0) top = v;
        if (j == s) {
            e = found;
            mine = v;
        }
        sum += expf(v - top);
    }
    if (block == 0) {
        if (!a.renormalize) sum = g.total(top);
        if (threadIdx.x == 0) {
            int* o = a.slots + pair * kSlotWords;
            o[0] = e;
            o[3] = __float_as_int(expf(mine - top) / sum);
        }
    }
    if (e < 0) return;
    expert_body<4, true, kF32, 2, WN, KW, UG, UG>(a, nullptr, e, 1, pair, block, lds);
}

// ---- down for few tokens -------------------------------------------------------------
// A workgroup: WN tiles of 16 outputs of one token (blockIdx.y).  The units (expert,
// UG groups of its hidden values) are one sequence of which each of the KW groups of
// waves takes every KW-th; a unit's product is weighted into the sum at once, and no
// pair's output goes through memory.
template <int WN, int KW, int UG>
struct One {
    static constexpr int PARTS = 3;
    static constexpr int kThreads = WN * KW * 64;
    static constexpr int kPieces = 16 * UG * PARTS;
    static constexpr int kStage = (kPieces + WN * 64 - 1) / (WN * 64) * (WN * 64) * 16;
    static constexpr int lds() {
        const int x = 2 * KW * kStage, red = KW * WN * PARTS * 64;
        return x > red ? x : red;
    }
};

template <Hidden F, int WN, int KW, int UG>
__global__ __launch_bounds__(WN* KW * 64) void down_one_kernel(MoeArgs a) {
    using X = One<WN, KW, UG>;
    constexpr bool kSplit = F == kF32;
    constexpr int PARTS = X::PARTS, kPart = 16 * UG;
    constexpr int V = kSplit ? values_each(kPart, WN * 64) : 8;
    constexpr int P = kSplit ? kPart * 8 / (V * WN * 64) : X::kStage / (WN * 64 * 16);
    static_assert(!kSplit || P * V * WN * 64 == kPart * 8, "every thread has as many");
    using Piece = std::conditional_t<kSplit, Values<V>, u32x4_t>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = w / WN, wn = w % WN;
    const int q = lane >> 4, first = blockIdx.y * a.top_k;      // the token's first pair
    const int G = (int)groups(a.I), Q = (int)quads(a.I), UI = (G + UG - 1) / UG;
    const int ht = a.H / 16;
    const int tile = blockIdx.x * WN + wn < ht ? blockIdx.x * WN + wn : ht - 1;
    const uint32_t lane16 = lane * 16, lane4 = lane * 4;

    // lane j holds the j-th expert and its share; the used ones come first
    int expert = -1;
    float share = 0.f;
    if (lane < a.top_k) {
        const int* s = a.slots + (first + lane) * kSlotWords;
        expert = s[0];
        share = __int_as_float(s[3]);
    }
    const int units = (int)__popcll(__ballot(expert >= 0)) * UI;
    const int its = (units + KW - 1) / KW;

    uint8_t* mine = lds + kw * 2 * X::kStage;
    u32x4_t wb[2][UG];
    Piece xb[P];
    uint32_t ws[2];
    bool xin[P];
    auto load = [&](int s, int it) {
        const int u = it * KW + kw;
        const int uc = u < units ? u : units - 1;
        const int sl = uc / UI, ui = uc % UI;
        const int64_t t = (int64_t)__builtin_amdgcn_readlane(expert, sl) * ht + tile;
        const uint8_t* wp = a.w2.codes + t * G * kCodeBlock;
        ws[s] = *reinterpret_cast<const uint32_t*>(
                    scalar(a.w2.scales + (t * Q + ui * UG / 4) * kScaleBlock) + lane4) >>
                (UG == 4 ? 0 : 8 * UG * (ui % (4 / UG)));
#pragma unroll
        for (int j = 0; j < UG; ++j) {
            const int g = ui * UG + j < G ? ui * UG + j : G - 1;
            wb[s][j] = load16_nt(scalar(wp + (int64_t)g * kCodeBlock) + lane16);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int value = ((i * WN + wn) * 64 + lane) * V, piece = value / 8;
            const int part = piece / kPart < PARTS ? piece / kPart : PARTS - 1;
            const int k = ui * UG * 128 + value % (128 * UG);
            xin[i] = u < units && k < a.I;
            using Value = std::conditional_t<kSplit, float, uint16_t>;
            const int64_t row = (kSplit ? 0 : (int64_t)part * a.T * a.top_k) + first + sl;
            const Value* p = static_cast<const Value*>(a.h) + row * a.I + (k < a.I ? k : 0);
            if constexpr (kSplit)
                xb[i].load(p);
            else
                xb[i] = *reinterpret_cast<const u32x4_t*>(p);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int value = ((i * WN + wn) * 64 + lane) * V;
            const auto place = [&](int p) {
                const int piece = value / 8 + p * kPart;
                const int at = (piece & ~15) + x_place(piece & 15, piece / kPart * 4);
                return mine + buf * X::kStage + at * 16 + value % 8 * 2;
            };
            if constexpr (kSplit) {
                xb[i].split(xin[i], place);
            } else {
                u32x4_t v;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = xin[i] ? xb[i][k] : 0u;
                *reinterpret_cast<u32x4_t*>(place(0)) = v;
            }
        }
    };
    // the first three columns of the operand hold the parts, the others the third again
    const int column = (lane & 15) < PARTS ? lane & 15 : PARTS - 1;
    f32x4_t sum = {0, 0, 0, 0};
    auto product = [&](auto sc, int it) {
        constexpr int s = decltype(sc)::value;
        const uint8_t* xl = mine + s * X::kStage;
        f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < UG; ++j) {
            const float f = scale_f32((ws[s] >> (8 * j)) & 255u);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const bf16x8_t wv = expand8(wb[s][j][b], f);
                const int at = column * kPart + 16 * j + x_place(q, b, column * 4);
                acc = mfma_bf16(wv, *reinterpret_cast<const bf16x8_t*>(xl + at * 16), acc);
            }
        }
        const int u = it * KW + kw;
        const float f = __int_as_float(__builtin_amdgcn_readlane(
            __float_as_int(share), (u < units ? u : units - 1) / UI));
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += u < units ? f * acc[i] : 0.f;
    };
    if (units > 0) {
        load(0, 0);
        stage(0);
        __syncthreads();
        auto step = [&](auto sc, int it) {
            constexpr int s = decltype(sc)::value;
            load(s ^ 1, it + 1);
            __builtin_amdgcn_sched_barrier(0);
            product(sc, it);
            __builtin_amdgcn_sched_barrier(0);
            stage(s ^ 1);
            __syncthreads();
        };
        for (int it = 0; it < its; it += 2) {
            step(std::integral_constant<int, 0>{}, it);
            if (it + 1 >= its) break;
            step(std::integral_constant<int, 1>{}, it + 1);
        }
    }
    __syncthreads();
    float* red = reinterpret_cast<float*>(lds);         // [KW][WN][PARTS][16]
    if ((lane & 15) < PARTS)
        *reinterpret_cast<f32x4_t*>(red + (w * PARTS + column) * 16 + 4 * q) = sum;
    __syncthreads();
    const int n = blockIdx.x * 16 * WN + tid;
    if (tid < 16 * WN && n < a.H) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < KW; ++k) {
            const float* r = red + ((k * WN + tid / 16) * PARTS) * 16 + tid % 16;
            v += r[0] + (r[16] + r[32]);
        }
        const int64_t at = blockIdx.y * a.ldy + n;
        if (a.y_f32)
            static_cast<float*>(a.y)[at] = v;
        else
            static_cast<uint16_t*>(a.y)[at] = bf16_bits(v);
    }
}

// y[t] = sum of its experts' outputs, weighted, in the order of their choice.
__global__ __launch_bounds__(256) void join_kernel(MoeArgs a) {
    const int n = (blockIdx.x * 256 + threadIdx.x) * 4, t = blockIdx.y;
    if (n >= a.H) return;
    f32x4_t s = {0, 0, 0, 0};
    for (int j = 0; j < a.top_k; ++j) {
        const int p = a.place[t * a.top_k + j];
        if (p < 0) continue;
        const float f = a.share[t * a.top_k + j];
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(a.out + (int64_t)p * a.H + n);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += f * v[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (a.y_f32)
            static_cast<float*>(a.y)[t * a.ldy + n + i] = s[i];
        else
            static_cast<uint16_t*>(a.y)[t * a.ldy + n + i] = bf16_bits(s[i]);
    }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Each token by itself, weights that several of them chose read again: two launches
// instead of four, at the cost of the repeated bytes.  Whole layer, us, so / by slots,
// and the bytes expected: 2 tokens, 2 of 8 experts, H = 5120, I = 1280 18.7 / 23.7 (5 MB);
// 4 tokens, 8 of 127, H = 2080, I = 736 31.3 / 31.6 (7 MB); 3 tokens, 6 of 64, H = 4096,
// I = 1408 42.0 / 46.8 (16 MB); 16 tokens, 4 of 64, H = 1024, I = 512 26.4 / 23.7 (25 MB);
// 4 tokens, 6 of 64, H = 5120, I = 1280 58.7 / 55.1 (35 MB); 32 tokens, 1 of 22,
// H = 800, I = 320 18.4 / 18.8 (9 MB), 64, 1 of 64, 31.1 / 21.8 (13 MB).
constexpr int kOneByOne = 32;               // tokens
constexpr int64_t kRepeatedBytes = 16 << 20;
bool one_by_one(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    if (T > kOneByOne) return false;
    // tokens that choose evenly: two of them share top_k^2 / E experts
    return T * (T - 1) / 2 * top_k * top_k * (3 * H * I / 32 * 17 / E) <= kRepeatedBytes;
}

int64_t max_slots(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    const int64_t pairs = T * top_k;
    return one_by_one(T, H, I, E, top_k) ? pairs : (E < pairs ? E : pairs) + pairs / 16;
}

template <bool UP, Hidden F, int R, int WN, int KW, int UG4, int UG16>
void launch_expert(const MoeArgs& a, hipStream_t s) {
    using X = Expert<UP, R, WN, KW, UG4, UG16>;
    static_assert(X::lds(16) <= 65536, "more LDS than a launch gets without asking");
    const int nt = (UP ? a.I : a.H) / 16, per = UP ? WN : WN * R;
    const int blocks = (nt + per - 1) / per;
    const dim3 grid((unsigned)((int64_t)a.max_slots * blocks)), block(X::kThreads);
    if (a.T <= 4)
        hipLaunchKernelGGL((expert_kernel<false, UP, F, R, WN, KW, UG4, UG16>), grid, block,
                           X::lds(4), s, a, blocks);
    else
        hipLaunchKernelGGL((expert_kernel<true, UP, F, R, WN, KW, UG4, UG16>), grid, block,
                           X::lds(16), s, a, blocks);
}

// Waves beside each other share a slot's rows, waves that split K let a few slots fill
// the GPU.  Up, H = 5120, I = 1280, 12 tokens, 2 of 8 experts (at most 360 workgroups of
// 2 x 2 waves): whole layer 38.0 us, with 1 x 4 waves 37.3; 48 tokens, 2 of 16 (880):
// 57.3 and 61.7.  Above four rows a slot units of two groups: 128 tokens, 4 of 16, 103
// with units of one, 96.
void launch_up(const MoeArgs& a, hipStream_t s) {
    if ((int64_t)a.max_slots * ((a.I + 31) / 32) < 512)
        launch_expert<true, kF32, 2, 1, 4, 2, 1>(a, s);
    else
        launch_expert<true, kF32, 2, 2, 2, 2, 2>(a, s);
}

// Down, by workgroups of 4 x 1 waves, 2 x 2 and 2 x 4, whole layer, us.  16 tokens, 6 of 64
// experts, H = 5120, I = 1280 (2800 of 4 x 1): 104.4 by the first, 106.5 by the second.
// 2 of 8 experts, H = 4096, I = 14336: 128 tokens (768) 337 by the first; 80 tokens (576)
// 293 by the second, 274 by the third; 12 tokens (288) 169 and 147.  H = 1024: 24 tokens,
// 2 of 8, I = 1024 24.5 and 23.4; 16 tokens, 4 of 64, I = 512 23.5 and 25.1; H = 2048,
// 16 tokens, 4 of 32, I = 768 32.6 and 33.5.
template <Hidden F>
void launch_down(const MoeArgs& a, hipStream_t s) {
    if ((int64_t)a.max_slots * ((a.H + 127) / 128) >= 640)
        launch_expert<false, F, 2, 4, 1, 1, 1>(a, s);
    else if (a.I >= 1024)
        launch_expert<false, F, 2, 2, 4, 1, 1>(a, s);
    else
        launch_expert<false, F, 2, 2, 2, 1, 1>(a, s);
}

template <int EV>
void launch_up_one(const MoeArgs& a, hipStream_t s) {
    constexpr int WN = 1, KW = 4, UG = 4;   // (1, 8, 2): 12.9 against 12.1 us at H = 5120, I = 1280
    using X = Expert<true, 2, WN, KW, UG, UG>;
    const int blocks = (a.I / 16 + WN - 1) / WN;
    const dim3 grid((unsigned)(a.top_k * blocks), (unsigned)a.T);
    hipLaunchKernelGGL((up_one_kernel<EV, WN, KW, UG>), grid, dim3(X::kThreads), X::lds(4), s, a,
                       blocks);
}

template <Hidden F, int WN, int KW, int UG>
void launch_down_one(const MoeArgs& a, hipStream_t s) {
    using X = One<WN, KW, UG>;
    static_assert(X::lds() <= 65536, "more LDS than a launch gets without asking");
    hipLaunchKernelGGL((down_one_kernel<F, WN, KW, UG>),
                       dim3((unsigned)((a.H / 16 + WN - 1) / WN), (unsigned)a.T),
                       dim3(X::kThreads), X::lds(), s, a);
}

template <int EV>
void launch_route(const MoeArgs& a, hipStream_t s) {
    if (a.T > kRouteTokens)
        hipLaunchKernelGGL(choose_kernel<EV>, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a);
    hipLaunchKernelGGL(route_kernel<EV>, dim3(1), dim3(kRouteThreads), 0, s, a);
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k, bool y_f32) {
    const int64_t pairs = T * top_k;
    const size_t slots = up256((size_t)max_slots(T, H, I, E, top_k) * kSlotWords * 4);
    const size_t h = (size_t)pairs * I * (y_f32 ? 6 : 4);
    if (one_by_one(T, H, I, E, top_k)) return slots + h;
    return slots + 2 * up256((size_t)pairs * 4) + up256((size_t)pairs * H * 4) + h;
}

hipError_t launch_moe(MoeArgs a, void* ws, hipStream_t s) {
    const int64_t pairs = (int64_t)a.T * a.top_k;
    a.max_slots = (int)max_slots(a.T, a.H, a.I, a.E, a.top_k);
    uint8_t* p = static_cast<uint8_t*>(ws);
    a.slots = reinterpret_cast<int*>(p);
    p += up256((size_t)a.max_slots * kSlotWords * 4);
    a.h = p;

    const int ev = a.E <= 64 ? 1 : a.E <= 128 ? 2 : a.E <= 256 ? 4 : 16;
    if (one_by_one(a.T, a.H, a.I, a.E, a.top_k)) {
        switch (ev) {
            case 1: launch_up_one<1>(a, s); break;
            case 2: launch_up_one<2>(a, s); break;
            case 4: launch_up_one<4>(a, s); break;
            default: launch_up_one<16>(a, s);
        }
        if (a.y_f32)
            launch_down_one<kParts, 1, 8, 2>(a, s);
        else
            launch_down_one<kF32, 1, 8, 2>(a, s);
        return hipGetLastError();
    }
    a.place = reinterpret_cast<int*>(p);
    p += up256((size_t)pairs * 4);
    a.share = reinterpret_cast<float*>(p);
    p += up256((size_t)pairs * 4);
    a.out = reinterpret_cast<float*>(p);
    p += up256((size_t)pairs * a.H * 4);
    a.h = p;
    switch (ev) {
        case 1: launch_route<1>(a, s); break;
        case 2: launch_route<2>(a, s); break;
        case 4: launch_route<4>(a, s); break;
        default: launch_route<16>(a, s);
    }
    launch_up(a, s);
    if (a.y_f32)
        launch_down<kParts>(a, s);
    else
        launch_down<kF32>(a, s);
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)((a.H + 1023) / 1024), (unsigned)a.T), dim3(256),
                       0, s, a);
    return hipGetLastError();
}

}  // namespace mx4
