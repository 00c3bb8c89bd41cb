// mx4_gemm.hip -- y = x W^T with W in MX4 and x in BF16 or MX4
// (../../include/mx4.h has the format).
#include <type_traits>

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
hipError_t launch_small(GemmArgs a, hipStream_t s) {
    const unsigned nb = (unsigned)((tiles(a.N) + R - 1) / R);
    const int M = a.M;
    const int most = 65535 * 16;            // rows one grid covers
    for (int m = 0; m < M; m += most) {
        a.M = M - m < most ? M - m : most;
        const dim3 grid(nb, (unsigned)tiles(a.M));
        if (a.x == nullptr) {
            hipLaunchKernelGGL((small_kernel<R, KW, D, true>), grid, dim3(KW * 64), 0, s, a);
            a.xm.codes += (int64_t)65535 * a.G * kCodeBlock;
            a.xm.scales += (int64_t)65535 * a.Q * kScaleBlock;
        } else {
            hipLaunchKernelGGL((small_kernel<R, KW, D, false>), grid, dim3(KW * 64), 0, s, a);
            a.x += (int64_t)most * a.ldx;
        }
        a.y = static_cast<uint8_t*>(a.y) + (int64_t)most * a.ldy * (a.y_f32 ? 4 : 2);
    }
    return hipGetLastError();
}

// A uniform pointer the compiler keeps in scalar registers: folded with the lane's
// offset it would hold two vector registers through the loop.
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
    asm volatile("" : "+s"(p));
    return p;
}

// ---- many rows of x -------------------------------------------------------------
// A workgroup of WM x WN waves computes 16 MT WM rows of x by 16 R WN weight
// rows; a wave 16 MT by 16 R, its sums in registers.  Weight pieces go from
// memory to registers in the layout the matrix instructions take them (a group
// ahead), x through LDS, double-buffered, where the WN waves share it.
// BF16 x: LDS row m holds 16 pieces of 8 values, piece p at place p ^ (m % 16),
// so that the 16 rows a read takes one piece from lie in 16 different places.
// MX4 x: its own blocks, in lane order.
// Steps run over whole quads of groups, as the scales do: a group past the last
// has zeros for x in LDS, the last weight block and its padding scale.
template <int MT, int R, int WM, int WN, bool XM>
struct Tile {
    static constexpr int kThreads = WM * WN * 64;
    static constexpr int BM = 16 * MT * WM, BN = 16 * R * WN;
    static constexpr int kAllPieces = BM * (XM ? 4 : 16);           // of x a group
    static constexpr int kPieces = (kAllPieces + kThreads - 1) / kThreads;  // a thread
    static constexpr int kStage = kPieces * kThreads * 16;          // bytes of LDS a group
};

template <int MT, int R, int WM, int WN, bool XM, int MIN_WAVES>
__global__ __launch_bounds__(WM* WN * 64, MIN_WAVES) void tile_kernel(GemmArgs a, int mb, int nb) {
    using T = Tile<MT, R, WM, WN, XM>;
    constexpr int P = T::kPieces;
    constexpr int H0 = XM ? P : (P + 1) / 2;    // x pieces in flight in the first half step
    __shared__ __align__(16) uint8_t xs[2][T::kStage];

    // Consecutive workgroups go to the 8 XCDs in turn: give each XCD a run of
    // neighbouring tiles, rows of x fastest, so that its L2 serves their x and W.
    const int total = mb * nb;
    int id = blockIdx.x;
    {
        const int per = total / 8, extra = total % 8, xcd = id % 8;
        id = xcd * per + (xcd < extra ? xcd : extra) + id / 8;
    }
    const int group_n = 8;                      // tiles of W beside each other
    const int band = group_n * mb;
    const int n_first = id / band * group_n;
    const int width = nb - n_first < group_n ? nb - n_first : group_n;
    const int bn = n_first + id % band % width;
    const int bm = id % band / width;
    const int slice = blockIdx.y;

    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = w / WN, wn = w % WN;
    const int c = lane & 15, q = lane >> 4;
    const int m0 = bm * T::BM;
    const int gb = slice * a.gs;                // first group, a multiple of 4
    const int ge = gb + a.gs < a.G ? gb + a.gs : a.G;
    const int steps = (ge - gb + 3) / 4 * 4;

    // weights
    const int64_t last_tile = tiles(a.N) - 1;
    const uint8_t* wp[R];
    const uint8_t* sp[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        int64_t t = (int64_t)bn * (T::BN / 16) + wn * R + r;
        if (t > last_tile) t = last_tile;
        wp[r] = a.w.codes + t * a.G * kCodeBlock;
        sp[r] = a.w.scales + t * a.Q * kScaleBlock;
    }
    // the pointers are uniform, the lanes' places 32-bit offsets
    const uint32_t lane16 = lane * 16, lane4 = lane * 4;
    // x
    uint32_t voff[P];
    const uint32_t row_last = (uint32_t)(a.M - 1 - m0);
    const uint8_t* xbase;
    const uint8_t* xsp[XM ? MT : 1];
    if constexpr (XM) {
        const int64_t last = tiles(a.M) - 1;
        xbase = a.xm.codes;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            int64_t t = m0 / 16 + w + i * (T::kThreads / 64);   // (not loaded past kAllPieces)
            if (t > last) t = last;
            voff[i] = (uint32_t)(t - m0 / 16);       // tile beside the first
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            int64_t t = m0 / 16 + wm * MT + i;
            if (t > last) t = last;
            xsp[i] = a.xm.scales + t * a.Q * kScaleBlock;
        }
        xbase += (int64_t)(m0 / 16) * a.G * kCodeBlock;
    } else {
        xbase = reinterpret_cast<const uint8_t*>(a.x + (int64_t)m0 * a.ldx);
    }

    u32x4_t wreg[2][R], xreg[P];
    bool xin = true;
    uint32_t ws[2][R], xsc[2][XM ? MT : 1];
    auto load_w = [&](int slot, int g) {
        const int gg = g < ge ? g : ge - 1;
#pragma unroll
        for (int r = 0; r < R; ++r)
            wreg[slot][r] = *reinterpret_cast<const u32x4_t*>(
                scalar(wp[r] + (int64_t)gg * kCodeBlock) + lane16);
    };
    auto load_scales = [&](int slot, int g) {
        const int64_t o = (int64_t)((g < ge ? g : ge - 1) >> 2) * kScaleBlock;
#pragma unroll
        for (int r = 0; r < R; ++r) 
            ws[slot][r] = *reinterpret_cast<const uint32_t*>(scalar(sp[r] + o) + lane4);
        if constexpr (XM) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
                xsc[slot][i] = *reinterpret_cast<const uint32_t*>(scalar(xsp[i] + o) + lane4);
        }
    };
    // (no branch: a load past the last group, row or K reads a valid place and is
    // replaced by zeros or, past the last tile and step, never used)
    auto load_x = [&](int i, int g) {
        const int gg = g < ge ? g : ge - 1;
        bool in = g < ge;
        if constexpr (XM) {
            xreg[i] = *reinterpret_cast<const u32x4_t*>(
                scalar(xbase + ((int64_t)voff[i] * a.G + gg) * kCodeBlock) + lane16);
        } else {
            const bool k_in = 128 * gg + 8 * (tid & 15) < a.K;
            in = in && k_in;
            // computed anew in every step: eight kept offsets would cost more registers
            // than there are
            uint32_t stride = 2u * (uint32_t)a.ldx;
            asm volatile("" : "+s"(stride));
            uint32_t r = (tid >> 4) + i * (T::kThreads / 16);
            r = r < row_last ? r : row_last;
            xreg[i] = *reinterpret_cast<const u32x4_t*>(
                xbase + 256 * (int64_t)gg + (__umul24(r, stride) + (k_in ? 16u * (tid & 15) : 0u)));
        }
        xin = in;
    };
    auto store_x = [&](int i, int buf) {
        int at;
        if constexpr (XM) {
            at = (tid + i * T::kThreads) * 16;
        } else {
            const int r = (tid >> 4) + i * (T::kThreads / 16);
            at = r * 256 + (((tid & 15) ^ (r & 15)) << 4);
        }
        u32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = xin ? xreg[i][e] : 0u;
        *reinterpret_cast<u32x4_t*>(&xs[buf][at]) = v;
    };

    f32x4_t acc[MT][R];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[i][r] = f32x4_t{0, 0, 0, 0};

    load_w(0, gb);
    load_scales(0, gb);
#pragma unroll
    for (int i = 0; i < P; ++i) load_x(i, gb);
#pragma unroll
    for (int i = 0; i < P; ++i) store_x(i, 0);
    __syncthreads();

    auto step = [&](auto jc, int g) {
        constexpr int J = decltype(jc)::value;
        constexpr int cur = J & 1, nxt = cur ^ 1;
        load_w(nxt, g + 1);
#pragma unroll
        for (int i = 0; i < H0; ++i) load_x(i, g + 1);
        // x operands are read two tiles (of 16 rows) ahead of the products on them
        constexpr int U = MT / 2;
        const uint8_t* xl = &xs[cur][0];
        if constexpr (XM) {
            u32x4_t xv[2][2];
            auto read = [&](int slot, int u) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    xv[slot][h] = *reinterpret_cast<const u32x4_t*>(
                        xl + (wm * MT + 2 * u + h) * 1024 + lane16);
            };
            read(0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u + 1 < U) read((u + 1) & 1, u + 1);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        acc[2 * u + h][r] =
                            mfma_mx4<J>(operand4(wreg[cur][r]), operand4(xv[u & 1][h]),
                                        acc[2 * u + h][r], ws[0][r], xsc[0][2 * u + h]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) store_x(i, nxt);
        } else {
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = scale_f32((ws[0][r] >> (8 * J)) & 255u);
            bf16x8_t xv[2][2], wv[R];
            const uint8_t* xrow = xl + (wm * MT * 16 + c) * 256;
            auto read = [&](int slot, int v) {
                const int b = v / U, u = v % U;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    xv[slot][h] = *reinterpret_cast<const bf16x8_t*>(
                        xrow + (2 * u + h) * 4096 + (((4 * q + b) ^ c) << 4));
            };
            read(0, 0);
#pragma unroll
            for (int v = 0; v < 4 * U; ++v) {
                const int b = v / U, u = v % U;
                if (u == 0) {
#pragma unroll
                    for (int r = 0; r < R; ++r) wv[r] = expand8(wreg[cur][r][b], s[r]);
                }
                if (v + 1 < 4 * U) read((v + 1) & 1, v + 1);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        acc[2 * u + h][r] = mfma_bf16(wv[r], xv[v & 1][h], acc[2 * u + h][r]);
                __builtin_amdgcn_sched_barrier(0);
                if (v == 2 * U - 1) {
#pragma unroll
                    for (int i = 0; i < H0; ++i) store_x(i, nxt);
#pragma unroll
                    for (int i = H0; i < P; ++i) load_x(i, g + 1);
                }
            }
#pragma unroll
            for (int i = H0; i < P; ++i) store_x(i, nxt);
        }
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int g = gb; g < gb + steps; g += 4) {
        load_scales(1, g + 4);
        step(std::integral_constant<int, 0>{}, g);
        step(std::integral_constant<int, 1>{}, g + 1);
        step(std::integral_constant<int, 2>{}, g + 2);
        step(std::integral_constant<int, 3>{}, g + 3);
#pragma unroll
        for (int r = 0; r < R; ++r) ws[0][r] = ws[1][r];
        if constexpr (XM) {
#pragma unroll
            for (int i = 0; i < MT; ++i) xsc[0][i] = xsc[1][i];
        }
    }

    // lane (c, q): row c of a 16-row tile of x, weight rows 4 q .. 4 q + 3
    const int64_t n0 = (int64_t)bn * T::BN + wn * R * 16 + 4 * q;
    const bool f32 = a.S > 1 || a.y_f32;
    const int64_t ld = a.S > 1 ? a.N : a.ldy;
    uint8_t* out = a.S > 1 ? reinterpret_cast<uint8_t*>(a.part + (int64_t)slice * a.M * a.N)
                           : static_cast<uint8_t*>(a.y);
    const int size = f32 ? 4 : 2;
    // four outputs in one store where every row of y starts on such a boundary
    const bool wide = ld % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (4 * size - 1)) == 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + (wm * MT + i) * 16 + c;
        uint8_t* o = out + (m * ld + n0) * size;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int left = m < a.M ? (int)(a.N - n0 - 16 * r < 4 ? a.N - n0 - 16 * r : 4) : 0;
            uint8_t* p = o + 16 * r * size;
            const f32x4_t v = acc[i][r];
            if (left == 4 && wide) {
                if (f32)
                    *reinterpret_cast<f32x4_t*>(p) = v;
                else
                    *reinterpret_cast<u32x2_t*>(p) =
                        u32x2_t{bf16_bits(v[0]) | (uint32_t)bf16_bits(v[1]) << 16,
                                bf16_bits(v[2]) | (uint32_t)bf16_bits(v[3]) << 16};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e >= left) continue;
                    if (f32)
                        reinterpret_cast<float*>(p)[e] = v[e];
                    else
                        reinterpret_cast<uint16_t*>(p)[e] = bf16_bits(v[e]);
                }
            }
        }
    }
}

// y = the slices' partial sums in slice order.
__global__ __launch_bounds__(256) void join_kernel(GemmArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t MN = (int64_t)a.M * a.N;
    if (i >= MN) return;
    float s = 0.f;
    for (int v = 0; v < a.S; ++v) s += a.part[v * MN + i];
    store_y(a, i / a.N, i % a.N, s);
}

template <int MT, int R, int WM, int WN, bool XM, int MIN_WAVES>
hipError_t launch_tile(GemmArgs& a, hipStream_t s) {
    using T = Tile<MT, R, WM, WN, XM>;
    const int mb = (a.M + T::BM - 1) / T::BM;
    const int nb = (int)((a.N + T::BN - 1) / T::BN);
    hipLaunchKernelGGL((tile_kernel<MT, R, WM, WN, XM, MIN_WAVES>),
                       dim3((unsigned)((int64_t)mb * nb), (unsigned)a.S), dim3(T::kThreads), 0, s,
                       a, mb, nb);
    if (a.S > 1) {
        const int64_t MN = (int64_t)a.M * a.N;
        hipLaunchKernelGGL(join_kernel, dim3((unsigned)((MN + 255) / 256)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

// Kernel and split of a product.
struct Plan {
    int bm;                 // rows of x a workgroup: 16 (few-row kernel), 32 .. 256
    int S, gs;
};

Plan plan_gemm(int64_t M, int64_t N, int64_t K, bool x_mx4) {
    Plan p{16, 1, (int)groups(K)};
    if (M <= 16) return p;
    p.bm = M <= 32 ? 32 : M <= 64 ? 64 : 128;
    if (x_mx4 && M > 128) p.bm = 256;
    const int64_t bn = p.bm >= 128 ? 256 : 128;
    const int64_t blocks = (M + p.bm - 1) / p.bm * ((N + bn - 1) / bn);
    const int Q = (int)quads(K);
    int64_t S = 512 / blocks;
    if (S > Q) S = Q;
    if (S < 1) S = 1;
    const int qs = (int)((Q + S - 1) / S);      // quads a slice
    p.S = (Q + qs - 1) / qs;
    p.gs = 4 * qs;
    return p;
}

}  // namespace

size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, bool x_mx4) {
    if (M == 0) return 0;
    const Plan p = plan_gemm(M, N, K, x_mx4);
    return p.S > 1 ? (size_t)p.S * M * N * 4 : 0;
}

hipError_t launch_gemm(GemmArgs a, void* ws, hipStream_t s) {
    const bool xm = a.x == nullptr;
    const Plan p = plan_gemm(a.M, a.N, a.K, xm);
    a.S = p.S;
    a.gs = p.gs;
    a.part = static_cast<float*>(ws);
    // the tile kernel's row offsets are products of 24-bit numbers
    const int bm = !xm && a.ldx >= (1 << 23) ? 16 : p.bm;
    switch (bm) {
        case 32:
            return xm ? launch_tile<2, 2, 1, 4, true, 2>(a, s) : launch_tile<2, 2, 1, 4, false, 2>(a, s);
        case 64:
            return xm ? launch_tile<4, 2, 1, 4, true, 2>(a, s) : launch_tile<4, 2, 1, 4, false, 2>(a, s);
        case 128:
            return xm ? launch_tile<8, 4, 1, 4, true, 2>(a, s) : launch_tile<8, 4, 1, 4, false, 2>(a, s);
        case 256: return launch_tile<8, 4, 2, 4, true, 2>(a, s);
        default: return launch_small<1, 8, 4>(a, s);
    }
}

}  // namespace mx4
