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

// ---- a few rows of x, read by every wave ----------------------------------------
// Up to 16 rows of x a workgroup: its KW waves split K between them and each
// streams R tiles of 16 weight rows, D groups in flight.  Lane 16 q + c holds
// piece (c, q) of the weight block and, of x, row c's values of the same 32 k:
// with W as the first operand a matrix instruction's lane needs 8 k of its row
// (BF16: four instructions a piece, k = 32 q + 8 b + e in instruction b -- any
// one-to-one assignment of k serves, as long as both operands share it) or the
// whole piece (MX4: one instruction a group).  The result has lane (c, q)
// holding weight rows 4 q .. 4 q + 3 for row c of x.  The waves' sums meet in
// LDS in wave order.  Loads take no branch (a row past M reads the last one's
// values, whose results are not stored): behind one, the compiler waits for
// loads it need not (QKV M = 1 9.1 -> 6.9 us with R = 2, KW = 4, D = 3).
// RAGGED: K % 128 != 0, blocks of x past K must be zero (their codes are, and
// nothing times zero but a finite number is).
template <int R, int KW, int D, bool XM, bool RAGGED>
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
    const uint16_t* xp = nullptr;
    const uint8_t* xcp = nullptr;
    const uint8_t* xsp = nullptr;
    if constexpr (XM) {
        xcp = a.xm.codes + (int64_t)blockIdx.y * a.G * kCodeBlock + lane * 16;
        xsp = a.xm.scales + (int64_t)blockIdx.y * a.Q * kScaleBlock + lane * 4;
    } else {
        const int m = m0 + c < a.M ? m0 + c : a.M - 1;
        xp = a.x + (int64_t)m * a.ldx + 32 * q;
    }

    constexpr int XV = XM ? 1 : 4;
    u32x4_t wb[D][R], xb[D][XV];
    uint32_t ws[D][R], xs[D];
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
            const bool in = !RAGGED || 128 * g + 32 * q < a.K;
            const uint16_t* p = xp + (in ? 128 * (int64_t)g : -32 * q);
#pragma unroll
            for (int b = 0; b < XV; ++b) {
                xb[d][b] = *reinterpret_cast<const u32x4_t*>(p + 8 * b);
                if constexpr (RAGGED) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) xb[d][b][e] = in ? xb[d][b][e] : 0u;
                }
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

template <int R, int KW, int D, bool XM>
hipError_t launch_small(const GemmArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((tiles(a.N) + R - 1) / R), (unsigned)tiles(a.M)), block(KW * 64);
    if (!XM && a.K % kGroup != 0)
        hipLaunchKernelGGL((small_kernel<R, KW, D, XM, !XM>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((small_kernel<R, KW, D, XM, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

// ---- a few rows of x, shared through LDS ------------------------------------------
// A workgroup: ROWS rows of x (4, or 16 and more) by 16 WN weight rows; KW
// groups of WN waves take every KW-th unit of UG groups of K.  A unit's weights
// come to registers one unit ahead of their products; its x goes through LDS,
// double-buffered, where the WN waves share it: with every wave reading x for
// itself, the caches deliver as many bytes of x as of weights (gate+up M = 16:
// 29.2 us there, 27.1 here; with x's reads left out, 18).  LDS row m of a
// group holds x's 16 pieces of 8 values, piece p at x_place(p, m), so that
// the rows one read takes a piece from lie in different places.  From 16
// rows on the weights are read through the caches: row blocks share them, and the
// weights of a small model stay in the last of them (gate+up M = 16 over 190 MB of
// weights 19.6 us, past the caches 20.8; over 760 MB 24.2 and 23.1).
template <int ROWS, int WN, int KW, int UG, bool XM>
struct Mid {
    static constexpr int kThreads = WN * KW * 64;
    static constexpr int MT = ROWS < 16 ? 1 : ROWS / 16;
    static constexpr int kAllPieces = XM ? MT * 64 * UG : ROWS * 16 * UG;   // of x a unit
    static constexpr int kPieces = (kAllPieces + WN * 64 - 1) / (WN * 64);  // a thread
    static constexpr int kStage = kAllPieces * 16;
    static constexpr int lds() {
        const int x = 2 * KW * kStage, red = KW * WN * MT * 1024;
        return x > red ? x : red;
    }
};

template <int ROWS, int WN, int KW, int UG, bool XM>
__global__ __launch_bounds__(WN* KW * 64) void mid_kernel(GemmArgs a, int mb, int nb) {
    using T = Mid<ROWS, WN, KW, UG, XM>;
    constexpr int MT = T::MT, P = T::kPieces;
    static_assert(!XM || UG == 4, "a scale's dword serves four groups");
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kw = w / WN, wn = w % WN;
    const int c = lane & 15, q = lane >> 4;
    // the row blocks of one weight block run side by side on one XCD (consecutive
    // workgroups go to the 8 XCDs in turn), so that its L2 serves the weights again
    int bm = 0, bn = blockIdx.x;
    if (mb > 1) {
        const int band = 8 * mb, b = blockIdx.x / band, i = blockIdx.x % band;
        const int width = nb - 8 * b < 8 ? nb - 8 * b : 8;
        bn = 8 * b + i % width;
        bm = i / width;
    }
    const int m0 = bm * (ROWS < 16 ? 16 : ROWS);
    const int U = (a.G + UG - 1) / UG;
    const int u0 = blockIdx.y * (a.gs / UG);
    const int u1 = u0 + a.gs / UG < U ? u0 + a.gs / UG : U;
    const int its = (u1 - u0 + KW - 1) / KW;
    const uint32_t lane16 = lane * 16, lane4 = lane * 4;

    const int64_t last_tile = tiles(a.N) - 1;
    int64_t tile = (int64_t)bn * WN + wn;
    if (tile > last_tile) tile = last_tile;
    const uint8_t* wp = a.w.codes + tile * a.G * kCodeBlock;
    const uint8_t* sp = a.w.scales + tile * a.Q * kScaleBlock;
    uint8_t* mine = lds + kw * 2 * T::kStage;
    auto at_piece = [&](int i) {
        int p = (i * WN + wn) * 64 + lane;
        if (T::kAllPieces % (WN * 64) != 0 && p > T::kAllPieces - 64 + lane)
            p = T::kAllPieces - 64 + lane;
        return p;
    };
    u32x4_t wb[2][UG], xb[P];
    uint32_t ws[2], xs[2][XM ? MT : 1];
    bool xin[P];
    // (no branch: a place past the last unit, group, row or K is a valid one whose x
    // is replaced by zeros, a piece past the last is the last once more)
    auto load_x = [&](int slot, int it) {
        const int u = u0 + it * KW + kw;
        const int uc = u < u1 ? u : u1 - 1;
        if constexpr (XM) {
            const int64_t so = (int64_t)uc * kScaleBlock;
            const int64_t last = tiles(a.M) - 1;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int block = i * WN + wn < MT * UG ? i * WN + wn : MT * UG - 1;
                const int64_t t = m0 / 16 + block / UG;     // (tile, group) of the unit
                const int g = u * UG + block % UG;
                xin[i] = u < u1 && g < a.G;
                xb[i] = *reinterpret_cast<const u32x4_t*>(
                    scalar(a.xm.codes + ((t < last ? t : last) * a.G + (g < a.G ? g : a.G - 1)) *
                                            kCodeBlock) + lane16);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t tt = m0 / 16 + t < last ? m0 / 16 + t : last;
                const uint8_t* p = scalar(a.xm.scales + tt * a.Q * kScaleBlock + so);
                xs[slot][t] = *reinterpret_cast<const uint32_t*>(p + lane4);
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int piece = at_piece(i);
                int m = m0 + piece / (16 * UG);
                if (m >= a.M) m = a.M - 1;
                const int k = u * UG * 128 + piece % (16 * UG) * 8;
                xin[i] = u < u1 && k < a.K;
                xb[i] = *reinterpret_cast<const u32x4_t*>(a.x + (int64_t)m * a.ldx +
                                                          (xin[i] ? k : 0));
            }
        }
    };
    auto load_w = [&](int slot, int it) {
        const int u = u0 + it * KW + kw;
        const int uc = u < u1 ? u : u1 - 1;
        const int64_t so = (int64_t)(uc * UG / 4) * kScaleBlock;
        const int shift = UG == 4 ? 0 : 8 * UG * (uc % (4 / UG));
        ws[slot] = *reinterpret_cast<const uint32_t*>(scalar(sp + so) + lane4) >> shift;
#pragma unroll
        for (int j = 0; j < UG; ++j) {
            const int g = uc * UG + j < a.G ? uc * UG + j : a.G - 1;
            wb[slot][j] = load16<ROWS == 4>(scalar(wp + (int64_t)g * kCodeBlock) + lane16);
        }
    };
    // x is waited for first; four rows of it arrive before the weights in any order,
    // and the weights come sooner if asked for first (gate+up M = 1 19.7 -> 18.4 us)
    auto load = [&](int slot, int it) {
        if (ROWS < 16) load_w(slot, it);
        load_x(slot, it);
        if (ROWS >= 16) load_w(slot, it);
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int piece = at_piece(i);
            int at = piece;
            if constexpr (!XM) {
                const int row = piece / (16 * UG), p = piece % (16 * UG);
                at = row * 16 * UG + (p & ~15) + x_place(p & 15, row);
            }
            u32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = xin[i] ? xb[i][e] : 0u;
            *reinterpret_cast<u32x4_t*>(mine + buf * T::kStage + at * 16) = v;
        }
    };
    f32x4_t acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4_t{0, 0, 0, 0};
    const int cr = ROWS < 16 ? c & (ROWS - 1) : c;
    auto product = [&](auto sc) {
        constexpr int slot = decltype(sc)::value;
        const uint8_t* xl = mine + slot * T::kStage;
        if constexpr (XM) {
            auto group = [&](auto jc) {
                constexpr int J = decltype(jc)::value;
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const u32x4_t xv = *reinterpret_cast<const u32x4_t*>(
                        xl + (t * UG + J) * kCodeBlock + lane16);
                    acc[t] = mfma_mx4<J>(operand4(wb[slot][J]), operand4(xv), acc[t], ws[slot],
                                         xs[slot][t]);
                }
            };
            group(std::integral_constant<int, 0>{});
            group(std::integral_constant<int, 1>{});
            group(std::integral_constant<int, 2>{});
            group(std::integral_constant<int, 3>{});
        } else {
#pragma unroll
            for (int j = 0; j < UG; ++j) {
                const float s = scale_f32((ws[slot] >> (8 * j)) & 255u);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    bf16x8_t xv[MT];
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const int row = t * 16 + cr;
                        xv[t] = *reinterpret_cast<const bf16x8_t*>(
                            xl + (row * 16 * UG + 16 * j + x_place(q, b, row)) * 16);
                    }
                    const bf16x8_t wv = expand8(wb[slot][j][b], s);
#pragma unroll
                    for (int t = 0; t < MT; ++t) acc[t] = mfma_bf16(wv, xv[t], acc[t]);
                }
            }
        }
    };
    load(0, 0);
    stage(0);
    __syncthreads();
    auto step = [&](auto sc, int it) {
        constexpr int slot = decltype(sc)::value;
        load(slot ^ 1, it + 1);
        __builtin_amdgcn_sched_barrier(0);
        product(sc);
        __builtin_amdgcn_sched_barrier(0);
        stage(slot ^ 1);
        __syncthreads();
    };
    for (int it = 0; it < its; it += 2) {
        step(std::integral_constant<int, 0>{}, it);
        if (it + 1 >= its) break;
        step(std::integral_constant<int, 1>{}, it + 1);
    }
    __syncthreads();

    // the k groups' sums in their order
    float* red = reinterpret_cast<float*>(lds);         // [KW][WN][MT][256]
#pragma unroll
    for (int t = 0; t < MT; ++t)
        *reinterpret_cast<f32x4_t*>(red + (w * MT + t) * 256 + lane * 4) = acc[t];
    __syncthreads();
    constexpr int kCols = 16 * WN;
    for (int i = tid; i < (ROWS < 16 ? ROWS : MT * 16) * kCols; i += T::kThreads) {
        const int m = i / kCols, col = i % kCols;
        const int64_t nn = (int64_t)bn * kCols + col;
        if (m0 + m >= a.M || nn >= a.N) continue;
        const int wr = col & 15, in = ((wr >> 2) * 16 + (m & 15)) * 4 + (wr & 3);
        const int at = ((col >> 4) * MT + (m >> 4)) * 256 + in;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < KW; ++k) s += red[k * WN * MT * 256 + at];
        if (a.S > 1)
            a.part[((int64_t)blockIdx.y * a.M + m0 + m) * a.N + nn] = s;
        else
            store_y(a, m0 + m, nn, s);
    }
}

// ---- many rows of x -------------------------------------------------------------
// A workgroup of WM x WN waves computes 16 MT WM rows of x by 16 R WN weight
// rows; a wave 16 MT by 16 R, its sums in registers.  Weight pieces go from
// memory to registers in the layout the matrix instructions take them, x through
// LDS, double-buffered, where the WN waves share it; both are asked for one group
// ahead, or two (DEEP) where the sums leave the registers for it.  64 x 128 tiles,
// us, one group ahead / two: gate+up M = 128 71 / 58, MX4 x 37.4 / 30.5; 128 x 256
// tiles of MX4 x, QKV M = 4096, 90.9 / 87.9.
// BF16 x: LDS row m holds 16 pieces of 8 values, piece p at x_place(p, m), so that
// the rows a read takes one piece from lie in different places.
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

template <int MT, int R, int WM, int WN, bool XM, bool DEEP>
__global__ __launch_bounds__(WM* WN * 64, 2) void tile_kernel(GemmArgs a, int mb, int nb) {
    using T = Tile<MT, R, WM, WN, XM>;
    constexpr int P = T::kPieces;
    // BF16 x comes in kRuns runs of H0 pieces a step, each asked for when the one before
    // is stored: no more in flight than the registers that 8 x 4 sums leave.  DEEP has
    // the registers to ask for all of them, a step earlier.
    constexpr int kRuns = XM || DEEP ? 1 : 4;
    constexpr int H0 = (P + kRuns - 1) / kRuns;
    constexpr int kAhead = DEEP ? 2 : 1;        // steps
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

    u32x4_t wreg[2 * kAhead][R], xreg[kAhead][P];
    bool xin[kAhead];
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
    auto load_x = [&](int set, int i, int g) {
        const int gg = g < ge ? g : ge - 1;
        bool in = g < ge;
        if constexpr (XM) {
            xreg[set][i] = *reinterpret_cast<const u32x4_t*>(
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
            xreg[set][i] = *reinterpret_cast<const u32x4_t*>(
                xbase + 256 * (int64_t)gg + (__umul24(r, stride) + (k_in ? 16u * (tid & 15) : 0u)));
        }
        xin[set] = in;
    };
    auto store_x = [&](int set, int i, int buf) {
        int at;
        if constexpr (XM) {
            at = (tid + i * T::kThreads) * 16;
        } else {
            const int r = (tid >> 4) + i * (T::kThreads / 16);
            at = r * 256 + (x_place(tid & 15, r) << 4);
        }
        u32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = xin[set] ? xreg[set][i][e] : 0u;
        *reinterpret_cast<u32x4_t*>(&xs[buf][at]) = v;
    };

    f32x4_t acc[MT][R];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[i][r] = f32x4_t{0, 0, 0, 0};

#pragma unroll
    for (int i = 0; i < P; ++i) load_x(0, i, gb);
    load_w(0, gb);
    load_scales(0, gb);
    if constexpr (DEEP) load_w(1, gb + 1);
#pragma unroll
    for (int i = 0; i < P; ++i) store_x(0, i, 0);
    if constexpr (DEEP) {
#pragma unroll
        for (int i = 0; i < P; ++i) load_x(1, i, gb + 1);
    }
    __syncthreads();

    auto step = [&](auto jc, int g) {
        constexpr int J = decltype(jc)::value;
        constexpr int cur = J & 1, nxt = cur ^ 1;
        // DEEP: the registers of x that hold this step's, stored before it, take the
        // step's after the next
        constexpr int set = DEEP ? cur : 0, next_set = DEEP ? nxt : 0;
        constexpr int wcur = J & (2 * kAhead - 1);
        load_w((J + kAhead) & (2 * kAhead - 1), g + kAhead);
#pragma unroll
        for (int i = 0; i < H0; ++i) load_x(set, i, g + kAhead);
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
                            mfma_mx4<J>(operand4(wreg[wcur][r]), operand4(xv[u & 1][h]),
                                        acc[2 * u + h][r], ws[0][r], xsc[0][2 * u + h]);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) store_x(next_set, i, nxt);
        } else {
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = scale_f32((ws[0][r] >> (8 * J)) & 255u);
            bf16x8_t xv[2][2], wv[2][R];
            const uint8_t* xrow = xl + (wm * MT * 16 + c) * 256;
            auto read = [&](int slot, int v) {
                const int b = v / U, u = v % U;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    xv[slot][h] = *reinterpret_cast<const bf16x8_t*>(
                        xrow + (2 * u + h) * 4096 + (x_place(q, b, c) << 4));
            };
            read(0, 0);
#pragma unroll
            for (int r = 0; r < R; ++r) wv[0][r] = expand8(wreg[wcur][r][0], s[r]);
#pragma unroll
            for (int v = 0; v < 4 * U; ++v) {
                const int b = v / U, u = v % U;
                if (v + 1 < 4 * U) read((v + 1) & 1, v + 1);
                if (b < 3) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (r * U / R == u)
                            wv[(b + 1) & 1][r] = expand8(wreg[wcur][r][b + 1], s[r]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        acc[2 * u + h][r] =
                            mfma_bf16(wv[b & 1][r], xv[v & 1][h], acc[2 * u + h][r]);
                __builtin_amdgcn_sched_barrier(0);
                if ((v + 1) % (4 * U / kRuns) == 0) {
                    constexpr int kLen = 4 * U / kRuns;
                    const int run = v / kLen;
#pragma unroll
                    for (int i = run * H0; i < (run + 1) * H0 && i < P; ++i)
                        store_x(next_set, i, nxt);
#pragma unroll
                    for (int i = (run + 1) * H0; i < (run + 2) * H0 && i < P; ++i)
                        load_x(set, i, g + 1);
                }
            }
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
    const int64_t n0 = (int64_t)bn * T::BN + wn * R * 16;
    const bool f32 = a.S > 1 || a.y_f32;
    const int64_t ld = a.S > 1 ? a.N : a.ldy;
    uint8_t* out = a.S > 1 ? reinterpret_cast<uint8_t*>(a.part + (int64_t)slice * a.M * a.N)
                           : static_cast<uint8_t*>(a.y);
    const int size = f32 ? 4 : 2;
    // 16 bytes at a time where every row of y starts on such a boundary
    const bool wide = ld % (16 / size) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + (wm * MT + i) * 16 + c;
        uint8_t* o = out + (m * ld + n0) * size;
#pragma unroll
        for (int r = 0; r < R; r += 2) {
            if (!f32 && wide && n0 + 16 * (r + 2) <= a.N) {
                // BF16: lanes q and q ^ 1 trade halves of two tiles, and hold eight outputs
                // in a row each (64 bytes of a row a store instead of 32)
                const f32x4_t v = acc[i][r], w2 = acc[i][r + 1];
                uint32_t p0 = bf16_bits(v[0]) | (uint32_t)bf16_bits(v[1]) << 16;
                uint32_t p1 = bf16_bits(v[2]) | (uint32_t)bf16_bits(v[3]) << 16;
                uint32_t p2 = bf16_bits(w2[0]) | (uint32_t)bf16_bits(w2[1]) << 16;
                uint32_t p3 = bf16_bits(w2[2]) | (uint32_t)bf16_bits(w2[3]) << 16;
                swap16(p0, p2);
                swap16(p1, p3);
                if (m < a.M)
                    *reinterpret_cast<u32x4_t*>(o + 2 * (16 * (r + (q & 1)) + 8 * (q >> 1))) =
                        u32x4_t{p0, p1, p2, p3};
                continue;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = 16 * (r + h) + 4 * q;
                const f32x4_t v = acc[i][r + h];
                const int64_t left = m < a.M ? a.N - n0 - n : 0;
                if (f32 && wide && left >= 4) {
                    *reinterpret_cast<f32x4_t*>(o + 4 * n) = v;
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e >= left) continue;
                    if (f32)
                        reinterpret_cast<float*>(o)[n + e] = v[e];
                    else
                        reinterpret_cast<uint16_t*>(o)[n + e] = bf16_bits(v[e]);
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
#pragma unroll 8
    for (int v = 0; v < a.S; ++v) s += a.part[v * MN + i];
    store_y(a, i / a.N, i % a.N, s);
}

hipError_t launch_join(const GemmArgs& a, hipStream_t s) {
    if (a.S > 1) {
        const int64_t MN = (int64_t)a.M * a.N;
        hipLaunchKernelGGL(join_kernel, dim3((unsigned)((MN + 255) / 256)), dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

template <int MT, int R, int WM, int WN, bool XM, bool DEEP>
hipError_t launch_tile(GemmArgs& a, hipStream_t s) {
    using T = Tile<MT, R, WM, WN, XM>;
    const int mb = (a.M + T::BM - 1) / T::BM;
    const int nb = (int)((a.N + T::BN - 1) / T::BN);
    hipLaunchKernelGGL((tile_kernel<MT, R, WM, WN, XM, DEEP>),
                       dim3((unsigned)((int64_t)mb * nb), (unsigned)a.S), dim3(T::kThreads), 0, s,
                       a, mb, nb);
    return launch_join(a, s);
}

template <int ROWS, int WN, int KW, int UG, bool XM>
hipError_t launch_mid(GemmArgs& a, hipStream_t s) {
    using T = Mid<ROWS, WN, KW, UG, XM>;
    static_assert(T::lds() <= 65536, "more LDS than a launch gets without asking");
    constexpr int bm = ROWS < 16 ? 16 : ROWS;
    const int mb = (a.M + bm - 1) / bm;
    const int nb = (int)((tiles(a.N) + WN - 1) / WN);
    hipLaunchKernelGGL((mid_kernel<ROWS, WN, KW, UG, XM>),
                       dim3((unsigned)((int64_t)mb * nb), (unsigned)a.S), dim3(T::kThreads),
                       T::lds(), s, a, mb, nb);
    return launch_join(a, s);
}

// Kernel and split of a product.
enum Kernel {
    kSmall, kMid4, kMid4Long, kMid16, kMid16x2, kMid32, kMid32x2, kMid64,
    kTileSmall, kTileMid, kTile128
};
struct Plan {
    Kernel kernel;
    int wn;                 // mid kernels: waves beside each other
    int S, gs;              // K slices, groups a slice (a multiple of 4)
};

// Waves beside each other that spread nt tiles best over 256 CUs: the CU with the
// most of them decides; up to 16 rows a CU with one workgroup, whose barriers nothing
// fills, counts a fifth more.  us (tiles of that CU): gate+up, 2176 tiles, M = 16,
// 5 waves 24.4 (2 x 5), 9 25.4 (9), 7 26.8 (2 x 7), 12 28.6 (12), 4 27.6 (3 x 4);
// M = 32, 9 waves 30.1, 5 31.3, 12 32.0, 7 35.0, 4 42.4; 1792 tiles, M = 16, 4 waves
// 15.5 (2 x 4), 7 17.6 (7).  Of equals the most waves, which share x.
int spread(int64_t nt, bool few_rows) {
    static const int kWaves[] = {12, 9, 7, 5, 4};
    int best = 4;
    int64_t least = -1;
    for (const int w : kWaves) {
        const int64_t most = ((nt + w - 1) / w + 255) / 256;
        const int64_t cost = most * w * (few_rows && most == 1 ? 6 : 5);
        if (least < 0 || cost < least) {
            least = cost;
            best = w;
        }
    }
    return best;
}

// By rows of x (M), tiles of 16 weight rows (nt) and groups of K (G).  Measured on
// QKV (nt = 448, G = 40), gate+up (2176, 40) and down (320, 136), us:
//   up to 16 rows, BF16 x: every wave on its own x for few tiles (QKV M = 1 6.9 against
//     7.8 through LDS, M = 16 9.8 against 11.1); shared through LDS for many tiles
//     (gate+up M = 1 18.5 against 22.1, M = 16 23.6 against 29.2) or a long K (down
//     M = 1 14.3 against 15.6, M = 16, K in six slices, 17.5 against 23.5).  MX4 x
//     is a quarter of the bytes: shared or not within 3%.  A long K for so few tiles
//     that they leave CUs idle is cut (M = 1, K = 17408, N = 1024 8.9, uncut 11.5; MX4 x
//     8.0 and 11.4).
//   above and few tiles: 16 (MX4 x: 16, 32) rows a workgroup, whose weights the row
//     blocks beside it find in L2, up to the grids that those fill (QKV M = 64 16.9,
//     M = 128 21.5; 64 x 128 tiles in four slices 21.2 and 24.9.  N = K = 1024, M = 512
//     6.0, tiles 9.2.  MX4 x: 16 rows at M = 48 10.4, 32 rows 11.1, at M = 128 17.6 and
//     14.4; N = 896 on K = 5120, M = 128, 6.3 and 8.7); a long K in slices (down M = 33 24.5,
//     MX4 x, M = 17, six slices, 16.3; 64 rows, five slices, 20.7).
//   17 to 32 and many tiles: 32 rows, waves as spread() says (MX4 x: four), unless BF16
//     tiles of 32 x 256 nearly fill the GPU (gate+up M = 32, 136 of them, 37.2, by waves
//     29.8; N = 65536 on K = 2048, 256 of them, 20.0 and 26.8).
//   33 to 64 and many tiles: the tiles below, BF16 x 64 x 256 from about one a CU on, else
//     32 x 256 (K = 5120, M = 64: N = 65536 53.5, 32 rows by two tiles a wave 72.1; N = 50000
//     51.4 and 65.0, N = 34816 42.3 and 41.7, N = 20480 31.4 and 35.7).
//   above: 128 x 256 if that gives 440 workgroups (QKV M = 2048 115, 64 x 256 125.5);
//     else, BF16 x, 64 x 256 if that gives 440 (QKV M = 1024 64.9, 128 x 256 75.5) or
//     nearly one a CU (QKV M = 512 39.2, 128 x 256 51.7), then 32 x 256 (QKV M = 256
//     29.2, 64 x 256 in two slices 32.4; gate+up M = 128 59.4, 64 x 256 on 272
//     workgroups 64.1); MX4 x 128 x 128, then 64 x 128 (QKV M = 512 21.8, 128 x 256
//     30.2).  Slices cost about 4 us to write, wait for and join: for a long K (down
//     M = 256, MX4 x, four slices of 64 x 128 37.2, one 60), and BF16 x on K = 4096 and more
//     where one slice leaves CUs idle (O M = 192 22.9 with three, 28.1 with one; K = 2560
//     18.9 and 16.7).
Plan plan_gemm(int64_t M, int64_t N, int64_t K, bool xm) {
    const int G = (int)groups(K), Q = (int)quads(K);
    const int64_t nt = tiles(N);
    const bool many = nt >= 1024, lengthy = G >= 64;
    const auto blocks = [&](int64_t bm, int64_t bn) {
        return (M + bm - 1) / bm * ((N + bn - 1) / bn);
    };
    Plan p{kSmall, 4, 1, 4 * Q};
    int64_t S = 1;
    const auto slices = [](int64_t want, int64_t have) { return (want + have / 2) / have; };
    if (M <= 16) {
        if (xm && lengthy && nt <= 160) {
            p.kernel = kMid16x2;
            S = slices(512, blocks(16, 32));
        } else if (xm || (!many && !lengthy)) {
            p.kernel = kSmall;
        } else if (M <= 4) {
            p.kernel = many ? kMid4 : kMid4Long;
            if (!many) S = slices(400, nt);
        } else {
            p.kernel = kMid16;
            if (many)
                p.wn = spread(nt, true);
            else
                S = slices(480, blocks(16, 64));
        }
    } else if (many && M <= 32 && (xm || blocks(32, 256) < 200)) {
        p.kernel = kMid32;
        p.wn = spread(nt, false);
    } else if (xm && !many &&
               (M <= (lengthy ? 192 : 256) || (!lengthy && blocks(32, 64) <= 640))) {
        if (lengthy) {
            p.kernel = M <= 64 ? kMid32 : kMid64;
            S = M <= 64 ? slices(480, blocks(32, 64)) : slices(640, blocks(64, 64));
        } else {
            p.kernel = blocks(16, 32) <= 1024  ? kMid16x2
                       : blocks(32, 64) <= 512 ? kMid32x2
                                               : kMid32;
        }
    } else if (!xm && !many &&
               (M <= (lengthy ? 64 : 128) || (!lengthy && blocks(16, 128) <= 448))) {
        p.kernel = !lengthy && (M <= 32 || blocks(16, 64) <= 256) ? kMid16x2 : kMid16;
        p.wn = 8;
        if (lengthy) S = slices(480, blocks(16, 128));
    } else if (M > 64 && blocks(128, 256) >= 440) {
        p.kernel = kTile128;
    } else if (xm) {
        p.kernel = M > 64 && blocks(128, 128) >= 440 ? kTileMid : kTileSmall;
        if (lengthy && p.kernel == kTileSmall) S = slices(640, blocks(64, 128));
    } else if (M > 32 && (blocks(64, 256) >= 440 ||
                          (blocks(64, 256) >= 200 && (lengthy || blocks(64, 256) <= 256)))) {
        p.kernel = kTileMid;
        if (lengthy && blocks(64, 256) < 440) S = slices(960, blocks(64, 256));
    } else {
        p.kernel = kTileSmall;
        if (lengthy)
            S = slices(480, blocks(32, 256));
        else if (G >= 32 && blocks(32, 256) < 200)
            S = 3;
    }
    if (S > Q) S = Q;
    if (S < 1) S = 1;
    const int qs = (int)((Q + S - 1) / S);      // quads a slice
    p.S = (Q + qs - 1) / qs;
    p.gs = 4 * qs;
    return p;
}

template <int ROWS>
hipError_t launch_mid_waves(int wn, GemmArgs& a, hipStream_t s) {
    switch (wn) {
        case 5: return launch_mid<ROWS, 5, 1, 4, false>(a, s);
        case 7: return launch_mid<ROWS, 7, 1, 4, false>(a, s);
        case 9: return launch_mid<ROWS, 9, 1, 4, false>(a, s);
        case 12: return launch_mid<ROWS, 12, 1, 4, false>(a, s);
        default: return launch_mid<ROWS, 4, 1, 4, false>(a, s);
    }
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
    Kernel k = p.kernel;
    if (!xm && k >= kTileSmall && a.ldx >= kFarRows) k = kSmall;
    if (k == kSmall) a.S = 1;
    if (xm) switch (k) {
        case kMid16x2: return launch_mid<16, 2, 2, 4, true>(a, s);
        case kMid32: return launch_mid<32, 4, 1, 4, true>(a, s);
        case kMid32x2: return launch_mid<32, 4, 2, 4, true>(a, s);
        case kMid64: return launch_mid<64, 4, 1, 4, true>(a, s);
        case kTileSmall: return launch_tile<4, 2, 1, 4, true, true>(a, s);
        case kTileMid: return launch_tile<8, 2, 1, 4, true, true>(a, s);
        case kTile128: return launch_tile<8, 4, 1, 4, true, true>(a, s);
        default: return launch_small<2, 8, 2, true>(a, s);
    }
    switch (k) {
        case kMid4: return launch_mid<4, 2, 2, 2, false>(a, s);
        case kMid4Long: return launch_mid<4, 1, 4, 4, false>(a, s);
        case kMid16:
            return p.wn == 8 ? launch_mid<16, 8, 1, 4, false>(a, s)
                             : launch_mid_waves<16>(p.wn, a, s);
        case kMid16x2: return launch_mid<16, 4, 2, 4, false>(a, s);
        case kMid32: return launch_mid_waves<32>(p.wn, a, s);
        case kTileSmall: return launch_tile<2, 4, 1, 4, false, true>(a, s);
        case kTileMid: return launch_tile<4, 4, 1, 4, false, true>(a, s);
        case kTile128: return launch_tile<8, 4, 1, 4, false, false>(a, s);
        default: return launch_small<2, 4, 3, false>(a, s);
    }
}

}  // namespace mx4
