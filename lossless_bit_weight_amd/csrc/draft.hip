// draft.hip -- verification of drafted tokens (../../include/draft.h states the
// operation).
//
// Two launches, three with the drafter's probabilities.  parts: every row of logits is
// read once, in chunks over the GPU, into registers; a chunk leaves its largest logit and
// its sum of powers (greedy: that logit's word).  rest (with probabilities): every
// workgroup of a sequence finds from the parts where it stops, and sums max(0, p - q) over
// its chunk of that row.  pick: one workgroup a sequence finds the chunk that the random
// number falls into, reads it again and finds the word.
// Powers, probabilities and sums are fp64: a word's border in the running sum of
// 10^5 words is then off by less than a random number of 24 bits can tell, so that
// the word does not depend on the order of summation.  The exponential costs 17 fp64
// instructions a word, which run at the rate of fp32's here, beside 2 or 4 bytes read.
// 32 sequences of 7 to 15 drafts, 129280 fp32 words, with probabilities: parts 48 us (204
// MB, 4.2 TB/s: the exponentials' time and the memory's overlap in part; without them 30),
// rest 13, pick 7; one sequence of 4 drafts, 32003 BF16 words: parts 4, pick 3 to 6: two
// launches' starts and ends and the ways to memory behind each other.
#include <type_traits>

#include "draft_internal.hpp"
#include "exp64.hpp"

namespace draft {
namespace {

constexpr int kThreads = 256;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kMaxRowsOf = 1024;            // of a sequence: DRAFT_MAX_D + 1

template <bool F32>
struct Row {
    static constexpr int VEC = F32 ? 4 : 8;     // words of 16 bytes
    const uint8_t* p;                           // word 0
    int head;                                   // words between a 16-byte boundary and p

    __device__ __forceinline__ Row(const void* base, int64_t at) {
        p = static_cast<const uint8_t*>(base) + at * (F32 ? 4 : 2);
        head = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (F32 ? 4 : 2);
    }
    __device__ __forceinline__ float one(int v) const {
        if constexpr (F32) return reinterpret_cast<const float*>(p)[v];
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[v] << 16);
    }
    // Words v .. v + VEC - 1, v on a 16-byte boundary.
    __device__ __forceinline__ void whole(int v, float* f) const {
        const u32x4_t d = *reinterpret_cast<const u32x4_t*>(p + (int64_t)v * (F32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (F32) {
                f[j] = __uint_as_float(d[j]);
            } else {
                f[2 * j] = __uint_as_float(d[j] << 16);
                f[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
            }
        }
    }
    // The same, those outside 0 .. V-1 as `none`.
    __device__ __forceinline__ void load(int v, int V, float none, float* f) const {
        if (v >= 0 && v + VEC <= V) {
            whole(v, f);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = v + j >= 0 && v + j < V ? one(v + j) : none;
        }
    }
};

// The sum over a workgroup of T threads, in every thread, in an order that depends on
// nothing.
template <int T>
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) v += part[w];
    return v;
}

__device__ __forceinline__ int length_of(const Args& a, int b) {
    const int n = a.lengths == nullptr ? a.D : a.lengths[b];
    return n < 0 ? 0 : n > a.D ? a.D : n;
}
// log2(e) / tau, or 0 for greedy
__device__ __forceinline__ double rate_of(float tau) {
    // (an infinite one: all words of finite logits alike)
    return tau > 0.f ? __builtin_fmax(kLog2E / (double)tau, 1e-300) : 0.0;
}
__device__ __forceinline__ float temperature_of(const Args& a, int b) {
    return a.temperature == nullptr ? 1.f : a.temperature[b];
}
__device__ __forceinline__ int64_t draft_of(const Args& a, int b, int i) {
    const int64_t at = (int64_t)b * a.D + i;
    return a.drafts_i64 ? static_cast<const int64_t*>(a.drafts)[at]
                        : static_cast<const int*>(a.drafts)[at];
}
// 2^((l - top) rate), 0 below 2^-1000 (least = -1000 / rate); selected, not branched to, so
// that a thread's words overlap.
__device__ __forceinline__ double power(float l, float top, double rate, double least) {
    const double d = (double)l - (double)top, p = exp2_64_low(d, rate, least);
    return d < least || l == -__builtin_inff() ? 0.0 : p;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    return a != a || b != b ? __builtin_nanf("") : a > b ? a : b;
}

// Chunk `chunk` of a row in the registers of T threads: NV vectors each, vector i of
// thread t at (NEAR: NV t + i; else t + T i) vectors behind the chunk's first.
template <bool F32, int NV, int T, bool NEAR>
struct Chunk {
    static constexpr int VEC = Row<F32>::VEC;
    static constexpr int kWords = T * VEC * NV;
    float f[NV][VEC];

    __device__ __forceinline__ static int word(const Row<F32>& r, int chunk, int i) {
        return chunk * kWords - r.head +
               (NEAR ? (int)threadIdx.x * NV + i : i * T + (int)threadIdx.x) * VEC;
    }
    __device__ __forceinline__ void load(const Row<F32>& r, int chunk, int V) {
        const int first = chunk * kWords - r.head;
        if (first >= 0 && first + kWords <= V) {    // (the same for all: loads side by side)
#pragma unroll
            for (int i = 0; i < NV; ++i) r.whole(word(r, chunk, i), f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) r.load(word(r, chunk, i), V, -__builtin_inff(), f[i]);
        }
    }
};

template <bool F32, int NV>
__global__ __launch_bounds__(kThreads) void parts_kernel(Args a) {
    constexpr int kWaves = kThreads / 64;
    __shared__ double sums[kWaves];
    __shared__ float tops[kWaves];
    __shared__ int words[kWaves];
    const int row = blockIdx.y * 32768 + blockIdx.z;
    const int chunk = blockIdx.x;
    const int b = row / (a.D + 1), i = row % (a.D + 1);
    if (row >= a.B * (a.D + 1)) return;
    const float tau = temperature_of(a, b);
    if (i > length_of(a, b)) return;
    const double rate = rate_of(tau);
    const Row<F32> r(a.logits, b * a.ldb + i * a.ldd);
    using C = Chunk<F32, NV, kThreads, false>;
    constexpr int VEC = C::VEC;
    C c;
    c.load(r, chunk, a.V);

    // the largest as a number, and as signed and unsigned bits: +inf and a positive NaN are
    // above all other signed numbers, a negative NaN above all other unsigned ones
    float top = -__builtin_inff();
    int sbits = (int)0x80000000;
    uint32_t ubits = 0;
    const auto larger = [](auto a, auto b) { return a > b ? a : b; };
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            const float f = c.f[k][j], g = c.f[k][j + 1];
            top = __builtin_fmaxf(top, __builtin_fmaxf(f, g));
            sbits = larger(sbits, larger(__float_as_int(f), __float_as_int(g)));
            ubits = larger(ubits, larger(__float_as_uint(f), __float_as_uint(g)));
        }
    if (sbits >= 0x7F800000 || ubits > 0xFF800000u) top = __builtin_nanf("");
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = max_nan(top, __shfl_xor(top, d));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = max_nan(top, tops[w]);

    double sum = 0.0;
    int word = 0x7FFFFFFF;
    if (rate == 0.0) {
#pragma unroll
        for (int k = NV - 1; k >= 0; --k)
#pragma unroll
            for (int j = VEC - 1; j >= 0; --j)
                word = c.f[k][j] == top ? C::word(r, chunk, k) + j : word;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const int o = __shfl_xor(word, d);
            word = o < word ? o : word;
        }
        if ((threadIdx.x & 63) == 0) words[threadIdx.x >> 6] = word;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) word = words[w] < word ? words[w] : word;
    } else if (top > -__builtin_inff()) {
        const double from = top, least = -1000.0 / rate;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                sum += exp2_64_low((double)c.f[k][j] - from, rate, least);
        sum = block_sum<kThreads>(sum, sums);
    }
    if (threadIdx.x == 0) a.parts[(int64_t)row * a.chunks + chunk] = Part{sum, top, word};
}

// From the row's chunks, by 16 lanes of a row (`lane` 0 .. 15 of them), in every one.
__device__ __forceinline__ Whole whole(const Args& a, int64_t row, double rate, double least,
                                       int lane) {
    const Part* p = a.parts + row * a.chunks;
    // one pass: the sum is kept in powers of the largest logit so far
    Whole w{0.0, -__builtin_inff(), 0x7FFFFFFF};
    for (int c = lane; c < a.chunks; c += 16) {
        const Part part = p[c];
        if (part.top > w.top || (part.top == w.top && part.word < w.word)) w.word = part.word;
        const float top = max_nan(w.top, part.top);
        if (rate != 0.0 && top > -__builtin_inff()) {
            const double old = w.sum > 0.0 ? w.sum * power(w.top, top, rate, least) : 0.0;
            w.sum = old + part.sum * (part.top == top ? 1.0 : power(part.top, top, rate, least));
        }
        w.top = top;
    }
    const float mine = w.top;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) {
        const float ot = __shfl_xor(w.top, d);
        const int ow = __shfl_xor(w.word, d);
        if (ot > w.top || (ot == w.top && ow < w.word)) w.word = ow;
        w.top = max_nan(w.top, ot);
    }
    if (rate == 0.0) return w;
    w.sum = w.good() && w.sum > 0.0 ? w.sum * power(mine, w.top, rate, least) : 0.0;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) w.sum += __shfl_xor(w.sum, d);
    return w;
}

template <bool F32>
__device__ __forceinline__ float value(const void* base, int64_t at) {
    return Row<F32>(base, at).one(0);
}
__device__ __forceinline__ float logit(const Args& a, int b, int i, int64_t v) {
    const int64_t at = b * a.ldb + i * a.ldd + v;
    return a.f32 ? value<true>(a.logits, at) : value<false>(a.logits, at);
}
__device__ __forceinline__ float prob(const Args& a, int b, int i, int64_t v) {
    const int64_t at = b * a.pdb + i * a.pdd + v;
    return a.probs_f32 ? value<true>(a.probs, at) : value<false>(a.probs, at);
}

// By the whole workgroup of T threads, 16 lanes a row; `space` has a place for each.
struct StopSpace {
    Whole rows[kMaxRowsOf];
    int refused;
};
template <int T>
__device__ __forceinline__ Stop stop_of(const Args& a, int b, StopSpace& space) {
    const int lane = threadIdx.x & 15;
    const int64_t row0 = (int64_t)b * (a.D + 1);
    // what depends on nothing first, together
    const float tau = temperature_of(a, b);
    const int n = length_of(a, b);
    int i = threadIdx.x / 16;
    int64_t x = i < a.D ? draft_of(a, b, i) : -1;
    const double rate = rate_of(tau), least = -1000.0 / rate;
    if (threadIdx.x == 0) space.refused = n;
    __syncthreads();
    for (; i <= n; i += T / 16) {
        if (i >= T / 16) x = i < n ? draft_of(a, b, i) : -1;
        // the draft's own word, beside the parts
        const bool in = i < n && x >= 0 && x < a.V;
        const float l = logit(a, b, i, in ? x : 0);
        const double q = a.probs != nullptr && in ? (double)prob(a, b, i, x) : 1.0;
        const double u = a.uniforms[row0 + i];
        const Whole r = whole(a, row0 + i, rate, least, lane);
        bool ok = r.good() && in;
        if (ok) ok = rate == 0.0 ? x == r.word : u * q * r.sum < power(l, r.top, rate, least);
        if (lane == 0) {
            space.rows[i] = r;
            if (i < n && !ok) atomicMin(&space.refused, i);
        }
    }
    __syncthreads();
    Stop s;
    s.n = space.refused;
    s.length = n;
    s.rate = rate;
    s.least = least;
    s.row = space.rows[s.n];
    return s;
}

// N values of a row from word v on, on no boundary but their own (those outside 0 .. V-1
// are some of the others).
template <int N>
__device__ __forceinline__ void probs_at(const Args& a, int64_t at, int v, float* q) {
    if (v >= 0 && v + N <= a.V) {
        if (a.probs_f32) {
            typedef float v_t __attribute__((ext_vector_type(N), aligned(4)));
            const v_t d = *reinterpret_cast<const v_t*>(static_cast<const float*>(a.probs) + at + v);
#pragma unroll
            for (int j = 0; j < N; ++j) q[j] = d[j];
        } else {
            typedef uint16_t v_t __attribute__((ext_vector_type(N), aligned(2)));
            const v_t d =
                *reinterpret_cast<const v_t*>(static_cast<const uint16_t*>(a.probs) + at + v);
#pragma unroll
            for (int j = 0; j < N; ++j) q[j] = __uint_as_float((uint32_t)d[j] << 16);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int in = v + j < 0 ? 0 : v + j < a.V ? v + j : a.V - 1;
            q[j] = a.probs_f32 ? value<true>(a.probs, at + in) : value<false>(a.probs, at + in);
        }
    }
}

// What the words of a chunk are drawn by behind the accepted tokens, times the row's sum.
template <bool F32, int NV, int T, bool NEAR>
struct Weights {
    using C = Chunk<F32, NV, T, NEAR>;
    static constexpr int VEC = C::VEC;
    double p[NV][VEC];
    int word[NV];               // the first of each vector

    // less: take off what the drafter had (refused: its one word, without probabilities)
    __device__ __forceinline__ void load(const Args& a, int b, const Stop& s, int chunk, bool less,
                                         int64_t refused) {
        const Row<F32> row(a.logits, b * a.ldb + s.n * a.ldd);
        C c;
        c.load(row, chunk, a.V);
        const bool off = less && a.probs != nullptr;
        float q[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            word[i] = C::word(row, chunk, i);
            if (off) probs_at<VEC>(a, b * a.pdb + s.n * a.pdd, word[i], q[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                double w = power(c.f[i][j], s.row.top, s.rate, s.least);
                if (off) {
                    // (one instruction in every kernel: whether it is above 0 has to agree)
                    const double d = __builtin_fma(-(double)q[i][j], s.row.sum, w);
                    w = w > 0.0 && d > 0.0 ? d : 0.0;
                } else if (less && word[i] + j == refused) {
                    w = 0.0;
                }
                p[i][j] = w;
            }
    }
    __device__ __forceinline__ double sum() const {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) s += p[i][j];
        return s;
    }
};

template <bool F32, int NV>
__global__ __launch_bounds__(kThreads) void rest_kernel(Args a) {
    __shared__ double sums[kThreads / 64];
    __shared__ StopSpace space;
    const int b = blockIdx.y * 32768 + blockIdx.z, chunk = blockIdx.x;
    if (b >= a.B) return;
    const Stop s = stop_of<kThreads>(a, b, space);
    if (chunk == 0 && threadIdx.x == 0) a.stops[b] = s;
    if (s.rate == 0.0 || s.n == s.length || !s.row.good()) return;
    Weights<F32, NV, kThreads, false> weights;
    weights.load(a, b, s, chunk, true, -1);
    const double sum = block_sum<kThreads>(weights.sum(), sums);
    if (threadIdx.x == 0) a.rest[(int64_t)b * a.chunks + chunk] = sum;
}

// Inclusive sum over the lanes of a wave: along the rows of 16 lanes, then over the rows.
__device__ __forceinline__ double wave_scan(double v) {
    const auto add = [&](auto ctrl, auto rows) {
        constexpr int C = decltype(ctrl)::value, R = decltype(rows)::value;
        const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), C, R, 0xF, false);
        const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), C, R, 0xF, false);
        v += __hiloint2double(hi, lo);
    };
    using std::integral_constant;
    add(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});    // row_shr:1
    add(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});    // row_shr:2
    add(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});    // row_shr:4
    add(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});    // row_shr:8
    add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});    // row_bcast:15
    add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});    // row_bcast:31
    return v;
}
// A lane's value, the same lane for all.
__device__ __forceinline__ double lane_value(double v, int lane) {
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                            __builtin_amdgcn_readlane(__double2loint(v), lane));
}

// A grid's x holds fewer than 2^32 work items: more sequences go along y.
constexpr int kGridX = 1 << 21;

// T threads of NV vectors: the chunks are those of parts_kernel.
template <bool F32, int NV, int T>
__global__ __launch_bounds__(T) void pick_kernel(Args a) {
    __shared__ double sums[T / 64];
    __shared__ StopSpace space;
    __shared__ int where, hit, final;
    __shared__ double below;
    const int b = blockIdx.y * kGridX + blockIdx.x;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    if (b >= a.B) return;
    const int64_t row0 = (int64_t)b * (a.D + 1);
    const double u = a.uniforms[row0 + a.D];
    Stop s;
    if (a.probs != nullptr)
        s = a.stops[b];             // as rest_kernel found it
    else
        s = stop_of<T>(a, b, space);
    int token = -1;
    using W = Weights<F32, NV, T, true>;
    if (s.row.good() && s.rate == 0.0) {
        token = s.row.word;
    } else if (s.row.good()) {
        const bool was_refused = s.n < s.length;
        // without probabilities: the refused word, if it is one
        int64_t x = -1;
        if (was_refused && a.probs == nullptr) {
            x = draft_of(a, b, s.n);
            if (x < 0 || x >= a.V) x = -1;
        }
        const bool less = was_refused && (a.probs != nullptr || x >= 0);
        const Part* part = a.parts + (row0 + s.n) * a.chunks;
        const double* rest = a.rest + (int64_t)b * a.chunks;
        // the refused word's chunk without it: their difference, but where that is next to
        // nothing (and would keep a rounding where nothing is left) added up again
        int cx = -1;
        double cx_sum = 0.0;
        if (x >= 0) {
            const Row<F32> row(a.logits, b * a.ldb + s.n * a.ldd);
            cx = (int)((x + row.head) / W::C::kWords);
            const double all = part[cx].sum * power(part[cx].top, s.row.top, s.rate, s.least);
            cx_sum = all - power(row.one((int)x), s.row.top, s.rate, s.least);
            if (!(cx_sum > 1e-6 * all)) {
                W weights;
                weights.load(a, b, s, cx, true, x);
                cx_sum = block_sum<T>(weights.sum(), sums);
            }
        }
        auto chunk_sum = [&](int c, bool off) {
            if (c >= a.chunks) return 0.0;
            if (off && a.probs != nullptr) return rest[c];
            if (off && c == cx) return cx_sum;
            return part[c].sum * power(part[c].top, s.row.top, s.rate, s.least);
        };
        // wave 0: the whole sum, then the chunk (64 chunks and fewer: both from one scan)
        if (w == 0) {
            double total = 0.0, v = 0.0, inc = 0.0;
            bool off = less;
            for (int pass = 0; pass < 2; ++pass) {
                total = 0.0;
                for (int c0 = 0; c0 < a.chunks; c0 += 64) {
                    v = chunk_sum(c0 + lane, off);
                    inc = wave_scan(v);
                    total += lane_value(inc, 63);
                }
                if (total > 0.0 || !off) break;
                off = false;
            }
            const double aim = u * total;
            double run = 0.0, before = 0.0;
            int at = -1;
            for (int c0 = 0; c0 < a.chunks && at < 0; c0 += 64) {
                if (a.chunks > 64) {
                    v = chunk_sum(c0 + lane, off);
                    inc = wave_scan(v);
                }
                const uint64_t found = __ballot(run + inc > aim && v > 0.0);
                if (found != 0) {
                    const int src = __builtin_ctzll(found);
                    at = c0 + src;
                    before = run + lane_value(inc - v, src);
                }
                run += lane_value(inc, 63);
            }
            bool last = false;
            if (at < 0) {           // the last word of the last chunk of positive weight
                last = true;
                for (int c0 = 0; c0 < a.chunks; c0 += 64) {
                    const uint64_t some = __ballot(chunk_sum(c0 + lane, off) > 0.0);
                    if (some != 0) at = c0 + 63 - __builtin_clzll(some);
                }
            }
            if (lane == 0) {
                where = off ? at : -1 - at;
                below = last ? __builtin_inf() : aim - before;
                hit = 0x7FFFFFFF;
                final = -1;
            }
        }
        __syncthreads();
        const bool off = where >= 0;
        W weights;
        weights.load(a, b, s, off ? where : -1 - where, off, x);
        const double mine = weights.sum(), inc = wave_scan(mine);
        if (lane == 63) sums[w] = inc;
        __syncthreads();
        double at = inc - mine;
#pragma unroll
        for (int k = 0; k < T / 64; ++k)
            if (k < w) at += sums[k];
        int first_hit = 0x7FFFFFFF, most = -1;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < W::VEC; ++j) {
                const double p = weights.p[i][j];
                const int v = weights.word[i] + j;
                at += p;
                if (p > 0.0) {
                    most = v;
                    if (at > below && v < first_hit) first_hit = v;
                }
            }
        // the words ascend with the lanes: of a wave one lane has its first, one its last
        const uint64_t hits = __ballot(first_hit != 0x7FFFFFFF), some = __ballot(most >= 0);
        if (hits != 0 && lane == __builtin_ctzll(hits)) atomicMin(&hit, first_hit);
        if (some != 0 && lane == 63 - __builtin_clzll(some)) atomicMax(&final, most);
        __syncthreads();
        token = hit != 0x7FFFFFFF ? hit : final;
    }
    for (int i = threadIdx.x; i <= a.D; i += T)
        a.tokens[row0 + i] = i < s.n ? (int)draft_of(a, b, i) : i == s.n ? token : -1;
    if (threadIdx.x == 0) a.accepted[b] = s.n;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Vectors of 16 bytes a thread holds of a chunk: as many as leave the GPU some chunks, four
// at most (32 x 16 rows of 129280 fp32 words 67 us, eight 69).
int vectors(int64_t rows, int64_t V, bool f32) {
    const int64_t words = kThreads * (f32 ? 4 : 8);
    int nv = 4;
    while (nv > 1 && rows * ((V + words * nv - 1) / (words * nv)) < 1024) nv /= 2;
    return nv;
}
int64_t chunk_count(int64_t rows, int64_t V, bool f32) {
    const int64_t size = (int64_t)vectors(rows, V, f32) * kThreads * (f32 ? 4 : 8);
    return (V + 7 + size - 1) / size;       // a row may start 7 words behind a boundary
}

template <bool F32, int NV>
hipError_t launch(const Args& a, hipStream_t s) {
    const auto grid = [&](int64_t rows) {
        const unsigned y = (unsigned)((rows + 32767) / 32768);
        return dim3((unsigned)a.chunks, y, (unsigned)(y > 1 ? 32768 : rows));
    };
    hipLaunchKernelGGL((parts_kernel<F32, NV>), grid((int64_t)a.B * (a.D + 1)), dim3(kThreads), 0,
                       s, a);
    if (a.probs != nullptr)
        hipLaunchKernelGGL((rest_kernel<F32, NV>), grid(a.B), dim3(kThreads), 0, s, a);
    constexpr int kWide = NV >= 4 ? 4 : 1;      // a long chunk over more threads
    const dim3 picks((unsigned)(a.B < kGridX ? a.B : kGridX),
                     (unsigned)((a.B + kGridX - 1) / kGridX));
    hipLaunchKernelGGL((pick_kernel<F32, NV / kWide, kThreads * kWide>), picks,
                       dim3(kThreads * kWide), 0, s, a);
    return hipGetLastError();
}

template <bool F32>
hipError_t launch_by(int nv, const Args& a, hipStream_t s) {
    switch (nv) {
        case 1: return launch<F32, 1>(a, s);
        case 2: return launch<F32, 2>(a, s);
        default: return launch<F32, 4>(a, s);
    }
}

}  // namespace

size_t workspace_bytes(int64_t B, int64_t D, int64_t V) {
    const int64_t rows = B * (D + 1);
    const int64_t c32 = chunk_count(rows, V, true), c16 = chunk_count(rows, V, false);
    const int64_t chunks = c32 > c16 ? c32 : c16;
    return up256((size_t)(rows * chunks) * sizeof(Part)) + up256((size_t)B * sizeof(Stop)) +
           (size_t)(B * chunks) * 8;
}

hipError_t launch_verify(Args a, void* ws, hipStream_t s) {
    const int64_t rows = (int64_t)a.B * (a.D + 1);
    a.chunks = (int)chunk_count(rows, a.V, a.f32);
    uint8_t* p = static_cast<uint8_t*>(ws);
    a.parts = reinterpret_cast<Part*>(p);
    p += up256((size_t)(rows * a.chunks) * sizeof(Part));
    a.stops = reinterpret_cast<Stop*>(p);
    p += up256((size_t)a.B * sizeof(Stop));
    a.rest = reinterpret_cast<double*>(p);
    const int nv = vectors(rows, a.V, a.f32);
    return a.f32 ? launch_by<true>(nv, a, s) : launch_by<false>(nv, a, s);
}

}  // namespace draft
