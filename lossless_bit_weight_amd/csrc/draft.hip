// draft.hip -- verification of drafted tokens (../../include/draft.h states the
// operation).
//
// Three launches.  parts: every row of logits is read once, in chunks over the GPU;
// a chunk leaves its largest logit and its sum of powers.  rest (with the drafter's
// probabilities): every workgroup of a sequence finds from the parts where it stops,
// and sums max(0, p - q) over its chunk of that row.  pick: one workgroup a sequence
// finds the chunk that the random number falls into, reads it again and finds the word.
// Powers, probabilities and sums are fp64: a word's border in the running sum of
// 10^5 words is then off by less than a random number of 24 bits can tell, so that
// the word does not depend on the order of summation.  The exponential costs 19 fp64
// instructions a word, which run at the rate of fp32's here, beside 2 or 4 bytes read.
#include "draft_internal.hpp"
#include "exp64.hpp"

namespace draft {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

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
    // Words v .. v + VEC - 1, v on a 16-byte boundary; those outside 0 .. V-1 are `none`.
    __device__ __forceinline__ void load(int v, int V, float none, float* f) const {
        if (v >= 0 && v + VEC <= V) {
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
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = v + j >= 0 && v + j < V ? one(v + j) : none;
        }
    }
};

// The sum over a workgroup, in every thread, in an order that depends on nothing.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w];
    return v;
}

__device__ __forceinline__ int length_of(const Args& a, int b) {
    if (a.lengths == nullptr) return a.D;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.D ? a.D : n;
}
// log2(e) / tau, or 0 for greedy
__device__ __forceinline__ double rate_of(const Args& a, int b) {
    if (a.temperature == nullptr) return kLog2E;
    const float tau = a.temperature[b];
    // (an infinite one: all words of finite logits alike)
    return tau > 0.f ? __builtin_fmax(kLog2E / (double)tau, 1e-300) : 0.0;
}
__device__ __forceinline__ int64_t draft_of(const Args& a, int b, int i) {
    const int64_t at = (int64_t)b * a.D + i;
    return a.drafts_i64 ? static_cast<const int64_t*>(a.drafts)[at]
                        : static_cast<const int*>(a.drafts)[at];
}
// 2^((l - top) rate)
__device__ __forceinline__ double power(float l, float top, double rate) {
    return l == -__builtin_inff() ? 0.0 : exp2_64(((double)l - (double)top) * rate);
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    return a != a || b != b ? __builtin_nanf("") : a > b ? a : b;
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void parts_kernel(Args a) {
    __shared__ double sums[kWaves];
    __shared__ float tops[kWaves];
    __shared__ int words[kWaves];
    const int row = blockIdx.y * 32768 + blockIdx.z;
    const int chunk = blockIdx.x;
    const int b = row / (a.D + 1), i = row % (a.D + 1);
    if (row >= a.B * (a.D + 1) || i > length_of(a, b)) return;
    const double rate = rate_of(a, b);
    const Row<F32> r(a.logits, b * a.ldb + i * a.ldd);
    constexpr int VEC = Row<F32>::VEC;
    const int first = chunk * a.size - r.head, last = first + a.size;

    float top = -__builtin_inff();
    int word = 0x7FFFFFFF;
    for (int v = first + (int)threadIdx.x * VEC; v < last && v < a.V; v += kThreads * VEC) {
        float f[VEC];
        r.load(v, a.V, -__builtin_inff(), f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if (f[j] != f[j] || f[j] == __builtin_inff()) {
                top = __builtin_nanf("");
            } else if (f[j] > top) {
                top = f[j];
                word = v + j;
            }
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const float ot = __shfl_xor(top, d);
        const int ow = __shfl_xor(word, d);
        if (ot > top || (ot == top && ow < word)) word = ow;
        top = max_nan(top, ot);
    }
    if ((threadIdx.x & 63) == 0) {
        tops[threadIdx.x >> 6] = top;
        words[threadIdx.x >> 6] = word;
    }
    __syncthreads();
    top = tops[0];
    word = words[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
        if (tops[w] > top || (tops[w] == top && words[w] < word)) word = words[w];
        top = max_nan(top, tops[w]);
    }
    double sum = 0.0;
    if (rate != 0.0 && top == top && top != -__builtin_inff()) {
        for (int v = first + (int)threadIdx.x * VEC; v < last && v < a.V; v += kThreads * VEC) {
            float f[VEC];
            r.load(v, a.V, -__builtin_inff(), f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += power(f[j], top, rate);
        }
    }
    sum = block_sum(sum, sums);
    if (threadIdx.x == 0) a.parts[(int64_t)row * a.chunks + chunk] = Part{sum, top, word};
}

// A row as a whole.
struct Whole {
    double sum;         // of 2^((l - top) rate)
    float top;          // NaN or -inf: no distribution
    int word;           // of the largest logit
    __device__ __forceinline__ bool good() const { return top > -__builtin_inff(); }
};

// The wave's: from the row's chunks, in every lane.
__device__ __forceinline__ Whole whole(const Args& a, int64_t row, double rate, int lane) {
    const Part* p = a.parts + row * a.chunks;
    Whole w{0.0, -__builtin_inff(), 0x7FFFFFFF};
    for (int c = lane; c < a.chunks; c += 64) {
        const float t = p[c].top;
        if (t > w.top || (t == w.top && p[c].word < w.word)) w.word = p[c].word;
        w.top = max_nan(w.top, t);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const float ot = __shfl_xor(w.top, d);
        const int ow = __shfl_xor(w.word, d);
        if (ot > w.top || (ot == w.top && ow < w.word)) w.word = ow;
        w.top = max_nan(w.top, ot);
    }
    if (!w.good() || rate == 0.0) return w;
    for (int c = lane; c < a.chunks; c += 64) w.sum += p[c].sum * power(p[c].top, w.top, rate);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) w.sum += __shfl_xor(w.sum, d);
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

// Where sequence b stops: its accepted tokens and the row behind them.
struct Stop {
    int n;              // accepted
    int length;
    Whole row;
};

// By the whole workgroup: wave w looks at the places w, w + kWaves, ...
__device__ __forceinline__ Stop stop_of(const Args& a, int b, double rate, int* refused,
                                        Whole* found) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int n = length_of(a, b);
    const int64_t row0 = (int64_t)b * (a.D + 1);
    if (threadIdx.x == 0) *refused = n;
    __syncthreads();
    for (int i = w; i < n; i += kWaves) {
        const Whole r = whole(a, row0 + i, rate, lane);
        const int64_t x = draft_of(a, b, i);
        bool ok = r.good() && x >= 0 && x < a.V;
        if (ok && rate == 0.0) {
            ok = x == r.word;
        } else if (ok) {
            const double q = a.probs == nullptr ? 1.0 : (double)prob(a, b, i, x);
            const double u = a.uniforms[row0 + i];
            ok = u * q * r.sum < power(logit(a, b, i, x), r.top, rate);
        }
        if (!ok) {
            if (lane == 0) atomicMin(refused, i);
            break;
        }
    }
    __syncthreads();
    Stop s;
    s.n = *refused;
    s.length = n;
    if (w == 0) {
        const Whole r = whole(a, row0 + s.n, rate, lane);
        if (lane == 0) *found = r;
    }
    __syncthreads();
    s.row = *found;
    return s;
}

// What a word is drawn by behind the accepted tokens, times the row's sum.
template <bool F32, int VEC>
struct Weights {
    const Args& a;
    const Stop& s;
    double rate;
    Row<F32> row;
    int64_t refused;            // without probabilities: the refused draft
    bool less;                  // take off what the drafter had
    int b;

    __device__ __forceinline__ Weights(const Args& args, const Stop& stop, double r, int seq,
                                       bool take)
        : a(args), s(stop), rate(r), row(args.logits, seq * args.ldb + stop.n * args.ldd),
          refused(-1), less(take), b(seq) {
        if (take && args.probs == nullptr) refused = draft_of(args, seq, stop.n);
    }
    __device__ __forceinline__ double of(int v, float l) const {
        double p = power(l, s.row.top, rate);
        if (less) {
            if (a.probs == nullptr) {
                if (v == refused) p = 0.0;
            } else {
                // (one instruction in every kernel: whether it is above 0 has to agree)
                const double d = __builtin_fma(-(double)prob(a, b, s.n, v), s.row.sum, p);
                p = d > 0.0 ? d : 0.0;
            }
        }
        return p;
    }
    // This thread's share of a chunk's sum.
    __device__ __forceinline__ double sum_of(int chunk) const {
        const int first = chunk * a.size - row.head, last = first + a.size;
        double sum = 0.0;
        for (int v = first + (int)threadIdx.x * VEC; v < last && v < a.V; v += kThreads * VEC) {
            float f[VEC];
            row.load(v, a.V, -__builtin_inff(), f);
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (f[j] != -__builtin_inff()) sum += of(v + j, f[j]);
        }
        return sum;
    }
};

template <bool F32>
__global__ __launch_bounds__(kThreads) void rest_kernel(Args a) {
    __shared__ double sums[kWaves];
    __shared__ int refused;
    __shared__ Whole found;
    const int b = blockIdx.y * 32768 + blockIdx.z, chunk = blockIdx.x;
    if (b >= a.B) return;
    const double rate = rate_of(a, b);
    const Stop s = stop_of(a, b, rate, &refused, &found);
    if (rate == 0.0 || s.n == s.length || !s.row.good()) return;
    constexpr int VEC = Row<F32>::VEC;
    const Weights<F32, VEC> weights(a, s, rate, b, true);
    const double sum = block_sum(weights.sum_of(chunk), sums);
    if (threadIdx.x == 0) a.rest[(int64_t)b * a.chunks + chunk] = sum;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ double wave_scan(double v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

template <bool F32>
__global__ __launch_bounds__(kThreads) void pick_kernel(Args a) {
    __shared__ double sums[kWaves];
    __shared__ int refused, where, final;
    __shared__ Whole found;
    __shared__ double below;
    const int b = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const double rate = rate_of(a, b);
    const Stop s = stop_of(a, b, rate, &refused, &found);
    const int64_t row0 = (int64_t)b * (a.D + 1);
    constexpr int VEC = Row<F32>::VEC;
    int token = -1;
    if (s.row.good() && rate == 0.0) {
        token = s.row.word;
    } else if (s.row.good()) {
        const bool was_refused = s.n < s.length;
        bool less = was_refused;
        if (less && a.probs == nullptr) {
            const int64_t x = draft_of(a, b, s.n);
            less = x >= 0 && x < a.V;
        }
        // sums of the chunks: kept (the rest), or the parts' rescaled
        const Part* part = a.parts + (row0 + s.n) * a.chunks;
        const double* rest = a.rest + (int64_t)b * a.chunks;
        const auto chunk_of = [&](int64_t v) {
            const Row<F32> r(a.logits, b * a.ldb + s.n * a.ldd);
            return (int)((v + r.head) / a.size);
        };
        const int64_t x = less && a.probs == nullptr ? draft_of(a, b, s.n) : -1;
        const int cx = x >= 0 ? chunk_of(x) : -1;
        // the refused draft's chunk without it: added up again, as a difference would leave
        // a rounding where nothing is left
        double cx_sum = 0.0;
        if (cx >= 0) {
            const Weights<F32, VEC> weights(a, s, rate, b, true);
            cx_sum = block_sum(weights.sum_of(cx), sums);
        }
        auto chunk_sum = [&](int c, bool off) {
            if (off && a.probs != nullptr) return rest[c];
            if (off && c == cx) return cx_sum;
            return part[c].sum * power(part[c].top, s.row.top, rate);
        };
        // wave 0: the whole sum, then the chunk
        if (w == 0) {
            double total = 0.0;
            bool off = less;
            for (int pass = 0; pass < 2; ++pass) {
                total = 0.0;
                for (int c0 = 0; c0 < a.chunks; c0 += 64)
                    total += __shfl(wave_scan(c0 + lane < a.chunks ? chunk_sum(c0 + lane, off) : 0.0,
                                              lane), 63);
                if (total > 0.0 || !off) break;
                off = false;
            }
            const double aim = (double)a.uniforms[row0 + a.D] * total;
            double run = 0.0, before = 0.0;
            int at = -1;
            for (int c0 = 0; c0 < a.chunks && at < 0; c0 += 64) {
                const double v = c0 + lane < a.chunks ? chunk_sum(c0 + lane, off) : 0.0;
                const double inc = wave_scan(v, lane);
                const uint64_t hit = __ballot(run + inc > aim && v > 0.0);
                if (hit != 0) {
                    const int src = __builtin_ctzll(hit);
                    at = c0 + src;
                    before = run + __shfl(inc - v, src);
                }
                run += __shfl(inc, 63);
            }
            if (at < 0) {           // the last chunk of positive weight
                for (int c0 = 0; c0 < a.chunks; c0 += 64) {
                    const double v = c0 + lane < a.chunks ? chunk_sum(c0 + lane, off) : 0.0;
                    const uint64_t some = __ballot(v > 0.0);
                    if (some != 0) at = c0 + 63 - __builtin_clzll(some);
                }
                before = -1.0;      // its last word
            }
            if (lane == 0) {
                where = off ? at : -1 - at;
                below = before < 0.0 ? __builtin_inf() : aim - before;
            }
        }
        __syncthreads();
        less = where >= 0;
        const int chunk = less ? where : -1 - where;
        const double aim = below;
        const Weights<F32, VEC> weights(a, s, rate, b, less);
        const int first = chunk * a.size - weights.row.head, last = first + a.size;
        double run = 0.0;
        int hit = 0x7FFFFFFF, most = -1;
        for (int v0 = first; v0 < last && v0 < a.V; v0 += kThreads * VEC) {
            const int v = v0 + (int)threadIdx.x * VEC;
            double p[VEC], mine = 0.0;
            float f[VEC];
            weights.row.load(v, v < last ? a.V : 0, -__builtin_inff(), f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                p[j] = f[j] != -__builtin_inff() ? weights.of(v + j, f[j]) : 0.0;
                mine += p[j];
            }
            const double inc = wave_scan(mine, lane);
            __syncthreads();
            if (lane == 63) sums[w] = inc;
            __syncthreads();
            double at = run + inc - mine;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) {
                if (k < w) at += sums[k];
                run += sums[k];
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                at += p[j];
                if (p[j] > 0.0) {
                    most = v + j;
                    if (at > aim && v + j < hit) hit = v + j;
                }
            }
        }
        if (threadIdx.x == 0) {
            refused = 0x7FFFFFFF;
            final = -1;
        }
        __syncthreads();
        atomicMin(&refused, hit);
        atomicMax(&final, most);
        __syncthreads();
        token = refused != 0x7FFFFFFF ? refused : final;
    }
    for (int i = threadIdx.x; i <= a.D; i += kThreads)
        a.tokens[row0 + i] = i < s.n ? (int)draft_of(a, b, i) : i == s.n ? token : -1;
    if (threadIdx.x == 0) a.accepted[b] = s.n;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Words of a chunk.
int chunk_size(int64_t rows, int64_t V) {
    int size = 8192;
    while (size > 2048 && rows * ((V + size - 1) / size) < 1024) size /= 2;
    return size;
}
int64_t chunk_count(int64_t rows, int64_t V) {
    const int size = chunk_size(rows, V);
    return (V + 7 + size - 1) / size;       // a row may start 7 words behind a boundary
}

template <bool F32>
hipError_t launch(const Args& a, hipStream_t s) {
    const auto grid = [&](int64_t rows) {
        const unsigned y = (unsigned)((rows + 32767) / 32768);
        return dim3((unsigned)a.chunks, y, (unsigned)(y > 1 ? 32768 : rows));
    };
    hipLaunchKernelGGL(parts_kernel<F32>, grid((int64_t)a.B * (a.D + 1)), dim3(kThreads), 0, s, a);
    if (a.probs != nullptr && a.D > 0)
        hipLaunchKernelGGL(rest_kernel<F32>, grid(a.B), dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(pick_kernel<F32>, dim3((unsigned)a.B), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t workspace_bytes(int64_t B, int64_t D, int64_t V) {
    const int64_t chunks = chunk_count(B * (D + 1), V);
    return up256((size_t)(B * (D + 1) * chunks) * sizeof(Part)) + (size_t)(B * chunks) * 8;
}

hipError_t launch_verify(Args a, void* ws, hipStream_t s) {
    const int64_t rows = (int64_t)a.B * (a.D + 1);
    a.size = chunk_size(rows, a.V);
    a.chunks = (int)chunk_count(rows, a.V);
    a.parts = static_cast<Part*>(ws);
    a.rest = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) +
                                       up256((size_t)(rows * a.chunks) * sizeof(Part)));
    return a.f32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace draft
