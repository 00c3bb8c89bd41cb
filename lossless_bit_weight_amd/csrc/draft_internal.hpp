// draft_internal.hpp -- arguments and launcher of the verification of drafted
// tokens (../../include/draft.h states the operation).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace draft {

// A chunk of a row: its largest logit (NaN: the chunk holds a NaN or +inf), that
// one's first word, and the sum of 2^((logit - largest) log2(e) / tau).
struct Part {
    double sum;
    float top;
    int word;
};

// A row as a whole.
struct Whole {
    double sum;         // of 2^((l - top) rate)
    float top;          // NaN or -inf: no distribution
    int word;           // of the largest logit
    __device__ __forceinline__ bool good() const { return top > -__builtin_inff(); }
};

// Where a sequence stops: its accepted tokens and the row behind them.
struct Stop {
    Whole row;
    double rate, least; // log2(e) / tau, 0: greedy; and -1000 / rate
    int n, length;      // accepted, drafted
};

struct Args {
    const void* logits;
    int f32;
    int B, D, V;
    int64_t ldb, ldd;
    const void* drafts;
    int drafts_i64;
    const float* uniforms;
    const void* probs;
    int probs_f32;
    int64_t pdb, pdd;
    const int* lengths;
    const float* temperature;
    int* tokens;
    int* accepted;
    int chunks;             // a row's
    // workspace
    Part* parts;            // [B (D + 1)][chunks]
    Stop* stops;            // [B], with probs
    double* rest;           // [B][chunks], with probs: sums of max(0, p - q)
};

size_t workspace_bytes(int64_t B, int64_t D, int64_t V);
hipError_t launch_verify(Args a, void* ws, hipStream_t s);

}  // namespace draft
