// Device helpers over the rows of a batch of sequences (fpstok_seqs), shared
// by the attention and the rotary-position kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "fpstok_attention.h"

namespace fpstok {

// Packed boundary b, clamped into the buffer.
__device__ __forceinline__ int64_t cu_at(const SeqArgs& s, int b) {
    const int64_t c = s.cu[b];
    return c < 0 ? 0 : c > s.rows ? s.rows : c;
}

// First row and length of sequence b; every value stays inside the buffer
// whatever cu / count hold.
__device__ __forceinline__ void seq_rows(const SeqArgs& s, int b, int64_t& start, int& len) {
    if (s.cu) {
        start = cu_at(s, b);
        const int64_t n = cu_at(s, b + 1) - start;
        len = n > 0 ? (int)n : 0;
    } else {
        start = (int64_t)b * s.cap;
        const int c = s.count[b];
        len = c < 0 ? 0 : c > s.cap ? s.cap : c;
    }
}

// Largest b in [0, B) with floor(cu[b] * G / tile) + b <= t, by the whole wave:
// each round tests 64 evenly spaced candidates at once.  In this numbering
// sequence b owns the slots from floor(cu[b] * G / tile) + b on, and it needs
// ceil(len * G / tile) of them, which end at or before the next sequence's
// first, so a grid of floor(rows * G / tile) + B slots covers every batch
// without knowing its lengths.  Every index stays in [0, B) for any cu.
__device__ __forceinline__ int find_seq(const SeqArgs& s, int64_t t, int G, int tile) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = s.B;
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int i = lane * step;
        const bool in = i < n && (cu_at(s, lo + i) * G) / tile + lo + i <= t;
        const int hits = __popcll(__ballot(in));
        const int k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        n = n - k * step < step ? n - k * step : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

__device__ __forceinline__ int64_t first_slot(const SeqArgs& s, int b, int G, int tile) {
    return (cu_at(s, b) * G) / tile + b;
}

}  // namespace fpstok
