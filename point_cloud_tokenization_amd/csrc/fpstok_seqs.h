// Device helpers over the rows of a batch of sequences (fpstok_seqs), shared
// by the attention and the rotary-position kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "fpstok_attention.h"

namespace fpstok {

// Packed boundary b, clamped into the buffer (rows < 2^31).
__device__ __forceinline__ int64_t cu_at(const SeqArgs& s, int b) {
    const int c = s.cu[b], rows = (int)s.rows;
    return c < 0 ? 0 : c > rows ? rows : c;
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

// Packed sequences in slots of 2^shift rows, `G` rows per buffer row: sequence
// b owns the slots from floor(cu[b] * G / 2^shift) + b on.  It needs
// ceil(len * G / 2^shift) of them, which end at or before the next sequence's
// first, so a grid of floor(rows * G / 2^shift) + B slots covers every batch
// without knowing its lengths.
__device__ __forceinline__ int64_t slot_of(int64_t cu, int b, int G, int shift) {
    if (G == 1) return (int64_t)((uint32_t)cu >> shift) + b;
    return (int64_t)((uint64_t)(cu * G) >> shift) + b;
}

// The sequence that owns `slot` (the largest b whose first slot is not past
// it), its rows, and the slot's number within it (negative if it is none's),
// by the whole wave: a round tests 64 evenly spaced candidates at once, and
// the last 256 adjacent ones, with both ends of each at hand.  Every index
// stays in [0, B] whatever cu holds.
__device__ __forceinline__ int find_seq(const SeqArgs& s, int64_t slot, int G, int shift,
                                        int64_t& start, int& len, int64_t& at) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = s.B;
    while (n > 256) {
        const int step = (n + 63) >> 6;
        const int i = lane * step;
        const int b = lo + (i < n ? i : 0);
        const int hits = __popcll(__ballot(i < n && slot_of(cu_at(s, b), b, G, shift) <= slot));
        const int k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        n = n - k * step < step ? n - k * step : step;
    }
    int c[5], hits = 0;  // (rows fit in 31 bits)
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        const int b = lo + 4 * lane + k;
        c[k] = (int)cu_at(s, b < s.B ? b : s.B);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = 4 * lane + k;
        hits += __popcll(__ballot(i < n && slot_of(c[k], lo + i, G, shift) <= slot));
    }
    const int k = __builtin_amdgcn_readfirstlane(hits > 0 ? hits - 1 : 0);
    const int sub = k & 3;
    const int c0 = sub == 0 ? c[0] : sub == 1 ? c[1] : sub == 2 ? c[2] : c[3];
    const int c1 = sub == 0 ? c[1] : sub == 1 ? c[2] : sub == 2 ? c[3] : c[4];
    start = __builtin_amdgcn_readlane(c0, k >> 2);
    const int left = __builtin_amdgcn_readlane(c1, k >> 2) - (int)start;
    len = left > 0 ? left : 0;
    lo = __builtin_amdgcn_readfirstlane(lo + k);
    at = slot - slot_of(start, lo, G, shift);
    return lo;
}

}  // namespace fpstok
