// Attention with a learned bias of the scores: the kernels of
// fpstok_attention_kernels.h with BIAS, and the sum of the tiles' parts of the
// table's gradient.
#include "fpstok_attention_kernels.h"

namespace fpstok {

// The plane of the pairs' entries: a workgroup takes 32 queries of a sequence, a
// thread a key at a time, up to the end of the last 32 keys (the last key again
// past the end, so every place that a block of 32 x 32 pairs reads holds an entry).
__global__ __launch_bounds__(256) void bias_plane_kernel(AttnArgs a, BiasArgs b) {
    __shared__ uint32_t own[kMaxAxes][32];
    const int tid = threadIdx.x;
    int64_t q0, k0, tile;
    int tq, tk, seq;
    const uint32_t slot = blockIdx.x;
    if (a.qs.cu) {
        seq = find_seq(a.qs, slot, 1, 5, q0, tq, tile);
        if (tile < 0) return;
    } else {
        const uint32_t per = (uint32_t)((a.qs.cap + 31) >> 5);
        seq = (int)(slot / per);
        tile = slot % per;
        seq_rows(a.qs, seq, q0, tq);
    }
    const int64_t left = tq - (tile << 5);
    if (a.same_seqs)
        k0 = q0, tk = tq;
    else
        seq_rows(a.ks, seq, k0, tk);
    if (left <= 0 || tk <= 0 || tk > b.pitch) return;
    const int rows = left < 32 ? (int)left : 32;
    const int64_t row0 = q0 + (tile << 5);
    for (int i = tid; i < 32 * kMaxAxes; i += 256) {
        const int r = i & 31, axis = i >> 5;
        if (axis < b.axes && r < rows) {
            const uint32_t x = ((const uint32_t*)b.q_pos)[(row0 + r) * b.axes + axis];
            own[axis][r] =
                b.ints ? x : __float_as_uint(__uint_as_float(x) * pick(b.rate, axis));
        }
    }
    __syncthreads();
    // 64 keys and every 4th row a wave
    const int lane = tid & 63, wave = tid >> 6;
    for (int j = lane; j < ((tk + 31) & ~31); j += 64) {
        uint32_t key[kMaxAxes];
#pragma unroll
        for (int axis = 0; axis < kMaxAxes; ++axis) {
            if (axis >= b.axes) break;
            const uint32_t x =
                ((const uint32_t*)b.k_pos)[(k0 + (j < tk ? j : tk - 1)) * b.axes + axis];
            key[axis] = b.ints ? x : __float_as_uint(__uint_as_float(x) * b.rate[axis]);
        }
        for (int r = wave; r < rows; r += 4) {
            uint32_t entries = 0;
#pragma unroll
            for (int axis = 0; axis < kMaxAxes; ++axis) {
                if (axis >= b.axes) break;
                by_kind(b.ints, b.log_shift[axis] >= 0, [&](auto ints, auto log) {
                    const int bucket = bucket_of<decltype(ints)::value, decltype(log)::value>(
                        key[axis], own[axis][r], b.rate[axis], b.shift[axis], b.top[axis],
                        b.log_shift[axis]);
                    entries |= (uint32_t)(b.first[axis] + bucket) << (8 * axis + 2);
                });
            }
            b.plane[(row0 + r) * b.pitch + j] = entries;
        }
    }
}

static void fill_plane(const AttnArgs& a, const BiasArgs& b, hipStream_t s) {
    if (!b.plane || a.qs.rows == 0) return;
    bias_plane_kernel<<<dim3((unsigned)row_slots(a.qs, 1, 5)), 256, 0, s>>>(a, b);
}

int32_t plan_plane(const AttnArgs& a, const BiasArgs& b, bool few, int32_t k_len) {
    if (few || b.entries > kTableEntries || a.H < 4 || k_len > 1024) return 0;
    // a window that hides most pairs of the plane
    if (a.left >= 0 && a.right >= 0 && 4 * ((int64_t)a.left + a.right + 1) < k_len) return 0;
    return (k_len + 31) & ~31;
}

// grad_table: the row tiles' parts in order, in 64 bits (a sum over every pair of
// the batch): 32 entries of one head per workgroup, 32 threads an entry.
__global__ __launch_bounds__(1024) void bias_table_kernel(BiasArgs b, int Hk, int G, int tiles) {
    __shared__ double sums[32][33];
    const int lane = threadIdx.x & 31, turn = threadIdx.x >> 5;
    const int h = blockIdx.x, hk = h / G, e = blockIdx.y * 32 + lane;
    const float* part =
        b.part + ((int64_t)hk * G + (h - hk * G)) * b.count + (e < b.count ? e : 0);
    const int64_t step = (int64_t)Hk * G * b.count;
    double sum = 0.0;
#pragma unroll 8
    for (int i = turn; i < tiles; i += 32) sum += (double)part[i * step];
    sums[turn][lane] = sum;
    __syncthreads();
    if (turn != 0 || e >= b.count) return;
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) total += sums[i][lane];
    b.grad[(int64_t)h * b.entries + b.from + e] = (float)total;
}

template <class T>
static hipError_t backward(const AttnArgs& a, BiasArgs b, hipStream_t s) {
    const bool rows = a.qs.rows > 0;
    fill_plane(a, b, s);
    if (!b.grad) {
        b.part = nullptr;
        if (rows) backward_q<T, true>(a, b, s);
    } else {
        // more than kTableEntries entries: a walk for each part of them
        const int tiles = rows ? (int)row_slots(a.qs, a.G, 7) : 0;
        for (b.from = 0; b.from < b.entries; b.from += b.count) {
            const int left = b.entries - b.from;
            b.count = left < kTableEntries ? left : kTableEntries;
            if (rows) backward_q<T, true>(a, b, s);
            bias_table_kernel<<<dim3((unsigned)a.H, (unsigned)((b.count + 31) / 32)), 1024, 0, s>>>(
                b, a.Hk, a.G, tiles);
        }
    }
    backward_kv<T, true>(a, b, s);
    return hipGetLastError();
}

hipError_t launch_attention_bias(const AttnArgs& a, const BiasArgs& b, const AttnPlan& plan,
                                 hipStream_t s) {
    fill_plane(a, b, s);
    return a.dtype == 0   ? forward<float, true>(a, b, plan, s)
           : a.dtype == 1 ? forward<_Float16, true>(a, b, plan, s)
                          : forward<__bf16, true>(a, b, plan, s);
}

hipError_t launch_attention_bias_backward(const AttnArgs& a, const BiasArgs& b, hipStream_t s) {
    return a.dtype == 0 ? backward<float>(a, b, s)
                        : a.dtype == 1 ? backward<_Float16>(a, b, s) : backward<__bf16>(a, b, s);
}

}  // namespace fpstok
