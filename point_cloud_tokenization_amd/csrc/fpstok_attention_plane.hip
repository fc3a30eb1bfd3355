// Attention with a learned bias whose pairs' entries are found once for all heads:
// the plane that holds them, and the kernels that read it.
#include "fpstok_attention_bias.h"

namespace fpstok {

// The plane of the pairs' entries: a workgroup takes 16 queries of a sequence, a
// thread a key at a time, up to the end of the last 32 keys (the last key again
// past the end, so every place that a block of 32 x 32 pairs reads holds an entry).
// Bound by the vector unit, about 6 instructions a pair and axis, once and not for
// every head: 256 events of up to 256 tokens, 4 axes, 24 us.  (12 heads of 64: with it,
// and tiles of 32 keys in grad_q's kernel, a training step took 1130 us instead of
// 1775.)
__global__ __launch_bounds__(256) void bias_plane_kernel(AttnArgs a, BiasArgs b) {
    __shared__ uint32_t own[kMaxAxes][16];
    const int tid = threadIdx.x;
    int64_t q0, k0, tile;
    int tq, tk, seq;
    const uint32_t slot = blockIdx.x;
    if (a.qs.cu) {
        seq = find_seq(a.qs, slot, 1, 4, q0, tq, tile);
        if (tile < 0) return;
    } else {
        const uint32_t per = (uint32_t)((a.qs.cap + 15) >> 4);
        seq = (int)(slot / per);
        tile = slot % per;
        seq_rows(a.qs, seq, q0, tq);
    }
    const int64_t left = tq - (tile << 4);
    if (a.same_seqs)
        k0 = q0, tk = tq;
    else
        seq_rows(a.ks, seq, k0, tk);
    if (left <= 0 || tk <= 0 || tk > b.pitch) return;
    const int rows = left < 16 ? (int)left : 16;
    const int64_t row0 = q0 + (tile << 4);
    const int keys = (tk + 31) & ~31;
    if (tid < 16 * kMaxAxes) {
        const int r = tid & 15, axis = tid >> 4;
        if (axis < b.axes && r < rows) {
            const uint32_t x = ((const uint32_t*)b.q_pos)[(row0 + r) * b.axes + axis];
            own[axis][r] =
                b.ints ? x : __float_as_uint(__uint_as_float(x) * pick(b.rate, axis));
        }
    }
    __syncthreads();
    // 4 rows and every 64th key a wave
    const int r0 = tid >> 6 << 2;
    if (r0 >= rows) return;
    const uint32_t joint_base = entry_base<true>(b), bytes_base = entry_base<false>(b);
    for (int j = tid & 63; j < keys; j += 64) {
        uint32_t joint[4], bytes[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) joint[r] = joint_base, bytes[r] = bytes_base;
#pragma unroll
        for (int axis = 0; axis < kMaxAxes; ++axis) {
            if (axis >= b.axes) break;
            const uint32_t x =
                ((const uint32_t*)b.k_pos)[(k0 + (j < tk ? j : tk - 1)) * b.axes + axis];
            const uint32_t key =
                b.ints ? x : __float_as_uint(__uint_as_float(x) * b.rate[axis]);
            const uint32_t unit = entry_unit<true>(b, axis);
            by_kind(b.ints, b.log_shift[axis] >= 0, [&](auto ints, auto log) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int bucket = bucket_of<decltype(ints)::value, decltype(log)::value>(
                        key, own[axis][r0 + r], b.rate[axis], b.shift[axis], b.top[axis],
                        b.log_shift[axis]);
                    joint[r] += (uint32_t)bucket * unit;
                    bytes[r] += (uint32_t)bucket * entry_unit<false>(b, axis);
                }
            });
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r0 + r >= rows) break;
            const int64_t at = (row0 + r0 + r) * b.pitch + j;
            b.plane[at] = joint[r];
            if (b.bytes) b.bytes[at] = bytes[r];
        }
    }
}

static void fill_plane(const AttnArgs& a, const BiasArgs& b, hipStream_t s) {
    if (!b.plane || a.qs.rows == 0) return;
    bias_plane_kernel<<<dim3((unsigned)row_slots(a.qs, 1, 4)), 256, 0, s>>>(a, b);
}

int32_t plan_plane(const AttnArgs& a, const BiasArgs& b, bool few, int32_t k_len) {
    // (64 padded float32 events of up to 128 tokens, 8 heads, 2 axes: 37 us without, 40
    // with it; 64 events, 12 heads, 4 axes: 34.7 and 31.8)
    if (few || b.entries > kTableEntries || a.H * b.axes < 24) return 0;
    // Longer sequences: two axes or more, planes of up to 1 GiB.  In bfloat16, with the
    // plane and by positions, us: 2 of 2500 rows, 12 heads of 64, 4 axes 224 and 352, a
    // training step 917 and 1455; 2 axes 197 and 227, 792 and 932; causal, whose plane is
    // half hidden, 177 and 203, 740 and 891.  6000 + 2111 + 64 rows, 16 heads on 8 of 128, 4
    // axes 1060 and 1476, 7.1 and 10.4 ms; 2 axes 968 and 920 (the one form that loses;
    // causal 548 and 488), 6.4 and 7.1 ms.  (One axis in order, 4000 causal rows, 24 heads
    // on 8 of 128: 1765 and 1371.)
    if (k_len > (b.axes > 1 ? 8192 : 1024) || a.qs.rows * ((k_len + 31) & ~31) > 1 << 28) return 0;
    if ((int64_t)a.G * table_size(b, true) > kGroupEntries) return 0;
    // a window that hides most pairs of the plane
    if (a.left >= 0 && a.right >= 0 && 4 * ((int64_t)a.left + a.right + 1) < k_len) return 0;
    return (k_len + 31) & ~31;
}

hipError_t launch_plane(const AttnArgs& a, const BiasArgs& b, const AttnPlan& plan, hipStream_t s) {
    fill_plane(a, b, s);
    return launch<kPlane>(a, b, plan, s);
}

hipError_t launch_plane_backward(const AttnArgs& a, const BiasArgs& b, hipStream_t s) {
    fill_plane(a, b, s);
    return launch_backward<kPlane>(a, b, s);
}

}  // namespace fpstok
