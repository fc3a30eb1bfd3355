// Attention with a learned bias of the scores: the kernels of
// fpstok_attention_kernels.h whose heads find the pairs' entries themselves, and
// the sum of the tiles' parts of the table's gradient.
#include "fpstok_attention_bias.h"

namespace fpstok {

// grad_table: the row tiles' parts in order, in 64 bits (a sum over every pair of
// the batch): 32 entries of one head per workgroup, 32 threads an entry.  A launch and
// the latency of its loads: 12 heads of 62 entries from 512 tiles, 5.8 us.
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

void launch_bias_table(const BiasArgs& b, const AttnArgs& a, int tiles, hipStream_t s) {
    const dim3 grid((unsigned)a.H, (unsigned)((b.count + 31) / 32));
    bias_table_kernel<<<grid, 1024, 0, s>>>(b, a.Hk, a.G, tiles);
}

hipError_t launch_attention_bias(const AttnArgs& a, const BiasArgs& b, const AttnPlan& plan,
                                 hipStream_t s) {
    return b.plane ? launch_plane(a, b, plan, s) : launch<kPositions>(a, b, plan, s);
}

hipError_t launch_attention_bias_backward(const AttnArgs& a, const BiasArgs& b, hipStream_t s) {
    return b.plane ? launch_plane_backward(a, b, s) : launch_backward<kPositions>(a, b, s);
}

}  // namespace fpstok
