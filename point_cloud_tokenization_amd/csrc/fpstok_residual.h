// Internal interface between the C ABI (fpstok_residual_api.cpp) and the gfx950
// kernels of the residual step (fpstok_residual.hip).  Not installed; not part
// of the ABI.
#pragma once

#include "fpstok_attention.h"

namespace fpstok {

struct RowsArg {
    void* data;  // null: not given
    int64_t row;  // stride in elements
};

constexpr int kResidualWeights = 5;  // post weight, post bias, scale, pre weight, pre bias

struct ResidualArgs {
    SeqArgs seqs;
    RowsArg x, y, gate, x_out, h;
    RowsArg grad_x_out, grad_h, grad_x, grad_y, grad_gate;
    const float* weights[kResidualWeights];  // null: ones, or zeros for a bias
    float* weight_grads[kResidualWeights];   // null: not formed
    float* stats;                            // [rows][4]: post mean, 1/std, pre mean, 1/std
    int32_t C, stream, branch;               // width, dtypes
    int32_t post, pre, gate_per, act;        // as in fpstok_residual_params
    float eps;
    // plan_residual: elements of a row that a thread holds, threads of a row, and
    // in how many runs of adjacent rows the rows are shared out
    int32_t elements, threads, runs;
    // backward: the workgroups' parts of the weights' gradients, [workgroups][given
    // weights][C], and of the gates of sequences, [runs + sequences][C]
    float* part;
    float* gate_part;
};

// The parts of a sequence's gate gradient: the rows start .. start + len - 1 of
// sequence b among rows first .. last - 1, shared out in runs of `per` adjacent
// ones.  In range whatever the boundaries are: sequences that run backwards may
// begin before the first one or end behind the last.
struct GateParts {
    int64_t first;
    int n;
};
__host__ __device__ inline GateParts gate_parts(int64_t start, int len, int64_t first,
                                                int64_t last, int per, int b) {
    const int64_t lo = start > first ? start : first;
    const int64_t hi = start + len < last ? start + len : last;
    if (lo >= hi) return GateParts{0, 0};
    const uint32_t run = (uint32_t)per, from = (uint32_t)(lo - first) / run;
    return GateParts{(int64_t)from + b, (int)((uint32_t)(hi - 1 - first) / run - from) + 1};
}

void plan_residual(ResidualArgs& a, bool backward);
int64_t residual_blocks(const ResidualArgs& a);  // workgroups
hipError_t launch_residual(const ResidualArgs& a, hipStream_t s);
hipError_t launch_residual_backward(const ResidualArgs& a, hipStream_t s);

}  // namespace fpstok
