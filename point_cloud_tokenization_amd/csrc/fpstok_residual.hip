// The residual step between two blocks of an encoder and its gradients:
//   u = post_norm(y),  z = act(gate) u,  xo = x + scale z,  h = pre_norm(xo).
#include "fpstok_mma.h"
#include "fpstok_residual.h"
#include "fpstok_seqs.h"

namespace fpstok {

// A row of C <= 8192 elements belongs to T threads (64 to 1024), 8 elements to
// each: 8 adjacent ones (VEC = 8: 16-byte accesses), or every T-th one where
// width, pointers or strides do not allow that (VEC = 1).
constexpr int kEl = 8;

template <int VEC, int T>
__device__ __forceinline__ int col(int t, int e) {
    return VEC == 8 ? t * 8 + e : t + e * T;
}

// A thread's elements of a row as they came from memory.  Threads and elements
// past the width load an element that exists (a load under a divergent branch
// would be waited for before the branch ends) and count as 0.
template <class E, int VEC, int T>
struct Raw {
    using V = uint32_t __attribute__((ext_vector_type(4)));
    V v[VEC == 8 ? sizeof(E) / 2 : 1];
    E e[VEC == 8 ? 1 : kEl];
    __device__ __forceinline__ void load(const E* p, int C, int t) {
        if constexpr (VEC == 8) {
            const int c = t * 8 < C ? t * 8 : 0;
#pragma unroll
            for (int i = 0; i < (int)sizeof(E) / 2; ++i) v[i] = ((const V*)(p + c))[i];
        } else {
#pragma unroll
            for (int i = 0; i < kEl; ++i) {
                const int c = col<VEC, T>(t, i);
                e[i] = p[c < C ? c : 0];
            }
        }
    }
    __device__ __forceinline__ void get(float* f, int C, int t) const {
        if constexpr (VEC == 8) {
            using E8 = E __attribute__((ext_vector_type(8)));
            const E8 x = *(const E8*)v;
            const bool in = t * 8 < C;
#pragma unroll
            for (int i = 0; i < kEl; ++i) f[i] = in ? (float)x[i] : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < kEl; ++i) f[i] = col<VEC, T>(t, i) < C ? (float)e[i] : 0.0f;
        }
    }
};

template <class E, int VEC, int T>
__device__ __forceinline__ void store(E* p, const float* f, int C, int t) {
    if constexpr (VEC == 8) {
        using V = uint32_t __attribute__((ext_vector_type(4)));
        using E8 = E __attribute__((ext_vector_type(8)));
        E8 x;
#pragma unroll
        for (int i = 0; i < kEl; ++i) x[i] = (E)f[i];
        if (t * 8 < C) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(E) / 2; ++i)
                ((V*)(p + t * 8))[i] = ((const V*)&x)[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kEl; ++i) {
            const int c = col<VEC, T>(t, i);
            if (c < C) p[c] = (E)f[i];
        }
    }
}

template <int VEC, int T>
__device__ __forceinline__ void load_weight(float* f, const float* w, float none, int C, int t) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < kEl; ++i) f[i] = none;
        return;
    }
    Raw<float, VEC, T> r;
    r.load(w, C, t);
    r.get(f, C, t);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __uint_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// The sum over a wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float x) {
    x += dpp<0xb1>(x);   // lanes l ^ 1
    x += dpp<0x4e>(x);   // l ^ 2
    x += dpp<0x141>(x);  // 7 - l % 8
    x += dpp<0x140>(x);  // 15 - l % 16
    const auto s =
        __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return pair_sum(__uint_as_float(s[0]) + __uint_as_float(s[1]));
}

// Sums over the T threads of a row.  A workgroup of T > 64 exchanges its waves'
// sums in LDS, in one of two places in turn: a wave that writes the third sum
// has passed the barrier of the second, which every wave reaches only after it
// has read the first.
template <int T>
struct RowSum {
    float (*lds)[2][16];
    int turn = 0;
    __device__ __forceinline__ void operator()(float& a, float& b) {
        a = wave_sum(a);
        b = wave_sum(b);
        if constexpr (T > 64) {
            const int wave = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) lds[turn][0][wave] = a, lds[turn][1][wave] = b;
            __syncthreads();
            a = 0.0f, b = 0.0f;
#pragma unroll
            for (int w = 0; w < T / 64; ++w) a += lds[turn][0][w], b += lds[turn][1][w];
            turn ^= 1;
        }
    }
    __device__ __forceinline__ void operator()(float& a) {
        float none = 0.0f;
        (*this)(a, none);
    }
};

// The sequence that holds a row, by the whole wave: the last of [0, B) that
// starts at or before it (64 evenly spaced candidates a round).  In range
// whatever cu holds.
__device__ __forceinline__ int seq_of_row(const SeqArgs& s, int64_t row) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = s.B;
    while (n > 1) {
        const int step = (n + 63) >> 6, i = lane * step;
        const int hits = __popcll(__ballot(i < n && cu_at(s, lo + (i < n ? i : 0)) <= row));
        const int k = hits > 0 ? hits - 1 : 0;
        lo += k * step;
        n = n - k * step < step ? n - k * step : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The rows of a run in order, and what is known of each: its sequence (packed:
// only if SEQ asks for it) and whether it is one of it.
struct RunRows {
    const SeqArgs& s;
    bool seq;
    int b = 0;
    int64_t lo, hi, end, live_end;  // rows of the run; where the sequence's slots and rows end
    __device__ __forceinline__ RunRows(const SeqArgs& s, int64_t run, int shift, bool seq)
        : s(s), seq(seq) {
        lo = run << shift;
        hi = lo + ((int64_t)1 << shift);
        if (hi > s.rows) hi = s.rows;
        if (s.cu) {
            const int64_t first = cu_at(s, 0), last = cu_at(s, s.B);
            if (lo < first) lo = first;
            if (hi > last) hi = last;
            end = live_end = hi;
            if (seq && lo < hi) {
                b = seq_of_row(s, lo);
                end = live_end = cu_at(s, b + 1);
            }
        } else if (lo < hi) {
            at_slot((int)((uint32_t)lo / (uint32_t)s.cap));
        }
    }
    __device__ __forceinline__ void at_slot(int seq_no) {
        b = seq_no;
        const int c = s.count[b];
        end = (int64_t)(b + 1) * s.cap;
        live_end = (int64_t)b * s.cap + (c < 0 ? 0 : c > s.cap ? s.cap : c);
    }
    // Moves on to the sequence that holds row r.
    __device__ __forceinline__ void to(int64_t r) {
        if (r < end) return;
        if (s.cu) {
            if (!seq) return;
            while (r >= end && b + 1 < s.B) end = cu_at(s, ++b + 1);
            live_end = end;
        } else {
            at_slot(b + 1 < s.B ? b + 1 : b);
        }
    }
};

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// Norms a row in place: (x - mean) / std with LAYER, x / rms without; `mean`
// and `r` = 1 / sqrt(mean square + eps) are returned.  The mean comes off
// before the squares are summed, in 32 bits; elements past the width stay 0.
template <int VEC, int T>
__device__ __forceinline__ void norm_row(float* x, bool layer, float inv_c, float eps, int C, int t,
                                         RowSum<T>& sum, float& mean, float& r) {
    mean = 0.0f;
    if (layer) {
#pragma unroll
        for (int i = 0; i < kEl; ++i) mean += x[i];
        sum(mean);
        mean *= inv_c;
#pragma unroll
        for (int i = 0; i < kEl; ++i) x[i] = col<VEC, T>(t, i) < C ? x[i] - mean : 0.0f;
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < kEl; ++i) q = __builtin_fmaf(x[i], x[i], q);
    sum(q);
    r = 1.0f / sqrtf(__builtin_fmaf(q, inv_c, eps));
#pragma unroll
    for (int i = 0; i < kEl; ++i) x[i] *= r;
}

template <int T>
constexpr int kThreads = T == 64 ? 256 : T;

// Forward.  The T threads of a row hold it in registers from the first load to
// the last store, so every operand is read and every result written once; a
// workgroup takes a run of adjacent rows, keeps the weights in registers and
// has the next row's loads on their way while it works on one.
template <class S, class B, int VEC, int T>
__global__ __launch_bounds__(kThreads<T>) void residual_kernel(ResidualArgs a) {
    __shared__ float lds[2][2][16];
    const int tid = threadIdx.x, t = tid % T, C = a.C;
    const int group = __builtin_amdgcn_readfirstlane(tid / T);
    const int64_t run = (int64_t)blockIdx.x * (kThreads<T> / T) + group;
    RowSum<T> sum{lds};
    RunRows rows(a.seqs, run, a.shift, a.gate_per == 2);
    if (rows.lo >= rows.hi) return;  // (the same for all threads of a row)
    const float inv_c = 1.0f / (float)C;
    const bool has_y = a.y.data != nullptr, gated = a.gate_per != 0;
    float wp[kEl], bp[kEl], sc[kEl], wh[kEl], bh[kEl];
    load_weight<VEC, T>(wp, a.weights[0], 1.0f, C, t);
    load_weight<VEC, T>(bp, a.weights[1], 0.0f, C, t);
    load_weight<VEC, T>(sc, a.weights[2], 1.0f, C, t);
    load_weight<VEC, T>(wh, a.weights[3], 1.0f, C, t);
    load_weight<VEC, T>(bh, a.weights[4], 0.0f, C, t);
    Raw<S, VEC, T> rx;
    Raw<B, VEC, T> ry, rg;
    auto load = [&](int64_t r) {
        rx.load((const S*)a.x.data + r * a.x.row, C, t);
        if (has_y) ry.load((const B*)a.y.data + r * a.y.row, C, t);
        if (gated)
            rg.load((const B*)a.gate.data + (a.gate_per == 2 ? rows.b : r) * a.gate.row, C, t);
    };
    load(rows.lo);
    for (int64_t r = rows.lo; r < rows.hi; ++r) {
        const bool live = r < rows.live_end;
        float x[kEl], y[kEl], g[kEl];
        rx.get(x, C, t);
        if (has_y) ry.get(y, C, t);
        if (gated) rg.get(g, C, t);
        if (r + 1 < rows.hi) {
            rows.to(r + 1);
            load(r + 1);
        }
        S* xo = a.x_out.data ? (S*)a.x_out.data + r * a.x_out.row : nullptr;
        B* h = a.h.data ? (B*)a.h.data + r * a.h.row : nullptr;
        float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!live) {
#pragma unroll
            for (int i = 0; i < kEl; ++i) x[i] = 0.0f;
            if (xo) store<S, VEC, T>(xo, x, C, t);
            if (h) store<B, VEC, T>(h, x, C, t);
            if (a.stats && t == 0) ((float4*)a.stats)[r] = st;
            continue;
        }
        if (has_y) {
            if (a.post != 0) {
                norm_row<VEC, T>(y, a.post == 2, inv_c, a.eps, C, t, sum, st.x, st.y);
#pragma unroll
                for (int i = 0; i < kEl; ++i) y[i] = __builtin_fmaf(y[i], wp[i], bp[i]);
            }
            if (gated) {
#pragma unroll
                for (int i = 0; i < kEl; ++i) {
                    if (a.act == 0)
                        y[i] *= g[i];
                    else
                        y[i] *= a.act == 1 ? sigmoid(g[i]) : g[i] * sigmoid(g[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kEl; ++i)
                x[i] = col<VEC, T>(t, i) < C ? __builtin_fmaf(y[i], sc[i], x[i]) : 0.0f;
        }
        if (xo) store<S, VEC, T>(xo, x, C, t);
        if (a.pre != 0) {
            norm_row<VEC, T>(x, a.pre == 2, inv_c, a.eps, C, t, sum, st.z, st.w);
#pragma unroll
            for (int i = 0; i < kEl; ++i) x[i] = __builtin_fmaf(x[i], wh[i], bh[i]);
            store<B, VEC, T>(h, x, C, t);
        }
        if (a.stats && t == 0) ((float4*)a.stats)[r] = st;
    }
}

// The gradients, from the same inputs and the rows' statistics: xo is formed
// again, so it enters unrounded and x, which the stream holds anyway, is all
// that is kept.  With xh the normed xo, yh the normed y, p = grad_h * pre
// weight:
//   gx = grad_x_out + rx (p - mean(p) - xh mean(p xh))     (mean(p): LAYER only)
//   gu = gx scale act(g),  grad_gate = gx scale u act'(g)
//   grad_y = ry (q - mean(q) - yh mean(q yh)),  q = gu * post weight
// A thread sums the weights' gradients of its columns over the rows of its
// run, in order; the workgroup adds its waves' and leaves one part, which the
// kernels below add in order: results are equal from run to run.
template <class S, class B, int VEC, int T>
__global__ __launch_bounds__(kThreads<T>) void residual_grad_kernel(ResidualArgs a) {
    __shared__ float lds[2][2][16];
    __shared__ float cols[T == 64 ? 3 : 1][T == 64 ? 64 * kEl : 1];
    const int tid = threadIdx.x, t = tid % T, C = a.C;
    const int group = __builtin_amdgcn_readfirstlane(tid / T);
    const int64_t run = (int64_t)blockIdx.x * (kThreads<T> / T) + group;
    RowSum<T> sum{lds};
    RunRows rows(a.seqs, run, a.shift, a.gate_per == 2);
    const float inv_c = 1.0f / (float)C;
    const bool has_y = a.y.data != nullptr, gated = a.gate_per != 0;
    const bool has_gx = a.grad_x_out.data != nullptr, has_gh = a.grad_h.data != nullptr;
    float wp[kEl], bp[kEl], sc[kEl], wh[kEl];
    load_weight<VEC, T>(wp, a.weights[0], 1.0f, C, t);
    load_weight<VEC, T>(bp, a.weights[1], 0.0f, C, t);
    load_weight<VEC, T>(sc, a.weights[2], 1.0f, C, t);
    load_weight<VEC, T>(wh, a.weights[3], 1.0f, C, t);
    float acc[kResidualWeights][kEl], gate_acc[kEl];
#pragma unroll
    for (int i = 0; i < kEl; ++i) {
#pragma unroll
        for (int k = 0; k < kResidualWeights; ++k) acc[k][i] = 0.0f;
        gate_acc[i] = 0.0f;
    }
    Raw<S, VEC, T> rx, rgx;
    Raw<B, VEC, T> ry, rg, rgh;
    float4 st_next = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto load = [&](int64_t r) {
        rx.load((const S*)a.x.data + r * a.x.row, C, t);
        if (has_y) ry.load((const B*)a.y.data + r * a.y.row, C, t);
        if (gated)
            rg.load((const B*)a.gate.data + (a.gate_per == 2 ? rows.b : r) * a.gate.row, C, t);
        if (has_gx) rgx.load((const S*)a.grad_x_out.data + r * a.grad_x_out.row, C, t);
        if (has_gh) rgh.load((const B*)a.grad_h.data + r * a.grad_h.row, C, t);
        if (a.stats) st_next = ((const float4*)a.stats)[r];
    };
    const bool gate_sums = a.gate_per == 2 && a.grad_gate.data != nullptr;
    if (rows.lo < rows.hi) load(rows.lo);
    for (int64_t r = rows.lo; r < rows.hi; ++r) {
        const bool live = r < rows.live_end;
        const int b = rows.b;
        const float4 st = st_next;
        float x[kEl], y[kEl], g[kEl], gx[kEl], gh[kEl];
        rx.get(x, C, t);
        if (has_y) ry.get(y, C, t);
        if (gated) rg.get(g, C, t);
        if (has_gh) rgh.get(gh, C, t);
#pragma unroll
        for (int i = 0; i < kEl; ++i) gx[i] = 0.0f;
        if (has_gx) rgx.get(gx, C, t);
        const bool more = r + 1 < rows.hi;
        if (more) {
            rows.to(r + 1);
            load(r + 1);
        }
        S* ox = a.grad_x.data ? (S*)a.grad_x.data + r * a.grad_x.row : nullptr;
        B* oy = a.grad_y.data ? (B*)a.grad_y.data + r * a.grad_y.row : nullptr;
        B* og = a.grad_gate.data && a.gate_per == 1
                    ? (B*)a.grad_gate.data + r * a.grad_gate.row
                    : nullptr;
        if (live) {
            float u[kEl], act[kEl], slope[kEl];
            if (has_y) {
                if (a.post != 0) {
#pragma unroll
                    for (int i = 0; i < kEl; ++i) {
                        y[i] = col<VEC, T>(t, i) < C ? (y[i] - st.x) * st.y : 0.0f;
                        u[i] = __builtin_fmaf(y[i], wp[i], bp[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kEl; ++i) u[i] = y[i];
                }
#pragma unroll
                for (int i = 0; i < kEl; ++i) {
                    act[i] = 1.0f, slope[i] = 1.0f;
                    if (gated && a.act == 0) act[i] = g[i];
                    if (gated && a.act != 0) {
                        const float s = sigmoid(g[i]);
                        act[i] = a.act == 1 ? s : g[i] * s;
                        slope[i] = s * (1.0f - s);
                        // silu: s (1 + g (1 - s))
                        if (a.act == 2) slope[i] = __builtin_fmaf(slope[i], g[i], s);
                    }
                    x[i] = __builtin_fmaf(u[i] * act[i], sc[i], x[i]);
                }
            }
            if (has_gh) {
                float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
                for (int i = 0; i < kEl; ++i) {
                    x[i] = col<VEC, T>(t, i) < C ? (x[i] - st.z) * st.w : 0.0f;
                    const float p = gh[i] * wh[i];
                    c1 = __builtin_fmaf(p, x[i], c1);
                    c2 += p;
                    acc[3][i] = __builtin_fmaf(gh[i], x[i], acc[3][i]);
                    acc[4][i] += gh[i];
                }
                sum(c1, c2);
                c1 *= inv_c;
                c2 = a.pre == 2 ? c2 * inv_c : 0.0f;
#pragma unroll
                for (int i = 0; i < kEl; ++i)
                    gx[i] = __builtin_fmaf(
                        st.w, __builtin_fmaf(-x[i], c1, gh[i] * wh[i] - c2), gx[i]);
            }
            if (ox) store<S, VEC, T>(ox, gx, C, t);
            if (has_y) {
                float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
                for (int i = 0; i < kEl; ++i) {
                    // (past the width gx is not 0)
                    const float d = col<VEC, T>(t, i) < C ? gx[i] : 0.0f;
                    acc[2][i] = __builtin_fmaf(d, act[i] * u[i], acc[2][i]);
                    const float gz = d * sc[i];
                    g[i] = gz * u[i] * slope[i];
                    gx[i] = gz * act[i];
                    acc[0][i] = __builtin_fmaf(gx[i], y[i], acc[0][i]);
                    acc[1][i] += gx[i];
                    if (a.post != 0) {
                        gx[i] *= wp[i];
                        c1 = __builtin_fmaf(gx[i], y[i], c1);
                        c2 += gx[i];
                    }
                }
                if (og) store<B, VEC, T>(og, g, C, t);
                if (gate_sums) {
#pragma unroll
                    for (int i = 0; i < kEl; ++i) gate_acc[i] += g[i];
                }
                if (a.post != 0) {
                    sum(c1, c2);
                    c1 *= inv_c;
                    c2 = a.post == 2 ? c2 * inv_c : 0.0f;
#pragma unroll
                    for (int i = 0; i < kEl; ++i)
                        gx[i] = st.y * __builtin_fmaf(-y[i], c1, gx[i] - c2);
                }
                if (oy) store<B, VEC, T>(oy, gx, C, t);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEl; ++i) gx[i] = 0.0f;
            if (ox) store<S, VEC, T>(ox, gx, C, t);
            if (oy) store<B, VEC, T>(oy, gx, C, t);
            if (og) store<B, VEC, T>(og, gx, C, t);
        }
        if (gate_sums && (!more || rows.b != b)) {
            // run + sequence is a number of its own: along the rows one of both grows
            store<float, VEC, T>(a.gate_part + (run + b) * C, gate_acc, C, t);
#pragma unroll
            for (int i = 0; i < kEl; ++i) gate_acc[i] = 0.0f;
        }
    }
    // the workgroup's part of every gradient that is asked for
    int given = 0;
#pragma unroll
    for (int k = 0; k < kResidualWeights; ++k) given += a.weight_grads[k] != nullptr;
    float* part = a.part + (int64_t)blockIdx.x * given * C;
#pragma unroll
    for (int k = 0; k < kResidualWeights; ++k) {
        if (a.weight_grads[k] == nullptr) continue;
        if constexpr (T == 64) {
            __syncthreads();
            if (group > 0) {
#pragma unroll
                for (int i = 0; i < kEl; ++i) cols[group - 1][i * 64 + t] = acc[k][i];
            }
            __syncthreads();
            if (group == 0) {
#pragma unroll
                for (int i = 0; i < kEl; ++i)
                    acc[k][i] = ((acc[k][i] + cols[0][i * 64 + t]) + cols[1][i * 64 + t]) +
                                cols[2][i * 64 + t];
            }
        }
        if (group == 0) store<float, VEC, T>(part, acc[k], C, t);
        part += C;
    }
}

// Adds the workgroups' parts of the weights' gradients in order: 32 columns of
// one weight per workgroup, 32 threads a column, in 64 bits (a sum over every
// row of the batch).
__global__ __launch_bounds__(1024) void residual_weights_kernel(ResidualArgs a, int blocks) {
    __shared__ double sums[32][33];
    const int lane = threadIdx.x & 31, turn = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    int given = 0, at = 0;
    float* out = nullptr;
#pragma unroll
    for (int k = 0; k < kResidualWeights; ++k)
        if (a.weight_grads[k] != nullptr) {
            if (given == (int)blockIdx.y) out = a.weight_grads[k], at = given;
            ++given;
        }
    const float* part = a.part + (int64_t)at * a.C + (c < a.C ? c : 0);
    double sum = 0.0;
#pragma unroll 8
    for (int i = turn; i < blocks; i += 32) sum += (double)part[(int64_t)i * given * a.C];
    sums[turn][lane] = sum;
    __syncthreads();
    if (turn != 0 || c >= a.C) return;
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) total += sums[i][lane];
    out[c] = (float)total;
}

// The gates' gradients of whole sequences: the runs' parts in order.
template <class B>
__global__ __launch_bounds__(256) void residual_gates_kernel(ResidualArgs a) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, turn = threadIdx.x >> 5;
    const int c = blockIdx.y * 32 + lane;
    for (int b = blockIdx.x; b < a.seqs.B; b += gridDim.x) {
        int64_t start;
        int len;
        seq_rows(a.seqs, b, start, len);
        float sum = 0.0f;
        if (len > 0) {
            const int64_t first = (start >> a.shift) + b;
            const int n = (int)(((start + len - 1) >> a.shift) + b - first) + 1;
            const float* part = a.gate_part + first * a.C + (c < a.C ? c : 0);
#pragma unroll 4
            for (int i = turn; i < n; i += 8) sum += part[(int64_t)i * a.C];
        }
        sums[turn][lane] = sum;
        __syncthreads();
        if (turn == 0 && c < a.C) {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) total += sums[i][lane];
            ((B*)a.grad_gate.data)[b * a.grad_gate.row + c] = (B)total;
        }
        __syncthreads();
    }
}

static int row_threads(int C) {
    int threads = 64;
    while (threads * kEl < C) threads *= 2;
    return threads;
}

int64_t residual_blocks(const ResidualArgs& a) {
    const int per = row_threads(a.C) == 64 ? 4 : 1;
    const int64_t runs = (a.seqs.rows + ((int64_t)1 << a.shift) - 1) >> a.shift;
    return (runs + per - 1) / per;
}

int residual_shift(const ResidualArgs& a, bool backward) {
    const int64_t runs = (backward ? 2048 : 4096) * 128 / row_threads(a.C);
    int shift = 0;
    while (shift < 20 && a.seqs.rows >> (shift + 1) >= runs) ++shift;
    return shift;
}

template <class S, class B, int VEC, int T>
static void launch(const ResidualArgs& a, bool backward, hipStream_t s) {
    const dim3 grid((unsigned)residual_blocks(a));
    if (backward)
        residual_grad_kernel<S, B, VEC, T><<<grid, kThreads<T>, 0, s>>>(a);
    else
        residual_kernel<S, B, VEC, T><<<grid, kThreads<T>, 0, s>>>(a);
}

template <class S, class B, int VEC>
static void by_width(const ResidualArgs& a, bool backward, hipStream_t s) {
    switch (row_threads(a.C)) {
        case 64: return launch<S, B, VEC, 64>(a, backward, s);
        case 128: return launch<S, B, VEC, 128>(a, backward, s);
        case 256: return launch<S, B, VEC, 256>(a, backward, s);
        case 512: return launch<S, B, VEC, 512>(a, backward, s);
        default: return launch<S, B, VEC, 1024>(a, backward, s);
    }
}

template <class S, class B>
static void by_alignment(const ResidualArgs& a, bool backward, hipStream_t s) {
    if (a.vec)
        by_width<S, B, 8>(a, backward, s);
    else
        by_width<S, B, 1>(a, backward, s);
}

static void by_type(const ResidualArgs& a, bool backward, hipStream_t s) {
    const bool wide = a.stream == 0;
    switch (a.branch) {
        case 0: return by_alignment<float, float>(a, backward, s);
        case 1:
            return wide ? by_alignment<float, _Float16>(a, backward, s)
                        : by_alignment<_Float16, _Float16>(a, backward, s);
        default:
            return wide ? by_alignment<float, __bf16>(a, backward, s)
                        : by_alignment<__bf16, __bf16>(a, backward, s);
    }
}

hipError_t launch_residual(const ResidualArgs& a, hipStream_t s) {
    by_type(a, false, s);
    return hipGetLastError();
}

hipError_t launch_residual_backward(const ResidualArgs& a, hipStream_t s) {
    const int64_t blocks = residual_blocks(a);
    if (blocks > 0) by_type(a, true, s);
    int given = 0;
    for (int k = 0; k < kResidualWeights; ++k) given += a.weight_grads[k] != nullptr;
    const unsigned columns = (unsigned)((a.C + 31) / 32);
    if (given > 0)
        residual_weights_kernel<<<dim3(columns, (unsigned)given), 1024, 0, s>>>(a, (int)blocks);
    if (a.gate_per == 2 && a.grad_gate.data && a.seqs.B > 0) {
        const dim3 grid(a.seqs.B < 16384 ? (unsigned)a.seqs.B : 16384u, columns);
        if (a.branch == 0)
            residual_gates_kernel<float><<<grid, 256, 0, s>>>(a);
        else if (a.branch == 1)
            residual_gates_kernel<_Float16><<<grid, 256, 0, s>>>(a);
        else
            residual_gates_kernel<__bf16><<<grid, 256, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace fpstok
