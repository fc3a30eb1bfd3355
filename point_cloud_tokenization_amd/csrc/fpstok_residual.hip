// The residual step between two blocks of an encoder and its gradients:
//   u = post_norm(y),  z = act(gate) u,  xo = x + scale z,  h = pre_norm(xo).
#include "fpstok_mma.h"
#include "fpstok_residual.h"
#include "fpstok_seqs.h"

namespace fpstok {

// A row of C elements belongs to T threads (64 to 1024, whole waves), EL adjacent
// elements to each, which come and go by 8- or 16-byte accesses (of any
// alignment).  Where EL does not divide C the last thread takes the row's last
// EL elements and leaves out the first of them, which are its neighbour's.
enum Fit {
    kNarrow,  // C < EL: elements one by one
    kTail,    // C > EL is no multiple of EL
    kWhole    // C is one
};

template <Fit FIT, int EL>
struct Cols {
    int C, base;  // this thread's first element
    int skip;     // of its EL elements, those that are not its own (EL: all)
    __device__ __forceinline__ Cols(int C, int t) : C(C) {
        base = t * EL < C ? t * EL : 0;
        skip = t * EL < C ? 0 : EL;
        if (FIT == kTail && skip == 0 && base + EL > C) {
            skip = base + EL - C;
            base = C - EL;
        }
    }
    __device__ __forceinline__ bool own(int e) const {
        return FIT == kNarrow ? skip == 0 && e < C : FIT == kTail ? e >= skip : skip == 0;
    }
    // What a thread adds to a sum over the row: threads past the width hold a
    // copy of the row's first elements.
    __device__ __forceinline__ float part(float x) const {
        return FIT != kWhole || skip == 0 ? x : 0.0f;
    }
    // An element that is not the thread's own counts as 0 in a sum over the row
    // where a thread may hold some of both.
    __device__ __forceinline__ float keep(float x, int e) const {
        return FIT == kWhole || own(e) ? x : 0.0f;
    }
};

// A thread's elements of a row as they came from memory.  Threads past the
// width load elements that exist (a load under a divergent branch would be
// waited for before the branch ends).
template <class E, Fit FIT, int EL>
struct Raw {
    using Vec = E __attribute__((ext_vector_type(EL)));
    using Loose = Vec __attribute__((aligned(sizeof(E))));  // of any alignment
    Vec v;
    __device__ __forceinline__ void load(const E* p, const Cols<FIT, EL>& c) {
        if constexpr (FIT != kNarrow) {
            v = *(const Loose*)(p + c.base);
        } else {
#pragma unroll
            for (int i = 0; i < EL; ++i) v[i] = p[i < c.C ? i : 0];
        }
    }
    __device__ __forceinline__ void get(float* f) const {
#pragma unroll
        for (int i = 0; i < EL; ++i) f[i] = (float)v[i];
    }
};

template <class E, Fit FIT, int EL>
__device__ __forceinline__ void store(E* p, const float* f, const Cols<FIT, EL>& c) {
    using R = Raw<E, FIT, EL>;
    typename R::Vec x;
#pragma unroll
    for (int i = 0; i < EL; ++i) x[i] = (E)f[i];
    if (FIT != kNarrow && c.skip == 0) {
        *(typename R::Loose*)(p + c.base) = x;
    } else if (FIT != kWhole && c.skip < EL) {
#pragma unroll
        for (int i = 0; i < EL; ++i)
            if (c.own(i)) p[c.base + i] = x[i];
    }
}

template <Fit FIT, int EL>
__device__ __forceinline__ void load_weight(float* f, const float* w, float none,
                                            const Cols<FIT, EL>& c) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < EL; ++i) f[i] = none;
        return;
    }
    Raw<float, FIT, EL> r;
    r.load(w, c);
    r.get(f);
}

// A workgroup's rows and threads: rows of one wave share a workgroup of four.
struct Threads {
    int T, t, group;
    int64_t run;
    __device__ __forceinline__ Threads(const ResidualArgs& a) {
        const int tid = threadIdx.x;
        T = a.threads;
        group = T == 64 ? __builtin_amdgcn_readfirstlane(tid >> 6) : 0;
        t = T == 64 ? tid & 63 : tid;
        run = T == 64 ? (int64_t)blockIdx.x * 4 + group : (int64_t)blockIdx.x;
    }
};

// A thread's weights of its own elements in LDS, [weight][4 elements][thread]: what
// is read again for every row need not stay in registers.
template <Fit FIT, int EL>
struct LdsWeights {
    using f4 = float __attribute__((ext_vector_type(4)));
    f4* at;
    int T;
    __device__ __forceinline__ LdsWeights(f4* lds, const Threads& th) : at(lds + th.t), T(th.T) {}
    __device__ __forceinline__ void put(int k, const float* w, float none,
                                        const Cols<FIT, EL>& c) {
        float f[EL];
        load_weight(f, w, none, c);
#pragma unroll
        for (int q = 0; q < EL / 4; ++q) {
            f4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f[q * 4 + i];
            at[(k * (EL / 4) + q) * T] = x;
        }
    }
    __device__ __forceinline__ void get(float* f, int k) const {
#pragma unroll
        for (int q = 0; q < EL / 4; ++q) {
            const f4 x = at[(k * (EL / 4) + q) * T];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[q * 4 + i] = x[i];
        }
    }
};

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
struct RowSum {
    float (*lds)[2][16];
    int waves, turn = 0;
    __device__ __forceinline__ RowSum(float (*lds)[2][16], int T) : lds(lds), waves(T >> 6) {}
    __device__ __forceinline__ void operator()(float& a, float& b) {
        a = wave_sum(a);
        b = wave_sum(b);
        if (waves > 1) {
            const int wave = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) lds[turn][0][wave] = a, lds[turn][1][wave] = b;
            __syncthreads();
            a = 0.0f, b = 0.0f;
            for (int w = 0; w < waves; ++w) a += lds[turn][0][w], b += lds[turn][1][w];
            turn ^= 1;
        }
    }
    __device__ __forceinline__ void operator()(float& a) {
        a = wave_sum(a);
        if (waves > 1) {
            const int wave = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) lds[turn][0][wave] = a;
            __syncthreads();
            a = 0.0f;
            for (int w = 0; w < waves; ++w) a += lds[turn][0][w];
            turn ^= 1;
        }
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

// How the rows are shared out: packed ones from the first sequence's first to
// the last one's last, padded ones all, in a.runs runs of as many adjacent rows.
struct Runs {
    int64_t first, last;
    int rows;  // of a run
    __device__ __forceinline__ Runs(const ResidualArgs& a) {
        first = a.seqs.cu ? cu_at(a.seqs, 0) : 0;
        last = a.seqs.cu ? cu_at(a.seqs, a.seqs.B) : a.seqs.rows;
        const uint32_t n = last > first ? (uint32_t)(last - first) : 0;
        rows = n > 0 ? (int)((n + (uint32_t)a.runs - 1) / (uint32_t)a.runs) : 1;
    }
};

// The rows of a run in order, and what is known of each: its sequence (packed:
// only if SEQ asks for it) and whether it is one of it.
struct RunRows {
    const SeqArgs& s;
    bool seq;
    int b = 0;
    int64_t lo, hi, end, live_end;  // rows of the run; where the sequence's slots and rows end
    __device__ __forceinline__ RunRows(const ResidualArgs& a, int64_t run)
        : s(a.seqs), seq(a.gate_per == 2) {
        const Runs runs(a);
        lo = runs.first + run * runs.rows;
        hi = lo + runs.rows < runs.last ? lo + runs.rows : runs.last;
        end = live_end = hi;
        if (run >= a.runs) lo = hi;
        if (lo >= hi) return;
        if (!s.cu) {
            at_slot((int)((uint32_t)lo / (uint32_t)s.cap));
        } else if (seq) {
            b = seq_of_row(s, lo);
            end = live_end = cu_at(s, b + 1);
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

// Off by |g| half steps of float32 from the product's rounding and a few from
// the instructions'.
__device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896f));
}

// Norms a row in place: (x - mean) / std with LAYER, x / rms without; `mean`
// and `r` = 1 / sqrt(mean square + eps) are returned.  The mean comes off
// before the squares are summed, in 32 bits.
template <Fit FIT, int EL>
__device__ __forceinline__ void norm_row(float* x, bool layer, float inv_c, float eps,
                                         const Cols<FIT, EL>& c, RowSum& sum, float& mean,
                                         float& r) {
    mean = 0.0f;
#pragma unroll
    for (int i = 0; i < EL; ++i) x[i] = c.keep(x[i], i);
    if (layer) {
#pragma unroll
        for (int i = 0; i < EL; ++i) mean += x[i];
        mean = c.part(mean);
        sum(mean);
        mean *= inv_c;
#pragma unroll
        for (int i = 0; i < EL; ++i) x[i] = c.keep(x[i] - mean, i);
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < EL; ++i) q = __builtin_fmaf(x[i], x[i], q);
    q = c.part(q);
    sum(q);
    r = __builtin_amdgcn_rsqf(__builtin_fmaf(q, inv_c, eps));
#pragma unroll
    for (int i = 0; i < EL; ++i) x[i] *= r;
}

// Forward.  The T threads of a row hold it in registers from the first load to
// the last store, so every operand is read and every result written once; a
// workgroup takes a run of adjacent rows, keeps the weights in registers and
// has the next row's loads on their way while it works on one.  Bound by HBM: 20,000
// rows of 5120 in bfloat16 are 206 us, 5.0 TB/s (a large copy: 5.2); one row of
// 768, 4.6 us, the launch.
// PLAIN: RMS norms without biases.
template <class S, class B, Fit FIT, int EL, int MAX_T, bool PLAIN>
__global__ __launch_bounds__(MAX_T) void residual_kernel(ResidualArgs a) {
    __shared__ float lds[2][2][16];
    const Threads th(a);
    const Cols<FIT, EL> c(a.C, th.t);
    RowSum sum(lds, th.T);
    RunRows rows(a, th.run);
    if (rows.lo >= rows.hi) return;  // (the same for all threads of a row)
    const float inv_c = 1.0f / (float)a.C;
    const bool has_y = a.y.data != nullptr, gated = a.gate_per != 0;
    float wp[EL], bp[EL], sc[EL], wh[EL], bh[EL];
    load_weight(wp, a.weights[0], 1.0f, c);
    if (!PLAIN) load_weight(bp, a.weights[1], 0.0f, c);
    load_weight(sc, a.weights[2], 1.0f, c);
    load_weight(wh, a.weights[3], 1.0f, c);
    if (!PLAIN) load_weight(bh, a.weights[4], 0.0f, c);
    Raw<S, FIT, EL> rx;
    Raw<B, FIT, EL> ry, rg;
    auto load = [&](int64_t r) {
        rx.load((const S*)a.x.data + r * a.x.row, c);
        if (has_y) ry.load((const B*)a.y.data + r * a.y.row, c);
        if (gated)
            rg.load((const B*)a.gate.data + (a.gate_per == 2 ? rows.b : r) * a.gate.row, c);
    };
    load(rows.lo);
    for (int64_t r = rows.lo; r < rows.hi; ++r) {
        const bool live = r < rows.live_end;
        float x[EL], y[EL], g[EL];
        rx.get(x);
        if (has_y) ry.get(y);
        if (gated) rg.get(g);
        if (r + 1 < rows.hi) {
            rows.to(r + 1);
            load(r + 1);
        }
        S* xo = a.x_out.data ? (S*)a.x_out.data + r * a.x_out.row : nullptr;
        B* h = a.h.data ? (B*)a.h.data + r * a.h.row : nullptr;
        float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!live) {
#pragma unroll
            for (int i = 0; i < EL; ++i) x[i] = 0.0f;
            if (xo) store(xo, x, c);
            if (h) store(h, x, c);
            if (a.stats && th.t == 0) ((float4*)a.stats)[r] = st;
            continue;
        }
        if (has_y) {
            if (a.post != 0) {
                norm_row(y, !PLAIN && a.post == 2, inv_c, a.eps, c, sum, st.x, st.y);
#pragma unroll
                for (int i = 0; i < EL; ++i)
                    y[i] = PLAIN ? y[i] * wp[i] : __builtin_fmaf(y[i], wp[i], bp[i]);
            }
            if (gated) {
                if (a.act != 0) {
#pragma unroll
                    for (int i = 0; i < EL; ++i) {
                        const float s = sigmoid(g[i]);
                        g[i] = a.act == 1 ? s : g[i] * s;
                    }
                }
#pragma unroll
                for (int i = 0; i < EL; ++i) y[i] *= g[i];
            }
#pragma unroll
            for (int i = 0; i < EL; ++i) x[i] = __builtin_fmaf(y[i], sc[i], x[i]);
        }
        if (xo) store(xo, x, c);
        if (a.pre != 0) {
            norm_row(x, !PLAIN && a.pre == 2, inv_c, a.eps, c, sum, st.z, st.w);
#pragma unroll
            for (int i = 0; i < EL; ++i)
                x[i] = PLAIN ? x[i] * wh[i] : __builtin_fmaf(x[i], wh[i], bh[i]);
            store(h, x, c);
        }
        if (a.stats && th.t == 0) ((float4*)a.stats)[r] = st;
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
// kernels below add in order: results are equal from run to run.  The weights lie in
// LDS and the branch is formed again after the sums, or too few rows would be on
// their way for HBM: 6000 rows of 5120, float32, RMS norms, 152 us instead of 225;
// 38,600 of 768 with a gate, 140 us.
// PLAIN: RMS norms without biases, which need neither means nor their sums.
template <class S, class B, Fit FIT, int EL, int MAX_T, bool PLAIN>
__global__ __launch_bounds__(MAX_T) void residual_grad_kernel(ResidualArgs a) {
    // rows of more than 4096 elements leave few registers: the next row is called
    // for when most of this one's are free again
    constexpr bool kLate = MAX_T > 512;
    __shared__ float lds[2][2][16];
    __shared__ float cols[3][64 * EL];
    const Threads th(a);
    const Cols<FIT, EL> c(a.C, th.t);
    RowSum sum(lds, th.T);
    RunRows rows(a, th.run);
    const float inv_c = 1.0f / (float)a.C;
    const bool has_y = a.y.data != nullptr, gated = a.gate_per != 0;
    const bool has_gx = a.grad_x_out.data != nullptr, has_gh = a.grad_h.data != nullptr;
    extern __shared__ __attribute__((aligned(16))) float fpstok_residual_lds[];
    enum { kPost, kScale, kPre, kPostBias };
    LdsWeights<FIT, EL> weights((typename LdsWeights<FIT, EL>::f4*)fpstok_residual_lds, th);
    if (th.group == 0) {
        weights.put(kPost, a.weights[0], 1.0f, c);
        weights.put(kScale, a.weights[2], 1.0f, c);
        weights.put(kPre, a.weights[3], 1.0f, c);
        if (!PLAIN) weights.put(kPostBias, a.weights[1], 0.0f, c);
    }
    __syncthreads();
    float acc[kResidualWeights][EL], gate_acc[EL];
#pragma unroll
    for (int i = 0; i < EL; ++i) {
#pragma unroll
        for (int k = 0; k < kResidualWeights; ++k) acc[k][i] = 0.0f;
        gate_acc[i] = 0.0f;
    }
    Raw<S, FIT, EL> rx, rgx;
    Raw<B, FIT, EL> ry, rg, rgh;
    float4 st_next = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto load = [&](int64_t r) {
        rx.load((const S*)a.x.data + r * a.x.row, c);
        if (has_y) ry.load((const B*)a.y.data + r * a.y.row, c);
        if (gated)
            rg.load((const B*)a.gate.data + (a.gate_per == 2 ? rows.b : r) * a.gate.row, c);
        if (has_gx) rgx.load((const S*)a.grad_x_out.data + r * a.grad_x_out.row, c);
        if (has_gh) rgh.load((const B*)a.grad_h.data + r * a.grad_h.row, c);
        if (a.stats) st_next = ((const float4*)a.stats)[r];
    };
    const bool gate_sums = a.gate_per == 2 && a.grad_gate.data != nullptr;
    if (rows.lo < rows.hi) load(rows.lo);
    for (int64_t r = rows.lo; r < rows.hi; ++r) {
        const bool live = r < rows.live_end;
        const int b = rows.b;
        const float4 st = st_next;
        float x[EL], y[EL], g[EL], gx[EL], gh[EL];
        rx.get(x);
        if (has_y) ry.get(y);
        if (gated) rg.get(g);
        if (has_gh) rgh.get(gh);
#pragma unroll
        for (int i = 0; i < EL; ++i) gx[i] = 0.0f;
        if (has_gx) rgx.get(gx);
        const bool more = r + 1 < rows.hi;
        bool called = false;
        auto call_next = [&]() {  // for the next row
            if (called || !more) return;
            called = true;
            rows.to(r + 1);
            load(r + 1);
        };
        if (!kLate) call_next();
        S* ox = a.grad_x.data ? (S*)a.grad_x.data + r * a.grad_x.row : nullptr;
        B* oy = a.grad_y.data ? (B*)a.grad_y.data + r * a.grad_y.row : nullptr;
        B* og = a.grad_gate.data && a.gate_per == 1
                    ? (B*)a.grad_gate.data + r * a.grad_gate.row
                    : nullptr;
        if (live) {
            // u = yh weight + bias, the gate and its derivative; formed twice, before and
            // after the sums, so that they need no registers in between
            auto branch = [&](float* u, float* act, float* slope) {
                asm volatile("" ::: "memory");
                if (a.post != 0) {
                    float wp[EL], bp[EL];
                    weights.get(wp, kPost);
                    if (!PLAIN) weights.get(bp, kPostBias);
#pragma unroll
                    for (int i = 0; i < EL; ++i)
                        u[i] = PLAIN ? y[i] * wp[i] : __builtin_fmaf(y[i], wp[i], bp[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < EL; ++i) u[i] = y[i];
                }
#pragma unroll
                for (int i = 0; i < EL; ++i) act[i] = 1.0f, slope[i] = 1.0f;
                if (!gated) return;
                if (a.act != 0) {
#pragma unroll
                    for (int i = 0; i < EL; ++i) {
                        const float s = sigmoid(g[i]);
                        act[i] = a.act == 1 ? s : g[i] * s;
                        slope[i] = s * (1.0f - s);
                        // silu: s (1 + g (1 - s))
                        if (a.act == 2) slope[i] = __builtin_fmaf(slope[i], g[i], s);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < EL; ++i) act[i] = g[i];
                }
            };
            if (has_y) {
                if (a.post != 0) {
#pragma unroll
                    for (int i = 0; i < EL; ++i) y[i] = PLAIN ? y[i] * st.y : (y[i] - st.x) * st.y;
                }
                float u[EL], act[EL], slope[EL], sc[EL];
                branch(u, act, slope);
                weights.get(sc, kScale);
#pragma unroll
                for (int i = 0; i < EL; ++i) x[i] = __builtin_fmaf(u[i] * act[i], sc[i], x[i]);
            }
            if (has_gh) {
                float c1 = 0.0f, c2 = 0.0f, wh[EL];
                weights.get(wh, kPre);
#pragma unroll
                for (int i = 0; i < EL; ++i) {
                    x[i] = PLAIN ? x[i] * st.w : (x[i] - st.z) * st.w;
                    gh[i] = c.keep(gh[i], i);
                    const float p = gh[i] * wh[i];
                    c1 = __builtin_fmaf(p, x[i], c1);
                    acc[3][i] = __builtin_fmaf(gh[i], x[i], acc[3][i]);
                    if (!PLAIN) {
                        c2 += p;
                        acc[4][i] += gh[i];
                    }
                }
                c1 = c.part(c1);
                if (PLAIN) {
                    sum(c1);
                } else {
                    c2 = c.part(c2);
                    sum(c1, c2);
                }
                c1 *= inv_c;
                c2 = a.pre == 2 ? c2 * inv_c : 0.0f;
#pragma unroll
                for (int i = 0; i < EL; ++i) {
                    const float p = gh[i] * wh[i];
                    gx[i] = __builtin_fmaf(st.w, __builtin_fmaf(-x[i], c1, PLAIN ? p : p - c2),
                                           gx[i]);
                }
            }
            if (ox) store(ox, gx, c);
            if (has_y) {
                float c1 = 0.0f, c2 = 0.0f, sc[EL], wp[EL], u[EL], act[EL], slope[EL];
                branch(u, act, slope);
                weights.get(sc, kScale);
                if (a.post != 0) weights.get(wp, kPost);
#pragma unroll
                for (int i = 0; i < EL; ++i) {
                    const float d = c.keep(gx[i], i);
                    acc[2][i] = __builtin_fmaf(d, act[i] * u[i], acc[2][i]);
                    const float gz = d * sc[i];
                    g[i] = gz * u[i] * slope[i];
                    gx[i] = gz * act[i];
                    acc[0][i] = __builtin_fmaf(gx[i], y[i], acc[0][i]);
                    if (!PLAIN) acc[1][i] += gx[i];
                    if (a.post != 0) {
                        gx[i] *= wp[i];
                        c1 = __builtin_fmaf(gx[i], y[i], c1);
                        if (!PLAIN) c2 += gx[i];
                    }
                }
                if (kLate) call_next();
                if (og) store(og, g, c);
                if (gate_sums) {
#pragma unroll
                    for (int i = 0; i < EL; ++i) gate_acc[i] += g[i];
                }
                if (a.post != 0) {
                    c1 = c.part(c1);
                    if (PLAIN) {
                        sum(c1);
                    } else {
                        c2 = c.part(c2);
                        sum(c1, c2);
                    }
                    c1 *= inv_c;
                    c2 = a.post == 2 ? c2 * inv_c : 0.0f;
#pragma unroll
                    for (int i = 0; i < EL; ++i)
                        gx[i] = st.y * __builtin_fmaf(-y[i], c1, PLAIN ? gx[i] : gx[i] - c2);
                }
                if (oy) store(oy, gx, c);
            }
        } else {
#pragma unroll
            for (int i = 0; i < EL; ++i) gx[i] = 0.0f;
            if (ox) store(ox, gx, c);
            if (oy) store(oy, gx, c);
            if (og) store(og, gx, c);
        }
        call_next();
        if (gate_sums && (!more || rows.b != b)) {
            // run + sequence is a number of its own: along the rows one of both grows
            store(a.gate_part + (th.run + b) * a.C, gate_acc, c);
#pragma unroll
            for (int i = 0; i < EL; ++i) gate_acc[i] = 0.0f;
        }
    }
    // the workgroup's part of every gradient that is asked for
    int given = 0;
#pragma unroll
    for (int k = 0; k < kResidualWeights; ++k) given += a.weight_grads[k] != nullptr;
    float* part = a.part + (int64_t)blockIdx.x * given * a.C;
#pragma unroll
    for (int k = 0; k < kResidualWeights; ++k) {
        if (a.weight_grads[k] == nullptr) continue;
        if (th.T == 64) {
            __syncthreads();
            if (th.group > 0) {
#pragma unroll
                for (int i = 0; i < EL; ++i) cols[th.group - 1][i * 64 + th.t] = acc[k][i];
            }
            __syncthreads();
            if (th.group == 0) {
#pragma unroll
                for (int i = 0; i < EL; ++i)
                    acc[k][i] = ((acc[k][i] + cols[0][i * 64 + th.t]) + cols[1][i * 64 + th.t]) +
                                cols[2][i * 64 + th.t];
            }
        }
        if (th.group == 0) store(part, acc[k], c);
        part += a.C;
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
    const Runs runs(a);
    for (int b = blockIdx.x; b < a.seqs.B; b += gridDim.x) {
        int64_t start;
        int len;
        seq_rows(a.seqs, b, start, len);
        const GateParts parts = gate_parts(start, len, runs.first, runs.last, runs.rows, b);
        const float* part = a.gate_part + parts.first * a.C + (c < a.C ? c : 0);
        float sum = 0.0f;
#pragma unroll 4
        for (int i = turn; i < parts.n; i += 8) sum += part[(int64_t)i * a.C];
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

// 4 elements a thread for gradients and a float32 stream, 8 else and for wide
// rows.  (float32 stream, 38,600 rows of 768: 4 elements 87 us forward and 140
// backward, 8 elements 102 and 197: half the registers, and 8 leave a quarter of the
// threads idle.  bfloat16, 34,000 of 512: 49 and 105 against 39 and 113; 11,700 of
// 2560 backward: 144 against 206, with a float32 stream and layer norms 229 against
// 189.)
static int residual_elements(const ResidualArgs& a, bool backward) {
    const int most = backward && a.stream != 0 ? 4096 : 2048;
    return a.C >= 4 && a.C <= most && (a.stream == 0 || backward) ? 4 : 8;
}

int64_t residual_blocks(const ResidualArgs& a) {
    const int per = a.threads == 64 ? 4 : 1;
    return (a.runs + per - 1) / per;
}

bool residual_plain(const ResidualArgs& a) {
    return a.post != 2 && a.pre != 2 && !a.weights[1] && !a.weights[4];
}

void plan_residual(ResidualArgs& a, bool backward) {
    a.elements = residual_elements(a, backward);
    a.threads = (a.C + 64 * a.elements - 1) / (64 * a.elements) * 64;
    // as many runs as the kernels' registers let run at once on 256 compute units
    const bool plain = residual_plain(a);
    int waves;
    if (!backward)
        waves = a.elements == 4 || plain ? 20 : 16;
    else if (a.elements == 4)
        waves = plain || a.stream != 0 ? 16 : 12;
    else
        waves = a.threads > 768 ? 16 : a.threads > 512 ? 12 : 8;
    const int per_unit = waves / (a.threads / 64);
    // (free slots leave some runs of padded rows little to do: shorter ones even that
    // out.  Backward a run leaves a part of the weights' gradients: 400 padded events, 512
    // wide, 102 us, with twice the runs 112)
    const int times = a.seqs.cu || backward ? 1 : 4;
    const int64_t runs = 256 * (int64_t)times * (per_unit < 1 ? 1 : per_unit);
    a.runs = (int32_t)(runs < a.seqs.rows ? runs : a.seqs.rows);
}

template <class S, class B, Fit FIT, int EL, int MAX_T>
static void launch(const ResidualArgs& a, bool backward, hipStream_t s) {
    const dim3 grid((unsigned)residual_blocks(a)), block(a.threads == 64 ? 256 : a.threads);
    const bool plain = residual_plain(a);
    if (!backward && plain)
        residual_kernel<S, B, FIT, EL, MAX_T, true><<<grid, block, 0, s>>>(a);
    else if (!backward)
        residual_kernel<S, B, FIT, EL, MAX_T, false><<<grid, block, 0, s>>>(a);
    else if (plain)
        residual_grad_kernel<S, B, FIT, EL, MAX_T, true>
            <<<grid, block, 3 * a.threads * EL * sizeof(float), s>>>(a);
    else
        residual_grad_kernel<S, B, FIT, EL, MAX_T, false>
            <<<grid, block, 4 * a.threads * EL * sizeof(float), s>>>(a);
}

template <class S, class B, Fit FIT>
static void by_width(const ResidualArgs& a, bool backward, hipStream_t s) {
    if (a.elements == 4 && a.threads <= 512)
        launch<S, B, FIT, 4, 512>(a, backward, s);
    else if (a.elements == 4)
        launch<S, B, FIT, 4, 1024>(a, backward, s);
    else if (a.threads <= 512)
        launch<S, B, FIT, 8, 512>(a, backward, s);
    else if (a.threads <= 768)
        launch<S, B, FIT, 8, 768>(a, backward, s);
    else
        launch<S, B, FIT, 8, 1024>(a, backward, s);
}

template <class S, class B>
static void by_fit(const ResidualArgs& a, bool backward, hipStream_t s) {
    if (a.C < a.elements)
        launch<S, B, kNarrow, 8, 512>(a, backward, s);
    else if (a.C % a.elements != 0)
        by_width<S, B, kTail>(a, backward, s);
    else
        by_width<S, B, kWhole>(a, backward, s);
}

static void by_type(const ResidualArgs& a, bool backward, hipStream_t s) {
    const bool wide = a.stream == 0;
    switch (a.branch) {
        case 0: return by_fit<float, float>(a, backward, s);
        case 1:
            return wide ? by_fit<float, _Float16>(a, backward, s)
                        : by_fit<_Float16, _Float16>(a, backward, s);
        default:
            return wide ? by_fit<float, __bf16>(a, backward, s)
                        : by_fit<__bf16, __bf16>(a, backward, s);
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
