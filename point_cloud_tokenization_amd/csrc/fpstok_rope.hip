// Rotary positions over several axes (fpstok_rope).
#include "fpstok_seqs.h"

namespace fpstok {

// sin and cos of an angle given in float64: k = the nearest multiple of
// pi/2, r = angle - k pi/2 by two fused multiply-adds (pi/2 split into its
// float64 rounding and the rest, so r is good to about 1e-16 + k 1e-33), then
// the Taylor polynomials on |r| <= pi/4, cut where the next term is below
// 2e-9 (sin) and 2e-10 (cos): below half a float32 step.
__device__ __forceinline__ void sincos_angle(double angle, float& sn, float& cs) {
    const double k = __builtin_rint(angle * 0.63661977236758134308);  // 2 / pi
    double r = __builtin_fma(-k, 1.57079632679489655800, angle);
    r = __builtin_fma(-k, 6.12323399573676603587e-17, r);
    const float x = (float)r;
    const float z = x * x;
    float s = __builtin_fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
    s = __builtin_fmaf(z, s, 8.33333333e-3f);
    s = __builtin_fmaf(z, s, -1.66666667e-1f);
    s = __builtin_fmaf(x * z, s, x);
    float c = __builtin_fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
    c = __builtin_fmaf(z, c, -1.38888889e-3f);
    c = __builtin_fmaf(z, c, 4.16666667e-2f);
    c = __builtin_fmaf(z, c, -0.5f);
    c = __builtin_fmaf(z, c, 1.0f);
    // quadrant: k mod 4, formed in float64 (k may pass 32 bits)
    const int quad = (int)(k - 4.0 * __builtin_floor(k * 0.25));
    const float a = (quad & 1) ? c : s;
    const float b = (quad & 1) ? s : c;
    sn = (quad & 2) ? -a : a;
    cs = ((quad + 1) & 2) ? -b : b;
}

// Angle of pair p on a row, as the kernel's sine and cosine.
__device__ __forceinline__ void row_sincos(const RopeArgs& a, int64_t row, int p, float& sn,
                                           float& cs) {
    int ax = 0;
    while (p >= a.first_pair[ax + 1]) ++ax;
    const int64_t at = row * a.axes + ax;
    const double pos = a.int_positions ? (double)((const int32_t*)a.positions)[at]
                                       : (double)((const float*)a.positions)[at];
    sincos_angle(pos * (double)a.freqs[p], sn, cs);
    if (a.inverse) sn = -sn;
}

// The rows ahead of the first packed sequence, and those up to the last one's
// end.
__device__ __forceinline__ int64_t rows_begin(const SeqArgs& s) { return s.cu ? cu_at(s, 0) : 0; }
__device__ __forceinline__ int64_t rows_end(const SeqArgs& s) {
    return s.cu ? cu_at(s, s.B) : s.rows;
}

// True if `row` is one of a sequence's; `skip`: it is not to be written.
__device__ __forceinline__ bool row_here(const SeqArgs& s, int64_t row, int64_t begin, int64_t end,
                                         bool& skip) {
    skip = row < begin || row >= end;
    return !skip && (s.cu || row % s.cap < s.count[row / s.cap]);
}

// Any alignment: a thread per (row, element pair), head after head.
template <class T>
__global__ __launch_bounds__(256) void rope_pair_kernel(RopeArgs a) {
    const int half = a.D / 2;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = t / half;
    const int p = (int)(t % half);
    bool skip;
    const bool here = row_here(a.seqs, row, rows_begin(a.seqs), rows_end(a.seqs), skip);
    if (skip) return;
    float sn = 0.0f, cs = 1.0f;
    const bool turn = p < a.R;
    if (turn && here) row_sincos(a, row, p, sn, cs);
    const int e1 = turn && !a.interleaved ? p : 2 * p;
    const int e2 = turn && !a.interleaved ? p + a.R : 2 * p + 1;
    for (int which = 0; which < 2; ++which) {
        const T* in = (const T*)a.in[which].data + row * a.in[which].row;
        T* out = (T*)a.out[which].data + row * a.out[which].row;
        for (int h = 0; h < a.heads[which]; ++h) {
            float y1 = 0.0f, y2 = 0.0f;
            if (here) {
                const float x1 = (float)in[e1], x2 = (float)in[e2];
                y1 = turn ? x1 * cs - x2 * sn : x1;
                y2 = turn ? x1 * sn + x2 * cs : x2;
            }
            out[e1] = (T)y1;
            out[e2] = (T)y2;
            in += a.in[which].head;
            out += a.out[which].head;
        }
    }
}

// Rows of heads aligned to 16 bytes.  A workgroup takes a.block_rows rows: their
// sines and cosines are formed once, in LDS, for all heads of q and k; then a
// thread turns 16 bytes (interleaved) or 16 bytes and their partners R
// elements further (half), kItems of them on their way at a time, adjacent
// threads adjacent in memory.  Rows of no sequence are not read: their items
// load a row of the workgroup that is one's (a load under a divergent branch
// would be waited for before the branch ends) and drop it, and their sines are not
// formed (1024 events of 4 rows in 128 slots: 74 us, 117 with them).  Bound by
// the bytes: 150,000 rows of 16 + 4 heads of 128 bfloat16 in 0.31 ms, 5.0 TB/s
// (a large copy's rate); 5,541 rows of 12 + 4 heads of 64 in 8 us, of which a
// launch is half; one event's 128 rows in 4.7 us, a launch.  One element pair per
// thread, above, took 362, 11 and 8.5 us.
template <class T, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
    constexpr int V = 16 / (int)sizeof(T), kItems = 4;
    using Vec = T __attribute__((ext_vector_type(V)));
    extern __shared__ float2 table[];  // [row][pair] cosine, sine
    const int R = a.R, tid = threadIdx.x;
    const int64_t begin = rows_begin(a.seqs), end = rows_end(a.seqs);
    const int64_t row0 = (int64_t)blockIdx.x * a.block_rows;
    const int rows = end - row0 < a.block_rows ? (int)(end - row0) : a.block_rows;
    if (rows <= 0) return;
    // a bit for each of the rows (at most 16) that is a sequence's
    uint32_t here = (1u << rows) - 1;
    if (a.seqs.cu) {
        if (begin - row0 >= rows) return;
        if (begin > row0) here &= ~0u << (begin - row0);
    } else {
        bool skip;
        const int r = tid & 63;
        here = (uint32_t)__ballot(
            r < rows && row_here(a.seqs, row0 + (r < rows ? r : 0), begin, end, skip));
    }
    const int some = __builtin_ctz(here | 1u << 31);
    const int turned = INTER ? 2 * R / V : R / V;  // turned items of a head
    const int per_head = turned + (a.D - 2 * R) / V, heads = a.heads[0] + a.heads[1];
    const int per_row = per_head * heads, total = per_row * rows;
    Vec x[kItems], y[kItems];
    T* to[kItems];
    int row[kItems], item[kItems];
    auto fetch = [&](int base) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (base - tid + i * 256 >= total) break;  // none of the workgroup's
            const uint32_t n = base + i * 256 < total ? base + i * 256 : total - 1;
            const uint32_t r = n / (uint32_t)per_row, m = n - r * per_row;
            const uint32_t h = m / (uint32_t)per_head, u = m - h * per_head;
            const bool k = (int)h >= a.heads[0];
            const HeadsArg& in = a.in[k];
            const HeadsArg& out = a.out[k];
            const int64_t hh = (int)h - (k ? a.heads[0] : 0);
            // first element: of the turned part, or of the rest of the head
            const int e = (int)u < turned ? (int)u * V : 2 * R + ((int)u - turned) * V;
            const int64_t read = row0 + (here >> r & 1 ? (int)r : some);
            const T* from = (const T*)in.data + read * in.row + hh * in.head + e;
            to[i] = (T*)out.data + (row0 + r) * out.row + hh * out.head + e;
            row[i] = (int)r;
            item[i] = (int)u;
            x[i] = y[i] = Vec{};
            if (here == 0) continue;
            x[i] = *(const Vec*)from;
            // (the rest of a head has no partner: its own element again)
            if constexpr (!INTER) y[i] = *(const Vec*)((int)u < turned ? from + R : from);
        }
    };
    fetch(tid);
    for (int n = tid; n < rows * R; n += 256) {
        const int r = n / R;
        float sn, cs;
        if (!(here >> r & 1)) continue;
        row_sincos(a, row0 + r, n - r * R, sn, cs);
        table[n] = make_float2(cs, sn);
    }
    __syncthreads();
    for (int base = tid; base - tid < total; base += 256 * kItems) {
        if (base != tid) fetch(base);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (base + i * 256 >= total) break;
            const bool live = here >> row[i] & 1;
            if (!live && a.seqs.cu) continue;
            const bool turn = item[i] < turned;
            if constexpr (INTER) {
                if (turn) {
                    const float2* cs = table + row[i] * R + item[i] * (V / 2);
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float2 c = cs[e / 2];
                        const float x1 = (float)x[i][e], x2 = (float)x[i][e + 1];
                        x[i][e] = (T)(x1 * c.x - x2 * c.y);
                        x[i][e + 1] = (T)(x1 * c.y + x2 * c.x);
                    }
                }
            } else {
                if (turn) {
                    const float2* cs = table + row[i] * R + item[i] * V;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float2 c = cs[e];
                        const float x1 = (float)x[i][e], x2 = (float)y[i][e];
                        x[i][e] = (T)(x1 * c.x - x2 * c.y);
                        y[i][e] = (T)(x1 * c.y + x2 * c.x);
                    }
                    *(Vec*)(to[i] + R) = live ? y[i] : Vec{};
                }
            }
            *(Vec*)to[i] = live ? x[i] : Vec{};
        }
    }
}

// 16-byte items need every head of every view, and the turned part of a head,
// to start and end on 16 bytes.
static bool by_16_bytes(const RopeArgs& a) {
    const int w = a.dtype == 0 ? 4 : 2, V = 16 / w;
    if ((a.interleaved ? 2 * a.R : a.R) % V != 0 || a.D % V != 0) return false;
    for (int i = 0; i < 2; ++i) {
        if (a.heads[i] == 0) continue;
        for (const HeadsArg* v : {&a.in[i], &a.out[i]})
            if ((uintptr_t)v->data % 16 != 0 || v->row * w % 16 != 0 || v->head * w % 16 != 0)
                return false;
    }
    return true;
}

template <class T>
static hipError_t rope(RopeArgs a, hipStream_t s) {
    if (!by_16_bytes(a)) {
        const int64_t threads = a.seqs.rows * (a.D / 2);
        rope_pair_kernel<T><<<dim3((unsigned)((threads + 255) / 256)), 256, 0, s>>>(a);
        return hipGetLastError();
    }
    // as many rows per workgroup as leave 1024 workgroups (on 5,541 rows: 256
    // workgroups 11.9 us, 512 10.7, 1024 9.8, 2048 9.8 to 10.7), at most 16,
    // and a table of at most 32 KB
    int64_t rows = a.seqs.rows / 1024;
    if (rows > 16) rows = 16;
    if (rows > 4096 / a.R) rows = 4096 / a.R;
    a.block_rows = rows < 1 ? 1 : (int32_t)rows;
    const dim3 grid((unsigned)((a.seqs.rows + a.block_rows - 1) / a.block_rows));
    const size_t lds = (size_t)a.block_rows * a.R * sizeof(float2);
    if (a.interleaved)
        rope_kernel<T, true><<<grid, 256, lds, s>>>(a);
    else
        rope_kernel<T, false><<<grid, 256, lds, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
    return a.dtype == 0   ? rope<float>(a, s)
           : a.dtype == 1 ? rope<_Float16>(a, s)
                          : rope<__bf16>(a, s);
}

}  // namespace fpstok
