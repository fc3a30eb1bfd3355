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

template <class T>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
    const int half = a.D / 2;
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = t / half;
    const int p = (int)(t % half);
    if (row >= a.seqs.rows) return;
    bool pad = false;
    if (a.seqs.cu) {
        if (row >= cu_at(a.seqs, a.seqs.B)) return;
    } else {
        pad = row % a.seqs.cap >= a.seqs.count[row / a.seqs.cap];
    }
    float sn = 0.0f, cs = 1.0f;
    const bool turn = p < a.R;
    if (turn && !pad) {
        int ax = 0;
        while (p >= a.first_pair[ax + 1]) ++ax;
        const int64_t at = row * a.axes + ax;
        const double pos = a.int_positions ? (double)((const int32_t*)a.positions)[at]
                                           : (double)((const float*)a.positions)[at];
        sincos_angle(pos * (double)a.freqs[p], sn, cs);
        if (a.inverse) sn = -sn;
    }
    const int e1 = turn && !a.interleaved ? p : 2 * p;
    const int e2 = turn && !a.interleaved ? p + a.R : 2 * p + 1;
    for (int which = 0; which < 2; ++which) {
        const T* in = (const T*)a.in[which].data + row * a.in[which].row;
        T* out = (T*)a.out[which].data + row * a.out[which].row;
        for (int h = 0; h < a.heads[which]; ++h) {
            float y1 = 0.0f, y2 = 0.0f;
            if (!pad) {
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

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
    const int64_t threads = a.seqs.rows * (a.D / 2);
    const dim3 grid((unsigned)((threads + 255) / 256));
    if (a.dtype == 0)
        rope_kernel<float><<<grid, 256, 0, s>>>(a);
    else if (a.dtype == 1)
        rope_kernel<_Float16><<<grid, 256, 0, s>>>(a);
    else
        rope_kernel<__bf16><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fpstok
