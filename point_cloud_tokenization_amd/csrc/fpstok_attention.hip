// Attention over the rows of variable-length sequences and its gradients.
#include "fpstok_seqs.h"

namespace fpstok {

// Keys a query at place p sees: [0, ns) and [lo, hi].
__device__ __forceinline__ void key_range(const AttnArgs& a, int64_t p, int tk, int& ns, int& lo,
                                          int& hi) {
    int64_t h = tk - 1, l = 0;
    if (a.right >= 0 && p + a.right < h) h = p + a.right;
    if (a.left >= 0 && p - a.left > 0) l = p - a.left;
    int64_t n = l < a.sinks ? l : a.sinks;
    if (n > h + 1) n = h + 1;
    if (n < 0) n = 0;
    if (l > h) { l = 1; h = 0; }
    ns = (int)n;
    lo = (int)l;
    hi = (int)h;
}

// Sequence and place in it of buffer row r; false if no sequence holds it.
__device__ __forceinline__ bool row_seq(const SeqArgs& s, int64_t r, int& b, int64_t& start,
                                        int& len) {
    b = s.cu ? 0 : (int)(r / s.cap);
    if (s.cu) {
        int lo = 0, n = s.B;  // largest b with cu[b] <= r
        while (n > 1) {
            const int m = n >> 1;
            if (cu_at(s, lo + m) <= r) { lo += m; n -= m; } else n = m;
        }
        b = lo;
    }
    seq_rows(s, b, start, len);
    return r >= start && r < start + len;
}

template <class T>
__device__ __forceinline__ float dot(const T* x, const T* y, int D) {
    float s = 0.0f;
    for (int d = 0; d < D; ++d) s = __builtin_fmaf((float)x[d], (float)y[d], s);
    return s;
}

__device__ __forceinline__ float wave_max(float x) {
    for (int o = 32; o; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}

__device__ __forceinline__ float wave_sum(float x) {
    for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
    return x;
}

// One wave per (query, head): lanes over keys for the scores and the
// softmax, over the head's elements for the weighted sum of v.
template <class T>
__global__ __launch_bounds__(256) void attention_kernel(AttnArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t r = w / a.H;
    const int h = (int)(w % a.H), hk = h / (a.H / a.Hk);
    if (r >= a.qs.rows) return;
    int b, tq, tk;
    int64_t q0, k0;
    const bool in = row_seq(a.qs, r, b, q0, tq);
    if (!in && a.qs.cu) return;
    float acc[2] = {0.0f, 0.0f}, m = -INFINITY, l = 0.0f;
    const T* q = (const T*)a.q.data + r * a.q.row + h * a.q.head;
    const T* kb = (const T*)a.k.data + hk * a.k.head;
    const T* vb = (const T*)a.v.data + hk * a.v.head;
    int ns = 0, lo = 1, hi = 0;
    if (in) {
        seq_rows(a.ks, b, k0, tk);
        key_range(a, (r - q0) + tk - tq, tk, ns, lo, hi);
    }
    const int n = ns + hi - lo + 1;
    for (int c = 0; c < n; c += 64) {
        const int t = c + lane;
        const int64_t j = k0 + (t < ns ? t : lo + t - ns);
        const float s = t < n ? dot(q, kb + j * a.k.row, a.D) * a.scale : -INFINITY;
        const float m2 = fmaxf(m, wave_max(s));
        const float f = expf(m - m2);
        const float p = t < n ? expf(s - m2) : 0.0f;
        l = l * f + wave_sum(p);
        m = m2;
        acc[0] *= f;
        acc[1] *= f;
        for (int u = 0; u < 64 && c + u < n; ++u) {
            const float pu = __shfl(p, u);
            const T* v = vb + (k0 + (c + u < ns ? c + u : lo + c + u - ns)) * a.v.row;
            for (int e = 0; e < 2; ++e)
                if (lane + 64 * e < a.D) acc[e] = __builtin_fmaf(pu, (float)v[lane + 64 * e], acc[e]);
        }
    }
    T* out = (T*)a.out.data + r * a.out.row + h * a.out.head;
    for (int e = 0; e < 2; ++e)
        if (lane + 64 * e < a.D) out[lane + 64 * e] = (T)(n > 0 ? acc[e] / l : 0.0f);
    if (a.lse && lane == 0) a.lse[r * a.H + h] = !in ? 0.0f : n > 0 ? m + logf(l) : -INFINITY;
}

// One wave per (query, head): grad_q, and delta for the kernel below.
template <class T>
__global__ __launch_bounds__(256) void attention_dq_kernel(AttnArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t r = w / a.H;
    const int h = (int)(w % a.H), hk = h / (a.H / a.Hk);
    if (r >= a.qs.rows) return;
    int b, tq, tk;
    int64_t q0, k0;
    const bool in = row_seq(a.qs, r, b, q0, tq);
    if (!in && a.qs.cu) return;
    float acc[2] = {0.0f, 0.0f}, delta = 0.0f, lse = 0.0f;
    const T* q = (const T*)a.q.data + r * a.q.row + h * a.q.head;
    const T* g = (const T*)a.grad_out.data + r * a.grad_out.row + h * a.grad_out.head;
    const T* o = (const T*)a.out.data + r * a.out.row + h * a.out.head;
    const T* kb = (const T*)a.k.data + hk * a.k.head;
    const T* vb = (const T*)a.v.data + hk * a.v.head;
    int ns = 0, lo = 1, hi = 0;
    if (in) {
        seq_rows(a.ks, b, k0, tk);
        key_range(a, (r - q0) + tk - tq, tk, ns, lo, hi);
        delta = dot(g, o, a.D);
        lse = a.lse[r * a.H + h];
    }
    if (in && lane == 0) a.delta[r * a.H + h] = delta;
    const int n = ns + hi - lo + 1;
    for (int c = 0; c < n; c += 64) {
        const int t = c + lane;
        const int64_t j = k0 + (t < ns ? t : lo + t - ns);
        float ds = 0.0f;
        if (t < n) {
            const float p = expf(dot(q, kb + j * a.k.row, a.D) * a.scale - lse);
            ds = p * (dot(g, vb + j * a.v.row, a.D) - delta);
        }
        for (int u = 0; u < 64 && c + u < n; ++u) {
            const float x = __shfl(ds, u);
            const T* k = kb + (k0 + (c + u < ns ? c + u : lo + c + u - ns)) * a.k.row;
            for (int e = 0; e < 2; ++e)
                if (lane + 64 * e < a.D) acc[e] = __builtin_fmaf(x, (float)k[lane + 64 * e], acc[e]);
        }
    }
    T* out = (T*)a.grad_q.data + r * a.grad_q.row + h * a.grad_q.head;
    for (int e = 0; e < 2; ++e)
        if (lane + 64 * e < a.D) out[lane + 64 * e] = (T)(acc[e] * a.scale);
}

// One wave per (key, key head): grad_k and grad_v over every query that sees
// the key, heads of the group one after another.
template <class T>
__global__ __launch_bounds__(256) void attention_dkv_kernel(AttnArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t r = w / a.Hk;
    const int hk = (int)(w % a.Hk), G = a.H / a.Hk;
    if (r >= a.ks.rows) return;
    int b, tq = 0, tk;
    int64_t q0 = 0, k0;
    const bool in = row_seq(a.ks, r, b, k0, tk);
    if (!in && a.ks.cu) return;
    float dk[2] = {0.0f, 0.0f}, dv[2] = {0.0f, 0.0f};
    const T* k = (const T*)a.k.data + r * a.k.row + hk * a.k.head;
    const T* v = (const T*)a.v.data + r * a.v.row + hk * a.v.head;
    int64_t i0 = 0, i1 = -1;
    if (in) {
        seq_rows(a.qs, b, q0, tq);
        const int64_t j = r - k0, off = (int64_t)tk - tq;
        i1 = tq - 1;
        if (a.right >= 0 && j - a.right - off > 0) i0 = j - a.right - off;
        if (a.left >= 0 && j >= a.sinks && j + a.left - off < i1) i1 = j + a.left - off;
    }
    for (int h = hk * G; h < (hk + 1) * G; ++h)
        for (int64_t c = i0; c <= i1; c += 64) {
            const int64_t i = q0 + c + lane;
            const T* q = (const T*)a.q.data + h * a.q.head;
            const T* g = (const T*)a.grad_out.data + h * a.grad_out.head;
            float p = 0.0f, ds = 0.0f;
            if (c + lane <= i1) {
                p = expf(dot(q + i * a.q.row, k, a.D) * a.scale - a.lse[i * a.H + h]);
                ds = p * (dot(g + i * a.grad_out.row, v, a.D) - a.delta[i * a.H + h]);
            }
            for (int u = 0; u < 64 && c + u <= i1; ++u) {
                const float pu = __shfl(p, u), du = __shfl(ds, u);
                const T* qu = q + (q0 + c + u) * a.q.row;
                const T* gu = g + (q0 + c + u) * a.grad_out.row;
                for (int e = 0; e < 2; ++e)
                    if (lane + 64 * e < a.D) {
                        dv[e] = __builtin_fmaf(pu, (float)gu[lane + 64 * e], dv[e]);
                        dk[e] = __builtin_fmaf(du, (float)qu[lane + 64 * e], dk[e]);
                    }
            }
        }
    T* ok = (T*)a.grad_k.data + r * a.grad_k.row + hk * a.grad_k.head;
    T* ov = (T*)a.grad_v.data + r * a.grad_v.row + hk * a.grad_v.head;
    for (int e = 0; e < 2; ++e)
        if (lane + 64 * e < a.D) {
            ok[lane + 64 * e] = (T)(dk[e] * a.scale);
            ov[lane + 64 * e] = (T)dv[e];
        }
}

template <class T>
static hipError_t forward(const AttnArgs& a, hipStream_t s) {
    attention_kernel<T><<<dim3((unsigned)((a.qs.rows * a.H + 3) / 4)), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <class T>
static hipError_t backward(const AttnArgs& a, hipStream_t s) {
    if (a.qs.rows > 0)
        attention_dq_kernel<T><<<dim3((unsigned)((a.qs.rows * a.H + 3) / 4)), 256, 0, s>>>(a);
    if (a.ks.rows > 0)
        attention_dkv_kernel<T><<<dim3((unsigned)((a.ks.rows * a.Hk + 3) / 4)), 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_attention(const AttnArgs& a, hipStream_t s) {
    return a.dtype == 0 ? forward<float>(a, s)
                        : a.dtype == 1 ? forward<_Float16>(a, s) : forward<__bf16>(a, s);
}

hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s) {
    return a.dtype == 0 ? backward<float>(a, s)
                        : a.dtype == 1 ? backward<_Float16>(a, s) : backward<__bf16>(a, s);
}

}  // namespace fpstok
