// Attention over the rows of variable-length sequences and its gradients.
#include "fpstok_mma.h"
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

// The rows of one workgroup's tile.  A row is a (query, head of the group) pair
// of one key head, numbered query * G + head: every row of a tile reads the
// same keys, so one query of 8 heads is 8 rows of a tile, and K and V are read
// once for the group.
struct RowTile {
    int64_t q0, k0;  // first buffer rows of the sequence
    int tq, tk, row0, rows;  // rows: those of the tile that exist
    int pad;                 // rows of the tile inside a padded sequence's slots
    int hk;
};

// Decodes a workgroup's place in the grid: heads fastest, so that with 8 key
// heads (or a multiple) a head's tiles stay on one of the 8 XCDs and share its
// L2.  Later tiles first where the mask is causal: they see more keys.
template <int BM>
__device__ __forceinline__ bool row_tile(const AttnArgs& a, const SeqArgs& s, int64_t block, int G,
                                         RowTile& t) {
    t.hk = (int)(block % a.Hk);
    const int64_t slot = block / a.Hk;
    int b;
    int64_t tile;
    if (s.cu) {
        b = find_seq(s, slot, G, BM);
        tile = slot - first_slot(s, b, G, BM);
        if (tile < 0) return false;
    } else {
        const int per = (int)(((int64_t)s.cap * G + BM - 1) / BM);
        b = (int)(slot / per);
        tile = slot % per;
    }
    seq_rows(a.qs, b, t.q0, t.tq);
    seq_rows(a.ks, b, t.k0, t.tk);
    const int len = &s == &a.qs ? t.tq : t.tk;
    const int64_t left = (int64_t)len * G - tile * BM;
    if (s.cu && left <= 0) return false;
    const int64_t pad = s.cu ? 0 : (int64_t)s.cap * G - tile * BM;
    t.row0 = (int)(tile * BM);
    t.rows = left < 0 ? 0 : left < BM ? (int)left : BM;
    t.pad = pad < BM ? (int)pad : BM;
    return true;
}

// Keys that some row with a place in [pa, pb] sees, in tiles of BN: `sink`
// tiles from key 0 on, then tiles first .. first + count - sink - 1.
template <int BN>
struct KeyTiles {
    int sink, first, count;
    __device__ __forceinline__ KeyTiles(const AttnArgs& a, int64_t pa, int64_t pb, int tk) {
        int64_t hi = tk - 1, lo = 0;
        if (a.right >= 0 && pb + a.right < hi) hi = pb + a.right;
        if (a.left >= 0 && pa - a.left > 0) lo = pa - a.left;
        first = (int)(lo / BN);
        sink = 0;
        count = 0;
        if (hi >= 0) {
            const int last = (int)(hi / BN);
            const int64_t n = a.sinks < hi + 1 ? a.sinks : hi + 1;
            sink = (int)((n + BN - 1) / BN);
            if (sink > first) sink = first;
            count = sink + (last >= first ? last - first + 1 : 0);
        }
    }
    __device__ __forceinline__ int tile(int i) const { return i < sink ? i : first + i - sink; }
};

// How the keys j0 .. j0 + BN - 1 look to rows with places in [pa, pb]: 0 no
// row sees any, 1 some rows hide some, 2 every row sees all.
template <int BN>
__device__ __forceinline__ int tile_view(const AttnArgs& a, int64_t pa, int64_t pb, int tk,
                                         int j0) {
    const int64_t j1 = (int64_t)j0 + BN - 1;
    const bool left_all = a.left < 0 || j0 >= pb - a.left || j1 < a.sinks;
    const bool left_none = a.left >= 0 && j1 < pa - a.left && j0 >= a.sinks;
    const bool right_all = j1 < tk && (a.right < 0 || j1 <= pa + a.right);
    const bool right_none = j0 >= tk || (a.right >= 0 && j0 > pb + a.right);
    return left_none || right_none ? 0 : left_all && right_all ? 2 : 1;
}

// Forward.  A workgroup of 4 waves takes 128 rows (32 per wave) of one key
// head and walks the tiles of BN keys they see.  Per tile a wave forms
// S^T = K Q^T (keys in registers, its 32 rows across the lanes), so a row's
// maximum and sum are a lane's own registers plus one exchange with lane ^ 32,
// its factor is one value per lane, and the weights, rounded to the type, are
// already the operand of O^T += V^T P^T.  The maximum a row subtracts is moved
// only when it grew by more than 2^8 (a rescale of O costs as many
// multiplications as it has registers; weights stay below 2^8).
template <class T, int DP, int BN>
__global__ __launch_bounds__(256) void attention_kernel(AttnArgs a) {
    constexpr int BM = 128, DB = DP / 32, KB = BN / 32, STEPS = DP / 16;
    using Tl = Tile<T, DP>;
    using Frag = typename Elem<T>::Frag;
    __shared__ __attribute__((aligned(16))) char smem[2 * 2 * BN * Tl::kPitch];
    __shared__ int bad_tag[2];
    FPSTOK_LDS char* lds = (FPSTOK_LDS char*)smem;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.H / a.Hk;
    RowTile t;
    if (!row_tile<BM>(a, a.qs, blockIdx.x, G, t)) return;

    // this lane's row
    const int r = wave * 32 + (lane & 31);
    const int qi = (t.row0 + r) / G, h = t.hk * G + (t.row0 + r) - qi * G;
    const bool live = r < t.rows;
    const int64_t qrow = t.q0 + qi;
    Frag qf[STEPS];
    {
        const T* q = (const T*)a.q.data + qrow * a.q.row + h * a.q.head;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int d = s * 16 + half * 8;
            Frag f = {};
            if (live && d < a.D) f = *(const Frag*)(q + d);
            qf[s] = f;
        }
    }
    // places of the workgroup's, the wave's and the lane's rows
    const int64_t off = (int64_t)t.tk - t.tq;
    const int last = t.rows > 0 ? t.rows - 1 : 0;
    const int64_t pa = t.row0 / G + off, pb = (t.row0 + last) / G + off;
    const int wl = wave * 32 + 31 < last ? wave * 32 + 31 : last;
    const int64_t wa = (t.row0 + wave * 32) / G + off, wb = (t.row0 + wl) / G + off;
    const bool wave_live = wave * 32 < t.rows;
    const int64_t p = qi + off;
    const int hi = (int)(a.right >= 0 && p + a.right < t.tk - 1 ? p + a.right : t.tk - 1);
    const int lo = (int)(a.left >= 0 && p - a.left > 0 ? p - a.left : 0);

    KeyTiles<BN> kt(a, pa, pb, t.tk);
    const int n = t.rows > 0 ? kt.count : 0;
    const T* kb = (const T*)a.k.data + t.k0 * a.k.row + t.hk * a.k.head;
    const T* vb = (const T*)a.v.data + t.k0 * a.v.row + t.hk * a.v.head;
    Stage<T, DP, BN, 256> sk, sv;
    if (tid < 2) bad_tag[tid] = 0;

    auto load = [&](int i) {
        const int64_t j0 = (int64_t)kt.tile(i) * BN;
        sk.load(kb + j0 * a.k.row, a.k.row, t.tk - (int)j0, a.D, tid);
        sv.load(vb + j0 * a.v.row, a.v.row, t.tk - (int)j0, a.D, tid);
    };
    auto store = [&](int i) {
        FPSTOK_LDS char* buf = lds + (i & 1) * 2 * BN * Tl::kPitch;
        sk.store(buf, tid);
        // a value that some row must not see is multiplied by a weight of 0
        // there: an infinite one has to leave the product
        if (tile_view<BN>(a, pa, pb, t.tk, kt.tile(i) * BN) == 1 && sv.clean())
            bad_tag[i & 1] = i + 1;
        sv.store(buf + BN * Tl::kPitch, tid);
    };

    f32x16 o[DB];
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = 0.0f;
    const float c = a.scale * 1.44269504088896f;  // log2 e
    float m = -INFINITY, mc = 0.0f, l = 0.0f;

    if (n > 0) {
        load(0);
        __syncthreads();
        store(0);
    }
    __syncthreads();
    for (int i = 0; i < n; ++i) {
        const int j0 = kt.tile(i) * BN;
        if (i + 1 < n) load(i + 1);
        const int view = wave_live ? tile_view<BN>(a, wa, wb, t.tk, j0) : 0;
        if (view != 0) {
            const FPSTOK_LDS char* kbuf = lds + (i & 1) * 2 * BN * Tl::kPitch;
            const FPSTOK_LDS char* vbuf = kbuf + BN * Tl::kPitch;
            float s[KB * 16];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                f32x16 x = 0.0f;
#pragma unroll
                for (int st = 0; st < STEPS; ++st)
                    x = Elem<T>::mma(Tl::row_frag(kbuf, b * 32 + (lane & 31), st, half), qf[st], x);
#pragma unroll
                for (int e = 0; e < 16; ++e) s[b * 16 + e] = x[e];
            }
            if (view == 1) {
#pragma unroll
                for (int e = 0; e < KB * 16; ++e) {
                    const int j = j0 + (e >> 4) * 32 + ((e >> 2) & 3) * 8 + half * 4 + (e & 3);
                    if (j > hi || (j < lo && j >= a.sinks)) s[e] = -INFINITY;
                }
            }
            float mx = s[0];
#pragma unroll
            for (int e = 1; e < KB * 16; ++e) mx = fmaxf(mx, s[e]);
            mx = pair_max(mx);
            if (__any(mx * c > mc + 8.0f || m == -INFINITY)) {
                const float m2 = fmaxf(m, mx);
                const float mc2 = m2 == -INFINITY ? 0.0f : m2 * c;
                const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mc - mc2);
                m = m2;
                mc = mc2;
                l *= f;
#pragma unroll
                for (int db = 0; db < DB; ++db) o[db] *= f;
            }
#pragma unroll
            for (int e = 0; e < KB * 16; ++e) {
                s[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], c, -mc));
                l += s[e];
            }
#pragma unroll
            for (int k = 0; k < KB * 2; ++k) {
                const Frag pf = to_frag<T>(s + k * 8);
#pragma unroll
                for (int db = 0; db < DB; ++db)
                    o[db] = Elem<T>::mma(Tl::col_frag(vbuf, k * 16, db, lane), pf, o[db]);
            }
            if (bad_tag[i & 1] == i + 1) {
                // rare: the rows that see an infinite value get it here
                for (int j = j0; j < j0 + BN && j <= hi; ++j) {
                    if (j < lo && j >= a.sinks) continue;
#pragma unroll
                    for (int db = 0; db < DB; ++db)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int d = db * 32 + (e >> 2) * 8 + half * 4 + (e & 3);
                            if (d < a.D) {
                                const float x = (float)vb[(int64_t)j * a.v.row + d];
                                if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u)
                                    o[db][e] += x;
                            }
                        }
                }
            }
        }
        if (i + 1 < n) store(i + 1);
        __syncthreads();
    }
    l = pair_sum(l);
    const bool some = m != -INFINITY || l != 0.0f;
    const float inv = live && some ? 1.0f / l : 0.0f;
    T* out = (T*)a.out.data + qrow * a.out.row + h * a.out.head;
    if (!some) {
#pragma unroll
        for (int db = 0; db < DB; ++db) o[db] = 0.0f;
    }
    store_row<T, DB>(o, inv, r < t.rows || r < t.pad ? out : nullptr, a.D, lane);
    if (a.lse && half == 0 && (live || r < t.pad))
        a.lse[qrow * a.H + h] =
            !live ? 0.0f
                  : some ? (mc + __builtin_amdgcn_logf(l)) * 0.693147180559945f : -INFINITY;
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

// Slots of a grid that covers every tile of BM rows of every sequence.
static int64_t row_slots(const SeqArgs& s, int G, int BM) {
    if (s.cu) return s.rows * G / BM + s.B;
    return (int64_t)s.B * (((int64_t)s.cap * G + BM - 1) / BM);
}

template <class T>
static hipError_t forward(const AttnArgs& a, hipStream_t s) {
    const int64_t blocks = row_slots(a.qs, a.H / a.Hk, 128) * a.Hk;
    if (a.D <= 64)
        attention_kernel<T, 64, 64><<<dim3((unsigned)blocks), 256, 0, s>>>(a);
    else
        attention_kernel<T, 128, sizeof(T) == 2 ? 64 : 32><<<dim3((unsigned)blocks), 256, 0, s>>>(a);
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
