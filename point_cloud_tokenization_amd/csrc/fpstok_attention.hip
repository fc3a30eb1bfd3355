// Attention over the rows of variable-length sequences and its gradients: the
// launches without a bias, the joins of split walks, and how a call is split.
#include "fpstok_attention_kernels.h"

namespace fpstok {

// Joins the parts of a row whose keys were split: a workgroup per (query,
// head).  Its threads take 4 elements each of every kGroups-th part, so a
// thread's loads do not wait for one another; the groups' sums are added in
// order.
template <class T>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
    using f4 = float __attribute__((ext_vector_type(4)));
    constexpr int kGroups = 8;
    __shared__ float factor[256];  // at most 256 parts
    __shared__ f4 sums[kGroups][32];
    __shared__ float wave_top[4], wave_sum[4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = blockIdx.x / a.H;
    const int h = (int)(blockIdx.x % a.H), G = a.G, hk = h / G;
    bool here = true;
    if (a.qs.cu) {
        if (row < cu_at(a.qs, 0) || row >= cu_at(a.qs, a.qs.B)) return;
    } else {
        here = row % a.qs.cap < a.qs.count[row / a.qs.cap];
    }
    const int64_t step = (int64_t)a.Hk * a.qs.rows * G;
    const int64_t at = ((int64_t)hk * a.qs.rows + row) * G + h - hk * G;
    float2 z = make_float2(-INFINITY, 0.0f);
    if (here && tid < a.splits) z = a.part_ml[tid * step + at];
    const bool seen = !(z.x == -INFINITY && z.y == 0.0f);
    float top = z.x;
#pragma unroll
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) wave_top[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
    const float f = seen ? __builtin_amdgcn_exp2f(z.x - top) : 0.0f;
    factor[tid] = f;
    float sum = z.y * f;
#pragma unroll
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) wave_sum[tid >> 6] = sum;
    __syncthreads();
    sum = (wave_sum[0] + wave_sum[1]) + (wave_sum[2] + wave_sum[3]);
    const int d = (tid & 31) * 4, group = tid >> 5;
    if (here) {
        f4 y = 0.0f;
        const float* part = a.part + at * a.D + (d < a.D ? d : 0);
        const int64_t stride = step * a.D;
#pragma unroll 4
        for (int s = group; s < a.splits; s += kGroups)
            y += factor[s] * *(const f4*)(part + s * stride);
        sums[group][tid & 31] = y;
    }
    __syncthreads();
    const bool some = here && (top != -INFINITY || sum != 0.0f);
    if (tid < 32 && d < a.D) {
        f4 y = 0.0f;
        if (some) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) y += sums[g][tid];
            y *= 1.0f / sum;
        }
        using T4 = T __attribute__((ext_vector_type(4)));
        *(T4*)((T*)a.out.data + row * a.out.row + h * a.out.head + d) =
            __builtin_convertvector(y, T4);
    }
    if (a.lse && tid == 0)
        a.lse[row * a.H + h] =
            !here ? 0.0f
                  : some ? (top + __builtin_amdgcn_logf(sum)) * 0.693147180559945f : -INFINITY;
}

// The same for many rows: 4 elements of one (query, head) per thread, its parts
// one after the other.
template <class T>
__global__ __launch_bounds__(256) void attention_join_rows_kernel(AttnArgs a) {
    using f4 = float __attribute__((ext_vector_type(4)));
    using T4 = T __attribute__((ext_vector_type(4)));
    const uint32_t per = (uint32_t)a.D / 4;
    const uint32_t x = blockIdx.x * 256u + threadIdx.x;
    const uint32_t rh = x / per;
    const int d = (int)(x - rh * per) * 4;
    const uint32_t row = rh / (uint32_t)a.H;
    if (row >= a.qs.rows) return;
    const int h = (int)(rh - row * (uint32_t)a.H), hk = h / a.G;
    bool here = true;
    if (a.qs.cu) {
        if (row < cu_at(a.qs, 0) || row >= cu_at(a.qs, a.qs.B)) return;
    } else {
        const uint32_t b = row / (uint32_t)a.qs.cap;
        here = (int)(row - b * (uint32_t)a.qs.cap) < a.qs.count[b];
    }
    const int64_t step = (int64_t)a.Hk * a.qs.rows * a.G;
    const int64_t at = ((int64_t)hk * a.qs.rows + row) * a.G + h - hk * a.G;
    float top = -INFINITY, sum = 0.0f;
    f4 y = 0.0f;
    if (here) {
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.part_ml[s * step + at].x);
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            const float2 z = a.part_ml[s * step + at];
            const float f =
                z.x == -INFINITY && z.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(z.x - top);
            sum += z.y * f;
            y += f * *(const f4*)(a.part + (s * step + at) * a.D + d);
        }
    }
    const bool some = here && (top != -INFINITY || sum != 0.0f);
    y *= some ? 1.0f / sum : 0.0f;
    if (!some) y = 0.0f;
    *(T4*)((T*)a.out.data + row * a.out.row + h * a.out.head + d) = __builtin_convertvector(y, T4);
    if (a.lse && d == 0)
        a.lse[(int64_t)row * a.H + h] = !here ? 0.0f : some ? log_sum(top, sum) : -INFINITY;
}

// Adds the parts of keys whose walk was split, in order: 4 elements of one key
// and head per thread.
template <class T>
__global__ __launch_bounds__(256) void attention_join_dkv_kernel(AttnArgs a) {
    using f4 = float __attribute__((ext_vector_type(4)));
    using T4 = T __attribute__((ext_vector_type(4)));
    const uint32_t per = (uint32_t)a.D / 4;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t at = x / per;
    const int d = (int)(x - at * per) * 4;
    const int64_t row = at / a.Hk;
    const int hk = (int)(at - row * a.Hk);
    if (row >= a.ks.rows) return;
    bool here = true;
    if (a.ks.cu) {
        if (row < cu_at(a.ks, 0) || row >= cu_at(a.ks, a.ks.B)) return;
    } else {
        here = row % a.ks.cap < a.ks.count[row / a.ks.cap];
    }
    f4 k = 0.0f, v = 0.0f;
    if (here) {
        const int64_t v_at = k_part_at(a, 0, a.Hk, 0);
#pragma unroll 4
        for (int s = 0; s < a.k_splits; ++s) {
            const float* part = a.k_part + k_part_at(a, s, hk, row) + d;
            k += *(const f4*)part;
            v += *(const f4*)(part + v_at);
        }
    }
    *(T4*)((T*)a.grad_k.data + row * a.grad_k.row + hk * a.grad_k.head + d) =
        __builtin_convertvector(k * a.scale, T4);
    *(T4*)((T*)a.grad_v.data + row * a.grad_v.row + hk * a.grad_v.head + d) =
        __builtin_convertvector(v, T4);
}

int64_t row_slots(const SeqArgs& s, int G, int shift) {
    if (s.cu) return (s.rows * G >> shift) + s.B;
    return (int64_t)s.B * (((int64_t)s.cap * G + (1 << shift) - 1) >> shift);
}

// Splits a row's keys until about `want` workgroups are there, into at least
// `least` keys each.
static int64_t key_splits(const AttnArgs& a, int64_t blocks, int64_t q_len, int64_t k_len,
                          int64_t want, int64_t least) {
    int64_t seen = k_len;
    if (a.left >= 0 && a.right >= 0 && seen > q_len + a.left + a.right + a.sinks)
        seen = q_len + a.left + a.right + a.sinks;
    int64_t n = blocks > 0 ? want / blocks : 1;
    if (n > seen / least) n = seen / least;
    return n < 1 ? 1 : n > 256 ? 256 : n;
}

AttnPlan plan_attention(const AttnArgs& a, int32_t q_len, int32_t k_len) {
    const int G = a.G;
    AttnPlan p;
    p.few = (int64_t)q_len * G <= 32;
    const int64_t blocks = row_slots(a.qs, G, p.few ? 5 : 7) * a.Hk;
    if (p.few) {
        p.splits = (int32_t)key_splits(a, blocks, q_len, k_len, 1024, 512);
    } else {
        // two workgroups per compute unit, unless nearly every one has a
        // workgroup already (5000 rows, 5 heads of 64: 200 workgroups, 2 parts
        // 74 us, unsplit 95; 2000 rows, 16 heads on 4, D = 128: 252 workgroups, 2
        // parts 59 us, unsplit 52).  How much 2 parts of 225 to 256 workgroups
        // would take goes by the keys: 1.16 times one part at 16 heads on 4 of
        // 128 and 1800 to 2050 rows, 0.97 with a causal mask; 0.95 and 0.76 at 8
        // heads of 128 and 3600 to 4100 rows; 0.77 and 0.64 at 5 heads of 64 and 5800
        // to 6500 rows, and from 257 workgroups on both are the same.  The step at
        // 224 keeps the first of these.  2500 rows of one head, parts of 256 keys
        // or more 19 us, of 512 21.  float32 tiles take 8 times as long, and four
        // workgroups even the compute units out (3000 rows, 12 heads of 64: 320
        // us, unsplit 450; 1500 rows: 114, with two 96).
        const int64_t want = a.dtype == 0 ? 1024 : blocks > 224 ? 0 : 512;
        p.splits = (int32_t)key_splits(a, blocks, 128 / G + 1, k_len, want, 256);
    }
    return p;
}

int plan_key_parts(const AttnArgs& a, int32_t q_len) {
    // workgroups of 128 keys, each with a walk of about this many queries, in at
    // most as many parts as all run at once (5000 rows, 8 heads on 1: 10 parts of
    // 40 workgroups 382 us a training step, 13 parts 430; 8 heads on 8, 320
    // workgroups: unsplit 397, 2 parts 412) and in
    // parts of 192 or more (a walk alone on its compute unit takes 1.6 us per 64
    // queries, the join 5 us.  One event of 110 tokens, 8 heads on 1, all of a
    // training step: parts of 512 or more 43 us, of 192 34; 21 padded events of
    // up to 256 tokens, 12 heads: of 192 43 us, of 128 54)
    const int64_t blocks = row_slots(a.ks, 1, 7) * a.Hk;
    int64_t walk = q_len;
    if (a.left >= 0 && a.right >= 0 && walk > 128 + a.left + a.right)
        walk = 128 + (int64_t)a.left + a.right;
    walk *= a.G;
    int64_t n = blocks > 0 ? 512 / blocks : 1;
    if (n > walk / 192) n = walk / 192;
    return n < 1 ? 1 : n > 64 ? 64 : (int)n;
}

void launch_join(const AttnArgs& a, hipStream_t s) {
    // a workgroup per (query, head) for few of them (one query on 131k keys
    // in 32 parts: 175 us against 180), a thread per 4 elements for many
    // (5000 rows, 3 heads: 48 us against 64)
    const int64_t joins = (a.qs.rows * a.H * (a.D / 4) + 255) / 256;
    auto by_type = [&](auto type) {
        using T = decltype(type);
        if (joins >= 128)
            attention_join_rows_kernel<T><<<dim3((unsigned)joins), 256, 0, s>>>(a);
        else
            attention_join_kernel<T><<<dim3((unsigned)(a.qs.rows * a.H)), 256, 0, s>>>(a);
    };
    a.dtype == 0 ? by_type(float{}) : a.dtype == 1 ? by_type(_Float16{}) : by_type(__bf16{});
}

void launch_join_dkv(const AttnArgs& a, hipStream_t s) {
    const int64_t threads = a.ks.rows * a.Hk * (a.D / 4);
    const dim3 grid((unsigned)((threads + 255) / 256));
    auto by_type = [&](auto type) {
        attention_join_dkv_kernel<decltype(type)><<<grid, 256, 0, s>>>(a);
    };
    a.dtype == 0 ? by_type(float{}) : a.dtype == 1 ? by_type(_Float16{}) : by_type(__bf16{});
}

template <class T>
static hipError_t backward(const AttnArgs& a, hipStream_t s) {
    if (a.qs.rows > 0) backward_q<T, kNoBias>(a, NoBias{}, s);
    backward_kv<T, kNoBias>(a, NoBias{}, s);
    return hipGetLastError();
}

hipError_t launch_attention(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
    return a.dtype == 0   ? forward<float, kNoBias>(a, NoBias{}, plan, s)
           : a.dtype == 1 ? forward<_Float16, kNoBias>(a, NoBias{}, plan, s)
                          : forward<__bf16, kNoBias>(a, NoBias{}, plan, s);
}

hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s) {
    return a.dtype == 0 ? backward<float>(a, s)
                        : a.dtype == 1 ? backward<_Float16>(a, s) : backward<__bf16>(a, s);
}

}  // namespace fpstok
