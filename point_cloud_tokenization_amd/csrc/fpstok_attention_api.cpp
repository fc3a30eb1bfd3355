// C ABI of attention and rotary positions (declared and documented in
// include/fpstok.h): argument validation, workspace carve-up and launches.
// Validation happens on the host before any HIP call.
#include "fpstok_attention.h"

#include <cmath>

#include "fpstok_host.h"

namespace fpstok {

static_assert(kMaxAxes == FPSTOK_MAX_AXES, "axes of the rotary positions");

static int elem_bytes(int dtype) { return dtype == FPSTOK_F32 ? 4 : 2; }

static fpstok_status check_seqs(const fpstok_seqs* s, const char* what) {
    if (!s) return fail(FPSTOK_EINVAL, "%s is NULL", what);
    if (s->num_seqs < 0) return fail(FPSTOK_EINVAL, "%s: num_seqs < 0", what);
    if (s->num_rows < 0) return fail(FPSTOK_EINVAL, "%s: num_rows < 0", what);
    if (s->max_len < 0) return fail(FPSTOK_EINVAL, "%s: max_len < 0", what);
    if (s->num_rows >= ((int64_t)1 << 31))
        return fail(FPSTOK_EUNSUPPORTED, "%s: num_rows >= 2^31", what);
    if (s->num_seqs > ((int64_t)1 << 24))
        return fail(FPSTOK_EUNSUPPORTED, "%s: num_seqs > 2^24", what);
    if (s->cu_seqlens && s->token_count)
        return fail(FPSTOK_EINVAL, "%s: give cu_seqlens or token_count, not both", what);
    if (((uintptr_t)s->cu_seqlens & 3u) != 0 || ((uintptr_t)s->token_count & 3u) != 0)
        return fail(FPSTOK_EINVAL, "%s: cu_seqlens and token_count must be 4-byte aligned", what);
    if (s->num_seqs == 0) return FPSTOK_OK;
    if (!s->cu_seqlens && !s->token_count)
        return fail(FPSTOK_EINVAL, "%s: cu_seqlens or token_count is required", what);
    if (s->token_count) {
        if (s->capacity < 1) return fail(FPSTOK_EINVAL, "%s: capacity must be >= 1", what);
        if (s->num_rows != s->num_seqs * s->capacity)
            return fail(FPSTOK_EINVAL, "%s: num_rows must be num_seqs * capacity", what);
    }
    return FPSTOK_OK;
}

static fpstok_status check_attn(const fpstok_seqs* qs, const fpstok_seqs* ks,
                                const fpstok_attn_params* p) {
    fpstok_status st = check_seqs(qs, "q_seqs");
    if (st != FPSTOK_OK) return st;
    if (ks != qs) {
        if ((st = check_seqs(ks, "k_seqs")) != FPSTOK_OK) return st;
        if (ks->num_seqs != qs->num_seqs)
            return fail(FPSTOK_EINVAL, "q_seqs and k_seqs hold %lld and %lld sequences",
                        (long long)qs->num_seqs, (long long)ks->num_seqs);
    }
    if (!p) return fail(FPSTOK_EINVAL, "params is NULL");
    if (p->num_heads < 1 || p->num_kv_heads < 1 || p->num_heads % p->num_kv_heads != 0)
        return fail(FPSTOK_EINVAL, "num_kv_heads must be a divisor of num_heads");
    if (p->num_heads > 65536) return fail(FPSTOK_EUNSUPPORTED, "num_heads > 65536");
    if (p->head_dim < 8 || p->head_dim > FPSTOK_MAX_HEAD_DIM || p->head_dim % 8 != 0)
        return fail(FPSTOK_EINVAL, "head_dim must be a multiple of 8 in [8, %d]",
                    FPSTOK_MAX_HEAD_DIM);
    if (p->dtype < FPSTOK_F32 || p->dtype > FPSTOK_BF16)
        return fail(FPSTOK_EINVAL, "dtype must be FPSTOK_F32, FPSTOK_F16 or FPSTOK_BF16");
    if (p->window_left < -1 || p->window_right < -1)
        return fail(FPSTOK_EINVAL, "window_left and window_right must be >= -1");
    if (p->num_sinks < 0 || p->num_sinks > FPSTOK_MAX_SINKS)
        return fail(FPSTOK_EINVAL, "num_sinks must be in [0, %d]", FPSTOK_MAX_SINKS);
    // (the factor that the kernels multiply scores by)
    if (!(p->scale > 0.0f) || !std::isfinite(p->scale * 1.44269504088896f))
        return fail(FPSTOK_EINVAL, "scale must be > 0, and scale * log2(e) finite in float32");
    // rows, places and windows are 32-bit numbers in the kernels
    if (qs->num_rows >= ((int64_t)1 << 30) || ks->num_rows >= ((int64_t)1 << 30))
        return fail(FPSTOK_EUNSUPPORTED, "num_rows >= 2^30");
    if (qs->num_rows * p->num_heads >= ((int64_t)1 << 31) ||
        ks->num_rows * p->num_kv_heads >= ((int64_t)1 << 31))
        return fail(FPSTOK_EUNSUPPORTED, "rows times heads >= 2^31");
    return FPSTOK_OK;
}

// One [rows][heads][D] view: pointer and strides aligned to `align` bytes,
// strides in range.
static fpstok_status check_heads(const fpstok_heads* v, const char* what, int64_t rows, int heads,
                                 int D, int dtype, uintptr_t align, bool output) {
    if (!v) return fail(FPSTOK_EINVAL, "%s is NULL", what);
    if (rows == 0) return FPSTOK_OK;
    if (!v->data) return fail(FPSTOK_EINVAL, "%s: data is NULL", what);
    const int w = elem_bytes(dtype);
    if (v->row_stride < 0 || v->head_stride < 0)
        return fail(FPSTOK_EINVAL, "%s: negative stride", what);
    if (v->row_stride > ((int64_t)1 << 23))  // a tile's rows within 32-bit byte offsets
        return fail(FPSTOK_EUNSUPPORTED, "%s: row_stride > 2^23", what);
    if (v->head_stride > ((int64_t)1 << 40))
        return fail(FPSTOK_EUNSUPPORTED, "%s: head_stride > 2^40", what);
    if (((uintptr_t)v->data % align) != 0 || ((uintptr_t)(v->row_stride * w) % align) != 0 ||
        ((uintptr_t)(v->head_stride * w) % align) != 0)
        return fail(FPSTOK_EINVAL, "%s: data and strides must be aligned to %d bytes", what,
                    (int)align);
    if (output) {
        // rows inside a head's span or heads inside a row's span, never both
        const bool rows_out =
            rows == 1 || v->row_stride >= (int64_t)(heads - 1) * v->head_stride + D;
        const bool heads_out =
            heads == 1 || v->head_stride >= (__int128)(rows - 1) * v->row_stride + D;
        const bool head_ok = heads == 1 || v->head_stride >= D;
        const bool row_ok = rows == 1 || v->row_stride >= D;
        if (!((rows_out && head_ok) || (heads_out && row_ok)))
            return fail(FPSTOK_EINVAL, "%s: rows or heads overlap", what);
    }
    return FPSTOK_OK;
}

static SeqArgs seq_args(const fpstok_seqs* s) {
    return SeqArgs{s->cu_seqlens, s->token_count, s->num_rows, (int32_t)s->num_seqs, s->capacity};
}

static HeadsArg heads_arg(const fpstok_heads* v) {
    return HeadsArg{v->data, v->row_stride, v->head_stride};
}

static AttnArgs attn_args(const fpstok_seqs* qs, const fpstok_seqs* ks,
                          const fpstok_attn_params* p) {
    AttnArgs a{};
    a.qs = seq_args(qs);
    a.ks = seq_args(ks);
    a.H = p->num_heads;
    a.Hk = p->num_kv_heads;
    a.G = a.H / a.Hk;
    a.g_shift = (a.G & (a.G - 1)) == 0 ? __builtin_ctz((unsigned)a.G) : -1;
    a.same_seqs = qs == ks;
    a.D = p->head_dim;
    a.dtype = p->dtype;
    // a window that reaches over every row hides nothing
    a.left = p->window_left < ks->num_rows ? p->window_left : -1;
    a.right = p->window_right < qs->num_rows ? p->window_right : -1;
    a.sinks = p->num_sinks;
    a.scale = p->scale;
    return a;
}

// A length to plan with: the caller's bound, or else the slots of a padded
// sequence or the mean length of packed ones.
static int32_t likely_len(const fpstok_seqs* s) {
    if (s->max_len > 0) return s->max_len;
    if (s->token_count) return s->capacity;
    return s->num_seqs > 0 ? (int32_t)((s->num_rows + s->num_seqs - 1) / s->num_seqs) : 0;
}

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Plans a call and lays out its workspace (pointers are offsets from `ws`);
// returns the bytes it needs.
static size_t lay_out(const fpstok_seqs* qs, const fpstok_seqs* ks, bool backward, void* ws,
                      AttnArgs& a, AttnPlan& plan) {
    const size_t rows = (size_t)qs->num_rows * a.H;
    char* at = (char*)ws;
    if (backward) {
        a.lse2 = (float*)at;
        a.delta = (float*)(at + align256(rows * sizeof(float)));
        size_t need = 2 * align256(rows * sizeof(float));
        a.k_splits = plan_key_parts(a, likely_len(qs));
        if (a.k_splits > 1) {
            a.k_part = (float*)(at + need);
            need += align256((size_t)a.k_splits * 2 * a.Hk * ks->num_rows * a.D * sizeof(float));
        }
        const int64_t q_blocks = row_slots(a.qs, a.G, 7) * a.Hk;
        const int64_t k_blocks = row_slots(a.ks, 1, 7) * a.Hk * a.k_splits;
        plan.blocks = q_blocks > k_blocks ? q_blocks : k_blocks;
        if (a.left < 0 || a.sinks == 0) return need;
        // about 512 workgroups of queries past the sinks, of 128 queries or more
        // (883 + 300 pulses, 16 heads on 4: 74 us a training step, of 256: 80)
        a.sink_shift = 7;
        while (qs->num_rows * a.Hk >> a.sink_shift > 512) ++a.sink_shift;
        a.sink_part = (float*)(at + need);
        const int64_t chunks = row_slots(a.qs, 1, a.sink_shift) * a.Hk;
        if (chunks > plan.blocks) plan.blocks = chunks;
        return need + align256((size_t)chunks * 2 * a.sinks * a.D * sizeof(float));
    }
    plan = plan_attention(a, likely_len(qs), likely_len(ks));
    a.splits = plan.splits;
    plan.blocks = row_slots(a.qs, a.G, plan.few ? 5 : 7) * a.Hk * a.splits;
    if (plan.splits == 1) return 0;
    const size_t ml = align256(rows * plan.splits * sizeof(float2));
    a.part_ml = (float2*)at;
    a.part = (float*)(at + ml);
    return ml + align256(rows * plan.splits * a.D * sizeof(float));
}

// A launch holds less than 2^32 threads, 256 a workgroup.
static fpstok_status check_grid(const AttnPlan& plan) {
    if (plan.blocks >= ((int64_t)1 << 24))
        return fail(FPSTOK_EUNSUPPORTED, "%lld workgroups, at most 2^24 - 1 in a launch",
                    (long long)plan.blocks);
    return FPSTOK_OK;
}

static fpstok_status check_attn_ws(size_t need, void* ws, size_t ws_bytes) {
    if (need == 0) return FPSTOK_OK;
    if (!ws) return fail(FPSTOK_EWORKSPACE, "workspace is NULL (need %zu bytes)", need);
    if (ws_bytes < need)
        return fail(FPSTOK_EWORKSPACE, "workspace has %zu bytes, need %zu", ws_bytes, need);
    if (((uintptr_t)ws & 255u) != 0)
        return fail(FPSTOK_EINVAL, "workspace must be 256-byte aligned");
    return FPSTOK_OK;
}

}  // namespace fpstok

using namespace fpstok;

FPSTOK_API size_t fpstok_attention_workspace_size(const fpstok_seqs* qs, const fpstok_seqs* ks,
                                                  const fpstok_attn_params* p, int32_t backward) {
    if (!ks) ks = qs;
    if (check_attn(qs, ks, p) != FPSTOK_OK) return 0;
    AttnArgs a = attn_args(qs, ks, p);
    AttnPlan plan;
    const size_t need = lay_out(qs, ks, backward != 0, nullptr, a, plan);
    return check_grid(plan) == FPSTOK_OK ? need : 0;
}

FPSTOK_API fpstok_status fpstok_attention(const fpstok_seqs* qs, const fpstok_seqs* ks,
                                          const fpstok_attn_params* p, const fpstok_heads* q,
                                          const fpstok_heads* k, const fpstok_heads* v,
                                          const fpstok_heads* out, float* lse, void* ws,
                                          size_t ws_bytes, void* stream) {
    if (!ks) ks = qs;
    fpstok_status st = check_attn(qs, ks, p);
    if (st != FPSTOK_OK) return st;
    const int64_t nq = qs->num_rows, nk = ks->num_rows;
    const int H = p->num_heads, Hk = p->num_kv_heads, D = p->head_dim, dt = p->dtype;
    if ((st = check_heads(q, "q", nq, H, D, dt, 16, false)) != FPSTOK_OK ||
        (st = check_heads(k, "k", nk, Hk, D, dt, 16, false)) != FPSTOK_OK ||
        (st = check_heads(v, "v", nk, Hk, D, dt, 16, false)) != FPSTOK_OK ||
        (st = check_heads(out, "out", nq, H, D, dt, 16, true)) != FPSTOK_OK)
        return st;
    if (((uintptr_t)lse & 3u) != 0) return fail(FPSTOK_EINVAL, "lse must be 4-byte aligned");
    AttnArgs a = attn_args(qs, ks, p);
    AttnPlan plan;
    const size_t need = lay_out(qs, ks, false, ws, a, plan);
    if ((st = check_grid(plan)) != FPSTOK_OK ||
        (st = check_attn_ws(need, ws, ws_bytes)) != FPSTOK_OK)
        return st;
    if (qs->num_seqs == 0 || nq == 0) return ok();
    a.q = heads_arg(q);
    a.k = heads_arg(k);
    a.v = heads_arg(v);
    a.out = heads_arg(out);
    a.lse = lse;
    const hipError_t e = launch_attention(a, plan, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "attention kernel launch");
    return ok();
}

FPSTOK_API fpstok_status fpstok_attention_backward(
    const fpstok_seqs* qs, const fpstok_seqs* ks, const fpstok_attn_params* p,
    const fpstok_heads* q, const fpstok_heads* k, const fpstok_heads* v, const fpstok_heads* out,
    const float* lse, const fpstok_heads* grad_out, const fpstok_heads* grad_q,
    const fpstok_heads* grad_k, const fpstok_heads* grad_v, void* ws, size_t ws_bytes,
    void* stream) {
    if (!ks) ks = qs;
    fpstok_status st = check_attn(qs, ks, p);
    if (st != FPSTOK_OK) return st;
    const int64_t nq = qs->num_rows, nk = ks->num_rows;
    const int H = p->num_heads, Hk = p->num_kv_heads, D = p->head_dim, dt = p->dtype;
    if ((st = check_heads(q, "q", nq, H, D, dt, 16, false)) != FPSTOK_OK ||
        (st = check_heads(k, "k", nk, Hk, D, dt, 16, false)) != FPSTOK_OK ||
        (st = check_heads(v, "v", nk, Hk, D, dt, 16, false)) != FPSTOK_OK ||
        (st = check_heads(out, "out", nq, H, D, dt, 16, false)) != FPSTOK_OK ||
        (st = check_heads(grad_out, "grad_out", nq, H, D, dt, 16, false)) != FPSTOK_OK ||
        (st = check_heads(grad_q, "grad_q", nq, H, D, dt, 16, true)) != FPSTOK_OK ||
        (st = check_heads(grad_k, "grad_k", nk, Hk, D, dt, 16, true)) != FPSTOK_OK ||
        (st = check_heads(grad_v, "grad_v", nk, Hk, D, dt, 16, true)) != FPSTOK_OK)
        return st;
    if (nq > 0 && !lse) return fail(FPSTOK_EINVAL, "lse is NULL");
    if (((uintptr_t)lse & 3u) != 0) return fail(FPSTOK_EINVAL, "lse must be 4-byte aligned");
    AttnArgs a = attn_args(qs, ks, p);
    AttnPlan plan;
    const size_t need = lay_out(qs, ks, true, ws, a, plan);
    if ((st = check_grid(plan)) != FPSTOK_OK ||
        (st = check_attn_ws(need, ws, ws_bytes)) != FPSTOK_OK)
        return st;
    if (qs->num_seqs == 0 || nq + nk == 0) return ok();
    a.q = heads_arg(q);
    a.k = heads_arg(k);
    a.v = heads_arg(v);
    a.out = heads_arg(out);
    a.grad_out = heads_arg(grad_out);
    a.grad_q = heads_arg(grad_q);
    a.grad_k = heads_arg(grad_k);
    a.grad_v = heads_arg(grad_v);
    a.lse = const_cast<float*>(lse);
    const hipError_t e = launch_attention_backward(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "attention gradient kernel launch");
    return ok();
}

FPSTOK_API fpstok_status fpstok_rope(const fpstok_seqs* seqs, const fpstok_rope_params* p,
                                     const void* positions, const float* freqs,
                                     const fpstok_heads* q_in, const fpstok_heads* q_out,
                                     const fpstok_heads* k_in, const fpstok_heads* k_out,
                                     void* stream) {
    fpstok_status st = check_seqs(seqs, "seqs");
    if (st != FPSTOK_OK) return st;
    if (!p) return fail(FPSTOK_EINVAL, "params is NULL");
    if (p->head_dim < 2 || p->head_dim > 1024 || p->head_dim % 2 != 0)
        return fail(FPSTOK_EINVAL, "head_dim must be even and in [2, 1024]");
    if (p->dtype < FPSTOK_F32 || p->dtype > FPSTOK_BF16)
        return fail(FPSTOK_EINVAL, "dtype must be FPSTOK_F32, FPSTOK_F16 or FPSTOK_BF16");
    if (p->positions_dtype != FPSTOK_F32 && p->positions_dtype != FPSTOK_I32)
        return fail(FPSTOK_EINVAL, "positions_dtype must be FPSTOK_F32 or FPSTOK_I32");
    if (p->num_axes < 1 || p->num_axes > FPSTOK_MAX_AXES)
        return fail(FPSTOK_EINVAL, "num_axes must be in [1, %d]", FPSTOK_MAX_AXES);
    if ((p->interleaved != 0 && p->interleaved != 1) || (p->inverse != 0 && p->inverse != 1))
        return fail(FPSTOK_EINVAL, "interleaved and inverse must be 0 or 1");
    RopeArgs a{};
    int64_t R = 0;
    for (int i = 0; i < p->num_axes; ++i) {
        if (p->pairs[i] < 0 || p->pairs[i] > p->head_dim)
            return fail(FPSTOK_EINVAL, "pairs[%d] out of range", i);
        a.first_pair[i] = (int32_t)R;
        R += p->pairs[i];
    }
    for (int i = p->num_axes; i <= kMaxAxes; ++i) a.first_pair[i] = (int32_t)R;
    if (R < 1 || 2 * R > p->head_dim)
        return fail(FPSTOK_EINVAL, "the axes' pairs must add up to 1 .. head_dim / 2");
    if ((k_in == nullptr) != (k_out == nullptr))
        return fail(FPSTOK_EINVAL, "give k_in and k_out, or neither");
    if (p->num_heads < 1 || p->num_heads > 65536)
        return fail(FPSTOK_EINVAL, "num_heads must be in [1, 65536]");
    if (k_in && (p->num_kv_heads < 1 || p->num_kv_heads > 65536))
        return fail(FPSTOK_EINVAL, "num_kv_heads must be in [1, 65536]");
    const int64_t n = seqs->num_rows;
    // a launch holds less than 2^32 threads: one per element pair of a row, or
    // 256 per 8 rows or more
    if (n * (p->head_dim > 64 ? p->head_dim : 64) >= ((int64_t)1 << 33))
        return fail(FPSTOK_EUNSUPPORTED, "num_rows * max(head_dim, 64) >= 2^33");
    const uintptr_t w = (uintptr_t)elem_bytes(p->dtype);
    const fpstok_heads* in[2] = {q_in, k_in};
    const fpstok_heads* out[2] = {q_out, k_out};
    const char* in_name[2] = {"q_in", "k_in"};
    const char* out_name[2] = {"q_out", "k_out"};
    for (int i = 0; i < (k_in ? 2 : 1); ++i) {
        const int heads = i == 0 ? p->num_heads : p->num_kv_heads;
        if ((st = check_heads(in[i], in_name[i], n, heads, p->head_dim, p->dtype, w, false)) !=
                FPSTOK_OK ||
            (st = check_heads(out[i], out_name[i], n, heads, p->head_dim, p->dtype, w, true)) !=
                FPSTOK_OK)
            return st;
        if (n > 0 && in[i]->data == out[i]->data &&
            (in[i]->row_stride != out[i]->row_stride || in[i]->head_stride != out[i]->head_stride))
            return fail(FPSTOK_EINVAL, "%s in place of %s needs the same strides", out_name[i],
                        in_name[i]);
        a.in[i] = heads_arg(in[i]);
        a.out[i] = heads_arg(out[i]);
        a.heads[i] = heads;
    }
    if (seqs->num_seqs == 0 || n == 0) return ok();
    if (!positions || !freqs) return fail(FPSTOK_EINVAL, "positions or freqs is NULL");
    if (((uintptr_t)positions & 3u) != 0 || ((uintptr_t)freqs & 3u) != 0)
        return fail(FPSTOK_EINVAL, "positions and freqs must be 4-byte aligned");
    a.seqs = seq_args(seqs);
    a.positions = positions;
    a.freqs = freqs;
    a.D = p->head_dim;
    a.dtype = p->dtype;
    a.int_positions = p->positions_dtype == FPSTOK_I32;
    a.axes = p->num_axes;
    a.R = (int32_t)R;
    a.interleaved = p->interleaved;
    a.inverse = p->inverse;
    const hipError_t e = launch_rope(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "rotary position kernel launch");
    return ok();
}
