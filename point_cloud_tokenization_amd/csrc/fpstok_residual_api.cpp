// C ABI of the residual step (declared and documented in include/fpstok.h):
// argument validation, workspace carve-up and launches.  Validation happens on
// the host before any HIP call.
#include "fpstok_residual.h"

#include <cmath>

#include "fpstok_seqs_host.h"

namespace fpstok {

static fpstok_status check_residual(const fpstok_seqs* s, const fpstok_residual_params* p) {
    fpstok_status st = check_seqs(s, "seqs");
    if (st != FPSTOK_OK) return st;
    if (!p) return fail(FPSTOK_EINVAL, "params is NULL");
    if (p->width < 1 || p->width > FPSTOK_MAX_WIDTH)
        return fail(FPSTOK_EINVAL, "width must be in [1, %d]", FPSTOK_MAX_WIDTH);
    if (p->branch_dtype < FPSTOK_F32 || p->branch_dtype > FPSTOK_BF16)
        return fail(FPSTOK_EINVAL, "branch_dtype must be FPSTOK_F32, FPSTOK_F16 or FPSTOK_BF16");
    if (p->stream_dtype != FPSTOK_F32 && p->stream_dtype != p->branch_dtype)
        return fail(FPSTOK_EINVAL, "stream_dtype must be FPSTOK_F32 or branch_dtype");
    if (p->post_norm < FPSTOK_NORM_NONE || p->post_norm > FPSTOK_NORM_LAYER ||
        p->pre_norm < FPSTOK_NORM_NONE || p->pre_norm > FPSTOK_NORM_LAYER)
        return fail(FPSTOK_EINVAL, "post_norm and pre_norm must be FPSTOK_NORM_*");
    if (p->gate_per < FPSTOK_GATE_NONE || p->gate_per > FPSTOK_GATE_SEQUENCE)
        return fail(FPSTOK_EINVAL, "gate_per must be FPSTOK_GATE_*");
    if (p->activation < FPSTOK_ACT_NONE || p->activation > FPSTOK_ACT_SILU)
        return fail(FPSTOK_EINVAL, "activation must be FPSTOK_ACT_*");
    if (!(p->eps >= 1.17549435e-38f) || !std::isfinite(p->eps))
        return fail(FPSTOK_EINVAL, "eps must be finite and at least 1.2e-38");
    return FPSTOK_OK;
}

// One [rows][width] view.
static fpstok_status check_rows(const fpstok_rows* v, const char* what, int64_t rows, int C,
                                int dtype, bool output, RowsArg& to) {
    if (!v) return fail(FPSTOK_EINVAL, "%s is NULL", what);
    to = RowsArg{v->data, rows > 1 ? v->row_stride : 0};
    if (rows == 0) return FPSTOK_OK;
    const int w = elem_bytes(dtype);
    if (!v->data) return fail(FPSTOK_EINVAL, "%s: data is NULL", what);
    if (((uintptr_t)v->data % (uintptr_t)w) != 0)
        return fail(FPSTOK_EINVAL, "%s: data must be aligned to %d bytes", what, w);
    if (to.row < 0) return fail(FPSTOK_EINVAL, "%s: negative stride", what);
    if (to.row > ((int64_t)1 << 23))
        return fail(FPSTOK_EUNSUPPORTED, "%s: row_stride > 2^23", what);
    if (output && rows > 1 && to.row < C) return fail(FPSTOK_EINVAL, "%s: rows overlap", what);
    return FPSTOK_OK;
}

// A view's rows in bytes, for the check of overlaps.
struct Span {
    const char* name;
    const char* data;
    int64_t rows, step, width;
    Span(const char* name, const RowsArg& v, int64_t rows, int C, int dtype)
        : name(name), data((const char*)v.data), rows(v.data ? rows : 0),
          step(v.row * elem_bytes(dtype)), width((int64_t)C * elem_bytes(dtype)) {
        if (step == 0 && this->rows > 1) this->rows = 1;  // (the same row again)
    }
    int64_t end() const { return (rows - 1) * step + width; }
};

// Whether two views share a byte.  Views of one stride may lie beside each other
// in wider rows; of two strides, every row of the one with fewer is looked at.
static bool overlap(const Span& a, const Span& b) {
    if (a.rows == 0 || b.rows == 0) return false;
    const int64_t d = b.data - a.data;  // (addresses, not one array's elements)
    if (d >= a.end() || -d >= b.end()) return false;
    if (a.rows > b.rows) return overlap(b, a);
    if (b.rows == 1) return true;
    if (a.rows == 1 || a.step == b.step) {
        // where a's row begins within b's step
        const int64_t at = ((-d) % b.step + b.step) % b.step;
        return !(at >= b.width && at + a.width <= b.step);
    }
    for (int64_t i = 0; i < a.rows; ++i) {
        const int64_t from = i * a.step - d;  // from b's first byte on
        // b's first row that ends behind it
        const int64_t k = from < b.width ? 0 : (from - b.width) / b.step + 1;
        if (k < b.rows && k * b.step < from + a.width) return true;
    }
    return false;
}

// Outputs may take an input's place row for row, and not overlap one, or one
// another, in any other way.
static fpstok_status check_overlaps(const Span* out, int outs, const Span* in, int ins) {
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < ins; ++j) {
            const bool same = out[i].data == in[j].data && out[i].step == in[j].step &&
                              out[i].rows == in[j].rows && out[i].width == in[j].width;
            if (!same && overlap(out[i], in[j]))
                return fail(FPSTOK_EINVAL, "%s overlaps %s", out[i].name, in[j].name);
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return fail(FPSTOK_EINVAL, "%s overlaps %s", out[i].name, out[j].name);
    }
    return FPSTOK_OK;
}

static fpstok_status check_weight(const float* w, const char* what, bool fits) {
    if (w && !fits) return fail(FPSTOK_EINVAL, "%s without what it belongs to", what);
    if (((uintptr_t)w & 3u) != 0) return fail(FPSTOK_EINVAL, "%s must be 4-byte aligned", what);
    return FPSTOK_OK;
}

// The operands that the step and its gradients share: x, y, gate and weights.
static fpstok_status check_inputs(const fpstok_seqs* s, const fpstok_residual_params* p,
                                  const fpstok_residual_weights* w, const fpstok_rows* x,
                                  const fpstok_rows* y, const fpstok_rows* gate,
                                  ResidualArgs& a) {
    fpstok_status st;
    const int64_t n = s->num_rows;
    a.seqs = seq_args(s);
    a.C = p->width;
    a.stream = p->stream_dtype;
    a.branch = p->branch_dtype;
    a.post = p->post_norm;
    a.pre = p->pre_norm;
    a.gate_per = p->gate_per;
    a.act = p->activation;
    a.eps = p->eps;
    if ((st = check_rows(x, "x", n, a.C, a.stream, false, a.x)) != FPSTOK_OK) return st;
    if (y) {
        if ((st = check_rows(y, "y", n, a.C, a.branch, false, a.y)) != FPSTOK_OK) return st;
    } else if (a.post != FPSTOK_NORM_NONE || a.gate_per != FPSTOK_GATE_NONE) {
        return fail(FPSTOK_EINVAL, "post_norm or gate_per without y");
    }
    if ((gate != nullptr) != (a.gate_per != FPSTOK_GATE_NONE))
        return fail(FPSTOK_EINVAL, "give gate with gate_per, or neither");
    if (!gate && a.act != FPSTOK_ACT_NONE)
        return fail(FPSTOK_EINVAL, "activation without a gate");
    if (gate && (st = check_rows(gate, "gate",
                                 a.gate_per == FPSTOK_GATE_ROW ? n : s->num_seqs, a.C, a.branch,
                                 false, a.gate)) != FPSTOK_OK)
        return st;
    if (!w) return FPSTOK_OK;
    const float* weights[kResidualWeights] = {w->post_weight, w->post_bias, w->scale,
                                              w->pre_weight, w->pre_bias};
    const char* names[kResidualWeights] = {"post_weight", "post_bias", "scale", "pre_weight",
                                           "pre_bias"};
    const bool fits[kResidualWeights] = {a.post != 0, a.post != 0, y != nullptr, a.pre != 0,
                                         a.pre != 0};
    for (int k = 0; k < kResidualWeights; ++k) {
        if ((st = check_weight(weights[k], names[k], fits[k])) != FPSTOK_OK) return st;
        a.weights[k] = weights[k];
    }
    return FPSTOK_OK;
}

// Lays out the workspace of the gradients and returns its bytes; `given`: the
// weights whose gradients are formed.
static size_t lay_out(ResidualArgs& a, int given, bool gates, void* ws) {
    const int64_t blocks = residual_blocks(a), runs = a.runs;
    const size_t row = (size_t)a.C * sizeof(float);
    a.part = (float*)ws;
    size_t need = align256((size_t)blocks * given * row);
    if (gates) {
        a.gate_part = (float*)((char*)ws + need);
        need += align256((size_t)(runs + a.seqs.B) * row);
    }
    return need;
}

}  // namespace fpstok

using namespace fpstok;

FPSTOK_API size_t fpstok_residual_workspace_size(const fpstok_seqs* s,
                                                 const fpstok_residual_params* p) {
    if (check_residual(s, p) != FPSTOK_OK) return 0;
    ResidualArgs a{};
    a.seqs = seq_args(s);
    a.C = p->width;
    a.stream = p->stream_dtype;
    a.post = a.pre = FPSTOK_NORM_RMS;  // (the most runs there can be)
    plan_residual(a, true);
    return lay_out(a, kResidualWeights, p->gate_per == FPSTOK_GATE_SEQUENCE, nullptr);
}

FPSTOK_API fpstok_status fpstok_residual(const fpstok_seqs* s, const fpstok_residual_params* p,
                                         const fpstok_residual_weights* w, const fpstok_rows* x,
                                         const fpstok_rows* y, const fpstok_rows* gate,
                                         const fpstok_rows* x_out, const fpstok_rows* h,
                                         float* stats, void* stream) {
    fpstok_status st = check_residual(s, p);
    if (st != FPSTOK_OK) return st;
    ResidualArgs a{};
    if ((st = check_inputs(s, p, w, x, y, gate, a)) != FPSTOK_OK) return st;
    const int64_t n = s->num_rows;
    if (!x_out && a.pre == FPSTOK_NORM_NONE)
        return fail(FPSTOK_EINVAL, "x_out is NULL and pre_norm is FPSTOK_NORM_NONE");
    if ((h != nullptr) != (a.pre != FPSTOK_NORM_NONE))
        return fail(FPSTOK_EINVAL, "give h with pre_norm, or neither");
    if (x_out &&
        (st = check_rows(x_out, "x_out", n, a.C, a.stream, true, a.x_out)) != FPSTOK_OK)
        return st;
    if (h && (st = check_rows(h, "h", n, a.C, a.branch, true, a.h)) != FPSTOK_OK) return st;
    const RowsArg* in[2] = {&a.x, &a.y};
    const RowsArg* out[2] = {&a.x_out, &a.h};
    for (int i = 0; i < 2; ++i)
        if (n > 1 && out[i]->data && out[i]->data == in[i]->data && out[i]->row != in[i]->row)
            return fail(FPSTOK_EINVAL, "%s in place needs the same stride", i ? "h" : "x_out");
    if (((uintptr_t)stats & 15u) != 0)
        return fail(FPSTOK_EINVAL, "stats must be 16-byte aligned");
    const int64_t gate_rows = a.gate_per == FPSTOK_GATE_SEQUENCE ? s->num_seqs : n;
    const Span ins[] = {{"x", a.x, n, a.C, a.stream},
                        {"y", a.y, n, a.C, a.branch},
                        {"gate", a.gate, gate_rows, a.C, a.branch}};
    const Span outs[] = {{"x_out", a.x_out, n, a.C, a.stream}, {"h", a.h, n, a.C, a.branch}};
    if ((st = check_overlaps(outs, 2, ins, 3)) != FPSTOK_OK) return st;
    if (s->num_seqs == 0 || n == 0) return ok();
    a.stats = stats;
    plan_residual(a, false);
    const hipError_t e = launch_residual(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "residual step kernel launch");
    return ok();
}

FPSTOK_API fpstok_status fpstok_residual_backward(
    const fpstok_seqs* s, const fpstok_residual_params* p, const fpstok_residual_weights* w,
    const fpstok_rows* x, const fpstok_rows* y, const fpstok_rows* gate, const float* stats,
    const fpstok_rows* grad_x_out, const fpstok_rows* grad_h, const fpstok_rows* grad_x,
    const fpstok_rows* grad_y, const fpstok_rows* grad_gate,
    const fpstok_residual_weight_grads* grads, void* ws, size_t ws_bytes, void* stream) {
    fpstok_status st = check_residual(s, p);
    if (st != FPSTOK_OK) return st;
    ResidualArgs a{};
    if ((st = check_inputs(s, p, w, x, y, gate, a)) != FPSTOK_OK) return st;
    const int64_t n = s->num_rows;
    if (!grad_x_out && !grad_h) return fail(FPSTOK_EINVAL, "grad_x_out and grad_h are NULL");
    if (grad_h && a.pre == FPSTOK_NORM_NONE)
        return fail(FPSTOK_EINVAL, "grad_h without pre_norm");
    if (grad_y && !y) return fail(FPSTOK_EINVAL, "grad_y without y");
    if (grad_gate && !gate) return fail(FPSTOK_EINVAL, "grad_gate without gate");
    const int64_t gate_rows = a.gate_per == FPSTOK_GATE_SEQUENCE ? s->num_seqs : n;
    struct {
        const fpstok_rows* v;
        const char* name;
        int64_t rows;
        int dtype;
        bool output;
        RowsArg* to;
    } views[] = {{grad_x_out, "grad_x_out", n, a.stream, false, &a.grad_x_out},
                 {grad_h, "grad_h", n, a.branch, false, &a.grad_h},
                 {grad_x, "grad_x", n, a.stream, true, &a.grad_x},
                 {grad_y, "grad_y", n, a.branch, true, &a.grad_y},
                 {grad_gate, "grad_gate", gate_rows, a.branch, true, &a.grad_gate}};
    for (const auto& v : views)
        if (v.v && (st = check_rows(v.v, v.name, v.rows, a.C, v.dtype, v.output, *v.to)) !=
                       FPSTOK_OK)
            return st;
    if (n > 1 && a.grad_x.data && a.grad_x.data == a.grad_x_out.data &&
        a.grad_x.row != a.grad_x_out.row)
        return fail(FPSTOK_EINVAL, "grad_x in place of grad_x_out needs the same stride");
    int given = 0;
    if (grads) {
        float* to[kResidualWeights] = {grads->post_weight, grads->post_bias, grads->scale,
                                       grads->pre_weight, grads->pre_bias};
        const char* names[kResidualWeights] = {"grad of post_weight", "grad of post_bias",
                                               "grad of scale", "grad of pre_weight",
                                               "grad of pre_bias"};
        for (int k = 0; k < kResidualWeights; ++k) {
            if ((st = check_weight(to[k], names[k], a.weights[k] != nullptr)) != FPSTOK_OK)
                return st;
            a.weight_grads[k] = to[k];
            given += to[k] != nullptr;
        }
    }
    if (n > 0 && s->num_seqs > 0 && !stats &&
        (a.post != FPSTOK_NORM_NONE || a.pre != FPSTOK_NORM_NONE))
        return fail(FPSTOK_EINVAL, "stats is NULL");
    if (((uintptr_t)stats & 15u) != 0)
        return fail(FPSTOK_EINVAL, "stats must be 16-byte aligned");
    a.stats = const_cast<float*>(stats);
    plan_residual(a, true);
    const bool gates = a.gate_per == FPSTOK_GATE_SEQUENCE;
    const size_t need = lay_out(a, kResidualWeights, gates, ws);
    if ((st = check_ws(need, ws, ws_bytes)) != FPSTOK_OK) return st;
    const Span ins[] = {{"x", a.x, n, a.C, a.stream},
                        {"y", a.y, n, a.C, a.branch},
                        {"gate", a.gate, gate_rows, a.C, a.branch},
                        {"grad_x_out", a.grad_x_out, n, a.C, a.stream},
                        {"grad_h", a.grad_h, n, a.C, a.branch}};
    const Span outs[] = {{"grad_x", a.grad_x, n, a.C, a.stream},
                         {"grad_y", a.grad_y, n, a.C, a.branch},
                         {"grad_gate", a.grad_gate, gate_rows, a.C, a.branch}};
    if ((st = check_overlaps(outs, 3, ins, 5)) != FPSTOK_OK) return st;
    lay_out(a, given, gates, ws);
    if (s->num_seqs == 0) a.runs = 0;  // no row is one of a sequence: zeros
    const hipError_t e = launch_residual_backward(a, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "residual step gradient kernel launch");
    return ok();
}
