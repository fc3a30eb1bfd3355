"""The residual step and its gradients from their definitions, in float64 on the
CPU, with the bound of tests/rounding.py on how far a result of the library may
be off."""
import numpy as np
import torch

from tests.attention_ref import half_step, tiny
from tests.rounding import F, Val

# a thread's 8 elements, 6 exchanges in a wave, 16 waves: the depth of a sum over columns
DEPTH = 8 + 6 + 16 + 2
KEYS = ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")


def _norm(x, kind, eps):
    """The normed rows and 1 / std (None without a norm)."""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(DEPTH)
    r = ((x * x).mean(DEPTH) + Val(np.float32(eps))).rsqrt()
    return x * r, r


def _affine(x, w, b):
    x = x if w is None else x * w
    return x if b is None else x + b


def _norm_grad(p, xh, r, kind):
    c1 = (p * xh).mean(DEPTH)
    if kind == "layer":
        p = p - p.mean(DEPTH)
    return r * (p - xh * c1)


def _act(g, name):
    """The gate and its derivative.  exp(-g) as 2^x with x = -g log2(e) rounded is off
    by |g| f, exp2 by a step, the sum by half a step, the reciprocal by a step:
    (|g| + 6) f at most; a result below 2^-126 may come out as 0."""
    if name == "none":
        return Val(g), Val(np.ones_like(g))
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    s = Val(s, (np.abs(np.clip(g, -200, 200)) + 6) * F * s + 2.0 ** -126)
    d = s * (Val(1.0) - s)
    if name == "sigmoid":
        return s, d
    return Val(g) * s, Val(g) * d + s


def residual(x, y, seqs, gate=None, gate_per="none", activation="none", post_norm="none",
             pre_norm="rms", eps=1e-6, grad_x_out=None, grad_h=None, **weights):
    """x, y, ... CPU tensors of the call's types; seqs: [(first row, length)].
    Returns {name: (value, bound)}: x_out, h and, with a gradient given, grad_*;
    rows in no sequence hold 0 with bound 0."""
    w = {k: None if weights.get(k) is None else Val(weights[k].double().numpy()) for k in KEYS}
    n, C = x.shape
    branch = x if y is None else y
    rows = np.concatenate([np.arange(r0, r0 + k) for r0, k in seqs] or [[]]).astype(np.int64)
    member = np.repeat(np.arange(len(seqs)), [k for _, k in seqs])
    get = lambda t: Val(t.double().numpy()[rows])  # noqa: E731
    res = {}

    def put(name, val, like):
        val = val.rounded(half_step(like.dtype), tiny(like.dtype))
        v, e = np.zeros((n, C)), np.zeros((n, C))
        v[rows], e[rows] = val.v, val.e
        res[name] = (v, e)

    xo, act, slope, u = get(x), None, None, None
    if y is not None:
        yh, ry = _norm(get(y), post_norm, eps)
        u = _affine(yh, w["post_weight"], w["post_bias"])
        z = u
        if gate is not None:
            g = gate.double().numpy()
            act, slope = _act(g[rows] if gate_per == "row" else g[member], activation)
            z = u * act
        xo = xo + (z if w["scale"] is None else z * w["scale"])
    put("x_out", xo, x)
    if pre_norm != "none":
        xh, rx = _norm(xo, pre_norm, eps)
        put("h", _affine(xh, w["pre_weight"], w["pre_bias"]), branch)
    if grad_x_out is None and grad_h is None:
        return res

    adds = max(1, len(rows)) + 8

    def weight(name, val):
        if w[name] is not None:
            s = val.sum(0, adds).rounded(F, 2.0 ** -150)
            res["grad_" + name] = (s.v, s.e)

    zero = Val(np.zeros((len(rows), C)))
    gx = zero if grad_x_out is None else get(grad_x_out)
    gh = zero
    if grad_h is not None:
        gh = get(grad_h)
        p = gh if w["pre_weight"] is None else gh * w["pre_weight"]
        gx = gx + _norm_grad(p, xh, rx, pre_norm)
    if pre_norm != "none":
        weight("pre_weight", gh * xh)
        weight("pre_bias", gh)
    put("grad_x", gx, x)
    if y is None:
        return res
    weight("scale", gx * (u if act is None else u * act))
    gz = gx if w["scale"] is None else gx * w["scale"]
    gu = gz
    if gate is not None:
        gg = gz * u * slope
        gu = gz * act
        if gate_per == "row":
            put("grad_gate", gg, gate)
        else:
            v, e = np.zeros((len(seqs), C)), np.zeros((len(seqs), C))
            for b, (_, k) in enumerate(seqs):
                part = Val(gg.v[member == b], gg.e[member == b]).sum(0, k + 8)
                part = part.rounded(half_step(gate.dtype), tiny(gate.dtype))
                v[b], e[b] = part.v, part.e
            res["grad_gate"] = (v, e)
    if post_norm != "none":
        weight("post_weight", gu * yh)
        weight("post_bias", gu)
        q = gu if w["post_weight"] is None else gu * w["post_weight"]
        gu = _norm_grad(q, yh, ry, post_norm)
    put("grad_y", gu, y)
    return res


def make(rows, C, sequences, stream, branch, gate_per, post_norm, pre_norm, scale, seed,
         block=True):
    """Random CPU operands of one call."""
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    o = dict(x=(2 * normal(rows, C)).to(stream),
             y=normal(rows, C).to(branch) if block else None,
             gate=None, gate_per=gate_per, post_norm=post_norm, pre_norm=pre_norm)
    if gate_per != "none":
        o["gate"] = normal(rows if gate_per == "row" else sequences, C).to(branch)
    if post_norm != "none":
        o["post_weight"] = 1 + 0.2 * normal(C)
    if post_norm == "layer":
        o["post_bias"] = 0.1 * normal(C)
    if scale:
        o["scale"] = 0.5 + 0.2 * normal(C)
    if pre_norm != "none":
        o["pre_weight"] = 1 + 0.2 * normal(C)
    if pre_norm == "layer":
        o["pre_bias"] = 0.1 * normal(C)
    grads = dict(grad_x_out=normal(rows, C).to(stream))
    if pre_norm != "none":
        grads["grad_h"] = normal(rows, C).to(branch)
    return o, grads
