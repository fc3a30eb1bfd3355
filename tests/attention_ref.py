"""Attention over sequences and rotary positions from their definitions, in
float64 on the CPU, with a bound on how far a result of the library may be
off.

The bounds count roundings.  With u = eps/2 of the views' type (one rounding
is off by at most u relative, plus half the smallest subnormal), f = 2^-24,
and, for a query i and the keys j it sees, E = scale * sum_d |q_d k_d|:

* a score is a float32 sum of D products and two multiplications:
  |ds| <= (D + 4) f E;  a weight exp(s - max) / sum adds the exponent's
  rounding (|s - max| f, at most 2 E f), exp2 and the sum's n additions:
  relative error r = 2 (D + 4) f E + 4 E f + (n + 16) f;
* out: weights rounded to the type (u; float32 keeps them), n additions, one
  final rounding:  (r + u_w + (n + 4) f) sum w |v| + u |out|;
* delta = sum g out inherits out's error; ds = w (g v - delta) adds its own
  rounding u_w; every gradient is a float32 sum of such terms, rounded once.

u_w is 0 for float32 views.  Every term enters with its absolute value, so the
bound holds whatever the order of the sums.
"""
import math

import numpy as np
import torch

F32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the smallest subnormal."""
    info = torch.finfo(dtype)
    return info.tiny * info.eps / 2


def visible(tq, tk, left, right, sinks):
    p = np.arange(tq)[:, None] + (tk - tq)
    j = np.arange(tk)[None]
    ok = np.ones((tq, tk), dtype=bool)
    if right >= 0:
        ok &= j <= p + right
    if left >= 0:
        ok &= (j >= p - left) | (j < sinks)
    return ok


def attention(q, k, v, q_seq, k_seq, left=-1, right=-1, sinks=0, scale=None, grad=None):
    """q [rows, H, D] etc. as CPU tensors of the call's dtype; q_seq, k_seq:
    lists of (first row, length).  Returns {name: (value, bound)} in float64
    numpy for out, lse and, with grad, grad_q, grad_k, grad_v; rows in no
    sequence hold 0 with bound 0."""
    dt = q.dtype
    u, t = half_step(dt), tiny(dt)
    uw, tw = (0.0, 0.0) if dt == torch.float32 else (u, t)
    Q, K, V = (x.double().numpy() for x in (q, k, v))
    H, Hk, D = Q.shape[1], K.shape[1], Q.shape[2]
    scale = np.float64(np.float32(1.0 / math.sqrt(D) if scale is None else scale))
    res = {n: np.zeros(s) for n, s in (("out", Q.shape), ("lse", Q.shape[:2]))}
    tol = {n: np.zeros_like(x) for n, x in res.items()}
    if grad is not None:
        Gr = grad.double().numpy()
        for n, x in (("grad_q", Q), ("grad_k", K), ("grad_v", V)):
            res[n], tol[n] = np.zeros_like(x), np.zeros_like(x)
    for (q0, tq), (k0, tk) in zip(q_seq, k_seq):
        if tq == 0:
            continue
        ok = visible(tq, tk, left, right, sinks)
        some = ok.any(1) if tk else np.zeros(tq, dtype=bool)
        n = max(1, int(ok.sum(1).max()) if tk else 1)
        for h in range(H):
            hk = h // (H // Hk)
            qs, ks, vs = Q[q0:q0 + tq, h], K[k0:k0 + tk, hk], V[k0:k0 + tk, hk]
            if not some.any():
                res["lse"][q0:q0 + tq, h] = -np.inf
                continue
            s = np.where(ok, qs @ ks.T * scale, -np.inf)
            E = scale * (np.abs(qs) @ np.abs(ks).T)
            E = np.where(ok, E, 0.0).max(1)
            top = np.where(some, s.max(1), 0.0)
            e = np.exp(s - top[:, None])
            tot = e.sum(1)
            w = e / np.where(some, tot, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                lse = np.where(some, top + np.log(tot), -np.inf)
            r = 2 * (D + 4) * F32 * E + 4 * E * F32 + (n + 16) * F32
            out = w @ vs
            absv = w @ np.abs(vs)
            e_out = (r + uw + (n + 4) * F32)[:, None] * absv + tw * np.abs(vs).sum(0) + \
                u * np.abs(out) + t
            e_out[~some] = 0.0
            res["out"][q0:q0 + tq, h] = out
            tol["out"][q0:q0 + tq, h] = e_out
            res["lse"][q0:q0 + tq, h] = lse
            tol["lse"][q0:q0 + tq, h] = np.where(
                some, (D + 4) * F32 * E + (n + 16) * F32 + 4 * F32 * (np.abs(lse) + E), 0.0)
            if grad is None:
                continue
            g = Gr[q0:q0 + tq, h]
            dp = g @ vs.T
            delta = (g * out).sum(1)
            ds = w * (dp - delta[:, None])
            e_delta = (np.abs(g) * e_out).sum(1) + (D + 4) * F32 * (np.abs(g) * np.abs(out)).sum(1)
            # the stored log-sum-exp's own error enters every weight
            rw = r + tol["lse"][q0:q0 + tq, h] + 4 * F32 * np.where(some, np.abs(lse), 0.0)
            e_ds = w * (rw[:, None] * np.abs(dp - delta[:, None]) +
                        (D + 4) * F32 * (np.abs(g) @ np.abs(vs).T) + e_delta[:, None] +
                        2 * F32 * (np.abs(dp) + np.abs(delta)[:, None]))
            e_ds = e_ds * (1 + uw) + uw * np.abs(ds) + np.where(ok, tw, 0.0)
            e_w = w * (rw[:, None] + uw) + np.where(ok, tw, 0.0)
            m = H // Hk * tq
            res["grad_q"][q0:q0 + tq, h] = dq = scale * (ds @ ks)
            tol["grad_q"][q0:q0 + tq, h] = scale * (
                (e_ds + (n + 4) * F32 * np.abs(ds)) @ np.abs(ks)) + u * np.abs(dq) + t
            res["grad_k"][k0:k0 + tk, hk] += scale * (ds.T @ qs)
            tol["grad_k"][k0:k0 + tk, hk] += scale * (
                (e_ds + (m + 4) * F32 * np.abs(ds)).T @ np.abs(qs))
            res["grad_v"][k0:k0 + tk, hk] += w.T @ g
            tol["grad_v"][k0:k0 + tk, hk] += (e_w + (m + 4) * F32 * w).T @ np.abs(g)
    if grad is not None:
        for n in ("grad_k", "grad_v"):
            inside = np.zeros(K.shape[0], dtype=bool)
            for k0, tk in k_seq:
                inside[k0:k0 + tk] = True
            tol[n] += np.where(inside[:, None, None], u * np.abs(res[n]) + t, 0.0)
    return {n: (res[n], tol[n]) for n in res}


def rope(x, positions, freqs, pairs, interleaved=False, inverse=False):
    """Value and bound of the rotation: cos and sin are off by at most 2^-23
    each (a float32 angle remainder and a polynomial), the turn is two
    products and a sum in float32, rounded once.  Each of the three float32
    operations may also round a subnormal result, off by at most 2^-150: a
    value near 8e-41 was off by 8.6e-46 = 0.6 * 2^-149 with a bound of one
    such rounding."""
    X = x.double().numpy()
    u, t = half_step(x.dtype), tiny(x.dtype)
    axis = np.repeat(np.arange(len(pairs)), pairs)
    R = axis.size
    ang = positions.double().numpy()[:, axis] * freqs.double().numpy()
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1.0 if inverse else 1.0)
    i1 = 2 * np.arange(R) if interleaved else np.arange(R)
    i2 = i1 + 1 if interleaved else i1 + R
    y, e = X.copy(), np.zeros_like(X)
    a, b = X[..., i1], X[..., i2]
    y[..., i1], y[..., i2] = a * c - b * s, a * s + b * c
    mag = (np.abs(a) + np.abs(b)) * (2.0 ** -23 + 3 * F32) + 3 * 2.0 ** -150
    for i in (i1, i2):
        e[..., i] = mag + u * np.abs(y[..., i]) + t
    return y, e


def check(got, ref, what):
    """got within ref's bound, element by element; infinities must agree."""
    val, tol = ref
    got = got.double().cpu().numpy()
    assert got.shape == val.shape, what
    inf = np.isinf(val)
    assert np.array_equal(got[inf], val[inf]), "%s: infinities differ" % what
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - val) <= tol) & ~inf
    if bad.any():
        at = np.argwhere(bad)
        i = tuple(at[0])
        raise AssertionError("%s: %d of %d outside the bound, first at %s: got %r ref %r bound %r" % (
            what, len(at), val.size, i, got[i], val[i], tol[i]))
