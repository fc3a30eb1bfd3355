"""Attention with a learned bias by buckets of distance from its definition, in
float64 on the CPU (buckets: the float32 operations that define them), with a
bound on how far a result of the library may be off.

The bounds are those of tests/attention_ref.py with the bias in the score: per
axis the entry is scaled and added (two roundings of at most E + B, where B
bounds the entries' sum), the score's own scaling one more.  grad_table is a
float32 result of unrounded terms: with n keys, off = the rows' sum of dS, which
takes delta's error back out, it is off by

* per pair w (r M + (D + 4) f |g| |v| + 4 f (|dp| + |delta| + e)), where e is
  the error of delta as formed from the rounded out and M = |dp - delta| + e;
* per row and pair of it w times what off is off by: the sum of those over the
  row and (n + 8) f sum w M, and r e for weights that do not add up to 1;
* (n + 140) f sum w M for the additions (up to n in a lane, 128 rows of a tile;
  tiles are added in float64), and one rounding;
* 2^-126 (M + 1) per pair: a weight, and a sum, below the smallest normal number
  may come out as 0.  (Entries 1000 apart: an entry's exact gradient is 1e-152
  where the weights, exp(-350) and less, are no float32 numbers.)
"""
import math

import numpy as np
import torch

from tests.attention_ref import F32, half_step, tiny, visible


def buckets(q_pos, k_pos, axis):
    """[Tq, Tk] buckets of one axis (a BiasAxis)."""
    f = np.float32
    rate, shift = f(axis.rate), f(axis.shift)
    with np.errstate(all="ignore"):
        if q_pos.dtype == np.int32:
            d = (k_pos[None].astype(np.int64) - q_pos[:, None]).astype(f) * rate
        else:
            d = (k_pos * rate)[None] - (q_pos * rate)[:, None]
        if axis.log_steps:
            m, e = np.frexp(f(1) + np.abs(d))  # t = m 2^e, m in [1/2, 1)
            L = (e - 1.0) * axis.log_steps + np.floor(axis.log_steps * (2.0 * m - 1.0))
            b = float(shift) + np.where(d < 0, -L, L)
        else:
            b = np.floor(d + shift).astype(np.float64)
    # (a distance that is not a number: any bucket)
    return np.clip(np.nan_to_num(b, nan=0.0), 0, axis.buckets - 1).astype(np.int64)


def attention(q, k, v, q_seq, k_seq, table, axes, q_pos, k_pos=None, left=-1, right=-1, sinks=0,
              scale=None, grad=None):
    """As attention_ref.attention, with table [H, buckets] and positions [rows,
    axes] as CPU tensors; also grad_table with a gradient."""
    dt = q.dtype
    u, t = half_step(dt), tiny(dt)
    uw, tw = (0.0, 0.0) if dt == torch.float32 else (u, t)
    Q, K, V = (x.double().numpy() for x in (q, k, v))
    T = table.double().numpy()
    T = np.where(T <= np.float64(np.float32(-1e30)), -np.inf, T)
    H, Hk, D = Q.shape[1], K.shape[1], Q.shape[2]
    A, first = len(axes), np.cumsum([0] + [a.buckets for a in axes])
    qp = q_pos.numpy()
    kp = qp if k_pos is None else k_pos.numpy()
    scale = np.float64(np.float32(1.0 / math.sqrt(D) if scale is None else scale))
    res = {n: np.zeros(s) for n, s in (("out", Q.shape), ("lse", Q.shape[:2]))}
    tol = {n: np.zeros_like(x) for n, x in res.items()}
    if grad is not None:
        Gr = grad.double().numpy()
        for n, x in (("grad_q", Q), ("grad_k", K), ("grad_v", V), ("grad_table", T)):
            res[n], tol[n] = np.zeros_like(x), np.zeros_like(x)
    for (q0, tq), (k0, tk) in zip(q_seq, k_seq):
        if tq == 0:
            continue
        seen = visible(tq, tk, left, right, sinks)
        entry = [first[a] + buckets(qp[q0:q0 + tq, a], kp[k0:k0 + tk, a], axes[a])
                 for a in range(A)]
        for h in range(H):
            hk = h // (H // Hk)
            qs, ks, vs = Q[q0:q0 + tq, h], K[k0:k0 + tk, hk], V[k0:k0 + tk, hk]
            bias = sum(T[h][e] for e in entry)
            ok = seen & (bias > -np.inf)
            some = ok.any(1) if tk else np.zeros(tq, dtype=bool)
            n = max(1, int(ok.sum(1).max()) if tk else 1)
            if not some.any():
                res["lse"][q0:q0 + tq, h] = -np.inf
                continue
            s = np.where(ok, qs @ ks.T * scale + np.where(ok, bias, 0.0), -np.inf)
            E = scale * (np.abs(qs) @ np.abs(ks).T)
            E = np.where(ok, E, 0.0).max(1)
            B = np.where(ok, sum(np.abs(T[h][e]) for e in entry), 0.0).max(1)
            EB = E + B
            top = np.where(some, s.max(1), 0.0)
            e = np.exp(s - top[:, None])
            tot = e.sum(1)
            w = e / np.where(some, tot, 1.0)[:, None]
            with np.errstate(divide="ignore"):
                lse = np.where(some, top + np.log(tot), -np.inf)
            e_s = (D + 4) * F32 * E + (2 * A + 4) * F32 * EB
            r = 2 * e_s + 4 * EB * F32 + (n + 16) * F32
            out = w @ vs
            absv = w @ np.abs(vs)
            e_out = (r + uw + (n + 4) * F32)[:, None] * absv + tw * np.abs(vs).sum(0) + \
                u * np.abs(out) + t
            e_out[~some] = 0.0
            res["out"][q0:q0 + tq, h] = out
            tol["out"][q0:q0 + tq, h] = e_out
            res["lse"][q0:q0 + tq, h] = lse
            tol["lse"][q0:q0 + tq, h] = e_lse = np.where(
                some, e_s + (n + 16) * F32 + 4 * F32 * (np.abs(lse) + EB), 0.0)
            if grad is None:
                continue
            g = Gr[q0:q0 + tq, h]
            dp = g @ vs.T
            delta = (g * out).sum(1)
            ds = w * (dp - delta[:, None])
            e_delta = (np.abs(g) * e_out).sum(1) + (D + 4) * F32 * (np.abs(g) * np.abs(out)).sum(1)
            # the stored log-sum-exp's own error enters every weight
            rw = r + e_lse + 4 * F32 * np.where(some, np.abs(lse), 0.0)
            gv = (D + 4) * F32 * (np.abs(g) @ np.abs(vs).T)
            e_ds = w * (rw[:, None] * np.abs(dp - delta[:, None]) + gv + e_delta[:, None] +
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
            M = np.abs(dp - delta[:, None]) + e_delta[:, None]
            pair = w * (rw[:, None] * M + gv + 4 * F32 * (np.abs(dp) + np.abs(delta)[:, None] +
                                                          e_delta[:, None]))
            pair += np.where(ok, 2.0 ** -126 * (M + 1), 0.0)
            e_off = pair.sum(1) + (n + 8) * F32 * (w * M).sum(1) + rw * e_delta
            term = pair + w * e_off[:, None] + (n + 140) * F32 * w * M
            for x in entry:
                res["grad_table"][h] += np.bincount(x.ravel(), ds.ravel(), T.shape[1])
                tol["grad_table"][h] += np.bincount(x.ravel(), term.ravel(), T.shape[1])
    if grad is not None:
        for n in ("grad_k", "grad_v"):
            inside = np.zeros(K.shape[0], dtype=bool)
            for k0, tk in k_seq:
                inside[k0:k0 + tk] = True
            tol[n] += np.where(inside[:, None, None], u * np.abs(res[n]) + t, 0.0)
        tol["grad_table"] += F32 * np.abs(res["grad_table"])
    return {n: (res[n], tol[n]) for n in res}
