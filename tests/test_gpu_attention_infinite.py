"""GPU tests of attention and its gradients where infinite inputs are seen.

A score of -infinity (a key or a query with one -infinite element that meets
elements of one sign) has weight 0: the key adds nothing to its queries, and a
query whose every visible score is -infinity counts as one that sees no key.
What is left is compared with the reference of the same inputs with those
pairs hidden, whether the kernels see a tile whole or in part."""
import numpy as np
import pytest
import torch

from tests import attention_ref as ref
from tests.gpu_util import log
from tests.test_gpu_attention import DT, F, layout, rand  # noqa: F401

pytestmark = pytest.mark.gpu

INF = float("inf")


def reference(hide, *args, **kw):
    """ref.attention with the pairs hide(tq, tk) (True: hidden) added to the
    mask."""
    keep = ref.visible
    try:
        ref.visible = lambda tq, tk, *w: keep(tq, tk, *w) & ~hide(tq, tk)
        return ref.attention(*args, **kw)
    finally:
        ref.visible = keep


# lengths, keys' lengths, H, Hk, window, sinks: one tile seen in part; whole
# tiles; several of them with a rest; masks; rows split over workgroups; sinks of
# rows past the window; a walk split over workgroups
SHAPES = [
    ([50], None, 4, 2, (-1, -1), 0),
    ([256], None, 4, 2, (-1, -1), 0),
    ([200], None, 3, 3, (-1, -1), 0),
    ([200], None, 4, 2, (-1, 0), 0),
    ([150], None, 2, 2, (8, 4), 2),
    ([700], None, 2, 1, (100, 0), 4),
    ([600], None, 8, 1, (-1, -1), 0),
    ([1], [900], 4, 2, (-1, -1), 0),
    ([3], [2500], 4, 1, (-1, -1), 0),
]


def inputs(F, shape, D, dtype, seed):  # noqa: F811
    lens, k_lens, H, Hk, window, sinks = shape
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    qs, q_seq, n = layout(F, lens, "packed")
    ks, k_seq, m = (None, q_seq, n) if k_lens is None else layout(F, k_lens, "packed")
    q, k, v, go = (rand(gen, (r, h, D), dt) for r, h in ((n, H), (m, Hk), (m, Hk), (n, H)))
    # element 3 of both is positive: an infinite one gives scores of one sign
    q[..., 3] = q[..., 3].abs() + 0.5
    k[..., 3] = k[..., 3].abs() + 0.5
    return qs, ks, q_seq, k_seq, q, k, v, go


def compute(F, shape, qs, ks, q, k, v, go):  # noqa: F811
    att = F.Attention(q.cuda(), k.cuda(), v.cuda(), qs, ks, shape[4], shape[5], None, True)
    out, lse = att()
    grads = att.backward(go.cuda())
    torch.cuda.synchronize()
    return dict(zip(("out", "lse", "grad_q", "grad_k", "grad_v"), (out, lse) + grads))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [40, 64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_seen_key_of_score_minus_infinity(F, shape, D, dtype):  # noqa: F811
    log("infinite key %s D=%d %s" % (shape, D, dtype))
    qs, ks, q_seq, k_seq, q, k, v, go = inputs(F, shape, D, dtype, 81)
    m = k.shape[0]
    keys = sorted({m // 3, m // 2, m - 1})
    fixed = k.clone()
    fixed[keys, :, 3] = 0.0
    k[keys, :, 3] = -INF

    def hide(tq, tk):
        h = np.zeros((tq, tk), dtype=bool)
        h[:, keys] = True
        return h

    got = compute(F, shape, qs, ks, q, k, v, go)
    want = reference(hide, q, fixed, v, q_seq, k_seq, *shape[4], shape[5], grad=go)
    # grad_q's own element 3 is 0 times -infinity in rows that see such a key
    # beside others, and no other element is touched
    sees = ref.visible(q.shape[0], m, *shape[4], shape[5])
    rows = sees[:, keys].any(1) & np.delete(sees, keys, 1).any(1)
    gq = got["grad_q"].float().cpu()
    assert bool(torch.isnan(gq[torch.from_numpy(rows)][..., 3]).all())
    val, tol = want["grad_q"]
    clean = gq.to(DT[dtype])
    clean[torch.from_numpy(rows), :, 3] = torch.from_numpy(val)[rows, :, 3].to(DT[dtype])
    got["grad_q"] = clean
    for name, t in got.items():
        ref.check(t, want[name], name)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [40, 64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("bad_grad", [False, True])
def test_query_whose_scores_are_minus_infinity(F, shape, D, dtype, bad_grad):  # noqa: F811
    """It gets 0 and -infinity, and adds nothing to any gradient, whatever its
    own gradient is."""
    log("infinite query %s D=%d %s %s" % (shape, D, dtype, bad_grad))
    qs, ks, q_seq, k_seq, q, k, v, go = inputs(F, shape, D, dtype, 82)
    n = q.shape[0]
    rows = sorted({n // 3, n // 2, n - 1})
    fixed, fixed_go = q.clone(), go.clone()
    q[rows, :, 3] = -INF
    fixed[rows, :, 3] = 0.0
    if bad_grad:
        go[rows[:1]], go[rows[1:], :, 5] = INF, float("nan")
        fixed_go[rows] = 0.0

    def hide(tq, tk):
        h = np.zeros((tq, tk), dtype=bool)
        h[rows] = True
        return h

    got = compute(F, shape, qs, ks, q, k, v, go)
    want = reference(hide, fixed, k, v, q_seq, k_seq, *shape[4], shape[5], grad=fixed_go)
    for name, t in got.items():
        ref.check(t, want[name], name)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [0, 2])
def test_key_seen_by_such_queries_only(F, D, dtype, sinks):  # noqa: F811
    """Its gradients are 0, whatever it and its value hold."""
    log("infinite pairs D=%d %s sinks %d" % (D, dtype, sinks))
    shape = ([300], None, 4, 2, (0, 0), sinks)
    qs, ks, q_seq, k_seq, q, k, v, go = inputs(F, shape, D, dtype, 85)
    rows = [5, 100, 131, 299]
    fixed = [t.clone() for t in (q, k, v, go)]
    q[rows, :, 3], k[rows[1:], :, 3] = -INF, INF
    v[rows, :, 4], go[rows, :, 5] = INF, -INF
    for t in fixed:
        t[rows] = 0.0

    def hide(tq, tk):
        h = np.zeros((tq, tk), dtype=bool)
        h[rows] = True
        return h

    got = compute(F, shape, qs, ks, q, k, v, go)
    want = reference(hide, *fixed[:3], q_seq, k_seq, *shape[4], shape[5], grad=fixed[3])
    for name, t in got.items():
        ref.check(t, want[name], name)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_such_a_query_sees_infinite_values(F, shape, D, dtype):  # noqa: F811
    """Its result is 0 whatever the values are."""
    log("infinite values %s D=%d %s" % (shape, D, dtype))
    qs, ks, _, _, q, k, v, _ = inputs(F, shape, D, dtype, 83)
    n = q.shape[0]
    rows = sorted({n // 3, n - 1})
    q[rows, :, 3] = -INF
    v[..., 1], v[..., 2] = INF, float("nan")
    att = F.Attention(q.cuda(), k.cuda(), v.cuda(), qs, ks, shape[4], shape[5])
    att.out.fill_(7.0)
    out, lse = att()
    torch.cuda.synchronize()
    assert bool((out[rows] == 0).all()) and bool((lse[rows] == -INF).all())
    others = [r for r in range(n) if r not in rows]
    if others:
        assert not bool(torch.isfinite(out[others][..., 1:3].float()).any())
        assert bool(torch.isfinite(out[others][..., 3:].float()).all())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_seen_infinite_element_of_grad_out(F, shape, D, dtype):  # noqa: F811
    """grad_v is infinite where the element meets a weight, grad_k wherever
    the row is seen, and nothing else is touched."""
    log("infinite gradient %s D=%d %s" % (shape, D, dtype))
    qs, ks, q_seq, k_seq, q, k, v, go = inputs(F, shape, D, dtype, 84)
    n, m, Hk = q.shape[0], k.shape[0], k.shape[1]
    row = n - 1 - n // 4
    go[row, 0, 7] = INF
    fixed = go.clone()
    fixed[row, 0, 7] = 0.0
    got = compute(F, shape, qs, ks, q, k, v, go)
    want = ref.attention(q, k, v, q_seq, k_seq, *shape[4], shape[5], grad=fixed)
    seen = torch.from_numpy(ref.visible(n, m, *shape[4], shape[5])[row])
    touched = torch.zeros((m, Hk), dtype=torch.bool)
    touched[:, 0] = seen
    gv, gk, gq = (got[x].float().cpu() for x in ("grad_v", "grad_k", "grad_q"))
    assert not bool(torch.isfinite(gv[touched][:, 7]).any())
    assert not bool(torch.isfinite(gk[touched]).any())
    assert not bool(torch.isfinite(gq[row, 0]).any())
    for name, t, hit in (("grad_v", gv, (touched, slice(7, 8))),
                         ("grad_k", gk, (touched, slice(None))),
                         ("grad_q", gq, None)):
        val, tol = (torch.from_numpy(x) for x in want[name])
        if hit is None:
            t[row, 0] = val[row, 0].float()
            tol[row, 0] = INF
        else:
            tol[hit[0]] = torch.where(torch.arange(D)[None].ge(hit[1].start or 0) &
                                      torch.arange(D)[None].lt(hit[1].stop or D),
                                      torch.full((1, D), INF, dtype=torch.float64), tol[hit[0]])
            t = torch.where(torch.isinf(tol), torch.zeros_like(t), t)
        ref.check(t, (val.numpy(), tol.numpy()), name)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [40, 64, 128])
def test_seen_sink_of_score_minus_infinity(F, D, dtype):  # noqa: F811
    """Among the sinks, whose gradients the rows past the window give in
    chunks, beside queries that add nothing."""
    log("infinite sink D=%d %s" % (D, dtype))
    shape = ([777], None, 4, 2, (60, 0), 5)
    qs, ks, q_seq, k_seq, q, k, v, go = inputs(F, shape, D, dtype, 86)
    keys, rows = [1, 3], [250, 640, 776]
    # (an element of their own for the queries: beside the keys' it would be +infinity)
    k[..., 5] = k[..., 5].abs() + 0.5
    fk, fq = k.clone(), q.clone()
    fk[keys, :, 3], fq[rows, :, 5] = 0.0, 0.0
    k[keys, :, 3], q[rows, :, 5] = -INF, -INF

    def hide(tq, tk):
        h = np.zeros((tq, tk), dtype=bool)
        h[:, keys], h[rows] = True, True
        return h

    got = compute(F, shape, qs, ks, q, k, v, go)
    want = reference(hide, fq, fk, v, q_seq, k_seq, *shape[4], shape[5], grad=go)
    sees = ref.visible(777, 777, 60, 0, 5)[:, keys].any(1)
    sees &= np.delete(ref.visible(777, 777, 60, 0, 5), keys, 1).any(1)
    sees[rows] = False
    sees = torch.from_numpy(sees)
    gq = got["grad_q"].cpu()
    assert bool(torch.isnan(gq[sees][..., 3].float()).all())
    gq[sees, :, 3] = torch.from_numpy(want["grad_q"][0])[sees, :, 3].to(DT[dtype])
    got["grad_q"] = gq
    for name, t in got.items():
        ref.check(t, want[name], name)
