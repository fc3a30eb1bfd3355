"""GPU tests that attention, its gradients and their workspace stay inside the
buffers whatever the lengths on the device say, and write where they are told
to."""
import ctypes

import numpy as np
import pytest
import torch

from tests.gpu_util import log
from tests.test_gpu_attention import DT, F, layout, rand  # noqa: F401

pytestmark = pytest.mark.gpu

GUARD, MARK = 64, 7.0


class Guarded:
    """A buffer of `shape` with rows of MARK around it."""

    def __init__(self, shape, dtype):
        self.store = torch.full((shape[0] + 2 * GUARD,) + tuple(shape[1:]), MARK, dtype=dtype,
                                device="cuda")
        self.t = self.store[GUARD:GUARD + shape[0]]

    def check(self, what):
        n = self.t.shape[0]
        assert bool((self.store[:GUARD] == MARK).all()), "%s: written ahead of it" % what
        assert bool((self.store[GUARD + n:] == MARK).all()), "%s: written behind it" % what


def call(F, qs, ks, q, k, v, go, window, sinks):  # noqa: F811
    """Forward and gradients through the C ABI into guarded buffers (the
    workspace of exactly the size asked for among them)."""
    (nq, H, D), (nk, Hk, _) = q.shape, k.shape
    pr = F.AttnParams(H, Hk, D, F._dtype_code(q, "q"), window[0], window[1], sinks, D ** -0.5)
    out = {n: Guarded(s, q.dtype) for n, s in (("out", q.shape), ("grad_q", q.shape),
                                               ("grad_k", k.shape), ("grad_v", k.shape))}
    out["lse"] = Guarded((nq, H), torch.float32)
    head = (ctypes.byref(qs), None if ks is None else ctypes.byref(ks), ctypes.byref(pr))
    h = {n: F.make_heads(t, n) for n, t in (("q", q), ("k", k), ("v", v), ("go", go))}
    h.update({n: F.make_heads(out[n].t, n) for n in ("out", "grad_q", "grad_k", "grad_v")})
    r = {n: ctypes.byref(x) for n, x in h.items()}
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    lse = ctypes.c_void_p(out["lse"].t.data_ptr())
    for backward in (0, 1):
        need = F.lib().fpstok_attention_workspace_size(*head, backward)
        ws = out["workspace %d" % backward] = Guarded((need // 256, 64), torch.float32)
        end = (ctypes.c_void_p(ws.t.data_ptr() if need else None), need, stream)
        assert ws.t.data_ptr() % 256 == 0 and need % 256 == 0
        if backward:
            F._check(F.lib().fpstok_attention_backward(
                *head, r["q"], r["k"], r["v"], r["out"], lse, r["go"], r["grad_q"], r["grad_k"],
                r["grad_v"], *end), "backward")
        else:
            F._check(F.lib().fpstok_attention(*head, r["q"], r["k"], r["v"], r["out"], lse, *end),
                     "forward")
    torch.cuda.synchronize()
    for n, x in out.items():
        x.check(n)
    return {n: x.t for n, x in out.items() if not n.startswith("workspace")}


# heads, window, sinks: whole; the sinks' rows in chunks; few key heads, so the
# walks of grad_k and grad_v are split
FORMS = [(4, 2, (-1, -1), 0), (2, 2, (30, 0), 2), (8, 1, (20, -1), 40), (8, 1, (-1, 0), 0)]
BAD_CU = [[0, 40, 20, 300], [-5, 50, 60, 900], [290, 10, 10, 10], [2**31 - 1, -2**31, 0, 5],
          [7, 7, 7, 7], [0, 300, 0, 300]]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [40, 128])
@pytest.mark.parametrize("H,Hk,window,sinks", FORMS)
def test_bad_packed_lengths(F, dtype, D, H, Hk, window, sinks):  # noqa: F811
    """Boundaries out of range or out of order, of the queries, the keys or
    both.  Rows of no sequence keep what they held."""
    gen = torch.Generator().manual_seed(91)
    n, m = 300, 270
    q, k, v, go = (rand(gen, s, DT[dtype]).cuda() for s in ((n, H, D), (m, Hk, D), (m, Hk, D),
                                                          (n, H, D)))
    good = torch.tensor([0, 90, 100, 250], dtype=torch.int32).cuda()
    for cu in BAD_CU:
        bad = torch.tensor(cu, dtype=torch.int32).cuda()
        for which, (qc, kc) in (("q", (bad, good)), ("k", (good, bad)), ("both", (bad, bad))):
            log("bad lengths %s of %s: %d/%d heads of %d %s" % (cu, which, H, Hk, D, dtype))
            got = call(F, F.make_seqs(n, cu_seqlens=qc), F.make_seqs(m, cu_seqlens=kc), q, k, v, go,
                       window, sinks)
            if which == "k":
                assert bool((got["out"][250:] == MARK).all())
                assert not bool((got["out"][:250] == MARK).all(-1).any())
            if which == "q":
                assert bool((got["grad_k"][250:] == MARK).all())
                assert not bool((got["grad_k"][:250] == MARK).all(-1).any())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [40, 128])
@pytest.mark.parametrize("H,Hk,window,sinks", FORMS)
def test_bad_padded_lengths(F, dtype, D, H, Hk, window, sinks):  # noqa: F811
    """Counts out of range: as if they were 0 or the capacity."""
    gen = torch.Generator().manual_seed(92)
    cap, lens = 70, [200, -3, 2**31 - 1, 40, -2**31]
    n = cap * len(lens)
    q, k, v, go = (rand(gen, (n, h, D), DT[dtype]).cuda() for h in (H, Hk, Hk, H))

    def seqs(x):
        return F.make_seqs(n, token_count=torch.tensor(x, dtype=torch.int32).cuda(), capacity=cap)

    log("bad counts %d/%d heads of %d %s" % (H, Hk, D, dtype))
    got = call(F, seqs(lens), None, q, k, v, go, window, sinks)
    want = call(F, seqs([min(max(x, 0), cap) for x in lens]), None, q, k, v, go, window, sinks)
    for name in got:
        assert torch.equal(got[name], want[name]), name
    live = np.repeat(np.clip(lens, 0, cap), cap) > np.tile(np.arange(cap), len(lens))
    assert bool((got["grad_q"][torch.from_numpy(~live).cuda()] == 0).all())
    assert bool((got["grad_v"][torch.from_numpy(live).cuda()] != 0).any(-1).all())


@pytest.mark.parametrize("how", ["argument", "assigned"])
def test_gradients_are_written_where_they_were_asked_for(F, how):  # noqa: F811
    log("gradient buffers %s" % how)
    gen = torch.Generator().manual_seed(93)
    qs, _, n = layout(F, [90, 5], "packed")
    q, k, v, go = (rand(gen, (n, h, 64), torch.bfloat16).cuda() for h in (4, 2, 2, 4))
    att = F.Attention(q, k, v, qs, training=True)
    att()
    want = [g.clone() for g in att.backward(go)]
    mine = [Guarded(t.shape, t.dtype) for t in (q, k, v)]
    views = tuple(x.t for x in mine)
    if how == "argument":
        att = F.Attention(q, k, v, qs, training=True, grads=views)
    else:
        att.grads = views
    att()
    got = att.backward(go)
    torch.cuda.synchronize()
    for g, w, m in zip(got, want, mine):
        assert g.data_ptr() == m.t.data_ptr() and torch.equal(g, w)
        m.check("gradient")


def test_gradient_buffers_are_checked(F):  # noqa: F811
    qs, _, n = layout(F, [9], "packed")
    q = torch.zeros((n, 2, 64), dtype=torch.bfloat16, device="cuda")
    att = F.Attention(q, q, q, qs, training=True)
    with pytest.raises(ValueError):
        att.grads = (q, q)
    with pytest.raises(ValueError):
        att.grads = (q, q[:3], q)
    with pytest.raises(TypeError):
        att.grads = (q, q.half(), q)
    with pytest.raises(ValueError):
        F.Attention(q, q, q, qs, grads=(q, q, q))
    with pytest.raises(ValueError):
        F.Attention(q, q, q, qs).grads = (q, q, q)
