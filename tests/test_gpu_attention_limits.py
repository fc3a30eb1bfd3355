"""GPU tests of attention at the ends of what its header allows: bounds on
the length that are too small, every head size, many heads, the largest
strides, and rows whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

from tests import attention_ref as ref
from tests.gpu_util import log
from tests.test_gpu_attention import DT, F, layout, rand, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("form", ["packed", "padded"])
@pytest.mark.parametrize("q_max,k_max", [(1, 1), (1, 5000), (5000, 1)])
@pytest.mark.parametrize("window,sinks", [((-1, -1), 0), ((60, 0), 3)])
def test_bounds_on_the_length_that_do_not_hold(  # noqa: F811
        F, dtype, form, q_max, k_max, window, sinks):  # noqa: F811
    log("wrong bounds %d %d %s %s %s" % (q_max, k_max, form, dtype, window))
    gen = torch.Generator().manual_seed(101)
    H, Hk, D = 4, 2, 64
    ql, kl = [300, 0, 40, 1], [170, 9, 0, 700]
    qs, q_seq, n = layout(F, ql, form, None, 0, q_max)
    ks, k_seq, m = layout(F, kl, form, None, 0, k_max)
    q, k, v, go = (rand(gen, (r, h, D), DT[dtype]) for r, h in ((n, H), (m, Hk), (m, Hk), (n, H)))
    att = F.Attention(q.cuda(), k.cuda(), v.cuda(), qs, ks, window, sinks, training=True)
    for t in (att.out, att.lse) + att.grads:
        t.fill_(7.0)
    out, lse = att()
    grads = att.backward(go.cuda())
    torch.cuda.synchronize()
    want = ref.attention(q, k, v, q_seq, k_seq, *window, sinks, grad=go)
    for name, t in zip(("out", "lse", "grad_q", "grad_k", "grad_v"), (out, lse) + grads):
        ref.check(t, want[name], name)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", list(range(8, 129, 8)))
def test_every_head_size(F, dtype, D):  # noqa: F811
    run(F, "head size", [70, 3, 129], D=D, dtype=dtype, H=2, Hk=1, left=40, right=7, sinks=2)
    run(F, "one query", [1, 1], [300, 40], D=D, dtype=dtype, H=2, Hk=1, hint=True)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H,Hk", [(300, 1), (200, 200), (129, 43)])
def test_many_heads(F, dtype, H, Hk):  # noqa: F811
    run(F, "many heads", [5, 0, 33], H=H, Hk=Hk, D=16, dtype=dtype, right=0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_row_stride(F, dtype):  # noqa: F811
    """Rows 2^23 elements apart, all views in one buffer, give what dense
    rows give."""
    log("row stride 2^23 %s" % dtype)
    gen = torch.Generator().manual_seed(102)
    H, Hk, D, n, step = 4, 2, 64, 150, 1 << 23
    qs, _, _ = layout(F, [n], "packed")
    q, k, v, go = (rand(gen, (n, h, D), DT[dtype]).cuda() for h in (H, Hk, Hk, H))
    dense = F.Attention(q, k, v, qs, None, (-1, 0), training=True)
    want = dense() + dense.backward(go)
    store = torch.empty(n * step, dtype=DT[dtype], device="cuda")
    wide, at = [], 0
    for t in (q, k, v, go, q, q, k, v):
        wide.append(store.as_strided(t.shape, (step, D, 1), at))
        at += t.shape[1] * D
    for w, t in zip(wide, (q, k, v, go)):
        w.copy_(t)
    att = F.Attention(*wide[:3], qs, None, (-1, 0), training=True, out=wide[4], grads=wide[5:])
    got = att() + att.backward(wide[3])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_past_32_bit_offsets(F, dtype):  # noqa: F811
    """A sequence whose keys begin more than 2^32 bytes (and 2^31 elements)
    into the buffer, behind one of 2.9 million keys."""
    log("rows past 32 bits %s" % dtype)
    H, Hk, D, far, near = 8, 8, 128, 2_900_000, 900
    ql, kl = [1, 150], [far, near]
    qs, q_seq, n = layout(F, ql, "packed")
    ks, k_seq, m = layout(F, kl, "packed", max_len=near)
    assert far * Hk * D > 1 << 31
    gen = torch.Generator().manual_seed(103)
    q, go = rand(gen, (n, H, D), DT[dtype]), rand(gen, (n, H, D), DT[dtype])
    tail = [rand(gen, (near, Hk, D), DT[dtype]) for _ in range(2)]
    k, v = (torch.zeros((m, Hk, D), dtype=DT[dtype], device="cuda") for _ in range(2))
    v[:far] = 1.0
    for t, x in zip((k, v), tail):
        t[far:] = x.cuda()
    att = F.Attention(q.cuda(), k, v, qs, ks, training=True)
    out, lse = att()
    gq, gk, gv = att.backward(go.cuda())
    torch.cuda.synchronize()
    # the first sequence: equal scores, values of 1
    assert bool((out[0] == 1.0).all())
    np.testing.assert_allclose(lse[0].cpu().numpy(), np.log(far), rtol=1e-6)
    want = ref.attention(q[1:], *tail, [(0, 150)], [(0, near)], grad=go[1:])
    for name, t in (("out", out[1:]), ("lse", lse[1:]), ("grad_q", gq[1:]), ("grad_k", gk[far:]),
                    ("grad_v", gv[far:])):
        ref.check(t, want[name], name)
