"""GPU tests of fpstok_attention, fpstok_attention_backward and fpstok_rope
through the C ABI, against their definitions in float64 within bounds that
count roundings (tests/attention_ref.py)."""
import numpy as np
import pytest
import torch

from point_cloud_tokenization_amd import synth
from tests import attention_ref as ref
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from point_cloud_tokenization_amd import fpstok

    fpstok.lib()
    return fpstok


def rand(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def layout(F, lens, form, cap=None, extra=0, max_len=0):
    """(Seqs, [(first row, length)], rows) of the given lengths."""
    n = torch.tensor(lens, dtype=torch.int32)
    if form == "padded":
        cap = max(max(lens), 1) if cap is None else cap
        rows = cap * len(lens)
        s = F.make_seqs(rows, token_count=n.cuda(), capacity=cap, max_len=max_len)
        return s, [(b * cap, x) for b, x in enumerate(lens)], rows
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(n, 0)
    rows = int(cu[-1]) + extra
    s = F.make_seqs(rows, cu_seqlens=cu.cuda(), max_len=max_len)
    return s, [(int(cu[b]), x) for b, x in enumerate(lens)], rows


def run(F, label, q_lens, k_lens=None, H=4, Hk=2, D=64, dtype="bf16", left=-1, right=-1, sinks=0,
        form="packed", train=True, scale=None, seed=1, spread=1.0, cap=None, extra=0,
        hint=False, big=1.0):
    log("attention case %s: q %s k %s H=%d/%d D=%d %s window (%d,%d) sinks %d %s" % (
        label, str(q_lens)[:60], str(k_lens)[:60], H, Hk, D, dtype, left, right, sinks, form))
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    kl = q_lens if k_lens is None else k_lens
    qs, q_seq, nq = layout(F, q_lens, form, cap, extra, max(q_lens) if hint else 0)
    ks, k_seq, nk = (None, q_seq, nq) if k_lens is None else \
        layout(F, k_lens, form, None, extra, max(kl) if hint else 0)
    q, k, v = rand(gen, (nq, H, D), dt, spread), rand(gen, (nk, Hk, D), dt), \
        rand(gen, (nk, Hk, D), dt, big)
    go = rand(gen, (nq, H, D), dt) if train else None
    att = F.Attention(q.cuda(), k.cuda(), v.cuda(), qs, ks, (left, right), sinks, scale, train)
    for t in (att.out, att.lse):
        t.fill_(7.0)
    out, lse = att()
    r = ref.attention(q, k, v, q_seq, k_seq, left, right, sinks, scale, go)
    if train:
        for t in att.grads:
            t.fill_(7.0)
        gq, gk, gv = att.backward(go.cuda())
        got = dict(out=out, lse=lse, grad_q=gq, grad_k=gk, grad_v=gv)
    else:
        got = dict(out=out, lse=lse)
    torch.cuda.synchronize()
    for name, t in got.items():
        val, tol = r[name]
        if form == "packed":
            # rows behind the last sequence keep what they held
            seq = k_seq if name in ("grad_k", "grad_v") else q_seq
            end = seq[-1][0] + seq[-1][1]
            val[end:], tol[end:] = 7.0, 0.0
        ref.check(t, (val, tol), "%s %s" % (label, name))
    return att


LENS = [1, 0, 5, 64, 33, 128, 129, 2, 200, 31]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [8, 40, 64, 72, 128])
def test_types_and_head_sizes(F, dtype, D):
    run(F, "head size", LENS, D=D, dtype=dtype, H=4, Hk=2, extra=5)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 2), (8, 1), (5, 1), (33, 1)])
def test_head_groups(F, dtype, H, Hk):
    run(F, "groups", [70, 1, 0, 130], H=H, Hk=Hk, dtype=dtype)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("left,right,sinks", [
    (-1, 0, 0), (0, 0, 0), (0, -1, 0), (10, 3, 0), (64, 64, 4), (31, 0, 1), (100, 0, 64),
    (5, 200, 17), (-1, 7, 3), (1000000000, 1000000000, 64), (0, 0, 64)])
def test_windows_and_sinks(F, dtype, left, right, sinks):
    run(F, "window", [300, 1, 64, 0, 65, 190], left=left, right=right, sinks=sinks, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["packed", "padded"])
@pytest.mark.parametrize("left,right,sinks", [(-1, -1, 0), (-1, 0, 0), (20, 5, 3)])
def test_more_keys_or_more_queries(F, dtype, form, left, right, sinks):
    """Lengths of zero on either side, and causal rows before the first key
    (more queries than keys), which see nothing."""
    run(F, "cross", [7, 100, 0, 1, 64, 150, 3], [90, 30, 12, 0, 64, 1, 300], left=left, right=right,
        sinks=sinks, dtype=dtype, form=form, cap=150)


@pytest.mark.parametrize("dtype", list(DT))
def test_padded_batch(F, dtype):
    run(F, "padded", [0, 128, 1, 77, 128, 64], dtype=dtype, form="padded", cap=128, H=3, Hk=3,
        D=40, hint=True)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H,Hk,D", [(12, 12, 64), (8, 1, 128), (32, 8, 64)])
def test_one_query_per_sequence(F, dtype, H, Hk, D):
    k = [1, 5000, 64, 0, 700, 2049]
    run(F, "one query", [1] * 6, k, H=H, Hk=Hk, D=D, dtype=dtype, train=False, hint=True)
    run(F, "one query padded", [1] * 6, k, H=H, Hk=Hk, D=D, dtype=dtype, train=False,
        form="padded")
    run(F, "one query window", [1] * 6, k, H=H, Hk=Hk, D=D, dtype=dtype, train=False, left=700,
        right=0, sinks=4)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nq", [1, 2, 5])
def test_few_queries_train(F, dtype, nq):
    run(F, "few queries", [nq] * 3, [900, 3, 1500], H=4, Hk=2, dtype=dtype, hint=True)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("left,right,sinks", [(-1, -1, 0), (-1, 0, 0), (90, 20, 8)])
def test_one_long_sequence(F, dtype, left, right, sinks):
    run(F, "long", [1500], H=2, Hk=1, D=64, left=left, right=right, sinks=sinks, dtype=dtype)


@pytest.mark.parametrize("dtype", list(DT))
def test_peaked_scores_and_large_values(F, dtype):
    # scores of tens: softmax close to one key, running maxima that grow
    run(F, "peaked", [257, 40], dtype=dtype, spread=20.0)
    run(F, "large values", [100], dtype=dtype, big=200.0)
    run(F, "flat", [300], dtype=dtype, scale=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_sequences(F, dtype):
    """More sequences than one wave tests at once, most of them tiny."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 6, 5000).tolist()
    lens[17], lens[4999], lens[64 * 64] = 150, 90, 70
    run(F, "many", lens, H=1, Hk=1, D=8, dtype=dtype)


@pytest.mark.parametrize("dtype", list(DT))
def test_strides(F, dtype):
    """q, k, v as slices of one projection; [heads, rows, D] storage; a
    query row shared by every sequence (stride 0)."""
    log("attention strides %s" % dtype)
    gen = torch.Generator().manual_seed(9)
    dt, lens, H, D = DT[dtype], [40, 100, 7], 3, 64
    qs, seq, n = layout(F, lens, "packed")
    qkv = rand(gen, (n, 3, H, D), dt)
    go = rand(gen, (n, H, D), dt)
    want = ref.attention(qkv[:, 0], qkv[:, 1], qkv[:, 2], seq, seq, 20, 0, 2, grad=go)
    dev = qkv.cuda()
    att = F.Attention(dev[:, 0], dev[:, 1], dev[:, 2], qs, None, (20, 0), 2, None, True)
    out, lse = att()
    grads = att.backward(go.cuda())
    for name, t in zip(("out", "lse", "grad_q", "grad_k", "grad_v"), (out, lse) + grads):
        ref.check(t, want[name], "qkv " + name)
    hm = [dev[:, i].transpose(0, 1).contiguous().transpose(0, 1) for i in range(3)]
    o2 = torch.zeros((H, n, D), dtype=dt, device="cuda").transpose(0, 1)
    att2 = F.Attention(*hm, qs, None, (20, 0), 2, None, True, out=o2)
    out2, _ = att2()
    go2 = go.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    g2 = att2.backward(go2)
    torch.cuda.synchronize()
    assert torch.equal(out2, out)
    for a, b in zip(g2, grads):
        assert torch.equal(a, b)
    q1 = rand(gen, (1, H, D), dt)
    one, one_seq, _ = layout(F, [1, 1, 1], "packed")
    att3 = F.Attention(q1.cuda().expand(3, H, D), dev[:, 1], dev[:, 2], one, qs, training=True)
    out3, lse3 = att3()
    g3 = att3.backward(go.cuda()[:1].expand(3, H, D))
    want = ref.attention(q1.expand(3, H, D), qkv[:, 1], qkv[:, 2], one_seq, seq,
                         grad=go[:1].expand(3, H, D))
    for name, t in zip(("out", "lse", "grad_q", "grad_k", "grad_v"), (out3, lse3) + g3):
        ref.check(t, want[name], "shared query " + name)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_hidden_values_never_reach_a_result(F, dtype, D, bad):
    """Rows of not-a-number or infinite values: in packed rows behind the last
    sequence, in padded slots, in another sequence, and in keys (queries)
    that a window hides."""
    log("attention hidden %s %d %r" % (dtype, D, bad))
    gen = torch.Generator().manual_seed(11)
    dt, H, Hk = DT[dtype], 4, 2
    for form in ("packed", "padded"):
        lens = [37, 90, 64, 130]
        qs, seq, n = layout(F, lens, form, cap=140, extra=9)
        q, k, v, go = (rand(gen, (n, h, D), dt) for h in (H, Hk, Hk, H))
        clean = ref.attention(q, k, v, seq, seq, 16, 4, 2, grad=go)
        inside = np.zeros(n, dtype=bool)
        for s, x in seq:
            inside[s:s + x] = True
        inside[seq[1][0]:seq[1][0] + lens[1]] = False  # sequence 1: bad throughout
        hide = torch.from_numpy(~inside)
        kb = k.clone()
        vb, qb, gb = v.clone(), q.clone(), go.clone()
        for t in (kb, vb, qb, gb):
            t[hide] = bad
        # one bad key and value, and one bad query and gradient, in the middle of
        # sequence 3: seen only inside the window
        j, i = seq[3][0] + 70, seq[3][0] + 100
        kb[j], vb[j], qb[i], gb[i] = bad, bad, bad, bad
        att = F.Attention(qb.cuda(), kb.cuda(), vb.cuda(), qs, None, (16, 4), 2, None, True)
        out, lse = att()
        grads = att.backward(gb.cuda())
        torch.cuda.synchronize()
        p = np.arange(lens[3])
        rows = inside.copy()
        touched = (p + 4 >= 70) & (p - 16 <= 70) | (p == 100)
        rows[seq[3][0]:][:lens[3]] &= ~touched
        keys = inside.copy()
        # keys that a touched query sees have touched gradients
        kt = np.zeros(lens[3], dtype=bool)
        for x in p[touched]:
            kt |= ref.visible(lens[3], lens[3], 16, 4, 2)[x]
        keys[seq[3][0]:][:lens[3]] &= ~kt
        for name, t, m in (("out", out, rows), ("lse", lse, rows), ("grad_q", grads[0], rows),
                           ("grad_k", grads[1], keys), ("grad_v", grads[2], keys)):
            val, tol = clean[name]
            ref.check(t[torch.from_numpy(m).cuda()], (val[m], tol[m]),
                      "%s %s hidden %s" % (form, name, bad))
        # what is seen is not lost
        assert torch.isnan(out[seq[3][0] + 70].float()).any() or bad == float("-inf")
        assert not torch.isfinite(grads[2][seq[3][0] + 100].float()).any()


def test_refuses_on_the_device_too(F):
    q = torch.zeros((4, 2, 60), dtype=torch.bfloat16, device="cuda")
    qs, _, _ = layout(F, [4], "packed")
    with pytest.raises(F.FpstokError):
        F.Attention(q, q, q, qs)()
    q = torch.zeros((4, 2, 64), device="cuda")
    with pytest.raises(TypeError):
        F.Attention(q, q.half(), q, qs)
    with pytest.raises(ValueError):
        F.Attention(q, q[:3], q, qs)
    with pytest.raises(ValueError):
        F.Attention(q, q, q, qs).backward(q)


def test_empty_batches(F):
    for lens, form in (([0], "packed"), ([0, 0], "padded")):
        qs, _, n = layout(F, lens, form, cap=4)
        q = torch.ones((n, 2, 64), dtype=torch.bfloat16, device="cuda")
        att = F.Attention(q, q, q, qs, training=True)
        out, lse = att()
        g = att.backward(q)
        torch.cuda.synchronize()
        assert float(out.float().abs().sum()) == 0.0
        assert all(float(x.float().abs().sum()) == 0.0 for x in g)
    # no keys at all: zeros and -inf; no queries at all: zero gradients
    some, _, _ = layout(F, [3, 2], "packed")
    none, _, _ = layout(F, [0, 0], "packed")
    q = torch.ones((5, 2, 64), dtype=torch.bfloat16, device="cuda")
    k = q[:0]
    att = F.Attention(q, k, k, some, none, training=True)
    att.out.fill_(3.0)
    out, lse = att()
    g = att.backward(q)
    torch.cuda.synchronize()
    assert float(out.float().abs().sum()) == 0.0 and bool((lse == -float("inf")).all())
    assert float(g[0].float().abs().sum()) == 0.0
    att = F.Attention(k, q, q, none, some, training=True)
    att()
    for x in att.grads:
        x.fill_(3.0)
    g = att.backward(k)
    torch.cuda.synchronize()
    assert float(g[1].float().abs().sum()) == 0.0 and float(g[2].float().abs().sum()) == 0.0


def test_bad_lengths_stay_inside_the_buffers(F):
    """Boundaries out of range or out of order are clamped: no access outside
    the buffers (guard rows around them keep their values)."""
    gen = torch.Generator().manual_seed(13)
    n, H, D = 100, 2, 64
    for cu in ([0, 40, 20, 100], [-5, 50, 60, 200], [90, 10, 10, 10], [2**31 - 1, -2**31, 0, 5]):
        store = [rand(gen, (n + 80, H, D), torch.bfloat16).cuda() for _ in range(8)]
        keep = [t.clone() for t in store]
        q, k, v, go, out, gq, gk, gv = (t[40:140] for t in store)
        qs = F.make_seqs(n, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
        log("bad lengths %s" % cu)
        att = F.Attention(q, k, v, qs, None, (30, 0), 2, None, True, out=out)
        att.grads = (gq, gk, gv)
        att()
        att.backward(go)
        torch.cuda.synchronize()
        for t, was in zip(store, keep):
            assert torch.equal(t[:40], was[:40]) and torch.equal(t[140:], was[140:])
    q = torch.zeros((12, 2, 64), dtype=torch.bfloat16, device="cuda")
    qs = F.make_seqs(12, token_count=torch.tensor([9, -3, 4], dtype=torch.int32).cuda(),
                     capacity=4)
    F.Attention(q, q, q, qs, training=True)()
    torch.cuda.synchronize()


# ------------------------------------------------- streams, graphs, repeats

def _plan(F, seed, lens=(60, 0, 128, 9), left=-1, right=-1, sinks=0, **kw):
    gen = torch.Generator().manual_seed(seed)
    qs, seq, n = layout(F, list(lens), "packed")
    q, k, v, go = (rand(gen, (n, h, 64), torch.bfloat16).cuda() for h in (4, 2, 2, 4))
    return F.Attention(q, k, v, qs, None, (left, right), sinks, None, True, **kw), go


def _all(att, go, stream=None):
    out, lse = att(stream)
    return [t.clone() for t in (out, lse) + att.backward(go, stream)]


@pytest.mark.parametrize("lens,left,right,sinks", [
    ((60, 0, 128, 9), -1, -1, 0), ((1800,), 100, 0, 4), ((1, 1), -1, -1, 0)])
def test_repeats_are_bit_identical(F, lens, left, right, sinks):
    att, go = _plan(F, 21, lens, left, right, sinks)
    first = _all(att, go)
    if att.ws is not None:
        att.ws.fill_(255)  # the workspace's old contents do not matter
    for _ in range(3):
        for a, b in zip(first, _all(att, go)):
            assert torch.equal(a, b)


def test_two_streams(F):
    """Two calls at once, each with its own buffers."""
    plans = [_plan(F, 31 + i, lens, 50, 0, 2) for i, lens in enumerate(((1500, 40), (900, 900)))]
    want = [_all(att, go) for att, go in plans]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in plans]
    for _ in range(5):
        for (att, go), s in zip(plans, streams):
            att(s)
            att.backward(go, s)
    torch.cuda.synchronize()
    for (att, go), w in zip(plans, want):
        for a, b in zip((att.out, att.lse) + att.grads, w):
            assert torch.equal(a, b)


def test_captured_and_replayed(F):
    """Forward, gradients and rotations in a graph, replayed on changed
    inputs with eager calls of another plan between the replays."""
    att, go = _plan(F, 41, (60, 0, 700, 9), 90, 0, 2)
    other, go2 = _plan(F, 42)
    n = att.q.shape[0]
    pos = torch.randn((n, 4), device="cuda")
    rope = F.Rope(att.q, att.k, pos, F.rope_frequencies((8, 8, 8, 8), device="cuda"), (8,) * 4,
                  att.q_seqs)
    rope()
    _all(att, go)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        rope()
        att()
        att.backward(go)
    for i in range(4):
        with torch.no_grad():
            att.q.copy_(torch.randn(att.q.shape, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (rope.q_out, rope.k_out, att.out, att.lse) + att.grads]
        rope()
        want = [rope.q_out.clone(), rope.k_out.clone()] + _all(att, go)
        _all(other, go2)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_directional_derivative(F):
    """float32 gradients against differences of the float32 forward: with step
    h the difference is off by h^2/6 of the third derivative and by the
    forward's rounding over h."""
    gen = torch.Generator().manual_seed(51)
    qs, seq, n = layout(F, [50, 20], "packed")
    q, k, v, go = (rand(gen, (n, h, 64), torch.float32) for h in (4, 2, 2, 4))
    dirs = [rand(gen, t.shape, torch.float32) for t in (q, k, v)]
    att = F.Attention(q.cuda(), k.cuda(), v.cuda(), qs, None, (12, 3), 2, None, True)
    att()
    grads = [g.double().cpu() for g in att.backward(go.cuda())]
    h = 2.0 ** -8
    for i, (t, d, g) in enumerate(zip((att.q, att.k, att.v), dirs, grads)):
        base = t.clone()
        vals = []
        for sign in (1, -1):
            t.copy_(base + sign * h * d.cuda())
            vals.append(float((att()[0].double().cpu() * go.double()).sum()))
        t.copy_(base)
        want = float((g * d.double()).sum())
        # |third derivative| of this sum stays under 1e4 (70 rows x 4 heads of
        # unit terms times |d|^3 on softmax weights); rounding: 2e4 elements of
        # about 2^-24 each, over 2 h
        assert abs((vals[0] - vals[1]) / (2 * h) - want) < h * h / 6 * 1e4 + 17920 * 2.0 ** -22 / h


# ------------------------------------------------------------------- rope

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("D,pairs", [(64, (8, 8, 8, 8)), (64, (5, 0, 9)), (128, (64,)), (2, (1,)),
                                     (72, (12, 12, 12)), (40, (4, 4)), (10, (2, 1))])
def test_rope(F, dtype, inter, inverse, D, pairs):
    log("rope case %s D=%d pairs %s inter %d inverse %d" % (dtype, D, pairs, inter, inverse))
    gen = torch.Generator().manual_seed(61)
    dt, lens = DT[dtype], [3, 0, 64, 50]
    fr = F.rope_frequencies(pairs, top=30.0)
    for form in ("packed", "padded"):
        qs, seq, n = layout(F, lens, form, cap=64, extra=6)
        q, k = rand(gen, (n, 6, D), dt), rand(gen, (n, 2, D), dt)
        pos = torch.randn((n, len(pairs)), generator=gen) * 2.0
        r = F.Rope(q.cuda(), k.cuda(), pos.cuda(), fr.cuda(), pairs, qs, inter)
        r.q_out.fill_(7.0)
        r.k_out.fill_(7.0)
        qo, ko = r(inverse)
        torch.cuda.synchronize()
        inside = np.zeros(n, dtype=bool)
        for s, x in seq:
            inside[s:s + x] = True
        for name, x, y in (("q", q, qo), ("k", k, ko)):
            val, tol = ref.rope(x, pos, fr, pairs, inter, inverse)
            val[~inside], tol[~inside] = 0.0 if form == "padded" else 7.0, 0.0
            ref.check(y, (val, tol), "rope %s %s" % (form, name))


@pytest.mark.parametrize("dtype", list(DT))
def test_rope_far_positions(F, dtype):
    """Integer positions up to 2^31 - 1 and angles up to 2^38."""
    gen = torch.Generator().manual_seed(62)
    n, D, pairs = 300, 64, (11, 11, 10)
    pos = torch.randint(-2**31, 2**31 - 1, (n, 3), generator=gen).to(torch.int32)
    pos[0], pos[1] = 2**31 - 1, -2**31
    fr = F.rope_frequencies(pairs, top=100.0)
    qs, _, _ = layout(F, [n], "packed")
    q = rand(gen, (n, 2, D), DT[dtype])
    r = F.Rope(q.cuda(), None, pos.cuda(), fr.cuda(), pairs, qs)
    qo, ko = r()
    torch.cuda.synchronize()
    assert ko is None
    # the reference's float64 cosine takes the exact product
    ref.check(qo, ref.rope(q, pos, fr, pairs), "far rope")


@pytest.mark.parametrize("n", [1, 2, 63, 1000, 5000])
def test_rope_sizes_strides_and_in_place(F, n):
    gen = torch.Generator().manual_seed(63)
    pairs = (10, 22)
    fr = F.rope_frequencies(pairs)
    pos = torch.randint(0, 3000, (n, 2), generator=gen).to(torch.int32)
    qs, _, _ = layout(F, [n], "packed")
    for dt in (torch.bfloat16, torch.float32):
        qkv = rand(gen, (n, 3, 4, 64), dt)
        dev = qkv.cuda()
        want = [ref.rope(qkv[:, i], pos, fr, pairs) for i in range(2)]
        r = F.Rope(dev[:, 0], dev[:, 1], pos.cuda(), fr.cuda(), pairs, qs)
        out = [t.clone() for t in r()]
        for o, w in zip(out, want):
            ref.check(o, w, "rope slices")
        r2 = F.Rope(dev[:, 0], dev[:, 1], pos.cuda(), fr.cuda(), pairs, qs, q_out=dev[:, 0],
                    k_out=dev[:, 1])
        r2()
        assert torch.equal(dev[:, 0], out[0]) and torch.equal(dev[:, 1], out[1])
        assert torch.equal(dev[:, 2].cpu(), qkv[:, 2])
        # an odd element offset: no 16-byte alignment
        flat = torch.zeros(n * 4 * 65 + 1, dtype=dt, device="cuda")[1:].view(n, 4, 65)
        flat[..., :64] = qkv[:, 0].cuda()
        odd = F.Rope(flat[..., :64], None, pos.cuda(), fr.cuda(), pairs, qs)()[0]
        assert torch.equal(odd, out[0])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("form", ["packed", "padded"])
@pytest.mark.parametrize("q_lens,k_lens,H,Hk,D,right", [
    ([700], None, 4, 2, 64, -1), ([601, 0, 77], None, 6, 2, 40, 0),
    ([40, 3], [2000, 0], 4, 2, 64, -1), ([1100], [900], 2, 1, 128, 0)])
def test_rows_whose_keys_are_split(F, dtype, form, q_lens, k_lens, H, Hk, D, right):
    """Few workgroups: several take parts of a row's keys, joined for few rows
    and for many."""
    run(F, "split", q_lens, k_lens, H=H, Hk=Hk, D=D, dtype=dtype, right=right, form=form,
        extra=5 if form == "packed" else 0)


# ------------------------------------------------ parts of larger batches

@pytest.mark.parametrize("H,Hk", [(4, 2), (8, 1)])
def test_rows_ahead_of_the_first_sequence(F, H, Hk):
    """cu_seqlens that starts past 0 (some events of a larger batch): nothing
    is read or written ahead of its rows."""
    gen = torch.Generator().manual_seed(64)
    cu = torch.tensor([37, 37, 140, 300], dtype=torch.int32)
    n, D, pairs = 320, 64, (8, 8, 8, 8)
    seq = [(37, 0), (37, 103), (140, 160)]
    inside = torch.zeros(n, dtype=torch.bool)
    inside[37:300] = True
    q, k, v, go = (rand(gen, (n, h, D), torch.bfloat16) for h in (H, Hk, Hk, H))
    for t in (q, k, v, go):
        t[~inside] = float("nan")
    pos = torch.randn((n, 4), generator=gen)
    qs = F.make_seqs(n, cu_seqlens=cu.cuda())
    fr = F.rope_frequencies(pairs)
    log("rows ahead: rotary positions")
    for width in (D, D - 1):  # 16 bytes at a time, and element by element
        x = torch.full((n, H, D + 1), 7.0, dtype=torch.bfloat16, device="cuda")
        x[..., :D] = q.cuda()
        src = q.cuda() if width == D else x[..., :D]
        r = F.Rope(src, None, pos.cuda(), fr.cuda(), pairs, qs)
        r.q_out.fill_(7.0)
        got = r()[0]
        torch.cuda.synchronize()
        val, tol = ref.rope(torch.where(inside[:, None, None], q, torch.zeros_like(q)), pos, fr,
                            pairs, False)
        val[~inside.numpy()], tol[~inside.numpy()] = 7.0, 0.0
        ref.check(got, (val, tol), "rope")
    log("rows ahead: attention")
    att = F.Attention(q.cuda(), k.cuda(), v.cuda(), qs, training=True)
    for t in (att.out, att.lse) + att.grads:
        t.fill_(7.0)
    out, lse = att()
    grads = att.backward(go.cuda())
    torch.cuda.synchronize()
    want = ref.attention(q, k, v, seq, seq, grad=go)
    for name, t in zip(("out", "lse", "grad_q", "grad_k", "grad_v"), (out, lse) + grads):
        assert bool((t[~inside] == 7.0).all()), name
        val, tol = want[name]
        ref.check(t[inside], (val[inside.numpy()], tol[inside.numpy()]), name)


def test_strides_of_single_rows_and_heads(F):
    """The stride of a dimension of one element is never used."""
    gen = torch.Generator().manual_seed(65)
    qs, seq, _ = layout(F, [1], "packed")
    for H in (1, 4):
        flat = rand(gen, (4 * 64,), torch.bfloat16)
        q = flat.as_strided((1, H, 64), (1 << 30, 64 if H > 1 else 3, 1))
        want = ref.attention(q, q, q, seq, seq)
        dev = flat.cuda().as_strided(q.shape, q.stride())
        out, _ = F.Attention(dev, dev, dev, qs)()
        torch.cuda.synchronize()
        ref.check(out, want["out"], "one row of %d heads" % H)


# ----------------------------------------------------------- used together

def test_tokens_through_a_layer(F):
    """Tokens of a batch: tokenize, pack features and centroids, project,
    rotate, attend, pool each event with one query, and unpack; gradients of
    the attention back through the rotation."""
    b = synth.make_batch("icecube_b64_voronoi", synth.parity_seed("icecube_b64_voronoi", 2))
    dev = torch.device("cuda:0")
    x, f, off = (torch.from_numpy(b[n]).to(dev) for n in ("coords", "features", "offsets"))
    t = F.tokenize(x, f, off, num_patches=128, charge_col=b["charge_col"])
    B, P, C = t["pooled"].shape
    gen = torch.Generator().manual_seed(71)
    H, Hk, D = 4, 2, 32
    w = [rand(gen, (C, h * D), torch.float32).cuda() * 0.3 for h in (H, Hk, Hk)]
    rows = torch.zeros((B * P, C), device=dev)
    cen = torch.zeros((B * P, 4), device=dev)
    cu = torch.empty(B + 1, dtype=torch.int32, device=dev)
    F.pack(t["token_count"], t["pooled"], rows, None, cu)
    F.pack(t["token_count"], t["centroids"], cen, None, cu)
    qs = F.make_seqs(B * P, cu_seqlens=cu, max_len=P)
    q, k, v = (torch.matmul(rows, m).view(B * P, h, D) for m, h in zip(w, (H, Hk, Hk)))
    fr = F.rope_frequencies((4, 4, 4, 4), base=100.0, top=20.0)
    r = F.Rope(q, k, cen, fr.to(dev), (4, 4, 4, 4), qs)
    rq, rk = r()
    att = F.Attention(rq, rk, v, qs, training=True)
    out, lse = att()
    go = rand(gen, out.shape, torch.float32)
    gq, gk, gv = att.backward(go.cuda())
    back = F.Rope(gq, gk, cen, fr.to(dev), (4, 4, 4, 4), qs)
    bq, bk = back(inverse=True)
    one = F.make_seqs(B, token_count=torch.ones(B, dtype=torch.int32, device=dev), capacity=1,
                      max_len=1)
    query = rand(gen, (1, H, D), torch.float32)
    keys = out.view(B * P, H, D)
    pooled, _ = F.Attention(query.cuda().expand(B, H, D), keys, keys, one, qs)()
    full = torch.empty((B, P, H * D), device=dev)
    F.unpack(t["token_count"], cu, out.view(B * P, H * D), full)
    torch.cuda.synchronize()
    # each step against the reference on that step's inputs
    c = cu.cpu().tolist()
    seq = [(c[i], c[i + 1] - c[i]) for i in range(B)]
    n = c[-1]
    cpu = lambda y: y.detach().cpu()  # noqa: E731
    for got, src in ((rq, q), (rk, k)):
        val, tol = ref.rope(cpu(src), cpu(cen), fr, (4, 4, 4, 4))
        ref.check(got[:n], (val[:n], tol[:n]), "layer rope")
    want = ref.attention(cpu(rq), cpu(rk), cpu(v), seq, seq, grad=go)
    for name, y in (("out", out), ("lse", lse), ("grad_q", gq), ("grad_k", gk), ("grad_v", gv)):
        ref.check(y, want[name], "layer " + name)
    for got, src in ((bq, gq), (bk, gk)):
        val, tol = ref.rope(cpu(src), cpu(cen), fr, (4, 4, 4, 4), inverse=True)
        ref.check(got[:n], (val[:n], tol[:n]), "layer rope gradient")
    want = ref.attention(query.expand(B, H, D), cpu(keys), cpu(keys), [(i, 1) for i in range(B)],
                         seq)
    ref.check(pooled, want["out"], "layer pooling")
    for i in range(B):
        m = c[i + 1] - c[i]
        assert torch.equal(full[i, :m], out.view(B * P, H * D)[c[i]:c[i + 1]])
        assert float(full[i, m:].abs().sum()) == 0.0


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("lens,k_lens,H,Hk,left,right,sinks", [
    ([700], None, 8, 1, -1, -1, 0), ([900, 3], None, 4, 1, 300, 0, 40),
    ([1500, 0, 40], [60, 5, 7], 4, 2, -1, -1, 0), ([1200], [130], 3, 1, -1, 0, 0)])
@pytest.mark.parametrize("form", ["packed", "padded"])
def test_few_keys_many_queries(F, dtype, lens, k_lens, H, Hk, left, right, sinks, form):
    """Walks of grad_k and grad_v that are split over workgroups."""
    run(F, "split walk", lens, k_lens, H=H, Hk=Hk, D=40, dtype=dtype, left=left, right=right,
        sinks=sinks, form=form, hint=True, extra=3 if form == "packed" else 0)
