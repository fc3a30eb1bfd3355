"""Attention with a learned bias and its gradients on the GPU against the float64
reference, each value within the bound of its roundings (tests/bias_ref.py)."""
import numpy as np
import pytest
import torch

from tests import bias_ref as ref
from tests.attention_ref import check

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32
NAMES = ("out", "lse", "grad_q", "grad_k", "grad_v", "grad_table")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def _axes(spec):
    """ "i" or "f" positions, then "n:rate[:steps[:shift]]" for each axis."""
    from point_cloud_tokenization_amd import fpstok as F

    kind, *axes = spec.split()
    out = []
    for a in axes:
        n, rate, *more = a.split(":")
        out.append(F.BiasAxis(int(n), float(rate), float(more[1]) if len(more) > 1 else None,
                              int(more[0]) if more else 0))
    return kind, out


def _layout(lens, form, dev):
    from point_cloud_tokenization_amd import fpstok as F

    if form == "padded":
        cap = max(lens) + 3
        t = torch.tensor(lens, dtype=torch.int32, device=dev)
        return ([(b * cap, n) for b, n in enumerate(lens)], cap * len(lens),
                F.make_seqs(cap * len(lens), token_count=t, capacity=cap))
    cu = 2 + np.concatenate([[0], np.cumsum(lens)])
    t = torch.tensor(cu, dtype=torch.int32, device=dev)
    rows = int(cu[-1]) + 5
    return ([(int(c), n) for c, n in zip(cu, lens)], rows, F.make_seqs(rows, cu_seqlens=t))


class Case:
    """Operands of one call on the CPU and the reference's results."""

    def __init__(self, dev, q_lens, k_lens, H, Hk, D, dt, spec, left=-1, right=-1, sinks=0,
                 form="packed", seed=1, train=True, table=None, spread=2.0):
        self.dev, self.dt = dev, dt
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.q_seq, qr, self.qs = _layout(q_lens, form, dev)
        self.k_seq, kr, self.ks = (self.q_seq, qr, self.qs) if k_lens is None else \
            _layout(k_lens, form, dev)
        self.same = k_lens is None
        self.kind, self.axes = _axes(spec)
        self.q, self.k, self.v = n(qr, H, D).to(dt), n(kr, Hk, D).to(dt), n(kr, Hk, D).to(dt)
        self.grad = n(qr, H, D).to(dt) if train else None
        A = len(self.axes)

        def positions(rows):
            if self.kind == "i":
                return torch.randint(-40, 40, (rows, A), generator=g, dtype=torch.int32) + \
                    2000000000 - 41
            return n(rows, A) * spread

        self.k_pos = positions(kr)
        self.q_pos = self.k_pos if self.same else positions(qr)
        self.table = n(H, sum(a.buckets for a in self.axes)) if table is None else table
        self.mask = dict(left=left, right=right, sinks=sinks)

    def reference(self):
        return ref.attention(self.q, self.k, self.v, self.q_seq, self.k_seq, self.table, self.axes,
                             self.q_pos, None if self.same else self.k_pos, grad=self.grad,
                             **self.mask)

    def call(self, **kw):
        from point_cloud_tokenization_amd import fpstok as F

        d = lambda t: t.to(self.dev)  # noqa: E731
        bias = F.RelativeBias(d(self.table), self.axes, d(self.q_pos),
                              None if self.same else d(self.k_pos))
        return F.Attention(d(self.q), d(self.k), d(self.v), self.qs,
                           None if self.same else self.ks,
                           window=(self.mask["left"], self.mask["right"]),
                           num_sinks=self.mask["sinks"], training=self.grad is not None,
                           bias=bias, **kw)

    def outputs(self, call):
        out = list(call())
        if self.grad is not None:
            out += call.backward(self.grad.to(self.dev))
        torch.cuda.synchronize()
        return out

    def run(self):
        want = self.reference()
        for name, t in zip(NAMES, self.outputs(self.call())):
            check(t, want[name], name)


FOUR = "f 9:1 9:1 9:1.5 14:2:2"


@pytest.mark.parametrize("dt", [FL, HF, BF])
@pytest.mark.parametrize("D", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("form", ["packed", "padded"])
def test_types_and_heads(dev, dt, D, form):
    Case(dev, [70, 1, 0, 130, 33], None, 4, 2, D, dt, FOUR, form=form).run()


@pytest.mark.parametrize("spec", [
    "f 1:1", "f 7:1", "f 64:8", "f 33:3:4", "f 65:8", "f 128:12", "f 32:4 32:4 32:4 32:4",
    "f 40:5 60:2:16 28:3", "i 31:1", "i 16:0.125:8:15", "i 12:0.5 40:1:8:0", "f 20:1:1:19",
    "f 8:1:0:-3", "f 8:1:0:30", "f 9:0", "f 9:-1"])
@pytest.mark.parametrize("dt", [BF, FL])
def test_axes(dev, spec, dt):
    """Every kind of axis, up to all entries there can be (beyond 64 the gradient
    takes two walks), shifts out of the buckets' range, no and negative rates."""
    Case(dev, [150, 20], None, 4, 2, 64, dt, spec).run()


@pytest.mark.parametrize("left,right,sinks", [(-1, 0, 0), (17, 0, 0), (0, 0, 0), (5, 9, 2),
                                              (40, 70, 16), (-1, 3, 0), (30, -1, 4)])
@pytest.mark.parametrize("dt,D", [(HF, 64), (BF, 128), (FL, 64)])
def test_windows(dev, left, right, sinks, dt, D):
    Case(dev, [300, 64, 7, 1], None, 4, 2, D, dt, "f 9:1 20:1:4", left, right, sinks).run()


@pytest.mark.parametrize("q_lens,k_lens", [([1, 1, 1], [5, 300, 1]), ([3, 0, 2], [2, 9, 0]),
                                           ([40, 5], [100, 3]), ([1], [2000])])
@pytest.mark.parametrize("H,Hk", [(6, 6), (8, 1), (8, 2)])
@pytest.mark.parametrize("right", [-1, 0])
def test_queries_beside_keys(dev, q_lens, k_lens, H, Hk, right):
    """A few queries, or one, against keys of their own; queries that see none."""
    for form in ("packed", "padded"):
        Case(dev, q_lens, k_lens, H, Hk, 64, HF, "i 24:0.25:4:23", right=right, form=form).run()


@pytest.mark.parametrize("dt,D", [(HF, 128), (BF, 64), (FL, 64), (FL, 128)])
def test_split_keys(dev, dt, D):
    """One query against many keys, and few rows of them, over several workgroups."""
    Case(dev, [1, 2], [5000, 1200], 8, 4, D, dt, "f 12:1 12:1:2", train=False).run()
    Case(dev, [900], None, 2, 1, D, dt, "f 12:1 12:1:2", right=0).run()


@pytest.mark.parametrize("H,Hk,spec", [(32, 1, "f 64:4 64:4"), (64, 2, "f 100:8 28:4"),
                                       (140, 1, "f 29:3"), (24, 24, "f 5:1")])
def test_many_heads(dev, H, Hk, spec):
    """Groups of many heads: up to 4096 entries of a key head's, heads that do not
    all fit in a tile of rows."""
    Case(dev, [33, 4], None, H, Hk, 32, BF, spec).run()


def test_many_rows(dev):
    Case(dev, [2500, 300], None, 2, 1, 64, BF, "f 20:1:2 16:2", 255, 0, 4).run()


def test_far_positions(dev):
    """int32 positions whose float32 values are the same, float32 ones far from 0
    and far apart, and ones that are not finite: no access out of range, and
    only the rows they belong to may differ."""
    c = Case(dev, [60, 50], None, 2, 2, 32, FL, "i 9:1 9:0.5")
    c.k_pos[:, 0] = 2000000000 + torch.arange(c.k_pos.shape[0], dtype=torch.int32) % 7
    c.run()
    c = Case(dev, [60, 50], None, 2, 2, 32, FL, "f 9:1 9:3:4", spread=1e30)
    c.run()
    c = Case(dev, [60, 50], None, 2, 2, 32, FL, "f 9:1 9:3:4")
    want = c.reference()
    row = c.q_seq[1][0] + 3
    c.k_pos[row, 0], c.k_pos[row + 1, 1], c.k_pos[row + 2, 0] = float("nan"), float("inf"), \
        float("-inf")
    got = dict(zip(NAMES, c.outputs(c.call())))
    first = slice(c.q_seq[0][0], c.q_seq[0][0] + 60)
    for name in NAMES[:-1]:
        check(got[name][first], tuple(x[first] for x in want[name]), name)
        assert bool(got[name].isfinite().all())


@pytest.mark.parametrize("dt,D,H,Hk", [(BF, 64, 12, 12), (HF, 128, 12, 6), (FL, 64, 12, 4)])
@pytest.mark.parametrize("window", [(-1, -1, 0), (-1, 0, 0), (500, 10, 5)])
@pytest.mark.parametrize("form", ["packed", "padded"])
def test_longer_sequences_of_several_heads(dev, dt, D, H, Hk, window, form):
    """(Padded, the plan's length is that of a slot; packed, it is the mean, which
    two sequences pass.)"""
    Case(dev, [5, 1311, 0, 1100, 1], None, H, Hk, D, dt, "f 9:0.3 12:1:2", *window,
         form=form).run()


@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2), (4, 1), (8, 1), (3, 1)])
@pytest.mark.parametrize("dt,D", [(BF, 64), (HF, 128), (FL, 64)])
@pytest.mark.parametrize("spec", ["i 12:0.25:4:11", "f 9:0.05 6:1:1", "f 20:-0.5:2"])
@pytest.mark.parametrize("window", [(100, 40, 3), (-1, 0, 0), (-1, -1, 0)])
def test_rows_in_order(dev, H, Hk, dt, D, spec, window):
    """Positions that grow along the sequence: most blocks of pairs fall into one
    bucket, the ones near the diagonal do not."""
    c = Case(dev, [260, 1, 140], None, H, Hk, D, dt, spec, *window)
    n = c.k_pos.shape[0]
    step = torch.arange(n)[:, None] * (3 if c.kind == "i" else 0.7)
    c.k_pos[:, :1] = (step + (2000000000 if c.kind == "i" else -90)).to(c.k_pos.dtype)
    c.run()


@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("spec", ["f 9:0.05", "f 12:0.5:2", "f 12:1:1:11"])
def test_position_that_is_not_finite_reaches_who_sees_it(dev, H, Hk, bad, spec):
    """Causal, positions in order: queries before the row do not see it, and their
    results do not change, though they share blocks of pairs with it."""
    for sign in (1, -1):
        c = Case(dev, [300], None, H, Hk, 64, BF, spec, right=0)
        c.k_pos[:, 0] = torch.arange(c.k_pos.shape[0]) * 0.5 * sign
        want = c.reference()
        r0 = c.q_seq[0][0]
        c.k_pos[r0 + 75] = bad
        c.q_pos = c.k_pos
        got = dict(zip(NAMES, c.outputs(c.call())))
        for name in ("out", "lse", "grad_q"):
            check(got[name][r0:r0 + 75], tuple(x[r0:r0 + 75] for x in want[name]), name)


@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 1)])
@pytest.mark.parametrize("spec", ["i 9:0.05", "i 12:0.5:2", "i 12:1:1:11"])
def test_distance_that_does_not_fit_is_of_its_pair_alone(dev, H, Hk, spec):
    """A row whose distance from others is no int32, hidden from all of them."""
    for sign in (1, -1):
        c = Case(dev, [300], None, H, Hk, 64, BF, spec, right=0)
        c.k_pos[:, 0] = (torch.arange(c.k_pos.shape[0]) - 2000) * sign
        want = c.reference()
        r0 = c.q_seq[0][0]
        c.k_pos[r0 + 75] = sign * (2 ** 31 - 1)
        c.q_pos = c.k_pos
        got = dict(zip(NAMES, c.outputs(c.call())))
        for name in ("out", "lse", "grad_q"):
            check(got[name][r0:r0 + 75], tuple(x[r0:r0 + 75] for x in want[name]), name)


@pytest.mark.parametrize("dt", [BF, FL])
@pytest.mark.parametrize("low", [float("-inf"), -3.4028234663852886e38, -1e30])
def test_hidden_by_the_table(dev, dt, low):
    """Entries that hide: some buckets, and all of one head's."""
    g = torch.Generator().manual_seed(8)
    table = torch.randn((4, 14), generator=g)
    table[0, :3] = low
    table[1, 9:] = low
    table[2] = low
    Case(dev, [90, 1, 40], None, 4, 2, 64, dt, "f 9:1 5:1", table=table).run()


def test_large_entries(dev):
    """Entries of +-1000: one bucket takes all."""
    g = torch.Generator().manual_seed(9)
    Case(dev, [90, 40], None, 4, 2, 64, BF, "f 9:1 5:1",
         table=1000 * torch.randn((4, 14), generator=g)).run()


@pytest.mark.parametrize("dt", [BF, FL])
def test_not_a_number_in_the_table(dev, dt):
    """One head's entry is not a number: other heads stay as they are."""
    c = Case(dev, [90, 40], None, 4, 4, 64, dt, "f 9:1 5:1")
    want = c.reference()
    c.table[3, 4] = float("nan")
    got = dict(zip(NAMES, c.outputs(c.call())))
    for name in NAMES[:-1]:
        check(got[name][:, :3], tuple(x[:, :3] for x in want[name]), name)
    check(got["grad_table"][:3], tuple(x[:3] for x in want["grad_table"]), "grad_table")
    assert bool(got["out"][:, 3].isnan().any())


@pytest.mark.parametrize("form", ["packed", "padded"])
@pytest.mark.parametrize("dt,D", [(HF, 64), (BF, 128), (FL, 64)])
def test_rows_of_no_sequence(dev, form, dt, D):
    """What rows of no sequence, and keys outside a window, hold reaches nothing."""
    c = Case(dev, [70, 0, 40], None, 4, 2, D, dt, "f 9:1 5:1", 20, 3, form=form)
    want = c.reference()
    dead = torch.ones(c.q.shape[0], dtype=torch.bool)
    for r0, n in c.q_seq:
        dead[r0:r0 + n] = False
    for t in (c.q, c.k, c.v, c.grad, c.k_pos):
        t[dead] = float("nan")
    call = c.call()
    marked = (call.out,) + call.grads[:3]
    if form == "packed":
        for t in marked:
            t.fill_(-7)
        for name in ("out", "grad_q", "grad_k", "grad_v"):
            want[name][0][dead.numpy()] = -7
    for name, t in zip(NAMES, c.outputs(call)):
        check(t, want[name], name)


@pytest.mark.parametrize("dt", [BF, HF])
def test_infinite_rows_outside_the_window(dev, dt):
    """An infinite value, key or gradient reaches only the rows that see it."""
    c = Case(dev, [200], None, 2, 1, 64, dt, "f 9:1 5:1", 10, 0)
    want = c.reference()
    r0 = c.q_seq[0][0]
    c.v[r0 + 50, 0, 3] = float("inf")
    c.k[r0 + 120, 0, 5] = float("nan")
    got = dict(zip(NAMES, c.outputs(c.call())))
    keep = np.zeros(c.q.shape[0], dtype=bool)
    keep[r0:r0 + 200] = True
    keep[r0 + 50:r0 + 61] = keep[r0 + 120:r0 + 131] = False
    for name in ("out", "lse", "grad_q"):
        check(got[name][torch.from_numpy(keep).to(dev)], tuple(x[keep] for x in want[name]), name)
    assert bool(got["out"][r0 + 55, :, 3].isinf().all())
    assert bool(got["lse"][r0 + 125].isnan().all())


def test_no_gradient_of_the_table(dev):
    """A table without a gradient: the others stay the same, bit for bit."""
    c = Case(dev, [200, 31], None, 4, 2, 64, BF, FOUR)
    a = c.outputs(c.call())
    call = c.call()
    call.grads = call.grads[:3] + (None,)
    b = c.outputs(call)
    assert b[-1] is None
    for x, y in zip(a[:-1], b[:-1]):
        assert torch.equal(x, y)


def test_nothing_written_elsewhere(dev):
    """Views inside larger buffers, a grad_table of one's own."""
    c = Case(dev, [200, 31], None, 4, 2, 64, BF, FOUR)
    want = c.reference()
    guard = torch.full((6, c.table.shape[1]), 5.0, device=dev)
    wide = torch.full((c.q.shape[0], 3, 4, 64), 5.0, dtype=BF, device=dev)
    call = c.call(out=wide[:, 1])
    call.grads = call.grads[:3] + (guard[1:5],)
    for name, t in zip(NAMES, c.outputs(call)):
        inside = torch.zeros(c.q.shape[0], dtype=torch.bool)
        for r0, n in c.q_seq:
            inside[r0:r0 + n] = True
        if name == "out":
            assert bool((t[~inside.to(dev)] == 5).all())
            check(t[inside.to(dev)], tuple(x[inside.numpy()] for x in want[name]), name)
        else:
            check(t, want[name], name)
    assert bool((guard[[0, 5]] == 5).all()) and bool((wide[:, ::2] == 5).all())


def test_empty(dev):
    """No rows in any sequence: the table's gradient is 0."""
    from point_cloud_tokenization_amd import fpstok as F

    c = Case(dev, [0, 0], None, 2, 2, 32, BF, "f 80:1")
    call = c.call()
    call.grads[3].fill_(3)
    assert bool((c.outputs(call)[-1] == 0).all())
    s = F.make_seqs(0, cu_seqlens=torch.zeros(1, dtype=torch.int32, device=dev))
    e = torch.zeros((0, 2, 32), device=dev)
    table = torch.ones((2, 4), device=dev)
    call = F.Attention(e, e, e, s, training=True, bias=F.RelativeBias(
        table, [F.BiasAxis(4)], torch.zeros((0, 1), device=dev)))
    call.grads[3].fill_(3)
    call()
    assert bool((call.backward(e)[-1] == 0).all())


def test_lengths_out_of_range(dev):
    """cu_seqlens outside the buffer, or running backwards, stay inside it."""
    from point_cloud_tokenization_amd import fpstok as F

    c = Case(dev, [40], None, 2, 1, 64, BF, "f 9:1 70:4")
    for cu in ([-5, 10, 90, 20, 1000], [30, 20, 10, 5, 0], [2 ** 31 - 1] * 5, [-2 ** 31] * 5):
        c.qs = F.make_seqs(c.q.shape[0], cu_seqlens=torch.tensor(cu, dtype=torch.int32,
                                                                 device=dev))
        c.outputs(c.call())


def test_same_result_every_run_and_on_another_stream(dev):
    c = Case(dev, [700, 1, 500], None, 4, 2, 64, BF, FOUR, 300, 20, 3)
    call = c.call()
    grad = c.grad.to(dev)
    first = [t.clone() for t in call()] + [t.clone() for t in call.backward(grad)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        out = list(call(stream)) + list(call.backward(grad, stream=stream))
        torch.cuda.synchronize()
        for a, b in zip(first, out):
            assert torch.equal(a, b)


def test_captured_graph(dev):
    """A captured step, replayed between eager calls on other inputs."""
    c = Case(dev, [150, 40], None, 4, 2, 64, BF, "f 40:5 60:2:16 28:3", 60, 0, 2)
    c2 = Case(dev, [150, 40], None, 4, 2, 64, BF, "f 40:5 60:2:16 28:3", 60, 0, 2, seed=2)
    call, other = c.call(), c2.call()
    grad, grad2 = c.grad.to(dev), c2.grad.to(dev)
    eager = [t.clone() for t in call()] + [t.clone() for t in call.backward(grad)]
    want2 = [t.clone() for t in other()] + [t.clone() for t in other.backward(grad2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call.backward(grad)
    outs = [call.out, call.lse] + list(call.grads)
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        got2 = list(other()) + list(other.backward(grad2))
        torch.cuda.synchronize()
        for a, b in zip(eager + want2, outs + got2):
            assert torch.equal(a, b)


def test_refusals_of_the_binding(dev):
    from point_cloud_tokenization_amd import fpstok as F

    c = Case(dev, [10], [10], 2, 2, 32, BF, "f 4:1 5:1")
    d = lambda t: t.to(dev)  # noqa: E731
    table, axes, qp, kp = d(c.table), c.axes, d(c.q_pos), d(c.k_pos)
    for args, err in (((table, axes[:1], qp, kp), ValueError), ((table, [], qp), ValueError),
                      ((table.bfloat16(), axes, qp), TypeError),
                      ((table, axes, qp.double()), TypeError),
                      ((table, axes, qp, kp.int()), TypeError),
                      ((table, axes, qp[:, :1]), ValueError)):
        with pytest.raises(err):
            F.RelativeBias(*args)
    ok = F.RelativeBias(table, axes, qp, kp)
    q, k = d(c.q), d(c.k)
    with pytest.raises(ValueError):  # keys of their own need positions
        F.Attention(q, k, k, c.qs, c.ks, bias=F.RelativeBias(table, axes, qp))
    with pytest.raises(ValueError):  # rows
        F.Attention(q, k, k, c.qs, c.ks, bias=F.RelativeBias(table, axes, qp[:5].contiguous(), kp))
    with pytest.raises(ValueError):  # heads
        F.Attention(q, k, k, c.qs, c.ks,
                    bias=F.RelativeBias(table[:1].contiguous(), axes, qp, kp))
    call = F.Attention(q, k, k, c.qs, c.ks, training=True, bias=ok)
    with pytest.raises(ValueError):
        call.grads = call.grads[:3]
    with pytest.raises(ValueError):
        call.grads = call.grads[:3] + (table[:, :4].contiguous(),)
