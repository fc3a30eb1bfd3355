"""Attention with a learned bias without a GPU: the float64 reference that the GPU
tests compare with (its buckets against the distances they begin at, its
gradients against differences), and what the C ABI refuses on the host before
touching the device."""
import ctypes
import math

import numpy as np
import pytest
import torch

from point_cloud_tokenization_amd import build as fbuild
from point_cloud_tokenization_amd import fpstok as F
from tests import attention_ref, bias_ref as ref


@pytest.fixture(scope="module")
def L():
    if fbuild.is_stale():
        fbuild.build()
    return F.lib()


# ------------------------------------------------------------- reference

def test_linear_buckets():
    got = ref.buckets(np.zeros(1, np.float32), np.array([-9, -1, -.5, 0, .49, .5, 2, 99],
                                                        np.float32), F.BiasAxis(5, 1.0))
    # shift 2.5: bucket 2 is the distances from -1/2 to 1/2
    assert got[0].tolist() == [0, 1, 2, 2, 2, 3, 4, 4]
    got = ref.buckets(np.array([10], np.int32), np.array([4, 9, 10, 11, 30], np.int32),
                      F.BiasAxis(6, 0.5, shift=3))
    assert got[0].tolist() == [0, 2, 3, 3, 5]


def test_log_buckets():
    """Places with rate 1/8 and 8 steps a doubling: exact up to 7, then two, four
    ... places a bucket."""
    d = np.arange(0, 120)
    got = ref.buckets(np.zeros(1, np.int32), d.astype(np.int32),
                      F.BiasAxis(64, 1 / 8, shift=0, log_steps=8))[0]
    want = [x if x < 8 else 8 * int(math.log2(1 + x / 8)) +
            int(8 * ((1 + x / 8) / 2 ** int(math.log2(1 + x / 8)) - 1)) for x in d]
    assert got.tolist() == want
    both = ref.buckets(np.array([50], np.float32), np.array([49, 50, 51], np.float32),
                       F.BiasAxis(9, 8.0, log_steps=1))[0]
    assert both.tolist() == [1, 4, 7]


def test_reference_without_a_bias():
    """A table of one value is no bias."""
    g = torch.Generator().manual_seed(2)
    q, go = torch.randn((7, 4, 8), generator=g), torch.randn((7, 4, 8), generator=g)
    k, v = torch.randn((7, 2, 8), generator=g), torch.randn((7, 2, 8), generator=g)
    seq = [(0, 4), (4, 3)]
    a = attention_ref.attention(q, k, v, seq, seq, 2, 0, 1, grad=go)
    b = ref.attention(q, k, v, seq, seq, torch.full((4, 5), 0.7), [F.BiasAxis(5)],
                      torch.randn((7, 1), generator=g), left=2, right=0, sinks=1, grad=go)
    for name in a:
        want = a[name][0] + (float(np.float32(0.7)) if name == "lse" else 0.0)
        np.testing.assert_allclose(b[name][0], want, atol=1e-12)
    # a row's ds add up to 0
    np.testing.assert_allclose(b["grad_table"][0].sum(1), 0.0, atol=1e-12)


@pytest.mark.parametrize("left,right,sinks", [(-1, -1, 0), (2, 0, 1)])
def test_reference_gradients_against_differences(left, right, sinks):
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k, v, go = n(9, 4, 8), n(10, 2, 8), n(10, 2, 8), n(9, 4, 8)
    axes = [F.BiasAxis(4, 1.0), F.BiasAxis(3, 2.0, log_steps=1)]
    table, qp, kp = n(4, 7), n(9, 2), n(10, 2)
    q_seq, k_seq = [(0, 4), (4, 0), (4, 5)], [(0, 6), (6, 1), (7, 3)]

    def run(q, k, v, table, grad=None):
        return ref.attention(q, k, v, q_seq, k_seq, table, axes, qp, kp, left, right, sinks,
                             scale=1.0 / math.sqrt(8), grad=grad)

    leaves = dict(q=q.double(), k=k.double(), v=v.double(), table=table.double())
    res = run(q, k, v, table, go)
    for name in leaves:
        d = n(*leaves[name].shape).double()
        step = 2.0 ** -12
        both = []
        for s in (step, -step):
            moved = dict(leaves, **{name: leaves[name] + s * d})
            both.append(float((run(**moved)["out"][0] * go.double().numpy()).sum()))
        want = (both[0] - both[1]) / (2 * step)
        got = float((res["grad_" + name][0] * d.numpy()).sum())
        # a central difference is off by step^2 / 6 times the third derivative
        # (a few units here): about 1e-6
        assert abs(got - want) < 1e-4 * max(1.0, abs(want)), name


# --------------------------------------------------------------- refusals

A = 0x100000


def _seqs(B=3, rows=100, cu=0x10000):
    return F.Seqs(B, rows, cu, None, 0, 0)


def _params(**kw):
    d = dict(num_heads=4, num_kv_heads=2, head_dim=64, dtype=F.BF16, window_left=-1,
             window_right=-1, num_sinks=0, scale=0.125)
    d.update(kw)
    return F.AttnParams(*[d[n] for n, _ in F.AttnParams._fields_])


def _bias(**kw):
    d = dict(q_positions=A, k_positions=None, table=A, positions_dtype=F.F32, num_axes=2,
             buckets=(8, 8), log_steps=(0, 4), rate=(1.0, 1.0), shift=(4.0, 4.0))
    d.update(kw)
    i4 = lambda v: (ctypes.c_int32 * 4)(*v)  # noqa: E731
    f4 = lambda v: (ctypes.c_float * 4)(*v)  # noqa: E731
    for n in ("buckets", "log_steps"):
        d[n] = i4(d[n])
    for n in ("rate", "shift"):
        d[n] = f4(d[n])
    return F.RelBias(*[d[n] for n, _ in F.RelBias._fields_])


def _by(x):
    return None if x is None else ctypes.byref(x)


def _forward(L, bias, ks=None, pr=None, ws=None, ws_bytes=0):
    h = F.Heads(A, 4096, 64)
    return L.fpstok_attention_bias(_by(_seqs()), _by(ks), _by(pr or _params()), _by(bias), _by(h),
                                   _by(h), _by(h), _by(h), A, ws, ws_bytes, None)


def _backward(L, bias, ks=None, pr=None, table=A, ws=A, ws_bytes=1 << 40):
    h = F.Heads(A, 4096, 64)
    return L.fpstok_attention_bias_backward(
        _by(_seqs()), _by(ks), _by(pr or _params()), _by(bias), _by(h), _by(h), _by(h), _by(h), A,
        _by(h), _by(h), _by(h), _by(h), table, ws, ws_bytes, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,expect", [
    (dict(positions_dtype=F.F16), F.EINVAL), (dict(num_axes=0), F.EINVAL),
    (dict(num_axes=5), F.EINVAL), (dict(buckets=(0, 8)), F.EINVAL),
    (dict(buckets=(8, -1)), F.EINVAL), (dict(buckets=(100, 29)), F.EINVAL),
    (dict(buckets=(2 ** 31 - 1, 2)), F.EINVAL),
    (dict(log_steps=(0, 3)), F.EINVAL), (dict(log_steps=(32, 0)), F.EINVAL),
    (dict(log_steps=(-1, 0)), F.EINVAL), (dict(rate=(NAN, 1.0)), F.EINVAL),
    (dict(rate=(1.0, INF)), F.EINVAL), (dict(shift=(INF, 4.0)), F.EINVAL),
    (dict(shift=(4.0, 4.5)), F.EINVAL), (dict(shift=(4.0, 2.0 ** 21)), F.EINVAL),
    (dict(q_positions=None), F.EINVAL), (dict(table=None), F.EINVAL),
    (dict(q_positions=A + 2), F.EINVAL), (dict(k_positions=A + 1), F.EINVAL),
    (dict(table=A + 2), F.EINVAL),
])
def test_bias_refusals(L, kw, expect):
    for call in (_forward, _backward):
        assert call(L, _bias(**kw)) == expect
        assert L.fpstok_last_error() != b""


def test_other_refusals(L):
    for call in (_forward, _backward):
        assert call(L, None) == F.EINVAL
        # keys of their own need positions of their own
        assert call(L, _bias(), ks=_seqs()) == F.EINVAL
        assert call(L, _bias(), pr=_params(head_dim=12)) == F.EINVAL
        # 64 heads on one of 128 buckets: 8192 entries
        assert call(L, _bias(num_axes=1, buckets=(128,), log_steps=(0,)),
                    pr=_params(num_heads=64, num_kv_heads=1)) == F.EUNSUPPORTED
    assert _backward(L, _bias(), table=A + 2) == F.EINVAL
    assert _backward(L, _bias(), ws=None) == F.EWORKSPACE
    assert _backward(L, _bias(), ws_bytes=1024) == F.EWORKSPACE
    assert _backward(L, _bias(), ws=A + 64) == F.EINVAL


def test_workspace_size(L):
    """The gradients' adds the row tiles' parts of the table's: 64 entries at most."""
    plain, size = L.fpstok_attention_workspace_size, L.fpstok_attention_bias_workspace_size
    s, p = _seqs(), _params()
    assert size(_by(s), None, _by(p), _by(_bias()), 0) == plain(_by(s), None, _by(p), 0)
    base = plain(_by(s), None, _by(p), 1)
    # at most 100 * 2 / 128 + 3 tiles of 4 heads
    parts = size(_by(s), None, _by(p), _by(_bias()), 1) - base
    assert 4 * 16 * 4 <= parts <= 256 * math.ceil(4 * 4 * 16 * 4 / 256)
    many = _bias(num_axes=1, buckets=(128,), log_steps=(0,))
    assert size(_by(s), None, _by(p), _by(many), 1) - base <= 256 * math.ceil(4 * 4 * 64 * 4 / 256)
    assert size(_by(s), None, _by(p), _by(_bias(num_axes=0)), 1) == 0


def test_struct_layout():
    assert ctypes.sizeof(F.RelBias) == 96 and F.RelBias.shift.offset == 80
