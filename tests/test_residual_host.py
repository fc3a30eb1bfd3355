"""The residual step without a GPU: the float64 reference that the GPU tests
compare with (its gradients against differences, its norms against their
definition), and what the C ABI refuses on the host before touching the
device."""
import ctypes

import numpy as np
import pytest
import torch

from point_cloud_tokenization_amd import build as fbuild
from point_cloud_tokenization_amd import fpstok as F
from tests import residual_ref as ref


@pytest.fixture(scope="module")
def L():
    if fbuild.is_stale():
        fbuild.build()
    return F.lib()


# ------------------------------------------------------------- reference

@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_reference_norms(kind):
    x = torch.randn((5, 12), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    got = ref.residual(x, None, [(0, 5)], pre_norm=kind, eps=0.25)["h"][0]
    if kind == "layer":
        want = torch.nn.functional.layer_norm(x, (12,), eps=0.25)
    else:
        want = x / torch.sqrt((x * x).mean(1, keepdim=True) + 0.25)
    np.testing.assert_allclose(got, want.numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("post,pre,gate,act,block", [
    ("rms", "rms", "row", "sigmoid", True), ("layer", "layer", "sequence", "silu", True),
    ("none", "rms", "row", "none", True), ("layer", "none", "none", "none", True),
    ("none", "layer", "none", "none", False)])
def test_reference_gradients_against_differences(post, pre, gate, act, block):
    seqs, rows, C = [(1, 3), (4, 0), (4, 2)], 7, 6
    f64 = torch.float64
    o, grads = ref.make(rows, C, 3, f64, f64, gate, post, pre, block, 3, block)
    o = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in o.items()}
    x, y = o.pop("x"), o.pop("y")
    res = ref.residual(x, y, seqs, activation=act, **o, **grads)

    def loss(x, y, o):
        r = ref.residual(x, y, seqs, activation=act, **o)
        total = (r["x_out"][0] * grads["grad_x_out"].numpy()).sum()
        return total + ((r["h"][0] * grads["grad_h"].numpy()).sum() if "h" in r else 0.0)

    g = torch.Generator().manual_seed(4)
    leaves = dict(o, x=x, y=y)
    checked = 0
    for name, t in leaves.items():
        if not isinstance(t, torch.Tensor):
            continue
        d = torch.randn(t.shape, generator=g, dtype=f64)
        step = 2.0 ** -16
        both = []
        for s in (step, -step):
            moved = dict(leaves, **{name: t + s * d})
            both.append(loss(moved.pop("x"), moved.pop("y"), moved))
        want = (both[0] - both[1]) / (2 * step)
        got = float((res["grad_" + name][0] * d.numpy()).sum())
        # a central difference is off by step^2 / 6 times the third derivative
        # (below 1e4 here) and by 2^-52 of the losses over the step
        assert abs(got - want) < 1e-5 * max(1.0, abs(want)), name
        checked += 1
    assert checked >= (2 if block else 1)


def test_reference_keeps_to_the_sequences():
    o, grads = ref.make(6, 5, 2, torch.float32, torch.float32, "none", "rms", "rms", True, 9)
    x, y = o.pop("x"), o.pop("y")
    a = ref.residual(x, y, [(1, 2), (4, 1)], **o, **grads)
    x[0] = y[3] = grads["grad_h"][5] = float("nan")
    b = ref.residual(x, y, [(1, 2), (4, 1)], **o, **grads)
    for name in a:
        np.testing.assert_array_equal(a[name][0], b[name][0])


# --------------------------------------------------------------- refusals

A = 0x100000


def _seqs(B=3, rows=100, cu=0x10000, tc=None, cap=0):
    return F.Seqs(B, rows, cu, tc, cap, 0)


def _params(**kw):
    d = dict(width=64, stream_dtype=F.F32, branch_dtype=F.BF16, post_norm=1, pre_norm=1,
             gate_per=1, activation=1, eps=1e-6)
    d.update(kw)
    return F.ResidualParams(*[d[n] for n, _ in F.ResidualParams._fields_])


def _by(x):
    return None if x is None else ctypes.byref(x)


def _views(names, kw):
    return [_by(kw[n] if n in kw else F.Rows(A, 64)) for n in names]


def _forward(L, s=None, p=None, w=None, stats=A, **kw):
    return L.fpstok_residual(_by(s or _seqs()), _by(p or _params()),
                             _by(w or F.ResidualWeights()),
                             *_views(("x", "y", "gate", "x_out", "h"), kw), stats, None)


def _backward(L, s=None, p=None, w=None, stats=A, grads=None, ws=A, ws_bytes=1 << 30, **kw):
    return L.fpstok_residual_backward(
        _by(s or _seqs()), _by(p or _params()), _by(w or F.ResidualWeights()),
        *_views(("x", "y", "gate"), kw), stats,
        *_views(("grad_x_out", "grad_h", "grad_x", "grad_y", "grad_gate"), kw),
        _by(grads or F.ResidualWeights()), ws, ws_bytes, None)


BOTH = [
    (dict(p=_params(width=0)), F.EINVAL), (dict(p=_params(width=8193)), F.EINVAL),
    (dict(p=_params(branch_dtype=3)), F.EINVAL), (dict(p=_params(branch_dtype=-1)), F.EINVAL),
    (dict(p=_params(stream_dtype=F.F16)), F.EINVAL),
    (dict(p=_params(post_norm=3)), F.EINVAL), (dict(p=_params(pre_norm=-1)), F.EINVAL),
    (dict(p=_params(gate_per=3)), F.EINVAL), (dict(p=_params(activation=3)), F.EINVAL),
    (dict(p=_params(eps=0.0)), F.EINVAL), (dict(p=_params(eps=1e-40)), F.EINVAL), (dict(p=_params(eps=float("nan"))), F.EINVAL),
    (dict(p=_params(eps=float("inf"))), F.EINVAL),
    (dict(s=_seqs(B=-1)), F.EINVAL), (dict(s=_seqs(cu=None)), F.EINVAL),
    (dict(s=_seqs(rows=1 << 31)), F.EUNSUPPORTED),
    (dict(s=_seqs(cu=None, tc=0x10000, cap=30)), F.EINVAL),
    (dict(x=None), F.EINVAL), (dict(x=F.Rows(None, 64)), F.EINVAL),
    (dict(x=F.Rows(A + 2, 64)), F.EINVAL), (dict(x=F.Rows(A, -64)), F.EINVAL),
    (dict(x=F.Rows(A, (1 << 23) + 1)), F.EUNSUPPORTED),
    (dict(y=F.Rows(A + 1, 64)), F.EINVAL), (dict(y=None), F.EINVAL),
    (dict(y=None, p=_params(post_norm=0)), F.EINVAL),
    (dict(gate=None), F.EINVAL), (dict(p=_params(gate_per=0, activation=0)), F.EINVAL),
    (dict(gate=None, p=_params(gate_per=0, activation=1)), F.EINVAL),
    (dict(w=F.ResidualWeights(post_weight=A + 2)), F.EINVAL),
    (dict(w=F.ResidualWeights(post_bias=A), p=_params(post_norm=0)), F.EINVAL),
]


@pytest.mark.parametrize("kw,expect", BOTH + [
    (dict(x_out=F.Rows(A, 63)), F.EINVAL), (dict(h=None), F.EINVAL),
    (dict(p=_params(pre_norm=0)), F.EINVAL),
    (dict(p=_params(pre_norm=0), x_out=None, h=None), F.EINVAL),
    (dict(x_out=F.Rows(A, 128)), F.EINVAL),  # in place with another stride
    (dict(stats=A + 4), F.EINVAL),
    (dict(w=F.ResidualWeights(pre_weight=A), p=_params(pre_norm=0), h=None), F.EINVAL),
])
def test_forward_refusals(L, kw, expect):
    assert _forward(L, **kw) == expect
    assert L.fpstok_last_error() != b""


@pytest.mark.parametrize("kw,expect", BOTH + [
    (dict(grad_x_out=None, grad_h=None), F.EINVAL),
    (dict(p=_params(pre_norm=0)), F.EINVAL),
    (dict(grad_x=F.Rows(A, 63)), F.EINVAL), (dict(grad_x=F.Rows(A, 128)), F.EINVAL),
    (dict(grad_y=F.Rows(A + 1, 64)), F.EINVAL),
    (dict(gate=None, p=_params(gate_per=0, activation=0)), F.EINVAL),  # grad_gate is given
    (dict(stats=None), F.EINVAL), (dict(stats=A + 8), F.EINVAL),
    (dict(grads=F.ResidualWeights(scale=A)), F.EINVAL),
    (dict(grads=F.ResidualWeights(scale=A + 2), w=F.ResidualWeights(scale=A)), F.EINVAL),
    (dict(ws=None), F.EWORKSPACE), (dict(ws_bytes=64), F.EWORKSPACE), (dict(ws=A + 16), F.EINVAL),
])
def test_backward_refusals(L, kw, expect):
    assert _backward(L, **kw) == expect
    assert L.fpstok_last_error() != b""


def test_nothing_to_do(L):
    """No rows, or no sequences: nothing is enqueued by the forward call."""
    none = F.Rows(None, 0)
    kw = dict(x=none, y=none, gate=none, x_out=none, h=none)
    assert _forward(L, s=_seqs(rows=0), **kw) == F.OK
    assert _forward(L, s=_seqs(B=0, rows=0, cu=None), **kw) == F.OK


def test_workspace_size(L):
    size = L.fpstok_residual_workspace_size
    s, p = _seqs(), _params(gate_per=0, activation=0)
    # at least one part of five weights; a gate per sequence adds its parts
    small = size(_by(s), _by(p))
    assert small >= 5 * 64 * 4 and small % 256 == 0
    assert size(_by(s), _by(_params(gate_per=2))) >= small + 3 * 64 * 4
    assert size(_by(s), _by(_params(width=0))) == 0
    assert size(_by(_seqs(rows=0)), _by(p)) == 0


def test_struct_layout():
    assert ctypes.sizeof(F.Rows) == 16 and ctypes.sizeof(F.ResidualParams) == 32
    assert ctypes.sizeof(F.ResidualWeights) == 40
