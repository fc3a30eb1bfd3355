"""Attention and rotary positions without a GPU: the float64 reference that the
GPU tests compare with (its gradients against differences, its masks against
their definition), and what the C ABI refuses on the host before touching the
device."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from point_cloud_tokenization_amd import build as fbuild
from point_cloud_tokenization_amd import fpstok as F
from tests import attention_ref as ref


@pytest.fixture(scope="module")
def L():
    if fbuild.is_stale():
        fbuild.build()
    return F.lib()


# ------------------------------------------------------------- reference

@pytest.mark.parametrize("tq,tk,left,right,sinks", [(5, 5, -1, -1, 0), (7, 4, 1, 0, 1),
                                                    (3, 9, 2, 1, 2), (6, 6, 0, -1, 3),
                                                    (4, 0, -1, -1, 0)])
def test_visible(tq, tk, left, right, sinks):
    got = ref.visible(tq, tk, left, right, sinks)
    for i in range(tq):
        for j in range(tk):
            p = i + tk - tq
            want = (right < 0 or j <= p + right) and (left < 0 or j >= p - left or j < sinks)
            assert bool(got[i, j]) == want


@pytest.mark.parametrize("left,right,sinks", [(-1, -1, 0), (2, 0, 1), (1, 1, 0)])
def test_reference_gradients_against_differences(left, right, sinks):
    g = torch.Generator().manual_seed(5)
    q = torch.randn((9, 4, 8), generator=g)
    k, v = torch.randn((10, 2, 8), generator=g), torch.randn((10, 2, 8), generator=g)
    go = torch.randn((9, 4, 8), generator=g)
    q_seq, k_seq = [(0, 4), (4, 0), (4, 5)], [(0, 6), (6, 1), (7, 3)]

    def loss(q, k, v):
        out = ref.attention(q, k, v, q_seq, k_seq, left, right, sinks)["out"][0]
        return float((out * go.double().numpy()).sum())

    r = ref.attention(q, k, v, q_seq, k_seq, left, right, sinks, grad=go)
    for name, t in (("grad_q", q), ("grad_k", k), ("grad_v", v)):
        d = torch.randn(t.shape, generator=g)
        step = 2.0 ** -12
        args = [x.double() if x is not t else None for x in (q, k, v)]
        hi = [t.double() + step * d.double() if a is None else a for a in args]
        lo = [t.double() - step * d.double() if a is None else a for a in args]
        diff = (loss64(hi, go, q_seq, k_seq, left, right, sinks) -
                loss64(lo, go, q_seq, k_seq, left, right, sinks)) / (2 * step)
        want = float((r[name][0] * d.double().numpy()).sum())
        # a central difference is off by step^2 / 6 times the third derivative
        # (a few units here): about 1e-6
        assert abs(diff - want) < 1e-4 * max(1.0, abs(want))
    assert loss(q, k, v) == pytest.approx(loss64([q.double(), k.double(), v.double()], go, q_seq,
                                                 k_seq, left, right, sinks), abs=1e-9)


def loss64(qkv, go, q_seq, k_seq, left, right, sinks):
    q, k, v = (x.numpy() for x in qkv)
    scale = float(np.float32(1.0 / math.sqrt(q.shape[2])))
    total = 0.0
    for (q0, tq), (k0, tk) in zip(q_seq, k_seq):
        ok = ref.visible(tq, tk, left, right, sinks)
        for h in range(q.shape[1]):
            hk = h // (q.shape[1] // k.shape[1])
            for i in range(tq):
                j = np.nonzero(ok[i])[0]
                if j.size == 0:
                    continue
                s = k[k0 + j, hk] @ q[q0 + i, h] * scale
                w = np.exp(s - s.max())
                total += float((w / w.sum()) @ (v[k0 + j, hk] @ go[q0 + i, h].double().numpy()))
    return total


def test_reference_rope_is_orthogonal():
    g = torch.Generator().manual_seed(6)
    x = torch.randn((5, 2, 12), generator=g, dtype=torch.float64)
    pos, fr = torch.randn((5, 2), generator=g), torch.rand(5, generator=g)
    for inter in (False, True):
        y, _ = ref.rope(x, pos, fr, [3, 2], inter)
        z, _ = ref.rope(torch.from_numpy(y), pos, fr, [3, 2], inter, inverse=True)
        np.testing.assert_allclose(z, x.numpy(), atol=1e-14)
        np.testing.assert_array_equal(y[..., 10:], x.numpy()[..., 10:])


# --------------------------------------------------------------- refusals

def _seqs(B=3, rows=100, cu=0x10000, tc=None, cap=0, max_len=0):
    return F.Seqs(B, rows, cu, tc, cap, max_len)


def _params(**kw):
    d = dict(num_heads=4, num_kv_heads=2, head_dim=64, dtype=F.BF16, window_left=-1,
             window_right=-1, num_sinks=0, scale=0.125)
    d.update(kw)
    return F.AttnParams(*[d[n] for n, _ in F.AttnParams._fields_])


def _heads(data=0x100000, row=256, head=64):
    return F.Heads(data, row, head)


def _forward(L, qs=None, ks=None, pr=None, lse=0x40000, ws=None, ws_bytes=0, **views):
    h = {n: _heads() for n in ("q", "k", "v", "out")}
    h.update(views)
    ref_ = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return L.fpstok_attention(ref_(qs or _seqs()), ref_(ks), ref_(pr or _params()),
                              *[ref_(h[n]) for n in ("q", "k", "v", "out")], lse, ws, ws_bytes,
                              None)


def _backward(L, qs=None, ks=None, pr=None, lse=0x40000, ws=0x1000000, ws_bytes=1 << 40, **views):
    names = ("q", "k", "v", "out", "grad_out", "grad_q", "grad_k", "grad_v")
    h = {n: _heads() for n in names}
    h.update(views)
    ref_ = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return L.fpstok_attention_backward(ref_(qs or _seqs()), ref_(ks), ref_(pr or _params()),
                                       *[ref_(h[n]) for n in names[:4]], lse,
                                       *[ref_(h[n]) for n in names[4:]], ws, ws_bytes, None)


BAD_SEQS = [dict(B=-1), dict(rows=-1), dict(max_len=-1), dict(cu=None), dict(tc=0x20000),
            dict(cu=0x10002), dict(cu=None, tc=0x20000, cap=0),
            dict(cu=None, tc=0x20000, cap=33), dict(cu=None, tc=0x20001, cap=33, rows=99)]
BAD_PARAMS = [dict(num_heads=0), dict(num_kv_heads=0), dict(num_kv_heads=3), dict(head_dim=0),
              dict(head_dim=60), dict(head_dim=136), dict(dtype=3), dict(dtype=-1),
              dict(window_left=-2), dict(window_right=-2), dict(num_sinks=-1),
              dict(num_sinks=65), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan),
              dict(scale=math.inf)]


@pytest.mark.parametrize("bad", BAD_SEQS)
def test_attention_refuses_sequences(L, bad):
    assert _forward(L, qs=_seqs(**bad)) == F.EINVAL
    assert _forward(L, ks=_seqs(**bad)) == F.EINVAL
    assert _backward(L, qs=_seqs(**bad)) == F.EINVAL
    assert F.lib().fpstok_last_error()


@pytest.mark.parametrize("bad", BAD_PARAMS)
def test_attention_refuses_params(L, bad):
    assert _forward(L, pr=_params(**bad)) == F.EINVAL
    assert _backward(L, pr=_params(**bad)) == F.EINVAL
    s = _seqs()
    assert L.fpstok_attention_workspace_size(ctypes.byref(s), None,
                                             ctypes.byref(_params(**bad)), 1) == 0


@pytest.mark.parametrize("name", ["q", "k", "v", "out"])
@pytest.mark.parametrize("bad", [dict(data=None), dict(data=0x100008), dict(row=252),
                                 dict(head=60), dict(row=-256)])
def test_attention_refuses_views(L, name, bad):
    assert _forward(L, **{name: _heads(**bad)}) == F.EINVAL
    assert _backward(L, **{name: _heads(**bad)}) == F.EINVAL


@pytest.mark.parametrize("name", ["grad_out", "grad_q", "grad_k", "grad_v"])
def test_attention_backward_refuses_views(L, name):
    assert _backward(L, **{name: _heads(data=0x100004)}) == F.EINVAL
    assert _backward(L, **{name: None}) == F.EINVAL


@pytest.mark.parametrize("bad", [dict(row=0), dict(row=64), dict(head=0), dict(head=56)])
def test_attention_refuses_overlapping_outputs(L, bad):
    assert _forward(L, out=_heads(**bad)) == F.EINVAL
    assert _backward(L, grad_q=_heads(**bad)) == F.EINVAL
    # heads outside rows ([heads, rows, D]) do not overlap: the call gets
    # past the views to the next check
    assert _backward(L, grad_q=_heads(row=64, head=6400), lse=None) == F.EINVAL
    assert b"lse" in L.fpstok_last_error()


def test_attention_refuses_counts_and_workspace(L):
    assert _forward(L, ks=_seqs(B=4)) == F.EINVAL
    assert _forward(L, lse=0x40002) == F.EINVAL
    assert _backward(L, ws=None) == F.EWORKSPACE
    assert _backward(L, ws_bytes=16) == F.EWORKSPACE
    assert _backward(L, ws=0x1000010) == F.EINVAL
    assert _forward(L, qs=_seqs(rows=1 << 31)) == F.EUNSUPPORTED
    assert _forward(L, qs=_seqs(B=(1 << 24) + 1)) == F.EUNSUPPORTED
    assert _forward(L, qs=_seqs(rows=(1 << 31) - 1), pr=_params(num_heads=64)) == F.EUNSUPPORTED
    assert _forward(L, q=_heads(row=1 << 24)) == F.EUNSUPPORTED
    assert _forward(L, q=_heads(head=1 << 41)) == F.EUNSUPPORTED


def test_attention_refuses_more_workgroups_than_a_launch_holds(L):
    """A launch holds 2^24 - 1 workgroups of 256 threads: one per 128 rows (32
    where sequences are short) and one per sequence, for every key head."""
    wide = _params(num_heads=64, num_kv_heads=64)
    fwd = {n: _heads(row=4096) for n in ("q", "k", "v", "out")}
    bwd = dict(fwd, **{n: _heads(row=4096) for n in ("grad_out", "grad_q", "grad_k", "grad_v")})
    for kw in (dict(qs=_seqs(B=1 << 20, rows=1 << 20), pr=wide),
               dict(qs=_seqs(B=1 << 18, rows=1 << 18), ks=_seqs(B=1 << 18, rows=1 << 18), pr=wide),
               dict(qs=_seqs(B=1 << 23, rows=100)),
               dict(qs=_seqs(B=1 << 20, rows=1 << 20, cu=None, tc=0x20000, cap=1), pr=wide)):
        assert _forward(L, **kw, **fwd) == F.EUNSUPPORTED
        assert b"workgroups" in L.fpstok_last_error()
        assert _backward(L, **kw, **bwd) == F.EUNSUPPORTED
        for backward in (0, 1):
            pr = kw.get("pr", _params())
            assert L.fpstok_attention_workspace_size(ctypes.byref(kw["qs"]), None,
                                                     ctypes.byref(pr), backward) == 0
    # the keys' gradients alone
    kw = dict(qs=_seqs(B=1 << 18, rows=1 << 18), ks=_seqs(B=1 << 18, rows=1 << 24), pr=wide)
    assert _backward(L, **kw, **bwd) == F.EUNSUPPORTED


def test_attention_nothing_to_do(L):
    assert _forward(L, qs=_seqs(B=0, rows=0, cu=None)) == F.OK
    assert _backward(L, qs=_seqs(B=0, rows=0, cu=None)) == F.OK


def _rope(L, seqs=None, pos=0x10000, freqs=0x20000, k=True, views=(), **kw):
    d = dict(num_heads=4, num_kv_heads=2, head_dim=64, dtype=F.F32, positions_dtype=F.F32,
             num_axes=4, pairs=(8, 8, 8, 8), interleaved=0, inverse=0)
    d.update(kw)
    d["pairs"] = (ctypes.c_int32 * 4)(*d["pairs"])
    pr = F.RopeParams(*[d[n] for n, _ in F.RopeParams._fields_])
    h = dict(q_in=_heads(), q_out=_heads(0x200000), k_in=_heads(0x300000), k_out=_heads(0x400000))
    if not k:
        h["k_in"] = h["k_out"] = None
    h.update(views)
    ref_ = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return L.fpstok_rope(ref_(seqs or _seqs()), ctypes.byref(pr), pos, freqs,
                         *[ref_(h[n]) for n in ("q_in", "q_out", "k_in", "k_out")], None)


@pytest.mark.parametrize("bad", [
    dict(num_heads=0), dict(num_kv_heads=0), dict(head_dim=63), dict(head_dim=0),
    dict(head_dim=1026), dict(dtype=3), dict(positions_dtype=1), dict(num_axes=0),
    dict(num_axes=5), dict(pairs=(8, 8, 8, 9)), dict(pairs=(0, 0, 0, 0)),
    dict(pairs=(-1, 8, 8, 8)), dict(interleaved=2), dict(inverse=-1), dict(pos=None),
    dict(freqs=None), dict(pos=0x10002), dict(seqs=_seqs(cu=None)),
    dict(views=dict(q_in=None)), dict(views=dict(q_out=None)), dict(views=dict(k_in=None)),
    dict(views=dict(k_out=None)), dict(views=dict(q_in=_heads(0x100002))),
    dict(views=dict(q_out=_heads(0x200000, row=64))),
    dict(views=dict(q_out=_heads(0x100000, row=512))),
])
def test_rope_refuses(L, bad):
    assert _rope(L, **bad) == F.EINVAL
    assert L.fpstok_last_error()


def test_rope_refuses_more_rows_than_a_launch_holds(L):
    assert _rope(L, seqs=_seqs(rows=1 << 27)) == F.EUNSUPPORTED
    assert _rope(L, seqs=_seqs(rows=1 << 27), head_dim=8, pairs=(1, 1, 1, 1)) == F.EUNSUPPORTED
    assert _rope(L, seqs=_seqs(rows=1 << 23), head_dim=1024, views=dict(
        q_out=_heads(0x200000, 4096, 1024), k_out=_heads(0x400000, 4096, 1024))) == F.EUNSUPPORTED


def test_rope_nothing_to_do(L):
    assert _rope(L, seqs=_seqs(B=0, rows=0, cu=None)) == F.OK
    assert _rope(L, seqs=_seqs(B=2, rows=0), k=False) == F.OK


def test_binding_refuses_before_the_library():
    q = torch.zeros((4, 2, 64))
    with pytest.raises(ValueError):
        F.make_heads(q, "q")
    with pytest.raises(ValueError):
        F.make_seqs(4)
    with pytest.raises(TypeError):
        F.make_seqs(4, cu_seqlens=torch.zeros(2))


def test_structs_match_the_header():
    assert ctypes.sizeof(F.Seqs) == 40 and ctypes.sizeof(F.Heads) == 24
    assert ctypes.sizeof(F.AttnParams) == 32 and ctypes.sizeof(F.RopeParams) == 48


def test_rope_frequencies():
    f = F.rope_frequencies((2, 0, 4), base=100.0, top=8.0)
    np.testing.assert_allclose(f.numpy(), [8, 0.8, 8, 8 / 100 ** 0.25, 0.8, 8 / 100 ** 0.75],
                               rtol=1e-6)


@pytest.mark.parametrize("scale", [2.36e38, 3.4e38])
def test_attention_refuses_scales_whose_kernel_factor_overflows(L, scale):
    """The kernels multiply scores by scale * log2(e) in float32."""
    assert _forward(L, pr=_params(scale=scale)) == F.EINVAL
    assert _backward(L, pr=_params(scale=scale)) == F.EINVAL
    # 2.35e38 log2(e) is 3.39e38, float32 ends at 3.403e38: past the parameters to the
    # next check
    assert _backward(L, pr=_params(scale=2.35e38), lse=None) == F.EINVAL
    assert b"lse" in L.fpstok_last_error()


def test_header_names_the_attention_for_a_c_caller(tmp_path):
    """A C program can ask whether the calls are declared."""
    src = tmp_path / "t.c"
    src.write_text('#include "fpstok.h"\n#if FPSTOK_ABI_VERSION != 3 || !FPSTOK_HAS_ATTENTION\n'
                   '#error old header\n#endif\nvoid *p = (void *)fpstok_attention;\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I",
                    os.path.dirname(F.HEADER), str(src)], check=True)
