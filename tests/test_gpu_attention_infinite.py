"""GPU tests of attention and its gradients where infinite inputs are seen.

A score of -infinity (a key or a query with one -infinite element that meets
elements of one sign) has weight 0: the key adds nothing to its queries, and a
query whose every visible score is -infinity counts as one that sees no key.
What is left is compared with the reference of the same inputs with those
pairs hidden, whether the kernels see a tile whole or in part."""
import pytest
import torch

from tests.gpu_util import log
from tests.test_gpu_attention import DT, F, layout, rand  # noqa: F401

pytestmark = pytest.mark.gpu

INF = float("inf")


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
