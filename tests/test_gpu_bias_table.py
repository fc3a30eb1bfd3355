"""The gradient of the bias's table where a bucket's weights are small beside the
row's, and where values are not finite: float32 sums of terms that are not rounded,
within the bounds of tests/bias_ref.py."""
import numpy as np
import pytest
import torch

from tests.attention_ref import check
from tests.test_gpu_bias import BF, FL, HF, NAMES, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


# by positions (few heads) with one, two and three axes, of over 64 buckets, from the plane
KINDS = [(4, 2, "f 9:1"), (4, 2, "f 9:1 5:1"), (2, 2, "f 9:1 7:1:2 5:1"), (2, 1, "f 9:1 70:4"),
         (12, 6, "f 9:1 5:1"), (12, 12, "f 9:1 9:1 7:1:2"), (12, 4, "f 9:1 9:1 9:1.5 14:2:2")]


@pytest.mark.parametrize("H,Hk,spec", KINDS)
@pytest.mark.parametrize("dt", [FL, BF])
@pytest.mark.parametrize("low", [-8.0, -12.0, -15.0, -18.0, -25.0, -30.0, -60.0])
def test_buckets_of_small_weights(dev, H, Hk, spec, dt, low):
    c = Case(dev, [200, 70], None, H, Hk, 64, dt, spec)
    c.table[:, 2] = low
    c.table[:, -1] = low + 1
    c.run()


@pytest.mark.parametrize("H,Hk,spec", KINDS)
@pytest.mark.parametrize("dt", [FL, BF])
@pytest.mark.parametrize("size", [1e6, 1e9])
@pytest.mark.parametrize("low", [float("-inf"), -90.0])
def test_large_value_behind_a_hidden_bucket(dev, H, Hk, spec, dt, size, low):
    """A key that the table hides from all others, or whose weights are 0 beside
    theirs, holds a value far larger than theirs.

    exp(-90) = 8e-40 is below 2^-126 = 1.2e-38, the smallest normal float32 number: such
    a weight may come out as 0, so it is off by up to 2^-126.  The bound of grad_table
    counts that; in out and grad_v (n terms of w times a value v or g) it is n 2^-126
    times the largest value, in grad_q and grad_k (n terms of scale w (dp - delta) times
    a value of k or q) with M = 2 D max|g| max|v| >= |dp - delta| it is scale n 2^-126 M
    times the largest one.  n: 100 pairs of a row, of a key 100 times its heads."""
    c = Case(dev, [100], None, H, Hk, 64, dt, spec, spread=1.0)
    r0 = c.q_seq[0][0]
    c.k_pos[r0 + 40, 0] = 1000.0  # (from it every distance falls into bucket 0, to it into the last)
    n0 = c.axes[0].buckets
    c.table[:, n0 - 1] = low
    c.v[r0 + 40] = size
    # a query of its own would see it whole: no gradient comes back there
    c.grad[r0 + 40] = 0
    top = {k: float(t.double().abs().max()) for k, t in (("q", c.q), ("k", c.k), ("v", c.v),
                                                        ("g", c.grad))}
    n, M = 100 * 2.0 ** -126, 2 * 64 * top["g"] * top["v"]
    off = dict(out=n * top["v"], grad_v=n * (H // Hk) * top["g"], grad_q=n * M * top["k"] / 8,
               grad_k=n * (H // Hk) * M * top["q"] / 8)
    want = c.reference()
    for name, t in zip(NAMES, c.outputs(c.call())):
        value, bound = want[name]
        check(t, (value, bound + off.get(name, 0.0) * (value != 0)), name)


@pytest.mark.parametrize("H,Hk,spec", [k for k in KINDS if k[0] != k[1]])
@pytest.mark.parametrize("dt", [FL, BF, HF])
@pytest.mark.parametrize("where", ["q", "k", "v", "grad", "table"])
def test_not_a_number_reaches_the_entries_it_adds_to(dev, H, Hk, spec, dt, where):
    c = Case(dev, [90, 40], None, H, Hk, 64, dt, spec)
    want = c.reference()
    r0, nan = c.q_seq[0][0], float("nan")
    heads = [3] if where in ("q", "table", "grad") and H > 3 else [0]
    if where == "table":
        c.table[heads[0], 4] = nan
    elif where in ("q", "grad"):
        (c.q if where == "q" else c.grad)[r0 + 30, heads[0], 5] = nan
    else:
        (c.k if where == "k" else c.v)[r0 + 30, 0, 5] = nan
        heads = list(range(H // Hk))
    got = dict(zip(NAMES, c.outputs(c.call())))
    keep = [h for h in range(H) if h not in heads]
    check(got["grad_table"][keep], tuple(x[keep] for x in want["grad_table"]), "grad_table")
    # the entries of the pairs that the row is in (all of its sequence for k and v)
    from tests import bias_ref

    p = c.q_pos.numpy()
    first = 0
    for a, axis in enumerate(c.axes):
        b = bias_ref.buckets(p[r0:r0 + 90, a], p[r0:r0 + 90, a], axis)
        if where in ("q", "grad"):
            b = b[30]
        elif where == "table":
            if a > 0:
                break
            b = b[(b == 4).any(1)]
        reached = np.unique(b) + first
        for h in heads:
            assert bool(got["grad_table"][h][torch.from_numpy(reached).to(dev)].isnan().all())
        first += axis.buckets
