"""Outputs of the residual step that overlap its inputs, and ones that lie beside
them in wider rows."""
import pytest
import torch

from tests import residual_ref as ref
from tests.test_gpu_residual import BF, FL, _compare, _layout

pytestmark = pytest.mark.gpu

C = 64


def test_training_beside_what_it_reads_again():
    from point_cloud_tokenization_amd import fpstok as F

    dev = torch.device("cuda:0")
    _, rows, s = _layout([50, 14], "packed", 0, 5, dev)
    wide = torch.zeros((rows + 1, C), device=dev)
    x, y = wide[:-1], torch.zeros((rows, C), dtype=BF, device=dev)
    pair = torch.zeros((rows, 2 * C), device=dev)
    for kw in (dict(x=x, x_out=wide[1:]), dict(x=wide[1:], x_out=x),
               dict(x=pair[:, :C], x_out=pair[:, 1:C + 1]),
               dict(x=pair[:, :C], x_out=pair[:, C - 1:2 * C - 1]),
               dict(x=x, h=wide.view(BF)[:-1, 8:C + 8]),
               dict(x=x, gate=y, gate_per="row", h=y)):
        with pytest.raises(ValueError, match="training"):
            F.Residual(kw.pop("x"), y, s, training=True, **kw)
    with pytest.raises(F.FpstokError, match="overlaps"):
        F.Residual(x, y, s, x_out=wide[1:])()


@pytest.mark.parametrize("side", [0, 1])
def test_side_by_side(side):
    """x and x_out as the two halves of wider rows, h between y's rows."""
    from point_cloud_tokenization_amd import fpstok as F

    dev = torch.device("cuda:0")
    seq, rows, s = _layout([30, 11], "packed", 1, 2, dev)
    o, grads = ref.make(rows, C, 2, FL, BF, "row", "rms", "rms", True, 31)
    want = ref.residual(seqs=seq, activation="silu", **o, **grads)
    d = {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in o.items()}
    pair = torch.zeros((rows, 2 * C), device=dev)
    two = torch.zeros((rows, 2 * C), dtype=BF, device=dev)
    cut = lambda t, k: t[:, C * k:C * (k + 1)]  # noqa: E731
    x, y = cut(pair, side), cut(two, side)
    x.copy_(d.pop("x"))
    y.copy_(d.pop("y"))
    call = F.Residual(x, y, s, activation="silu", training=True, x_out=cut(pair, 1 - side),
                      h=cut(two, 1 - side), **d)
    _compare(call, grads, want, dev)
