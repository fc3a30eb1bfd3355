"""Gradients of gates per sequence where the sequences run backwards: nothing
outside the buffers is read or written (what the gates of such sequences get is not
said)."""
import pytest
import torch

from tests import residual_ref as ref
from tests.test_gpu_residual import BF, FL, _call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cu", [[20, 0, 40, 40, 40], [0, 40, 10, 5, 20], [39, 0, 1, 0, 40],
                                [10, 40, 0, 40, 12], [2 ** 31 - 1, 0, 40, -1, 40]])
def test_sequences_that_run_backwards(cu):
    from point_cloud_tokenization_amd import fpstok as F

    dev, rows, C = torch.device("cuda:0"), 40, 64
    o, grads = ref.make(rows, C, 4, FL, BF, "sequence", "rms", "rms", True, 24)
    s = F.make_seqs(rows, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev))
    guard = torch.full((rows + 8, C), 3.0, device=dev)
    call = _call(o, s, dev, "silu", x_out=guard[4:-4])
    call()
    call.backward(**{k: v.to(dev) for k, v in grads.items()})
    torch.cuda.synchronize()
    assert bool((guard[:4] == 3).all()) and bool((guard[-4:] == 3).all())
