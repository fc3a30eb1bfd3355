"""Attention whose pairs' entries lie in the plane, with sequences that end at the
buffer's last row and in any half of a tile of 64 keys."""
import numpy as np
import pytest
import torch

from tests import test_gpu_bias as base

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _tight(lens, form, dev):
    """No slot or row behind the last sequence."""
    from point_cloud_tokenization_amd import fpstok as F

    if form == "padded":
        cap = max(lens)
        t = torch.tensor(lens, dtype=torch.int32, device=dev)
        return ([(b * cap, n) for b, n in enumerate(lens)], cap * len(lens),
                F.make_seqs(cap * len(lens), token_count=t, capacity=cap))
    cu = np.concatenate([[0], np.cumsum(lens)])
    t = torch.tensor(cu, dtype=torch.int32, device=dev)
    return ([(int(c), n) for c, n in zip(cu, lens)], int(cu[-1]),
            F.make_seqs(int(cu[-1]), cu_seqlens=t, max_len=max(lens)))


@pytest.mark.parametrize("lens", [[1], [20], [7, 32], [40, 96], [64, 65], [33, 128, 160]])
@pytest.mark.parametrize("dt,D", [(BF, 128), (HF, 72), (BF, 64)])
@pytest.mark.parametrize("form", ["packed", "padded"])
@pytest.mark.parametrize("right", [-1, 0])
def test_last_row_of_the_buffer(monkeypatch, lens, dt, D, form, right):
    monkeypatch.setattr(base, "_layout", _tight)
    base.Case(torch.device("cuda:0"), lens, None, 12, 6, D, dt, "f 9:1 12:1:2", right=right,
              form=form).run()
