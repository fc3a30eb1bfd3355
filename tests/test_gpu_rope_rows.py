"""GPU tests of rotary positions where a workgroup has rows of several
sequences and of none."""
import numpy as np
import pytest
import torch

from tests import attention_ref as ref
from tests.gpu_util import log
from tests.test_gpu_attention import DT, F, rand  # noqa: F401

pytestmark = pytest.mark.gpu

PAIRS = (8, 8, 8, 8)


def turn(F, x, pos, fr, seqs, inter, in_place):  # noqa: F811
    src = x.cuda()
    r = F.Rope(src, None, pos.cuda(), fr.cuda(), PAIRS, seqs, inter,
               q_out=src if in_place else None)
    if not in_place:
        r.q_out.fill_(7.0)
    out = r()[0]
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cap,seqs,empty", [(5, 1000, 0.3), (3, 9000, 0.9), (64, 300, 0.7)])
def test_padded_slots(F, dtype, inter, in_place, cap, seqs, empty):  # noqa: F811
    """Slots of no row, whole workgroups of them among these, hold
    not-a-number values and positions, and get 0."""
    log("rope padded %d x %d, %s in place %s" % (seqs, cap, dtype, in_place))
    rng = np.random.default_rng(97)
    gen = torch.Generator().manual_seed(97)
    count = rng.integers(0, cap + 1, seqs)
    count[rng.random(seqs) < empty] = 0
    n = cap * seqs
    live = torch.from_numpy((np.arange(cap)[None] < count[:, None]).reshape(-1))
    x, pos = rand(gen, (n, 2, 72), DT[dtype]), torch.randn((n, 4), generator=gen)
    fr = F.rope_frequencies(PAIRS, top=20.0)
    val, tol = ref.rope(x, pos, fr, PAIRS, inter)
    val[~live.numpy()], tol[~live.numpy()] = 0.0, 0.0
    x[~live], pos[~live] = float("nan"), float("nan")
    s = F.make_seqs(n, token_count=torch.from_numpy(count).to(torch.int32).cuda(), capacity=cap)
    ref.check(turn(F, x, pos, fr, s, inter, in_place), (val, tol), "padded")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("first,last", [(0, 5000), (1, 4999), (2047, 2049), (4998, 5000),
                                        (333, 334), (17, 17)])
def test_packed_rows_in_the_middle(F, dtype, inter, first, last):  # noqa: F811
    log("rope packed rows %d to %d, %s" % (first, last, dtype))
    gen = torch.Generator().manual_seed(98)
    n = 5000
    live = np.zeros(n, dtype=bool)
    live[first:last] = True
    x, pos = rand(gen, (n, 2, 72), DT[dtype]), torch.randn((n, 4), generator=gen)
    fr = F.rope_frequencies(PAIRS, top=20.0)
    val, tol = ref.rope(x, pos, fr, PAIRS, inter)
    val[~live], tol[~live] = 7.0, 0.0
    hide = torch.from_numpy(~live)
    x[hide], pos[hide] = float("nan"), float("nan")
    cu = torch.tensor([first, (first + last) // 2, last], dtype=torch.int32)
    s = F.make_seqs(n, cu_seqlens=cu.cuda())
    ref.check(turn(F, x, pos, fr, s, inter, False), (val, tol), "packed")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n", [3, 2500])
@pytest.mark.parametrize("D,pairs", [(1024, (512,)), (1024, (100, 0, 21)), (1022, (511,)),
                                     (2, (1,)), (256, (1, 1, 1, 1))])
def test_largest_and_smallest_heads(F, dtype, inter, n, D, pairs):  # noqa: F811
    log("rope %d rows of %d, pairs %s, %s" % (n, D, pairs, dtype))
    gen = torch.Generator().manual_seed(99)
    q, k = rand(gen, (n, 3, D), DT[dtype]), rand(gen, (n, 1, D), DT[dtype])
    pos = torch.randn((n, len(pairs)), generator=gen)
    fr = F.rope_frequencies(pairs, top=20.0)
    s = F.make_seqs(n, cu_seqlens=torch.tensor([0, n], dtype=torch.int32).cuda())
    r = F.Rope(q.cuda(), k.cuda(), pos.cuda(), fr.cuda(), pairs, s, inter)
    for t, x in zip(r(), (q, k)):
        ref.check(t, ref.rope(x, pos, fr, pairs, inter), "heads of %d" % D)


def test_rows_past_32_bit_offsets(F):  # noqa: F811
    n, live = 2_900_000, 40
    log("rope %d rows" % n)
    gen = torch.Generator().manual_seed(100)
    x, pos = rand(gen, (live, 8, 128), torch.bfloat16), torch.randn((live, 4), generator=gen)
    far, where = torch.zeros((n, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        (n, 4), device="cuda")
    far[n - live:], where[n - live:] = x.cuda(), pos.cuda()
    fr = F.rope_frequencies(PAIRS, top=20.0)
    s = F.make_seqs(n, cu_seqlens=torch.tensor([0, n], dtype=torch.int32).cuda())
    out = F.Rope(far, None, where, fr.cuda(), PAIRS, s)()[0]
    torch.cuda.synchronize()
    ref.check(out[n - live:], ref.rope(x, pos, fr, PAIRS), "far rows")
    assert not bool(out[:n - live].any())
