"""GPU tests of attention and rotary positions constructed on one stream and
called on another."""
import pytest
import torch

from tests import attention_ref as ref
from tests.gpu_util import log
from tests.test_gpu_attention import F, layout, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def occupy(n=40):
    """Some milliseconds of work on the current stream."""
    x = torch.ones((4096, 4096), device="cuda")
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    for _ in range(n):
        torch.matmul(x, x, out=y)


@pytest.mark.parametrize("given", [False, True])
def test_first_call_on_another_stream(F, given):  # noqa: F811
    """The constructor's fills are queued behind other work on its stream: a
    call on a stream that does not wait by itself gives whole results, before and
    after they ran."""
    log("first call on another stream, output given: %s" % given)
    gen = torch.Generator().manual_seed(95)
    lens, H, Hk, D, pairs = [200, 0, 77], 4, 2, 64, (8, 8, 8, 8)
    qs, seq, n = layout(F, lens, "packed")
    q, k, v, go = (rand(gen, (n, h, D), torch.bfloat16) for h in (H, Hk, Hk, H))
    pos, fr = torch.randn((n, 4), generator=gen), F.rope_frequencies(pairs)
    dq, dk, dv, dgo, dpos, dfr = (t.cuda() for t in (q, k, v, go, pos, fr))
    outs = [torch.empty_like(dq) for _ in range(2)] if given else [None] * 2
    side = torch.cuda.Stream()
    F.Attention(dq, dk, dv, qs, training=True).backward(dgo, side)  # (loads the kernels)
    occupy()
    rope = F.Rope(dq, dk, dpos, dfr, pairs, qs, q_out=outs[0])
    turned = rope(stream=side)
    att = F.Attention(dq, dk, dv, qs, training=True, out=outs[1])
    occupied = not torch.cuda.current_stream().query()
    got = att(side) + att.backward(dgo, side)
    torch.cuda.synchronize()
    assert occupied, "the first stream was done too early to tell"
    for t, x in zip(turned, (q, k)):
        ref.check(t, ref.rope(x, pos, fr, pairs), "rope")
    want = ref.attention(q, k, v, seq, seq, grad=go)
    for name, t in zip(("out", "lse", "grad_q", "grad_k", "grad_v"), got):
        ref.check(t, want[name], name)


def test_captured_on_another_stream_than_constructed(F):  # noqa: F811
    """Constructed inside a capture, or ahead of one without a call in between;
    called on a third stream afterwards."""
    gen = torch.Generator().manual_seed(96)
    qs, seq, n = layout(F, [60, 130], "packed")
    q, k, v, go = (rand(gen, (n, h, 64), torch.bfloat16) for h in (4, 2, 2, 4))
    dev = [t.cuda() for t in (q, k, v)]
    dgo = go.cuda()
    want = ref.attention(q, k, v, seq, seq, grad=go)
    F.Attention(*dev, qs, training=True)()  # (loads the kernels)
    before = F.Attention(*dev, qs, training=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        inside = F.Attention(*dev, qs, training=True)
        for att in (before, inside):
            att()
            att.backward(dgo)
    side = torch.cuda.Stream()
    for turn in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for att in (before, inside):
            for name, t in zip(("out", "lse", "grad_q", "grad_k", "grad_v"),
                               (att.out, att.lse) + att.grads):
                ref.check(t, want[name], "replay %d %s" % (turn, name))
        for t in (before.out, before.lse) + before.grads:
            t.fill_(9.0)
        torch.cuda.synchronize()
        got = before(side) + before.backward(dgo, side)
        torch.cuda.synchronize()
        for name, t in zip(("out", "lse", "grad_q", "grad_k", "grad_v"), got):
            ref.check(t, want[name], "eager %d %s" % (turn, name))


def test_buffers_outlive_the_object_on_another_stream(F):  # noqa: F811
    """The memory of a plan that is dropped while its call waits on another
    stream is not given to a new tensor."""
    qs, _, n = layout(F, [700], "packed")
    q = torch.ones((n, 2, 64), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    F.Attention(q, q, q, qs, training=True)()  # (loads the kernels)
    torch.cuda.synchronize()
    att = F.Attention(q, q, q, qs, training=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        occupy()
    att(side)
    att.backward(q, side)
    held = {t.data_ptr(): t.numel() * t.element_size()
            for t in (att.ws, att.lse, att.out) + att.grads}
    del att
    new = [torch.empty(size, dtype=torch.uint8, device="cuda") for size in held.values()]
    busy = not side.query()
    torch.cuda.synchronize()
    assert busy, "the other stream was done too early to tell"
    assert not any(t.data_ptr() in held for t in new)
