"""The pieces of an encoder layer together, as a model runs them on the tokens of a
batch of events: tokenize, pack, norm, rotary positions, attention with the bias,
the residual step, and the gradients back through all of it.  Every stage is
checked against its reference on what the stage before it really wrote, so each
bound is that of one stage; then the layer is captured and replayed."""
import numpy as np
import pytest
import torch

from tests import attention_ref, bias_ref, residual_ref
from tests.attention_ref import check

pytestmark = pytest.mark.gpu

H, D, PATCHES = 4, 32, 16
C = H * D


def _events(dev):
    """Packed tokens and centroids of a tokenized batch, in buffers of B * P rows."""
    from point_cloud_tokenization_amd import fpstok as F
    from point_cloud_tokenization_amd import synth

    b = synth.make_batch("tiny_uniform")
    t = lambda k: torch.from_numpy(b[k]).to(dev)  # noqa: E731
    out = F.tokenize(t("coords"), t("features"), t("offsets"), num_patches=PATCHES, pool="mean",
                     charge_col=b["charge_col"])
    count, B = out["token_count"], out["token_count"].numel()
    w = torch.randn((out["pooled"].shape[2], C), generator=torch.Generator().manual_seed(3))
    rows = (out["pooled"].reshape(B * PATCHES, -1) @ w.to(dev)).view(B, PATCHES, C).contiguous()
    tokens, places = torch.zeros((B * PATCHES, C), device=dev), torch.zeros((B * PATCHES, 4),
                                                                            device=dev)
    cu = torch.zeros(B + 1, dtype=torch.int32, device=dev)
    F.pack(count, rows, tokens, None, cu)
    F.pack(count, out["centroids"], places, None, cu)
    torch.cuda.synchronize()
    first = cu.cpu().tolist()
    return tokens, places, F.make_seqs(B * PATCHES, cu_seqlens=cu), \
        [(a, b - a) for a, b in zip(first, first[1:])]


class Layer:
    def __init__(self, tokens, places, seqs, dt):
        from point_cloud_tokenization_amd import fpstok as F

        dev, rows, B = tokens.device, tokens.shape[0], seqs.num_seqs
        g = torch.Generator().manual_seed(4)
        n = lambda *s: torch.randn(s, generator=g).to(dev)  # noqa: E731
        self.tokens, self.places = tokens, places
        self.w_first = dict(pre_norm="layer", pre_weight=1 + 0.1 * n(C), pre_bias=0.1 * n(C))
        self.h = torch.zeros((rows, C), dtype=dt, device=dev)
        self.norm = F.Residual(tokens, None, seqs, h=self.h, training=True, **self.w_first)
        heads = self.h.view(rows, H, D)
        self.pairs = [4, 4, 4, 4]
        self.freqs = F.rope_frequencies(self.pairs, top=4.0, device=dev)
        self.rope = F.Rope(heads, None, places, self.freqs, self.pairs, seqs)
        self.turned = self.rope.q_out
        self.axes = [F.BiasAxis(9, 4.0) for _ in range(3)] + [F.BiasAxis(12, 8.0, log_steps=2)]
        self.table = 0.5 * n(H, 39)
        self.attn = F.Attention(self.turned, self.turned, heads, seqs, training=True,
                                bias=F.RelativeBias(self.table, self.axes, places))
        self.gate = n(B, C).to(dt)
        self.w_step = dict(post_norm="rms", post_weight=1 + 0.1 * n(C), scale=0.5 + 0.1 * n(C),
                           pre_norm="rms", pre_weight=1 + 0.1 * n(C))
        self.step = F.Residual(tokens, self.attn.out.view(rows, C), seqs, gate=self.gate,
                               gate_per="sequence", activation="sigmoid", training=True,
                               **self.w_step)
        # what comes back to the heads is turned back in place
        self.back = torch.zeros((rows, H, D), dtype=dt, device=dev)
        self.unrope = F.Rope(self.back, None, places, self.freqs, self.pairs, seqs,
                             q_out=torch.zeros_like(self.back))
        self.grad_h = torch.zeros((rows, C), dtype=dt, device=dev)

    def forward(self):
        self.norm()
        self.rope()
        self.attn()
        return self.step()

    def backward(self, gx, gh):
        g = self.step.backward(gx, gh)
        q, k, v, _ = self.attn.backward(g["y"].view(self.turned.shape))
        torch.add(q, k, out=self.back)
        self.unrope(inverse=True)
        torch.add(self.unrope.q_out.view_as(self.grad_h), v.view_as(self.grad_h), out=self.grad_h)
        return self.norm.backward(g["x"], self.grad_h)

    def results(self):
        return [self.h, self.turned, self.attn.out, self.attn.lse, self.step.x_out, self.step.h,
                self.back, self.grad_h] + list(self.attn.grads) + \
            [t for g in (self.step.grads, self.norm.grads) for t in g.values()]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_layer(dt):
    dev = torch.device("cuda:0")
    tokens, places, seqs, seq = _events(dev)
    assert 0 < sum(n for _, n in seq) <= tokens.shape[0] and len(seq) == 4
    layer = Layer(tokens, places, seqs, dt)
    g = torch.Generator().manual_seed(5)
    gx = torch.randn(tokens.shape, generator=g).to(dev)
    gh = torch.randn(tokens.shape, generator=g).to(dev).to(dt)
    layer.forward()
    layer.backward(gx, gh)
    torch.cuda.synchronize()
    cpu = lambda t: t.detach().cpu().clone()  # noqa: E731
    weights = lambda w: {k: cpu(v) if isinstance(v, torch.Tensor) else v  # noqa: E731
                         for k, v in w.items()}
    rows = tokens.shape[0]

    want = residual_ref.residual(cpu(tokens), None, seq, grad_x_out=cpu(layer.step.grads["x"]),
                                 grad_h=cpu(layer.grad_h), **weights(layer.w_first))
    # (its branch type is h's, the reference's the stream's: round h once more)
    u, tiny = attention_ref.half_step(dt), attention_ref.tiny(dt)
    value, bound = want["h"]
    check(layer.h, (value, bound + u * (np.abs(value) + bound) + tiny * (value != 0)), "h")
    for name, got in layer.norm.grads.items():
        check(got, want["grad_" + name], "norm " + name)

    heads = cpu(layer.h).view(rows, H, D)
    inside = np.zeros(rows, dtype=bool)
    for r0, n in seq:
        inside[r0:r0 + n] = True
    for x, got, inverse in ((heads, layer.turned, False),
                            (cpu(layer.back), layer.unrope.q_out, True)):
        y, e = attention_ref.rope(x, cpu(places), cpu(layer.freqs), layer.pairs, inverse=inverse)
        check(got[torch.from_numpy(inside).to(dev)], (y[inside], e[inside]), "rope")

    t = cpu(layer.turned)
    want = bias_ref.attention(t, t, heads, seq, seq, cpu(layer.table), layer.axes, cpu(places),
                              grad=cpu(layer.step.grads["y"]).view(rows, H, D))
    check(layer.attn.out, want["out"], "out")
    for name, got in zip(("grad_q", "grad_k", "grad_v", "grad_table"), layer.attn.grads):
        check(got, want[name], name)

    want = residual_ref.residual(cpu(tokens), cpu(layer.attn.out).view(rows, C), seq,
                                 gate=cpu(layer.gate), gate_per="sequence", activation="sigmoid",
                                 grad_x_out=cpu(gx), grad_h=cpu(gh), **weights(layer.w_step))
    check(layer.step.x_out, want["x_out"], "x_out")
    check(layer.step.h, want["h"], "h")
    for name, got in layer.step.grads.items():
        check(got, want["grad_" + name], "step " + name)

    eager = [cpu(x) for x in layer.results()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward()
        layer.backward(gx, gh)
    for _ in range(3):
        for x in layer.results():
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, layer.results()):
            assert torch.equal(a, b.cpu())
        layer.forward()
        layer.backward(gx, gh)
