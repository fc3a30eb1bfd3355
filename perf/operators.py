"""Cases that measure fpstok_rope, fpstok_attention and fpstok_attention_backward.

Each case is one call a point transformer makes on tokens (or on raw pulses):
rotate queries and keys by the tokens' positions, attend inside every event,
and, in training, the gradients.  ``run`` takes the library's kernels where
``own`` is true and a plain form in elementary torch operations (float32,
rounded once) where it is false; ``exact`` is the definition in float64.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------- cases

def _rope(name, rows, heads, kv_heads, dim, dtype, axes, layout, inverse):
    c = dict(op="rope", rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
             axes=axes, layout=layout, inverse=inverse)
    if name:
        c["name"] = name
    return c


def _attn(name, op, q_lens, k_lens, heads, kv_heads, dim, dtype, left=-1, right=-1, sinks=0,
          form="packed"):
    """q_lens / k_lens: "B:median:sigma:lo:hi:seed" (log-normal lengths),
    a comma-separated list, "NxL" (N equal lengths) or "=" (k as q)."""
    c = dict(op=op, q_lens=q_lens, k_lens=k_lens, heads=heads, kv_heads=kv_heads, dim=dim,
             dtype=dtype, left=left, right=right, sinks=sinks, form=form)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the tokens of one event, rotated by their 4D centroids: latency of a single call
        _rope("rope_event", 128, 12, 12, 64, "bf16", "f32:8,8,8,8", "half", False),
        # the packed tokens of a batch of events, float16, grouped key heads
        _rope("rope_batch", 5541, 12, 4, 64, "fp16", "f32:8,8,8,8", "interleaved", False),
        # gradient of a rotation by (time, height, width) over a long packed batch
        _rope("rope_grid_grad", 150000, 16, 4, 128, "bf16", "i32:20,22,22", "half", True),
        # 64 IceCube-sized events of at most 128 tokens: one encoder layer's attention
        _attn("events", "forward", "64:100:1.0:5:128:1001", "=", 12, 12, 64, "bf16"),
        # float32 tokens as the tokenizer returns them, padded to 128 slots per event
        _attn("events_fp32_padded", "forward", "64:100:1.0:1:128:1002", "=", 8, 8, 40, "fp32",
              form="padded"),
        # raw pulses of high-energy events in time order, a window and 4 register tokens
        _attn("pulses_window", "forward", "84240,20011,4097,1000,64,1,0,2049", "=", 8, 2, 64,
              "fp16", 128, 128, 4),
        # long sequences, causal, grouped heads
        _attn("long_causal", "forward", "16384,5000,777", "=", 16, 4, 128, "bf16", -1, 0),
        # attention pooling: one query per event over its padded tokens
        _attn("pool_query", "forward", "256x1", "256:500:0.8:1:1024:1003", 12, 12, 64, "bf16",
              form="padded"),
        # one new token per sequence against long keys and values
        _attn("token_long", "forward", "4x1", "131072,70001,20000,513", 32, 8, 128, "fp16"),
        # one training step of an encoder layer's attention on 256 events
        _attn("train_events", "train", "256:150:1.0:5:256:1004", "=", 12, 12, 64, "bf16"),
        # training on raw pulses in time order: causal window, register tokens, grouped heads
        _attn("train_pulses", "train", "40003,12000,2500,333,1,0", "=", 8, 4, 64, "fp16", 255, 0,
              4),
        # training on long sequences, full attention
        _attn("train_long", "train", "6000,2111,64", "=", 16, 8, 128, "bf16"),
    ]


def _loguniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "events", "events", "pulses", "long", "token", "train",
                       "train", "train_window"])
    dtype = rng.choice(["bf16", "fp16", "bf16", "fp32"])
    if kind == "rope":
        rows = _loguniform(rng, 1, 120000)
        heads, kv = rng.choice([(12, 12), (16, 4), (8, 1), (6, 3), (4, 4)])
        dim = rng.choice([32, 64, 72, 128])
        axes = rng.choice([1, 2, 3, 4])
        total = rng.choice([dim // 2, dim // 4])
        pairs = [total // axes + (1 if a < total % axes else 0) for a in range(axes)]
        spec = "%s:%s" % (rng.choice(["f32", "i32"]), ",".join(str(p) for p in pairs))
        return _rope(None, rows, heads, kv, dim, dtype, spec,
                     rng.choice(["half", "interleaved"]), rng.random() < 0.5)
    shape = rng.randrange(1, 100000)
    form = rng.choice(["packed", "padded"])
    heads, kv = rng.choice([(12, 12), (8, 2), (16, 4), (6, 6), (8, 1)])
    dim = rng.choice([32, 40, 64, 64, 96, 128])
    if kind == "events":
        B, hi = _loguniform(rng, 1, 400), rng.choice([64, 128, 200, 256, 1024])
        return _attn(None, "forward", "%d:%d:1.0:1:%d:%d" % (B, rng.randrange(20, 300), hi, shape),
                     "=", heads, kv, dim, dtype, form=form)
    if kind == "pulses":
        lens = ",".join(str(_loguniform(rng, 1, 40000)) for _ in range(rng.randrange(1, 6)))
        return _attn(None, "forward", lens, "=", heads, kv, rng.choice([32, 64]), dtype,
                     rng.choice([17, 64, 128, 300]), rng.choice([0, 31, 128]),
                     rng.choice([0, 1, 4, 16]))
    if kind == "long":
        lens = ",".join(str(_loguniform(rng, 300, 6000)) for _ in range(rng.randrange(1, 4)))
        return _attn(None, "forward", lens, "=", heads, kv, dim, dtype, -1, rng.choice([-1, 0]))
    if kind == "token":
        B, hi = _loguniform(rng, 1, 256), rng.choice([300, 1024, 20000])
        B = min(B, 2000000 // hi)
        return _attn(None, "forward", "%dx%d" % (B, rng.choice([1, 1, 2, 5])),
                     "%d:%d:0.8:5:%d:%d" % (B, hi // 2, hi, shape), heads, kv, dim, dtype,
                     -1, rng.choice([-1, 0]), form=form)
    if kind == "train":
        B, hi = _loguniform(rng, 1, 256), rng.choice([64, 128, 256, 700])
        return _attn(None, "train", "%d:%d:1.0:1:%d:%d" % (B, rng.randrange(20, 200), hi, shape),
                     "=", heads, kv, dim, dtype, form=form)
    lens = ",".join(str(_loguniform(rng, 1, 15000)) for _ in range(rng.randrange(1, 6)))
    return _attn(None, "train", lens, "=", heads, kv, rng.choice([32, 64]), dtype,
                 rng.choice([17, 64, 128, 300]), rng.choice([0, 31, 128]),
                 rng.choice([0, 1, 4, 16]))


def _lens(text, other=None):
    if text == "=":
        return other
    if "x" in text:
        n, length = text.split("x")
        return [int(length)] * int(n)
    if ":" in text:
        B, median, sigma, lo, hi, seed = text.split(":")
        z = np.random.default_rng(int(seed)).standard_normal(int(B))
        n = np.rint(np.exp(math.log(float(median)) + float(sigma) * z))
        return [int(x) for x in np.clip(n, int(lo), int(hi))]
    return [int(x) for x in text.split(",")]


def _case_lens(case):
    q = _lens(case["q_lens"])
    return q, _lens(case["k_lens"], q)


def _capacity(text, lens):
    """Slots per sequence of the padded form."""
    if ":" in text:
        return int(text.split(":")[4])
    return max(lens)


def _visible_pairs(tq, tk, left, right, sinks):
    if tq == 0 or tk == 0:
        return 0
    p = np.arange(tq, dtype=np.int64) + (tk - tq)
    hi = np.minimum(tk - 1, p + right) if right >= 0 else np.full(tq, tk - 1)
    lo = np.maximum(0, p - left) if left >= 0 else np.zeros(tq, dtype=np.int64)
    n = np.maximum(0, hi - lo + 1)
    # sinks below the window, up to the right bound
    n = n + np.maximum(0, np.minimum(np.minimum(lo, sinks), hi + 1))
    return int(n.sum())


def work(case):
    w = _BYTES[case["dtype"]]
    if case["op"] == "rope":
        n, hd = case["rows"], (case["heads"] + case["kv_heads"]) * case["dim"]
        kind, pairs = case["axes"].split(":")
        pairs = [int(x) for x in pairs.split(",")]
        return {"bytes": 2 * n * hd * w + 4 * n * len(pairs) + 4 * sum(pairs),
                "flops": 6 * n * sum(pairs) * (case["heads"] + case["kv_heads"])}
    ql, kl = _case_lens(case)
    q = sum(ql) * case["heads"] * case["dim"] * w
    kv = sum(kl) * case["kv_heads"] * case["dim"] * w
    pairs = sum(_visible_pairs(a, b, case["left"], case["right"], case["sinks"])
                for a, b in zip(ql, kl)) * case["heads"]
    if case["op"] == "forward":
        # q, k, v in; the output and its log-sum-exp out
        return {"bytes": 2 * q + 2 * kv + 4 * sum(ql) * case["heads"],
                "flops": 4 * case["dim"] * pairs}
    # q, k, v and the output's gradient in; the output and three gradients out
    return {"bytes": 4 * q + 4 * kv, "flops": 14 * case["dim"] * pairs}


# ------------------------------------------------------------------ inputs

class _State:
    pass


def _layout(lens, form, text, dev):
    """Row starts, buffer rows and the device description of the sequences."""
    n = torch.tensor(lens, dtype=torch.int32)
    if form == "padded":
        cap = _capacity(text, lens)
        return ([b * cap for b in range(len(lens))], len(lens) * cap, n.to(dev), cap)
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(n, 0)
    return cu[:-1].tolist(), int(cu[-1]), cu.to(dev), 0


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    st = _State()
    st.case = case
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        n = case["rows"]
        kind, pairs = case["axes"].split(":")
        st.pairs = [int(x) for x in pairs.split(",")]
        st.q, st.k = normal(n, H, D), normal(n, Hk, D)
        if kind == "f32":
            # standardized positions: a few units wide, some far out
            st.pos = torch.randn((n, len(st.pairs)), generator=gen, device=dev) * 1.5
            top = 200.0
        else:
            # long sequences of frames: a far-running first axis, a grid in the others
            st.pos = torch.randint(0, 1000, (n, len(st.pairs)), generator=gen, device=dev,
                                   dtype=torch.int32)
            st.pos[:, 0] *= 1000
            top = 1.0
        st.freqs = torch.cat([top * 10000.0 ** (-torch.arange(m, dtype=torch.float64) / max(m, 1))
                              for m in st.pairs]).to(torch.float32).to(dev)
        if own:
            from point_cloud_tokenization_amd import fpstok as F

            cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
            st.call = F.Rope(st.q, st.k, st.pos, st.freqs, st.pairs,
                             F.make_seqs(n, cu_seqlens=cu),
                             interleaved=case["layout"] == "interleaved")
        return st
    st.ql, st.kl = _case_lens(case)
    same = case["k_lens"] == "="
    st.q_start, q_rows, q_dev, q_cap = _layout(st.ql, case["form"], case["q_lens"], dev)
    st.k_start, k_rows, k_dev, k_cap = (st.q_start, q_rows, q_dev, q_cap) if same else \
        _layout(st.kl, case["form"], case["k_lens"], dev)
    st.q, st.k, st.v = normal(q_rows, H, D), normal(k_rows, Hk, D), normal(k_rows, Hk, D)
    st.grad = normal(q_rows, H, D) if case["op"] == "train" else None
    if own:
        from point_cloud_tokenization_amd import fpstok as F

        def seqs(rows, d, cap, lens):
            if cap:
                return F.make_seqs(rows, token_count=d, capacity=cap, max_len=max(lens))
            return F.make_seqs(rows, cu_seqlens=d, max_len=max(lens))

        st.call = F.Attention(st.q, st.k, st.v, seqs(q_rows, q_dev, q_cap, st.ql),
                              None if same else seqs(k_rows, k_dev, k_cap, st.kl),
                              window=(case["left"], case["right"]), num_sinks=case["sinks"],
                              training=case["op"] == "train")
    return st


# --------------------------------------------------------------------- run

def run(st):
    case = st.case
    if own:
        if case["op"] == "rope":
            return st.call(inverse=case["inverse"])
        out = st.call()
        if case["op"] == "forward":
            return out
        grads = st.call.backward(st.grad)
        return [out[0]] + list(grads)
    if case["op"] == "rope":
        return _plain_rope(st)
    return _plain_attention(st)


def _plain_rope(st):
    pairs, R = st.pairs, sum(st.pairs)
    axis = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs)).to(st.q.device)
    ang = st.pos.double()[:, axis] * st.freqs.double()
    c, s = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    if st.case["inverse"]:
        s = -s
    out = []
    for x in (st.q, st.k):
        y = x.float().clone()
        if st.case["layout"] == "half":
            a, b = y[..., :R].clone(), y[..., R:2 * R].clone()
            y[..., :R] = a * c - b * s
            y[..., R:2 * R] = a * s + b * c
        else:
            a, b = y[..., 0:2 * R:2].clone(), y[..., 1:2 * R:2].clone()
            y[..., 0:2 * R:2] = a * c - b * s
            y[..., 1:2 * R:2] = a * s + b * c
        out.append(y.to(x.dtype))
    return out


def _plain_attention(st):
    """Sequence after sequence, in blocks of queries against the slice of the
    keys that the block can see."""
    case = st.case
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G, left, right, sinks = H // Hk, case["left"], case["right"], case["sinks"]
    scale, dev, dt = 1.0 / math.sqrt(D), st.q.device, st.q.dtype
    train = case["op"] == "train"
    out = torch.zeros(st.q.shape, device=dev)
    lse = torch.zeros(st.q.shape[:2], device=dev)
    if train:
        gq, gk, gv = (torch.zeros(t.shape, device=dev) for t in (st.q, st.k, st.v))
    for q0, tq, k0, tk in zip(st.q_start, st.ql, st.k_start, st.kl):
        if tq == 0 or tk == 0:
            continue
        k = st.k[k0:k0 + tk].float().permute(1, 0, 2).contiguous()
        v = st.v[k0:k0 + tk].float().permute(1, 0, 2).contiguous()
        block = tq if left < 0 and right < 0 and tq * tk <= 1 << 22 else \
            1024 if left >= 0 and right >= 0 else 2048
        for a in range(0, tq, block):
            b = min(tq, a + block)
            p0, p1 = a + tk - tq, b - 1 + tk - tq
            lo = max(0, p0 - left) if left >= 0 else 0
            hi = max(0, min(tk, p1 + right + 1)) if right >= 0 else tk
            lo = min(lo, hi)
            n0 = min(sinks, lo)
            kb = torch.cat([k[:, :n0], k[:, lo:hi]], 1) if n0 else k[:, lo:hi]
            vb = torch.cat([v[:, :n0], v[:, lo:hi]], 1) if n0 else v[:, lo:hi]
            qb = st.q[q0 + a:q0 + b].float().reshape(b - a, Hk, G, D).permute(1, 2, 0, 3)
            qb = qb.reshape(Hk, G * (b - a), D)
            s = torch.matmul(qb, kb.transpose(1, 2).contiguous()) * scale
            if left >= 0 or right >= 0:
                col = torch.arange(lo, hi, device=dev)
                if n0:
                    col = torch.cat([torch.arange(0, n0, device=dev), col])
                p = torch.arange(p0, p1 + 1, device=dev)[:, None]
                hide = torch.zeros((b - a, col.numel()), dtype=torch.bool, device=dev)
                if right >= 0:
                    hide |= col > p + right
                if left >= 0:
                    hide |= (col < p - left) & (col >= sinks)
                s.view(Hk, G, b - a, -1).masked_fill_(hide, -math.inf)
            top = s.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            e = torch.exp(s - top)
            total = e.sum(-1, keepdim=True)
            e = e / torch.where(total == 0, torch.ones_like(total), total)
            o = torch.matmul(e, vb)

            def back(x):
                return x.reshape(Hk, G, b - a, -1).permute(2, 0, 1, 3).reshape(b - a, H, -1)

            out[q0 + a:q0 + b] = back(o)
            lse[q0 + a:q0 + b] = back(top + torch.log(total))[..., 0]
            if train:
                g = st.grad[q0 + a:q0 + b].float().reshape(b - a, Hk, G, D).permute(1, 2, 0, 3)
                g = g.reshape(Hk, G * (b - a), D)
                dp = torch.matmul(g, vb.transpose(1, 2).contiguous())
                ds = e * (dp - (e * dp).sum(-1, keepdim=True)) * scale
                gq[q0 + a:q0 + b] = back(torch.matmul(ds, kb))
                dk = torch.matmul(ds.transpose(1, 2).contiguous(), qb).permute(1, 0, 2)
                dv = torch.matmul(e.transpose(1, 2).contiguous(), g).permute(1, 0, 2)
                for dst, d in ((gk, dk), (gv, dv)):
                    dst[k0:k0 + n0] += d[:n0]
                    dst[k0 + lo:k0 + hi] += d[n0:]
    if train:
        return [out.to(dt), gq.to(dt), gk.to(dt), gv.to(dt)]
    return [out.to(dt), lse]


# ------------------------------------------------------------------- exact

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "rope":
        res = []
        col = 0
        ang = []
        for a, m in enumerate(st.pairs):
            for _ in range(m):
                ang.append(st.pos[:, a].double() * float(st.freqs[col]))
                col += 1
        ang = torch.stack(ang, 1)
        if case["inverse"]:
            ang = -ang
        rot = torch.polar(torch.ones_like(ang), ang)[:, None]
        R = col
        for x in (st.q, st.k):
            y = x.double()
            if case["layout"] == "half":
                z = torch.complex(y[..., :R].contiguous(), y[..., R:2 * R].contiguous()) * rot
                res.append(torch.cat([z.real, z.imag, y[..., 2 * R:]], -1))
            else:
                z = torch.complex(y[..., 0:2 * R:2].contiguous(), y[..., 1:2 * R:2].contiguous())
                z = torch.view_as_real(z * rot).flatten(-2)
                res.append(torch.cat([z, y[..., 2 * R:]], -1))
        return res
    return _exact_attention(st)


def _exact_attention(st):
    """Head after head in float64: every block of rows gathers the keys its
    rows can see by index, and softmax is taken over the visible entries."""
    case = st.case
    H, G, D = case["heads"], case["heads"] // case["kv_heads"], case["dim"]
    left, right, sinks = case["left"], case["right"], case["sinks"]
    dev = st.q.device
    train = case["op"] == "train"
    f64 = dict(dtype=torch.float64, device=dev)
    out = torch.zeros(st.q.shape, **f64)
    lse = torch.zeros(st.q.shape[:2], **f64)
    dq, dk, dv = (torch.zeros(t.shape, **f64) for t in (st.q, st.k, st.v)) if train else \
        (None, None, None)
    for b in range(len(st.ql)):
        tq, tk = st.ql[b], st.kl[b]
        if tq == 0 or tk == 0:
            continue
        rows = 4096 if tk * 4096 <= 1 << 27 else 1024
        if left >= 0 and (right >= 0 or sinks == 0):
            rows = 1024
        for i0 in range(0, tq, rows):
            i = torch.arange(i0, min(tq, i0 + rows), device=dev)
            pos = i + (tk - tq)
            first, last = int(pos[0]), int(pos[-1])
            j = torch.arange(tk, device=dev)
            keep = torch.ones(tk, dtype=torch.bool, device=dev)
            if left >= 0:
                keep &= (j >= first - left) | (j < sinks)
            if right >= 0:
                keep &= j <= last + right
            j = j[keep]
            if j.numel() == 0:
                continue
            ok = torch.ones((i.numel(), j.numel()), dtype=torch.bool, device=dev)
            if left >= 0:
                ok &= (j[None] >= pos[:, None] - left) | (j[None] < sinks)
            if right >= 0:
                ok &= j[None] <= pos[:, None] + right
            qi, kj = st.q_start[b] + i, st.k_start[b] + j
            for h in range(H):
                q = st.q[qi, h].double()
                k = st.k[kj, h // G].double()
                v = st.v[kj, h // G].double()
                z = (q @ k.T) / math.sqrt(D)
                z = torch.where(ok, z, torch.full_like(z, -math.inf))
                norm = torch.logsumexp(z, 1)
                some = ok.any(1)
                w = torch.exp(z - torch.where(some, norm, torch.zeros_like(norm))[:, None])
                o = w @ v
                out[qi, h] = o
                lse[qi, h] = norm
                if train:
                    g = st.grad[qi, h].double()
                    dw = g @ v.T
                    dz = w * (dw - (g * o).sum(1)[:, None])
                    dq[qi, h] = (dz @ k) / math.sqrt(D)
                    dk[kj, h // G] += (dz.T @ q) / math.sqrt(D)
                    dv[kj, h // G] += w.T @ g
    if train:
        return [out, dq, dk, dv]
    return [out, lse]
