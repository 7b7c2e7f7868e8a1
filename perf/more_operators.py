"""Cases of what training a draft needs beside the packed attention core, for
measurement: the per-head norm and rotation of queries and keys with its
gradient, the cross entropy of a linear head over a large vocabulary with its
gradient, and the global gradient norm with clipping.

``run`` computes one pass of a case: with ``own`` false in plain torch, with
``own`` true through the library.  The operators:

rotate  y = rotation(position) (gain * x / rms(x)) of every query and key head,
        or the gradients of x and of the gains from those of y.
loss    nll = logsumexp(x w^T) - (x w^T)[target] of every row, and, where
        asked, the gradients of sum(d_nll * nll) in x (and w).
clip    norm = sqrt(sum of all squares) over many tensors, which are scaled by
        max_norm / norm where the norm is above max_norm.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6          # of the head norms
THETA = 1e6         # rotation base
POSITIONS = 131072  # positions that a layer's rotation table holds


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one draft block of one sequence, slices of a fused projection's
        # output: the smallest call, latency alone
        dict(name="rotate one block", op="rotate", batch=1, rows=16, heads=32, kv_heads=8,
             dim=128, dtype="bfloat16", backward=False, fused=True, packed=0, lens=1),
        # the block rows of a training step, keys written into the packed
        # attention core's buffer behind 4096 context rows
        dict(name="rotate training", op="rotate", batch=2, rows=4096, heads=32, kv_heads=8,
             dim=128, dtype="bfloat16", backward=False, fused=True, packed=4096, lens=2),
        # the same rows on the way back
        dict(name="rotate training backward", op="rotate", batch=2, rows=4096, heads=32,
             kv_heads=8, dim=128, dtype="bfloat16", backward=True, fused=True, packed=4096,
             lens=3),
        # a small layer in 32 bits, odd row count, head size 64
        dict(name="rotate fp32 backward", op="rotate", batch=3, rows=1001, heads=4, kv_heads=2,
             dim=64, dtype="float32", backward=True, fused=False, packed=0, lens=4),
        # scoring one block of drafted tokens: bound by one read of the head
        dict(name="loss one block", op="loss", rows=16, vocab=150000, hidden=4096, grad="none",
             ignored=0.0, lens=5),
        # a validation pass over a few sequences' blocks, an odd row count
        dict(name="loss validation", op="loss", rows=1000, vocab=150000, hidden=4096,
             grad="none", ignored=0.2, lens=6),
        # a training step whose head is the target model's and stays fixed
        dict(name="loss frozen head", op="loss", rows=4096, vocab=150000, hidden=4096, grad="x",
             ignored=0.0, lens=7),
        # a training step that trains a head over a reduced vocabulary too
        dict(name="loss trained head", op="loss", rows=2048, vocab=64000, hidden=4096,
             grad="xw", ignored=0.0, lens=8),
        # odd sizes, two rows in five without a target
        dict(name="loss ragged", op="loss", rows=777, vocab=50001, hidden=1000, grad="xw",
             ignored=0.4, lens=9),
        # the gradients of one decoder layer's norms: small tensors, latency
        dict(name="clip small", op="clip", tensors=8, lo=128, hi=4096, layers=0, f32=0.5,
             clipped=True, odd=False, lens=10),
        # one decoder layer in bf16, clipped into the optimizer's buffers
        dict(name="clip one layer", op="clip", tensors=0, lo=0, hi=0, layers=1, f32=0.0,
             clipped=True, odd=False, lens=11),
        # the norm of five layers' gradients (what a step that need not clip does)
        dict(name="norm five layers", op="clip", tensors=0, lo=0, hi=0, layers=5, f32=0.0,
             clipped=False, odd=False, lens=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    lens = rng.randrange(1, 1 << 30)
    op = rng.choice(["rotate", "loss", "loss", "clip"])
    if op == "rotate":
        batch = _log_int(rng, 1, 32)
        kv_heads = rng.choice([1, 2, 4, 8])
        dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
        return dict(op=op, batch=batch, rows=_log_int(rng, 1, 8192 // batch),
                    heads=kv_heads * rng.choice([1, 2, 4, 7] if kv_heads < 8 else [1, 2, 4]),
                    kv_heads=kv_heads, dim=128 if dtype == "bfloat16" else rng.choice([32, 64, 80]),
                    dtype=dtype, backward=rng.random() < 0.5, fused=rng.random() < 0.5,
                    packed=rng.choice([0, _log_int(rng, 1, 4096)]), lens=lens)
    if op == "loss":
        rows = _log_int(rng, 1, 4096)
        hidden = 8 * _log_int(rng, 8, 512)
        vocab = _log_int(rng, 100, max(101, min(150000, 1_000_000_000_000 // (rows * hidden))))
        return dict(op=op, rows=rows, vocab=vocab, hidden=hidden,
                    grad=rng.choice(["none", "x", "xw"]),
                    ignored=rng.choice([0.0, 0.0, rng.uniform(0.0, 0.9)]), lens=lens)
    tensors = _log_int(rng, 1, 60)
    return dict(op=op, tensors=tensors, lo=1, hi=_log_int(rng, 16, 400_000_000 // tensors),
                layers=0, f32=rng.choice([0.0, 0.3, 1.0]), clipped=rng.random() < 0.7,
                odd=rng.random() < 0.5, lens=lens)


# -------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rotate_inputs(case, seed):
    """What the projections leave, the positions, the gains, and for the
    gradient what comes back from the attention core."""
    gen = _generator(seed)
    B, R, nq, nkv, d = (case[n] for n in ("batch", "rows", "heads", "kv_heads", "dim"))
    dt = getattr(torch, case["dtype"])
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    # heads of one row differ in size, rows too
    size = torch.exp(0.5 * rand(B, R, nq + nkv, 1))
    x = (rand(B, R, nq + nkv, d) * size).to(dt)
    if case["fused"]:  # [Q heads | K heads | V heads] of one projection
        wide = torch.zeros(B, R, nq + 2 * nkv, d, device="cuda", dtype=dt)
        wide[:, :, :nq + nkv] = x
        q, k = wide[:, :, :nq], wide[:, :, nq:nq + nkv]
    else:
        q, k = x[:, :, :nq].contiguous(), x[:, :, nq:].contiguous()
    r = random.Random(case["lens"])
    first = torch.tensor([r.randrange(0, POSITIONS - R) for _ in range(B)], device="cuda")
    shift = torch.arange(R, device="cuda")
    if R >= 64:  # blocks of 16 behind their anchors
        shift = (shift // 16) * 7 + shift % 16
    positions = (first[:, None] + shift).clamp(max=POSITIONS - 1).int()
    s = dict(q=q, k=k, positions=positions, q_norm=(1 + 0.1 * rand(d)).to(dt),
             k_norm=(1 + 0.1 * rand(d)).to(dt))
    if case["backward"]:
        s["d_q"] = rand(B, R, nq, d).to(dt)
        s["d_k"] = rand(B, nkv, case["packed"] + R, d).to(dt)[:, :, case["packed"]:].transpose(1, 2)
    return s


def _loss_inputs(case, seed):
    """Hidden rows that point to their targets by a varying amount (some are
    sure, some are not), a head of N(0, 0.02), weights that fall along the
    blocks; targets of -100 are ignored."""
    gen = _generator(seed)
    N, V, H = case["rows"], case["vocab"], case["hidden"]
    w = (0.02 * torch.randn(V, H, device="cuda", generator=gen)).bfloat16()
    target = torch.randint(0, V, (N,), device="cuda", generator=gen)
    pull = 12.0 * torch.rand(N, 1, device="cuda", generator=gen) / (0.0004 * H)
    x = torch.randn(N, H, device="cuda", generator=gen)
    x = (x + pull * w[target].float()).bfloat16()
    drop = torch.randperm(N, device="cuda", generator=gen)[:_dropped(case)]
    target[drop] = -100
    d = torch.exp(-torch.arange(N, device="cuda") % 16 / 7.0) / max(1, N - _dropped(case))
    return dict(x=x, w=w, target=target.int(), d_nll=d.float())


def _dropped(case):
    return int(case["rows"] * case["ignored"])


def _layer_sizes(layers):
    """Weights of decoder layers: hidden 4096, 32 query and 8 KV heads of 128,
    MLP width 12288."""
    H, I, d = 4096, 12288, 128
    return layers * [H * H, 1024 * H, 1024 * H, H * H, d, d, I * H, I * H, H * I, H, H]


def _clip_sizes(case):
    """(elements, 32 bits?) of every tensor: they belong to the case."""
    if case["layers"]:
        return [(n, False) for n in _layer_sizes(case["layers"])]
    r = random.Random(case["lens"])
    return [(_log_int(r, case["lo"], case["hi"]), r.random() < case["f32"])
            for _ in range(case["tensors"])]


def _clip_inputs(case, seed):
    """Gradients of unlike sizes; `odd`: slices that start anywhere."""
    gen = _generator(seed)
    r = random.Random(case["lens"] + 1)
    grads = []
    for n, wide in _clip_sizes(case):
        skip = r.randrange(8) if case["odd"] else 0
        dt = torch.float32 if wide else torch.bfloat16
        size = math.exp(r.uniform(-6.0, 1.0))
        g = torch.empty(n + skip, device="cuda", dtype=dt).normal_(0.0, size, generator=gen)
        grads.append(g[skip:])
    return grads


def prepare(case, seed):
    op, s = case["op"], {"case": case}
    if op == "rotate":
        s.update(_rotate_inputs(case, seed))
        B, R, nq, nkv, d = (case[n] for n in ("batch", "rows", "heads", "kv_heads", "dim"))
        dt = s["q"].dtype
        if own:
            from block_diffusion_draft_gb300 import DFlashAttention
            z = lambda *n: torch.zeros(*n, device="cuda", dtype=dt)  # noqa: E731
            h = 128
            w = dict(wq=z(nq * d, h), wk=z(nkv * d, h), wv=z(nkv * d, h), wo=z(h, nq * d),
                     q_norm=z(d), k_norm=z(d))
            s["attn"] = DFlashAttention(w, hidden=h, n_heads=nq, n_kv_heads=nkv, head_dim=d,
                                        rms_eps=EPS, rope_theta=THETA, max_position=POSITIONS,
                                        dtype=dt)
        else:
            f = torch.tensor([THETA ** (-2.0 * j / d) for j in range(d // 2)]).float().double()
            angle = torch.arange(POSITIONS, device="cuda").double()[:, None] * f.cuda()
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        # where the results go: the attention core's layouts, or the fused
        # projection's gradient
        empty = lambda *n: torch.zeros(*n, device="cuda", dtype=dt)  # noqa: E731
        if case["backward"] and case["fused"]:
            wide = empty(B, R, nq + 2 * nkv, d)
            s["q_out"], s["k_out"] = wide[:, :, :nq], wide[:, :, nq:nq + nkv]
        else:
            s["q_out"] = empty(B, R, nq, d)
            keys = empty(B, nkv, (0 if case["backward"] else case["packed"]) + R, d)
            s["k_out"] = keys[:, :, keys.shape[2] - R:].transpose(1, 2)
        return s
    if op == "loss":
        s.update(_loss_inputs(case, seed))
        return s
    s["grads"] = _clip_inputs(case, seed)
    total = math.sqrt(sum(float(g.double().square().sum()) for g in s["grads"]))
    s["max_norm"] = (0.3 if case["clipped"] else 3.0) * total
    if case["clipped"]:
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
    return s


# --------------------------------------------------------------- plain forms
def _turn(x, cos, sin, back=False):
    """Rotation of the pairs (j, j + d/2)."""
    a, b = x.chunk(2, -1)
    if back:
        return torch.cat([a * cos + b * sin, b * cos - a * sin], -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_rotate(s, x, gain, out):
    at = s["positions"].long()
    cos, sin = s["cos"][at].unsqueeze(2), s["sin"][at].unsqueeze(2)
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()
    out.copy_(_turn(y, cos, sin))
    return out


def _plain_rotate_back(s, x, gain, d_y, out):
    at = s["positions"].long()
    cos, sin = s["cos"][at].unsqueeze(2), s["sin"][at].unsqueeze(2)
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * r
    z = _turn(d_y.float(), cos, sin, back=True)
    d_gain = (z * x).sum((0, 1, 2), dtype=torch.float64).float()
    z = z * gain.float()
    out.copy_(r * (z - x * (z * x).mean(-1, keepdim=True)))
    return out, d_gain


def _plain_loss(s):
    x, w, grad = s["x"].float(), s["w"].float(), s["case"]["grad"]
    held = s["target"] >= 0
    t = s["target"].long().clamp(min=0)[:, None]
    z = x @ w.t()
    top = z.amax(-1, keepdim=True)
    z_t = z.gather(1, t)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True, dtype=torch.float64)
    lse = top.double() + total.log()
    nll = (lse - z_t.double()).float().squeeze(1)
    zero = torch.zeros((), device=x.device)
    res = {"nll": torch.where(held, nll, zero),
           "lse": torch.where(held, lse.float().squeeze(1), zero)}
    if grad != "none":
        p = p.div_(total.float())
        p.scatter_add_(1, t, torch.full_like(z_t, -1.0))
        p *= torch.where(held, s["d_nll"], zero)[:, None]
        res["dx"] = (p @ w).bfloat16()
        if grad == "xw":
            res["dw"] = (p.t() @ x).bfloat16()
    return res


def _plain_clip(s):
    total = sum(g.square().sum(dtype=torch.float64) if g.dtype == torch.float32
                else g.double().square().sum() for g in s["grads"])
    norm = total.sqrt()
    if not s["case"]["clipped"]:
        return {"norm": norm.float()}
    scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0).float()
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * scale)
    return {"norm": norm.float(), "out": s["out"]}


# ----------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if op == "rotate":
        if s["case"]["backward"]:
            if own:
                dq, dk, dgq, dgk = s["attn"].qk_norm_rope_backward(
                    s["q"], s["k"], s["positions"], s["q_norm"], s["k_norm"], s["d_q"], s["d_k"],
                    s["q_out"], s["k_out"])
            else:
                dq, dgq = _plain_rotate_back(s, s["q"], s["q_norm"], s["d_q"], s["q_out"])
                dk, dgk = _plain_rotate_back(s, s["k"], s["k_norm"], s["d_k"], s["k_out"])
            return {"dq": dq, "dk": dk, "d_q_norm": dgq, "d_k_norm": dgk}
        if own:
            q, k = s["attn"].qk_norm_rope(s["q"], s["k"], s["positions"], s["q_norm"],
                                          s["k_norm"], s["q_out"], s["k_out"])
        else:
            q = _plain_rotate(s, s["q"], s["q_norm"], s["q_out"])
            k = _plain_rotate(s, s["k"], s["k_norm"], s["k_out"])
        return {"q": q, "k": k}
    if op == "loss":
        if not own:
            return _plain_loss(s)
        from block_diffusion_draft_gb300 import linear_cross_entropy, linear_cross_entropy_grad
        if s["case"]["grad"] == "none":
            nll, lse = linear_cross_entropy(s["x"], s["w"], s["target"])
            return {"nll": nll, "lse": lse}
        nll, lse, dx, dw = linear_cross_entropy_grad(s["x"], s["w"], s["target"], s["d_nll"],
                                                     need_dw=s["case"]["grad"] == "xw")
        res = {"nll": nll, "lse": lse, "dx": dx}
        return res if dw is None else {**res, "dw": dw}
    if not own:
        return _plain_clip(s)
    from block_diffusion_draft_gb300 import clip_grad_norm, grad_norm
    if not s["case"]["clipped"]:
        return {"norm": grad_norm(s["grads"])}
    return {"norm": clip_grad_norm(s["grads"], s["max_norm"], s["out"]), "out": s["out"]}


def work(case):
    if case["op"] == "rotate":
        # rows in and out (for the gradient also those that came back), and
        # one position and rotation row each
        rows, d = case["batch"] * case["rows"], case["dim"]
        size = 2 if case["dtype"] == "bfloat16" else 4
        values = rows * (case["heads"] + case["kv_heads"]) * d
        return {"bytes": values * size * (3 if case["backward"] else 2) + rows * 4,
                "flops": values * (20 if case["backward"] else 8)}
    if case["op"] == "loss":
        # the logits once, and one product for each gradient
        n, V, H = case["rows"] - _dropped(case), case["vocab"], case["hidden"]
        products = {"none": 1, "x": 2, "xw": 3}[case["grad"]]
        moved = n * H + V * H + (case["rows"] * H if products > 1 else 0) + (
            V * H if products > 2 else 0)
        return {"bytes": 2 * moved + case["rows"] * 16, "flops": 2.0 * products * n * V * H}
    size = sum(n * (4 if wide else 2) for n, wide in _clip_sizes(case))
    values = sum(n for n, _ in _clip_sizes(case))
    # clipping needs the norm first: a second read, and the write
    return {"bytes": size * (3 if case["clipped"] else 1) + 4,
            "flops": values * (3 if case["clipped"] else 2)}


# --------------------------------------------------------------------- exact
def _exact_rotate(x, gain, positions, d_y=None):
    """One head at a time as complex numbers: pair (j, j + d/2) times
    exp(i * position * f_j); the gradient by the chain rule written out."""
    x, gain, d = x.double(), gain.double(), x.shape[-1]
    f = np.float32(np.power(THETA, -2.0 * np.arange(d // 2) / d)).astype(np.float64)
    angle = positions.double()[..., None, None] * torch.from_numpy(f).to(x.device)
    spin = torch.complex(torch.cos(angle), torch.sin(angle))
    pair = lambda v: torch.complex(v[..., :d // 2], v[..., d // 2:])  # noqa: E731
    flat = lambda c: torch.cat([c.real, c.imag], -1)  # noqa: E731
    rms = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    if d_y is None:
        return flat(pair(gain * x / rms) * spin)
    d_z = flat(pair(d_y.double()) * spin.conj())
    d_gain = (d_z * x / rms).sum(dim=(0, 1, 2))
    inner = (d_z * gain * x).sum(-1, keepdim=True)
    return d_z * gain / rms - x * inner / (d * rms ** 3), d_gain


def exact(case, seed):
    if case["op"] == "rotate":
        s = _rotate_inputs(case, seed)
        if not case["backward"]:
            return {"q": _exact_rotate(s["q"], s["q_norm"], s["positions"]),
                    "k": _exact_rotate(s["k"], s["k_norm"], s["positions"])}
        dq, dgq = _exact_rotate(s["q"], s["q_norm"], s["positions"], s["d_q"])
        dk, dgk = _exact_rotate(s["k"], s["k_norm"], s["positions"], s["d_k"])
        return {"dq": dq, "dk": dk, "d_q_norm": dgq, "d_k_norm": dgk}
    if case["op"] == "loss":
        s = _loss_inputs(case, seed)
        N, V, H = case["rows"], case["vocab"], case["hidden"]
        w = s["w"].double()
        res = {n: torch.zeros(N, device="cuda", dtype=torch.float64) for n in ("nll", "lse")}
        if case["grad"] != "none":
            res["dx"] = torch.zeros(N, H, device="cuda", dtype=torch.float64)
        if case["grad"] == "xw":
            res["dw"] = torch.zeros(V, H, device="cuda", dtype=torch.float64)
        keep = torch.nonzero(s["target"] >= 0).flatten()
        for at in keep.split(1024):
            x, t = s["x"][at].double(), s["target"][at].long()
            z = torch.mm(x, w.t())
            lse = torch.logsumexp(z, 1)
            res["lse"][at] = lse
            res["nll"][at] = lse - z[torch.arange(len(at), device="cuda"), t]
            if case["grad"] == "none":
                continue
            g = torch.exp(z - lse[:, None])
            g[torch.arange(len(at), device="cuda"), t] -= 1.0
            g *= s["d_nll"][at].double()[:, None]
            res["dx"][at] = torch.mm(g, w)
            if case["grad"] == "xw":
                res["dw"].addmm_(g.t(), x)
        return res
    grads = _clip_inputs(case, seed)
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in grads))
    res = {"norm": torch.tensor(norm, dtype=torch.float64)}
    if case["clipped"]:
        # 0.3 of the norm is what the cases clip to
        res["out"] = [g.double() * 0.3 for g in grads]
    return res
