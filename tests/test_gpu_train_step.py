"""One training step of a small draft: projections, head norm and rotation, the
packed attention core, the head's cross entropy, every gradient, clipping; as a
user runs them together, against the same step in 64 bits with autograd.

Tolerance: the step rounds to bf16 thirteen times between its inputs and the
earliest gradients (projection, norm and rotation, Q', P and the output of the
core, x, the factors and the result of dx, d_o, P, dS and the results of the
core's gradient, the rotation's gradient), each by at most 2^-8 relative to the
2-norm of what it rounds; sums keep that relation as long as their terms do not
cancel, for which a factor of two is left: 26 * 2^-8."""
import torch

from block_diffusion_draft_gb300 import (DFlashAttention, clip_grad_norm, grad_norm,
                                         linear_cross_entropy, linear_cross_entropy_grad)
import train_reference as R

B, S, NB, BS, H, NQ, NKV, D, V = 2, 70, 3, 16, 256, 8, 2, 128, 500
T = NB * BS
TOL = 26 * 2.0 ** -8


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = dict(block=rand(B, T, H), ctx=rand(B, S, H), wqkv=rand((NQ + 2 * NKV) * D, H) / H ** 0.5,
             wo=rand(H, NQ * D) / (NQ * D) ** 0.5, q_norm=1 + 0.2 * rand(D),
             k_norm=1 + 0.2 * rand(D), head=2 * rand(V, H) / H ** 0.5)
    x = {k: v.bfloat16() for k, v in x.items()}
    x["anchors"] = torch.tensor([[3, 40, 70], [0, 17, 33]], dtype=torch.int32)
    t = torch.randint(0, V, (B, T), generator=g, dtype=torch.int32)
    t[:, ::BS] = -100  # the anchors themselves are given
    x["targets"] = t
    x["weights"] = torch.exp(-(torch.arange(T) % BS) / 7.0).expand(B, T).contiguous() / (B * T)
    return x


def positions(x):
    block = (x["anchors"].unsqueeze(-1) + torch.arange(BS)).view(B, T)
    return torch.arange(S).expand(B, S).contiguous().int(), block.int()


def reference(x):
    p = {k: x[k].double().requires_grad_() for k in ("wqkv", "wo", "q_norm", "k_norm", "head")}
    block, ctx = x["block"].double(), x["ctx"].double()
    pos_c, pos_b = positions(x)
    rot = lambda t, gain, pos: R.qk_rope(t, gain, pos, 1e6, 1e-6)[0]  # noqa: E731
    qkv = (block @ p["wqkv"].t()).view(B, T, NQ + 2 * NKV, D)
    kv = (ctx @ p["wqkv"][NQ * D:].t()).view(B, S, 2 * NKV, D)
    q = rot(qkv[:, :, :NQ], p["q_norm"], pos_b)
    k = torch.cat([rot(kv[:, :, :NKV], p["k_norm"], pos_c),
                   rot(qkv[:, :, NQ:NQ + NKV], p["k_norm"], pos_b)], 1)
    v = torch.cat([kv[:, :, NKV:], qkv[:, :, NQ + NKV:]], 1)
    k, v = (t.repeat_interleave(NQ // NKV, 2) for t in (k, v))
    of = torch.arange(T) // BS
    seen = torch.zeros(B, T, S + T, dtype=torch.bool)
    for b in range(B):
        seen[b, :, :S] = torch.arange(S) < x["anchors"][b][of].unsqueeze(-1)
        seen[b, :, S:] = of.unsqueeze(-1) == of
    z = torch.einsum("bthd,bkhd->bhtk", q, k) / D ** 0.5
    z = z.masked_fill(~seen.unsqueeze(1), float("-inf"))
    o = torch.einsum("bhtk,bkhd->bthd", torch.softmax(z, -1), v).reshape(B, T, NQ * D)
    y = o @ p["wo"].t() + block
    logits = (y @ p["head"].t()).view(-1, V)
    t = x["targets"].view(-1).long()
    nll = torch.nn.functional.cross_entropy(logits, t, ignore_index=-100, reduction="none")
    (nll * x["weights"].double().view(-1)).sum().backward()
    return nll.detach(), {k: v.grad for k, v in p.items()}


class Step:
    def __init__(self, x):
        self.x = {k: v.cuda() for k, v in x.items()}
        x = self.x
        w = dict(wq=x["wqkv"][:NQ * D], wk=x["wqkv"][NQ * D:(NQ + NKV) * D],
                 wv=x["wqkv"][(NQ + NKV) * D:], wo=x["wo"], q_norm=x["q_norm"],
                 k_norm=x["k_norm"])
        self.attn = DFlashAttention(w, hidden=H, n_heads=NQ, n_kv_heads=NKV, head_dim=D,
                                    max_position=256)
        pos = positions({k: v.cpu() for k, v in x.items()})
        self.pos_c, self.pos_b = (p.cuda() for p in pos)

    def run(self):
        x, attn = self.x, self.attn
        qkv = (x["block"] @ x["wqkv"].t()).view(B, T, NQ + 2 * NKV, D)
        kv = (x["ctx"] @ x["wqkv"][NQ * D:].t()).view(B, S, 2 * NKV, D)
        q, k = qkv[:, :, :NQ], qkv[:, :, NQ:NQ + NKV]
        keys = torch.empty(B, NKV, S + T, D, device="cuda", dtype=torch.bfloat16)
        vals = torch.cat([kv[:, :, NKV:], qkv[:, :, NQ + NKV:]], 1).transpose(1, 2).contiguous()
        attn.qk_norm_rope(None, kv[:, :, :NKV], self.pos_c, k_norm=x["k_norm"],
                          k_out=keys[:, :, :S].transpose(1, 2))
        qr, _ = attn.qk_norm_rope(q, k, self.pos_b, x["q_norm"], x["k_norm"],
                                  k_out=keys[:, :, S:].transpose(1, 2))
        o, lse = attn.packed_core(qr, keys, vals, x["anchors"], S, BS)
        y = (o.view(B, T, NQ * D) @ x["wo"].t() + x["block"]).view(-1, H)
        nll, _, dy, d_head = linear_cross_entropy_grad(y, x["head"], x["targets"].view(-1),
                                                       x["weights"].view(-1))
        d_o = (dy @ x["wo"]).view(B, T, NQ, D)
        d_wo = dy.t() @ o.view(-1, NQ * D)
        dq, dk, dv = attn.packed_core_backward(qr, keys, vals, o, lse, d_o, x["anchors"], S, BS)
        d_qkv, d_kv = torch.empty_like(qkv), torch.empty_like(kv)
        _, _, dgq, dgk = attn.qk_norm_rope_backward(
            q, k, self.pos_b, x["q_norm"], x["k_norm"], dq, dk[:, :, S:].transpose(1, 2),
            d_qkv[:, :, :NQ], d_qkv[:, :, NQ:NQ + NKV])
        _, _, _, dgk_c = attn.qk_norm_rope_backward(
            None, kv[:, :, :NKV], self.pos_c, None, x["k_norm"], None,
            dk[:, :, :S].transpose(1, 2), dk_out=d_kv[:, :, :NKV])
        d_qkv[:, :, NQ + NKV:] = dv[:, :, S:].transpose(1, 2)
        d_kv[:, :, NKV:] = dv[:, :, :S].transpose(1, 2)
        d_wqkv = d_qkv.view(-1, (NQ + 2 * NKV) * D).t() @ x["block"].view(-1, H)
        d_wqkv[NQ * D:] += d_kv.view(-1, 2 * NKV * D).t() @ x["ctx"].view(-1, H)
        grads = dict(wqkv=d_wqkv, wo=d_wo, q_norm=dgq, k_norm=dgk + dgk_c, head=d_head)
        return nll, grads, y


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return float((a - b).norm() / b.norm())


def test_a_step_of_training_against_autograd_in_64_bits():
    x = inputs(1)
    nll_ref, want = reference(x)
    s = Step(x)
    nll, grads, y = s.run()
    torch.cuda.synchronize()
    assert s.attn.device_error() == 0
    assert rel(nll, nll_ref) <= TOL
    assert (nll.view(B, T)[:, ::BS] == 0).all()
    for k, g in grads.items():
        assert rel(g, want[k]) <= TOL, (k, rel(g, want[k]))
    # the loss alone is the same
    assert torch.equal(linear_cross_entropy(y, s.x["head"], s.x["targets"].view(-1))[0] == 0,
                       nll == 0)
    # clipping the step's gradients
    total = float(sum(v.square().sum() for v in want.values())) ** 0.5
    parts = list(grads.values())
    norm = grad_norm(parts)
    assert abs(float(norm) - total) <= TOL * total
    before = [p.clone() for p in parts]
    assert float(clip_grad_norm(parts, 0.5 * float(norm))) == float(norm)
    for p, b in zip(parts, before):
        assert rel(p, b.double() * 0.5) <= 2.0 ** -8
    assert abs(float(grad_norm(parts)) - 0.5 * float(norm)) <= 2.0 ** -8 * float(norm)


def test_a_captured_step_equals_the_eager_one():
    s = Step(inputs(2))
    nll, want, _ = s.run()
    want = {k: v.clone() for k, v in want.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nll_g, grads, _ = s.run()
        norm = clip_grad_norm(list(grads.values()), 1e30)
    for _ in range(3):
        for g in grads.values():
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(nll_g, nll)
        assert all(torch.equal(grads[k], want[k]) for k in want)
    assert float(norm) == float(grad_norm(list(want.values())))


def test_first_calls_of_a_process_may_be_captured():
    """Nothing of the training calls needs an eager call before a capture."""
    code = """
import torch
from block_diffusion_draft_gb300 import (DFlashAttention, clip_grad_norm, grad_norm,
                                         linear_cross_entropy, linear_cross_entropy_grad)
z = lambda *s: torch.randn(*s, device="cuda").bfloat16()
attn = DFlashAttention(dict(wq=z(256, 128), wk=z(128, 128), wv=z(128, 128), wo=z(128, 256),
                            q_norm=z(128), k_norm=z(128)), hidden=128, n_heads=2, n_kv_heads=1,
                       head_dim=128, max_position=64)
q, k, pos = z(1, 5, 2, 128), z(1, 5, 1, 128), torch.arange(5, device="cuda").int().view(1, 5)
x, w = z(300, 64), z(700, 64)
t, d = torch.arange(300, device="cuda").int(), torch.ones(300, device="cuda")
few, many = [z(99)], [z(3000000), z(7)]
def calls():
    out = list(attn.qk_norm_rope(q, k, pos)) + list(attn.qk_norm_rope_backward(
        q, k, pos, None, None, q, k))
    out += linear_cross_entropy(x, w, t)
    for need in (True, False):
        out += [o for o in linear_cross_entropy_grad(x, w, t, d, need) if o is not None]
        out += [o for o in linear_cross_entropy_grad(x[:9], w, t[:9], d[:9], need)
                if o is not None]
    return out + [grad_norm(few), grad_norm(many), clip_grad_norm(many, 1e30)]
s = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    got = calls()
graph.replay()
torch.cuda.synchronize()
want = calls()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("captured")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
