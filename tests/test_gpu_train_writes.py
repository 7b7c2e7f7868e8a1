"""What the training calls write into tensors of the caller's, as autograd sees
it: a tensor saved for a backward pass must not change without a word."""
import pytest
import torch

from block_diffusion_draft_gb300 import DFlashAttention, clip_grad_norm, grad_norm

pytestmark = pytest.mark.gpu

NQ, NKV, D = 4, 2, 128


def test_autograd_sees_that_a_saved_tensor_was_written():
    """Tensors that a call overwrites and that autograd has saved before: the
    backward pass refuses them; given tensors that are only read still pass."""
    zeros = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    attn = DFlashAttention(dict(wq=zeros(NQ * D, 128), wk=zeros(NKV * D, 128),
                                wv=zeros(NKV * D, 128), wo=zeros(128, NQ * D), q_norm=zeros(D) + 1,
                                k_norm=zeros(D) + 1), hidden=128, n_heads=NQ, n_kv_heads=NKV,
                           head_dim=D, max_position=64)
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    pos = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    q, k, d_q, d_k = rand(1, 6, NQ, D), rand(1, 6, NKV, D), rand(1, 6, NQ, D), rand(1, 6, NKV, D)
    grads = [rand(100), rand(7, 9).float()]
    outs = [torch.empty_like(t) for t in (q, k, d_q, d_k, *grads)]
    leaf = torch.ones((), device="cuda", requires_grad=True)

    def saved(*tensors):
        return sum((t.detach().float() * 0 + leaf * t).sum() for t in tensors)

    def back(tensors):
        return attn.qk_norm_rope_backward(q, k, pos, None, None, d_q, d_k, *tensors)

    for call, written, read in (
            (lambda: attn.qk_norm_rope(q, k, pos), [], [q, k]),
            (lambda: attn.qk_norm_rope(q, k, pos, q_out=outs[0], k_out=outs[1]), outs[:2], [q, k]),
            (lambda: attn.qk_norm_rope(None, k, pos, k_out=k), [k], [q]),
            (lambda: back(outs[2:4]), outs[2:4], [q, k, d_q, d_k]),
            (lambda: back((d_q, d_k)), [d_q, d_k], [q, k]),
            (lambda: grad_norm(grads), [], grads),
            (lambda: clip_grad_norm(grads, 1e-3, outs[4:]), outs[4:], grads),
            (lambda: clip_grad_norm(grads, 1e-3), grads, [])):
        kept, lost = saved(*read) if read else None, [saved(t) for t in written]
        call()
        if kept is not None:
            kept.backward()
        for y in lost:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()
    with torch.inference_mode():  # tensors without a version
        t = [torch.ones(50, device="cuda")]
        clip_grad_norm(t, 1.0)
