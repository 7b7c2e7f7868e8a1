"""Training operators beside the packed core: what is refused on the host (no
GPU), and the references' own pins."""
import ctypes

import pytest
import torch

from block_diffusion_draft_gb300 import build
from block_diffusion_draft_gb300 import dflash_attn as D

import train_reference as R


@pytest.fixture(scope="module")
def L():
    build.build()
    return D.lib()


FAKE = 0x1000


def test_norm_and_rotation_reject_null_handles(L):
    h = (ctypes.c_int64 * 4)(FAKE, 0, 0, 0)
    h = ctypes.cast(h, ctypes.c_void_p)
    n = ctypes.c_size_t(0)
    assert L.dflash_qk_norm_rope(None, 1, 1, h, h, None, None, FAKE, h, h, None) == -1
    assert b"null" in L.dflash_last_error()
    assert L.dflash_qk_norm_rope_backward(None, 1, 1, h, h, None, None, FAKE, h, h, h, h, FAKE,
                                          FAKE, FAKE, 1 << 20, None) == -1
    assert L.dflash_qk_norm_rope_workspace(None, ctypes.byref(n)) == -1


def _clip(L, **kw):
    a = dict(g=[0x10000, 0x20000], out=None, n=[64, 64], t=[0, 1], max_norm=1.0, norm=FAKE,
             ws=FAKE, bytes=1 << 24)
    a.update(kw)
    k = len(a["n"])
    arr = lambda t, xs: None if xs is None else (t * max(1, len(xs)))(*xs)  # noqa: E731
    return L.dflash_clip_grad_norm(kw.get("k", k), arr(ctypes.c_void_p, a["g"]),
                                   arr(ctypes.c_void_p, a["out"]), arr(ctypes.c_int64, a["n"]),
                                   arr(ctypes.c_int32, a["t"]), a["max_norm"], a["norm"], a["ws"],
                                   a["bytes"], None)


@pytest.mark.parametrize("kw,rc", [
    (dict(k=-1), -1), (dict(g=None), -1), (dict(norm=None), -1), (dict(ws=None), -1),
    (dict(bytes=64), -3), (dict(ws=FAKE + 4), -1), (dict(norm=FAKE + 2), -1),
    (dict(t=[0, 2]), -1), (dict(n=[64, -1]), -1), (dict(g=[0x10000, None]), -1),
    (dict(g=[0x10001, 0x20000]), -1), (dict(g=[0x10000, 0x20002]), -1),
    (dict(max_norm=-1.0), -1), (dict(max_norm=float("nan")), -1),
    (dict(g=[0x10000, 0x10000]), -1), (dict(g=[0x10000, 0x10000 + 124]), -1),
    (dict(out=[0x30000, 0x30000]), -1), (dict(out=[0x20000, 0x10000]), -1),
    (dict(out=[0x10002, 0x40000]), -1), (dict(out=[0x10000, None]), -1)])
def test_clipping_checks_its_arguments_on_the_host(L, kw, rc):
    assert _clip(L, **kw) == rc


def test_grad_norm_checks_its_arguments(L):
    n = ctypes.c_size_t(0)
    assert L.dflash_grad_norm_workspace(-1, ctypes.byref(n)) == -1
    assert L.dflash_grad_norm_workspace(3, None) == -1
    assert L.dflash_grad_norm_workspace(3, ctypes.byref(n)) == 0 and n.value > 0
    assert L.dflash_grad_norm(1, None, None, None, FAKE, FAKE, 1 << 20, None) == -1
    for f in (lambda: D.grad_norm([]), lambda: D.grad_norm([torch.zeros(3)]),
              lambda: D.clip_grad_norm([torch.zeros(3)], 1.0)):
        with pytest.raises(ValueError):
            f()


def test_dense_means_one_run_of_memory():
    t = torch.zeros(4, 6, 8)
    assert D._dense(t) and D._dense(t.permute(2, 0, 1)) and D._dense(t[:1]) and D._dense(t[:, :1])\
        is False
    assert not D._dense(t[..., ::2]) and not D._dense(torch.zeros(3, 1).expand(3, 4))
    assert D._dense(torch.zeros(()))


def _differences(f, x, h=1e-5):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        g.view(-1)[i] = (f(x + e.view_as(x)) - f(x - e.view_as(x))) / (2 * h)
    return g


def test_reference_rotation_gradient_equals_differences():
    g = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, gain, dy = rand(1, 2, 2, 6), 1 + 0.3 * rand(6), rand(1, 2, 2, 6)
    pos = torch.tensor([[3, 1000]])
    loss = lambda x, gain: (R.qk_rope(x, gain, pos, 1e4, 1e-6)[0] * dy).sum()  # noqa: E731
    dx, dg, _, _ = R.qk_rope_backward(x, gain, pos, 1e4, 1e-6, dy)
    assert torch.allclose(dx, _differences(lambda v: loss(v, gain), x), atol=1e-8)
    assert torch.allclose(dg, _differences(lambda v: loss(x, v), gain), atol=1e-8)
    # the rotation keeps a pair's length and turns by the position
    y, _ = R.qk_rope(x, torch.ones(6).double(), pos, 1e4, 0.0)
    assert torch.allclose(y.square().mean(-1), torch.ones(1, 2, 2).double())


def test_reference_cross_entropy_gradient_equals_differences():
    g = torch.Generator().manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, d = rand(5, 4), rand(7, 4), rand(5)
    t = torch.tensor([2, -100, 6, 7, 0])
    loss = lambda x, w: (R.linear_cross_entropy(x, w, t, d)[0] * d).sum()  # noqa: E731
    nll, lse, dx, dw = R.linear_cross_entropy(x, w, t, d)
    assert (nll[[1, 3]] == 0).all() and (dx[[1, 3]] == 0).all()
    assert torch.allclose(dx, _differences(lambda v: loss(v, w), x), atol=1e-8)
    assert torch.allclose(dw, _differences(lambda v: loss(x, v), w), atol=1e-8)
    want = torch.nn.functional.cross_entropy(x @ w.t(), torch.where(t == 7, -100, t),
                                             reduction="none")
    assert torch.allclose(nll, want)


def _ce(L, grad, **kw):
    a = dict(rows=4, vocab=100, hidden=64, x=FAKE, xs=64, w=FAKE, ws=64, targets=FAKE, d_nll=FAKE,
             nll=FAKE, lse=FAKE, dx=FAKE, dw=None, space=FAKE, bytes=1 << 40)
    a.update(kw)
    head = [a[k] for k in ("rows", "vocab", "hidden", "x", "xs", "w", "ws", "targets")]
    tail = [a["space"], a["bytes"], None]
    if grad:
        return L.dflash_linear_ce_grad(*head, *[a[k] for k in ("d_nll", "nll", "lse", "dx", "dw")],
                                       *tail)
    return L.dflash_linear_ce(*head, a["nll"], a["lse"], *tail)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("kw,rc", [
    (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(hidden=0), -1), (dict(hidden=60), -2),
    (dict(rows=(1 << 20) + 1), -2), (dict(vocab=(1 << 24) + 1), -2),
    (dict(hidden=(1 << 16) + 8), -2), (dict(x=None), -1), (dict(w=None), -1),
    (dict(targets=None), -1), (dict(nll=None), -1), (dict(lse=None), -1), (dict(x=FAKE + 8), -1),
    (dict(w=FAKE + 2), -1), (dict(targets=FAKE + 2), -1), (dict(nll=FAKE + 1), -1),
    (dict(xs=56), -1), (dict(xs=68), -1), (dict(ws=0), -1), (dict(ws=66), -1),
    (dict(xs=1 << 33), -2), (dict(space=None), -1), (dict(space=FAKE + 16), -1),
    (dict(bytes=100), -3)])
def test_cross_entropy_checks_its_arguments_on_the_host(L, grad, kw, rc):
    assert _ce(L, grad, **kw) == rc


@pytest.mark.parametrize("kw", [dict(d_nll=None), dict(dx=None), dict(dx=FAKE + 8),
                                dict(dw=FAKE + 4), dict(d_nll=FAKE + 2)])
def test_cross_entropy_gradient_checks_its_arguments(L, kw):
    assert _ce(L, True, **kw) == -1


def test_cross_entropy_workspace(L):
    n = ctypes.c_size_t(0)
    f = lambda *a: L.dflash_linear_ce_workspace(*a, ctypes.byref(n))  # noqa: E731
    assert L.dflash_linear_ce_workspace(1, 1, 8, 0, None) == -1
    assert f(1, 1, 8, 3) == -1 and f(1, 1, 9, 0) == -2 and f(0, 1, 8, 2) == 0
    size = {}
    for grads in range(3):
        assert f(4096, 150000, 4096, grads) == 0
        size[grads] = n.value
    assert size[0] < size[1] <= size[2]
    # a piece's exponentials, not the vocabulary's
    assert f(16384, 1000000, 4096, 2) == 0 and n.value < 8 << 30


def test_cross_entropy_checks_its_tensors():
    x, w = torch.zeros(3, 16).bfloat16(), torch.zeros(5, 16).bfloat16()
    t, d = torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    for f in (lambda: D.linear_cross_entropy(x, w, t), lambda: D.linear_cross_entropy(x[0], w, t),
              lambda: D.linear_cross_entropy_grad(x, w[:, :8], t, d)):
        with pytest.raises(ValueError):
            f()
