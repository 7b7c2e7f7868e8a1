"""Calls over the 8-bit cache captured into CUDA graphs and replayed between
other calls."""
import pytest
import torch

from block_diffusion_draft_gb300 import DraftCache, Q8Cache
from block_diffusion_draft_gb300 import workloads as W

import helpers as T

pytestmark = pytest.mark.gpu


def small_layer():
    sp = W.spec("qwen3_8b_single", hidden=512, n_heads=8, n_kv_heads=2, n_target_layers=1,
                max_position=4096)
    return T.gpu_layer(sp, W.weights(sp, 3, with_fc=False)), sp


def step_inputs(sp, n_ctx, q_len, L, seed):
    th = torch.cat([W.hidden_rows(sp, seed, "hidden", 0, b, n) for b, n in enumerate(n_ctx)])
    nz = torch.stack([W.hidden_rows(sp, seed, "noise", 0, b, q_len) for b in range(len(n_ctx))])
    pos = torch.cat([W.window_positions(L[b], n, q_len) for b, n in enumerate(n_ctx)])
    return nz.cuda(), th.cuda(), n_ctx, pos.cuda()


def test_a_captured_step_survives_larger_ones():
    """A step captured at a small size is replayed after steps that need far
    more scratch of the cache and of the layer."""
    attn, sp = small_layer()
    cache = Q8Cache(attn, 2, 2000, "int8")
    held = [30, 5]
    first = step_inputs(sp, held, 1, [0, 0], 1)
    attn.forward_q8(cache, *first)
    cache.crop(held)
    args = step_inputs(sp, [3, 2], 8, held, 2)
    want = attn.forward_q8(cache, *args).clone()
    rows = [x.clone() for x in cache.read()]
    cache.crop(held)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = attn.forward_q8(cache, *args)
    for n, q_len in ((40, 16), (300, 16), (900, 64)):
        cache.crop([0, 0])
        big = Q8Cache(attn, 2, 2000, "int8")
        attn.forward_q8(big, *step_inputs(sp, [n, n], q_len, [0, 0], 3))
        attn.forward_q8(cache, *step_inputs(sp, [n, n // 2], q_len, [0, 0], 4))
        cache.crop([0, 0])
        attn.forward_q8(cache, *first)
        cache.crop(held)
        fill = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        cache.crop([0, 0])
        attn.forward_q8(cache, *first)
        cache.crop(held)
        assert torch.equal(attn.forward_q8(cache, *args), want)
        assert all(torch.equal(x, y) for x, y in zip(cache.read(), rows))
        del fill, big
    assert attn.device_error() == 0


def test_a_captured_step_over_the_bf16_cache_survives_larger_8_bit_ones():
    """The two kinds of steps share the layer's scratch."""
    attn, sp = small_layer()
    held = [30, 5]
    cache, big = DraftCache(attn, 2, 200), Q8Cache(attn, 2, 2000, "e4m3")
    attn.forward(cache, *step_inputs(sp, held, 1, [0, 0], 1))
    cache.crop(held)
    args = step_inputs(sp, [3, 2], 8, held, 2)
    want = attn.forward(cache, *args).clone()
    cache.crop(held)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = attn.forward(cache, *args)
    for n, q_len in ((300, 16), (900, 64)):
        attn.forward_q8(big, *step_inputs(sp, [n, n], q_len, [0, 0], 3))
        big.crop([0, 0])
        other = DraftCache(attn, 2, 2000)  # takes what was freed
        torch.cuda.synchronize()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        cache.crop(held)
        assert torch.equal(attn.forward(cache, *args), want)
        assert all(not x.any() for x in other.read())
    assert attn.device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_replayed_append_keeps_what_is_known_of_other_rows(fmt):
    """An append captured at row 0 is replayed after rows of larger and smaller
    scales came behind it: they read as before."""
    attn, _ = small_layer()
    cache = Q8Cache(attn, 2, 600, fmt)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda n: torch.randn(n, 2, 128, device="cuda", generator=gen).bfloat16()  # noqa: E731
    k, v = rand(20), rand(20)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.append(k, v, [15, 5])
    g.replay()
    more, tiny = rand(400) * 64, rand(40) * 2.0 ** -9
    more[100:200, :, :64] = 0
    cache.append(torch.cat([more, tiny]), torch.cat([tiny, more]), [400, 40])
    q = torch.randn(2, 4, 8, 128, device="cuda", generator=gen).bfloat16()
    want = attn.q8_core(cache, q)
    ref = Q8Cache(attn, 2, 600, fmt)
    ref.append(torch.cat([k[:15], more, k[15:], tiny]), torch.cat([v[:15], tiny, more[:360],
                                                                    v[15:], more[360:]]), [415, 45])
    assert all(torch.equal(x, y) for x, y in zip(cache.read(), ref.read()))
    assert all(torch.equal(x, y) for x, y in zip(want, attn.q8_core(ref, q)))
    for _ in range(2):
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(attn.q8_core(cache, q), want))
