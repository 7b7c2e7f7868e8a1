"""Global gradient norm and clipping on the GPU, against 64 bits.

Tolerance: a group of 64 squares added in fp32 is off by at most 66 * 2^-24 of
itself (64 products and additions, the conversion), the root halves that, and
the norm is rounded once: 34 * 2^-24.  A clipped value passes the factor (that
error and its rounding) and one product, then its type's half step."""
import math

import pytest
import torch

from block_diffusion_draft_gb300 import DFlashError, clip_grad_norm, grad_norm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def make(sizes, seed, skip=False):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        off = i % 8 if skip else 0
        dt = torch.bfloat16 if (i + seed) % 3 else torch.float32
        t = torch.randn(n + off, generator=g) * math.exp(float(torch.randn(1, generator=g)))
        out.append(t.to(dt).cuda()[off:])
    return out


def check_clipped(got, grads, factor):
    for o, g in zip(got, grads):
        want = g.double() * factor
        assert ((o.double() - want).abs() <= (HALF[g.dtype] * 1.01 + 37 * U) * want.abs()).all()


SIZES = [[1], [7], [8], [9], [15, 16, 17], [2047, 2048, 2049], [16384], [16383, 16385, 1, 3],
         [0, 5, 0], [0], [100000, 3, 262144, 1, 77777], [300001]]


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_norm_and_clipping(sizes, skip):
    grads = make(sizes, len(sizes), skip)
    want = norm64(grads)
    n = grad_norm(grads)
    assert n.shape == () and n.dtype == torch.float32
    assert abs(float(n) - want) <= 34 * U * want
    before = [g.clone() for g in grads]
    out = [torch.full_like(g, 9.0) for g in grads]
    for max_norm, factor in ((0.25 * want, 0.25), (2 * want + 1, 1.0), (math.inf, 1.0), (0.0, 0.0)):
        m = clip_grad_norm(grads, max_norm, out)
        assert float(m) == float(n)
        check_clipped(out, before, factor)
        if factor == 1.0:
            assert all(torch.equal(o, b) for o, b in zip(out, before))
        assert all(torch.equal(g, b) for g, b in zip(grads, before))
    assert float(clip_grad_norm(grads, 2 * want + 1)) == float(n)
    assert all(torch.equal(g, b) for g, b in zip(grads, before))
    assert float(clip_grad_norm(grads, 0.25 * want)) == float(n)
    check_clipped(grads, before, 0.25)


def test_many_tensors_take_several_launches():
    grads = make([(i * 37) % 301 for i in range(2500)], 4, True)
    want = norm64(grads)
    before = [g.clone() for g in grads]
    assert abs(float(clip_grad_norm(grads, 0.5 * want)) - want) <= 34 * U * want
    check_clipped(grads, before, 0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e30, 3e38, 1e-30, 1e-38, 2e-42])
def test_magnitudes_at_the_ends_of_the_range(dtype, size):
    g = torch.Generator().manual_seed(1)
    t = (torch.rand(5000, generator=g) * size).to(dtype).cuda()
    want = norm64([t])
    if want < 3.4e38:
        assert abs(float(grad_norm([t])) - want) <= 34 * U * want + 2.0 ** -149
    else:
        assert math.isinf(float(grad_norm([t])))
    out = [torch.empty_like(t)]
    clip_grad_norm([t], 0.5 * want, out)  # a norm above fp32's range clips, too
    tiny = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    ref = t.double() * 0.5
    assert ((out[0].double() - ref).abs() <= (HALF[dtype] * 1.01 + 37 * U) * ref + tiny).all()
    if size >= 1e30:  # to a small norm: the factor is below the normal numbers
        clip_grad_norm([t], 1e-3, out)
        ref = t.double() * (1e-3 / want)
        assert ((out[0].double() - ref).abs() <= (HALF[dtype] * 1.01 + 40 * U) * ref + tiny).all()


@pytest.mark.parametrize("bit", range(23))
def test_single_bits_below_the_normal_numbers(bit):
    """Every value the same power of two: 2500 of them, whose root is 50."""
    t = torch.full((2500,), 1 << bit, dtype=torch.int32, device="cuda").view(torch.float32)
    assert float(grad_norm([t])) == 50 * 2.0 ** (bit - 149)
    b = torch.full((2500,), 1 << bit % 7, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    assert float(grad_norm([b])) == 50 * 2.0 ** (bit % 7 - 133)


def test_zeros_and_a_single_value():
    z = torch.zeros(100000, device="cuda")
    assert float(grad_norm([z])) == 0.0
    assert float(clip_grad_norm([z], 1.0)) == 0.0 and (z == 0).all()
    z[54321] = 3e-30
    assert abs(float(grad_norm([z])) - 3e-30) <= 40 * U * 3e-30


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_non_finite_gradients_stay_as_they_are(value):
    grads = make([5000, 40000, 3], 2)
    grads[1][12345] = value
    before = [g.clone() for g in grads]
    n = float(clip_grad_norm(grads, 1e-3))
    assert (math.isnan(n) if math.isnan(value) else n == math.inf)
    out = [torch.empty_like(g) for g in grads]
    clip_grad_norm(grads, 1e-3, out)
    for g, b, o in zip(grads, before, out):
        assert torch.equal(g.nan_to_num(7.0), b.nan_to_num(7.0))
        assert torch.equal(o.nan_to_num(7.0), b.nan_to_num(7.0))


def test_the_same_in_every_run_on_streams_and_in_graphs():
    grads = make([70000, 123, 262144, 9999], 6)
    want = norm64(grads)
    out = [torch.empty_like(g) for g in grads]
    n = float(clip_grad_norm(grads, 0.1 * want, out))
    ref = [o.clone() for o in out]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = []
    for s in (side, other):
        with torch.cuda.stream(s):
            o = [torch.empty_like(g) for g in grads]
            m = clip_grad_norm(grads, 0.1 * want, o)
            runs.append((m, o))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m = clip_grad_norm(grads, 0.1 * want, out)
    for o in out:
        o.zero_()
    m.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for m, o in runs + [(m, out)]:
        assert float(m) == n and all(torch.equal(a, b) for a, b in zip(o, ref))


def test_dense_tensors_in_any_order_of_axes():
    a = torch.randn(30, 50, device="cuda").t()
    b = torch.randn(4, 6, 8, device="cuda").permute(2, 0, 1)
    want = norm64([a, b])
    before = [a.clone(), b.clone()]
    clip_grad_norm([a, b], 0.5 * want)
    check_clipped([a, b], before, 0.5)


def test_neighbouring_slices_of_one_buffer():
    """Tensors that touch, at any offset: nothing of a neighbour is written."""
    for dtype in (torch.bfloat16, torch.float32):
        flat = torch.randn(60000, device="cuda").to(dtype)
        cuts = [3, 4, 21, 22, 1000, 1007, 30001, 59990]
        parts = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
        rest = [flat[:3].clone(), flat[59990:].clone()]
        before = [p.clone() for p in parts]
        want = norm64(parts)
        clip_grad_norm(parts[::2] + parts[1::2], 0.5 * want)
        check_clipped(parts, before, 0.5)
        assert torch.equal(flat[:3], rest[0]) and torch.equal(flat[59990:], rest[1])


def test_one_gradient_into_two_buffers():
    g = torch.randn(5001, device="cuda")
    out = [torch.empty_like(g), torch.empty_like(g)]
    want = norm64([g, g])
    clip_grad_norm([g, g], 0.25 * want, out)
    check_clipped(out, [g, g], 0.25)


def test_refusals():
    a, b = torch.randn(64, device="cuda"), torch.randn(64, device="cuda")
    for f in (lambda: grad_norm([]), lambda: grad_norm([a.half()]), lambda: grad_norm([a.cpu()]),
              lambda: grad_norm([a[::2]]), lambda: clip_grad_norm([a], 1.0, [a, b]),
              lambda: clip_grad_norm([a], 1.0, [b[:32]]),
              lambda: clip_grad_norm([a], 1.0, [b.bfloat16()]),
              lambda: grad_norm([a, b.cpu()])):
        with pytest.raises(ValueError):
            f()
    keep = a.clone()
    for f in (lambda: clip_grad_norm([a, a], 1.0), lambda: clip_grad_norm([a[:40], a[32:]], 1.0),
              lambda: clip_grad_norm([a, b], 1.0, [b, a]), lambda: clip_grad_norm([a], -1.0),
              lambda: clip_grad_norm([a], math.nan),
              lambda: clip_grad_norm([a[:32]], 1.0, [a[8:40]]),
              lambda: clip_grad_norm([a, b], 1.0, [torch.empty_like(a), a])):
        with pytest.raises(DFlashError, match="ARG"):
            f()
    assert torch.equal(a, keep)
    assert float(grad_norm([a, a])) > 0  # reading twice is allowed


def test_a_tensor_of_more_than_2_31_values():
    """Ones but for two values: their squares' sum and its root are exact."""
    n = (1 << 31) + 12345
    t = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    t[-1], t[12345] = 1024.0, -512.0
    want = math.sqrt(n - 2 + 2.0 ** 20 + 2.0 ** 18)
    assert abs(float(grad_norm([t])) - want) <= 34 * U * want
    # a factor of a half, but for its rounding, gives halves in bf16
    assert abs(float(clip_grad_norm([t], want / 2)) - want) <= 34 * U * want
    assert float(t[-1]) == 512.0 and float(t[12345]) == -256.0
    t[-1] = t[12345] = 0.5
    assert float(t.min()) == 0.5 and float(t.max()) == 0.5
