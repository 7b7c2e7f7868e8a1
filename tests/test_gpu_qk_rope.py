"""Per-head norm and rotation of queries and keys and its gradient on the GPU,
against the definition in 64 bits.

Tolerance: a stored value is off by half a step of its type.  Before that, in
fp32 (step 2^-24 of the value): the sum of squares takes at most 13 additions
and products, halved by the root, then mean, eps, root and quotient (4), gain
and 1/rms (2), the rotation's factor, product and addition (3): below 20 * 2^-24
of |z_j| + |z_{j+d/2}|.  The gradient's terms pass the same steps once more and
the sum of products: below 40 * 2^-24 of the terms' sizes.  A gain's gradient
adds 64 sums of at most 4 such terms in sequence: 128 * 2^-24 of the terms'
sizes together."""
import pytest
import torch

from block_diffusion_draft_gb300 import DFlashAttention
import train_reference as R

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24
MAXPOS, THETA, EPS = 70000, 1e6, 1e-6


def layer(nq, nkv, d, dtype):
    z = lambda *s: torch.zeros(*s, dtype=dtype)  # noqa: E731
    g = torch.Generator().manual_seed(nq + d)
    gain = lambda: (1 + 0.2 * torch.randn(d, generator=g)).to(dtype)  # noqa: E731
    w = dict(wq=z(nq * d, 128), wk=z(nkv * d, 128), wv=z(nkv * d, 128), wo=z(128, nq * d),
             q_norm=gain(), k_norm=gain())
    return DFlashAttention(w, hidden=128, n_heads=nq, n_kv_heads=nkv, head_dim=d, rms_eps=EPS,
                           rope_theta=THETA, max_position=MAXPOS, dtype=dtype), w


def close(got, want, size, dtype, steps, what):
    got = got.detach().double().cpu()
    tol = HALF[dtype] * want.abs() * (1 + 2 ** -8) + steps * U * size
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{what}: {((got - want).abs() / tol).max()} of the tolerance"


def case(B, rows, nq, nkv, d, dtype, layout, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, rows, nq + 2 * nkv, d, generator=g)
    x = (x * torch.exp(torch.randn(B, rows, nq + 2 * nkv, 1, generator=g))).to(dtype).cuda()
    q, k = x[:, :, :nq], x[:, :, nq:nq + nkv]
    if layout == "dense":
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, MAXPOS, (B, rows), generator=g, dtype=torch.int32)
    dq = torch.randn(B, rows, nq, d, generator=g).to(dtype).cuda()
    dk = torch.randn(B, nkv, rows + 3, d, generator=g).to(dtype).cuda()[:, :, 3:].transpose(1, 2)
    return q, k, pos, dq, dk


SHAPES = [(1, 1, 1, 1, 128, torch.bfloat16), (1, 16, 32, 8, 128, torch.bfloat16),
          (3, 37, 7, 1, 128, torch.bfloat16), (2, 129, 9, 3, 128, torch.bfloat16),
          (1, 1, 4, 2, 64, torch.float32), (2, 65, 6, 2, 64, torch.float32),
          (1, 33, 5, 5, 128, torch.float32), (2, 19, 4, 2, 80, torch.float32),
          (1, 7, 3, 1, 2, torch.float32), (1, 5, 2, 1, 256, torch.float32),
          (2, 11, 3, 3, 34, torch.float32)]


@pytest.mark.parametrize("layout", ["dense", "slices"])
@pytest.mark.parametrize("B,rows,nq,nkv,d,dtype", SHAPES)
def test_forward_and_gradient_equal_the_definition(B, rows, nq, nkv, d, dtype, layout):
    attn, w = layer(nq, nkv, d, dtype)
    q, k, pos, dq, dk = case(B, rows, nq, nkv, d, dtype, layout, B + rows)
    gq, gk = w["q_norm"].cuda(), w["k_norm"].cuda()
    keys = torch.full((B, nkv, rows + 5, d), 7.0, device="cuda", dtype=dtype)
    q_out, k_out = attn.qk_norm_rope(q, k, pos.cuda(), gq, gk,
                                     k_out=keys[:, :, 5:].transpose(1, 2))
    same = attn.qk_norm_rope(q, k, pos.cuda())  # the layer's own gains
    res = attn.qk_norm_rope_backward(q, k, pos.cuda(), gq, gk, dq, dk)
    again = attn.qk_norm_rope_backward(q, k, pos.cuda(), None, None, dq, dk)
    torch.cuda.synchronize()
    assert (keys[:, :, :5] == 7.0).all()
    assert torch.equal(same[0], q_out) and torch.equal(same[1], k_out)
    assert all(torch.equal(a, b) for a, b in zip(res, again))
    f = lambda t: t.double().cpu()  # noqa: E731
    for x, gain, dy, y, dx, dg, name in ((q, gq, dq, q_out, res[0], res[2], "q"),
                                         (k, gk, dk, k_out, res[1], res[3], "k")):
        want, size = R.qk_rope(f(x), f(gain), pos, THETA, EPS)
        close(y, want, size, dtype, 20, name)
        want, wdg, size, gsize = R.qk_rope_backward(f(x), f(gain), pos, THETA, EPS, f(dy))
        close(dx, want, size, dtype, 40, "d" + name)
        close(dg, wdg, gsize, torch.float32, 128, "gain of " + name)
    assert attn.device_error() == 0


def test_unaligned_fp32_rows_and_odd_strides():
    attn, w = layer(3, 1, 64, torch.float32)
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(2, 9, 4 * 64 + 3, generator=g).cuda()
    x = wide[:, :, 1:1 + 256].unflatten(-1, (4, 64))
    q, k = x[:, :, :3], x[:, :, 3:]
    pos = torch.randint(0, MAXPOS, (2, 9), generator=g, dtype=torch.int32)
    q_out, k_out = attn.qk_norm_rope(q, k, pos.cuda())
    dense = attn.qk_norm_rope(q.contiguous(), k.contiguous(), pos.cuda())
    for x, gain, y in ((q, "q_norm", q_out), (k, "k_norm", k_out), (q, "q_norm", dense[0])):
        want, size = R.qk_rope(x.double().cpu(), w[gain].double(), pos, THETA, EPS)
        close(y, want, size, torch.float32, 20, gain)


def test_only_keys_in_place_and_broadcast_gradient():
    attn, w = layer(4, 2, 128, torch.bfloat16)
    q, k, pos, _, _ = case(2, 21, 4, 2, 128, torch.bfloat16, "dense", 3)
    none, k_out = attn.qk_norm_rope(None, k, pos.cuda())
    both = attn.qk_norm_rope(q, k, pos.cuda())
    assert none is None and torch.equal(k_out, both[1])
    kk = k.clone()
    attn.qk_norm_rope(None, kk, pos.cuda(), k_out=kk)
    assert torch.equal(kk, both[1])
    one = torch.ones(1, 1, 1, 128, device="cuda", dtype=torch.bfloat16)
    wide, dense = one.expand(2, 21, 4, 128), one.repeat(2, 21, 4, 1)
    a = attn.qk_norm_rope_backward(q, None, pos.cuda(), None, None, wide, None)
    b = attn.qk_norm_rope_backward(q, None, pos.cuda(), None, None, dense, None, dq_out=dense)
    assert a[1] is None and a[3] is None
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_nothing_to_do_and_positions_outside():
    attn, _ = layer(4, 2, 128, torch.bfloat16)
    z = torch.zeros(0, 5, 4, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(0, 5, device="cuda", dtype=torch.int32)
    q_out, _ = attn.qk_norm_rope(z, None, pos)
    assert q_out.shape == z.shape
    _, _, dg, _ = attn.qk_norm_rope_backward(z, None, pos, None, None, z, None)
    assert (dg == 0).all()
    q = torch.randn(1, 3, 4, 128, device="cuda").bfloat16()
    far = torch.tensor([[-5, MAXPOS - 1, MAXPOS + 7]], device="cuda", dtype=torch.int32)
    near = torch.tensor([[0, MAXPOS - 1, MAXPOS - 1]], device="cuda", dtype=torch.int32)
    a, b = attn.qk_norm_rope(q, None, far)[0], attn.qk_norm_rope(q, None, near)[0]
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    assert attn.device_error() == 2 and attn.device_error() == 0


def test_non_finite_heads_stay_by_themselves():
    attn, _ = layer(4, 2, 128, torch.bfloat16)
    q, k, pos, dq, dk = case(2, 9, 4, 2, 128, torch.bfloat16, "dense", 8)
    clean = attn.qk_norm_rope(q, k, pos.cuda())[0].clone()
    q[1, 3, 2, 5] = float("nan")
    q[0, 2, 0, 0] = float("inf")
    got = attn.qk_norm_rope(q, k, pos.cuda())[0]
    bad = torch.zeros(2, 9, 4, dtype=torch.bool, device="cuda")
    bad[1, 3, 2] = bad[0, 2, 0] = True
    assert torch.equal(got[~bad], clean[~bad])
    assert torch.isnan(got[bad]).any(-1).all()


def test_another_stream_and_a_replayed_graph():
    attn, _ = layer(8, 2, 128, torch.bfloat16)
    q, k, pos, dq, dk = case(2, 50, 8, 2, 128, torch.bfloat16, "slices", 9)
    p = pos.cuda()
    want = attn.qk_norm_rope(q, k, p) + attn.qk_norm_rope_backward(q, k, p, None, None, dq, dk)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = attn.qk_norm_rope(q, k, p) + attn.qk_norm_rope_backward(q, k, p, None, None, dq, dk)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):  # two graphs, replayed on two streams at a time
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = attn.qk_norm_rope(q, k, p)
            out += attn.qk_norm_rope_backward(q, k, p, None, None, dq, dk)
        graphs.append((graph, out))
    other = torch.cuda.Stream()
    for _ in range(20):
        for t in graphs[0][1] + graphs[1][1]:
            t.zero_()
        torch.cuda.synchronize()
        for (graph, _), s in zip(graphs, (side, other)):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    attn, _ = layer(4, 2, 128, torch.bfloat16)
    q, k, pos, dq, dk = case(2, 9, 4, 2, 128, torch.bfloat16, "dense", 8)
    p = pos.cuda()
    bad = [lambda: attn.qk_norm_rope(None, None, p), lambda: attn.qk_norm_rope(q, k, p.long()),
           lambda: attn.qk_norm_rope(q, k, p[:1]), lambda: attn.qk_norm_rope(q.float(), k, p),
           lambda: attn.qk_norm_rope(q[:, :, :3], k, p), lambda: attn.qk_norm_rope(q.cpu(), k, p),
           lambda: attn.qk_norm_rope(q.transpose(2, 3).contiguous().transpose(2, 3), k, p),
           lambda: attn.qk_norm_rope(None, k, p, q_out=q),
           lambda: attn.qk_norm_rope(q, k, p, torch.ones(64, device="cuda").bfloat16()),
           lambda: attn.qk_norm_rope_backward(q, k, p, None, None, dq, None)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    from block_diffusion_draft_gb300 import DFlashError
    wide = torch.zeros(2, 9, 4 * 128 + 4, device="cuda", dtype=torch.bfloat16)
    odd = wide[:, :, 4:].unflatten(-1, (4, 128))
    for f in (lambda: attn.qk_norm_rope(odd, None, p),
              lambda: attn.qk_norm_rope(q, None, p, q_out=q[:, :1].expand(2, 9, 4, 128)),
              lambda: attn.qk_norm_rope(q, None, p, q_out=wide.view(-1).as_strided(
                  (2, 9, 4, 128), (9 * 512, 448, 128, 1)))):
        with pytest.raises(DFlashError, match="ARG"):
            f()


@pytest.mark.parametrize("axis", [0, 1, 2])
def test_offsets_above_32_bits(axis):
    """One axis of every tensor strides over 2^31 elements and more: the same
    results as of dense tensors."""
    attn, _ = layer(2, 2, 128, torch.bfloat16)
    shape = (2, 2, 2, 128)
    g = torch.Generator().manual_seed(axis)
    dense = [torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(4)]
    pos = torch.tensor([[5, 60000], [17, 3]], dtype=torch.int32, device="cuda")
    want = attn.qk_norm_rope(dense[0], dense[1], pos)
    back = attn.qk_norm_rope_backward(dense[0], dense[1], pos, None, None, dense[2], dense[3])
    space = torch.zeros((1 << 31) + 4096 * 6, device="cuda", dtype=torch.bfloat16)
    strides = [1024, 512, 256, 1]
    strides[axis] = 1 << 31
    far = [space[i * 4096:].as_strided(shape, strides) for i in range(6)]
    for f, x in zip(far, dense):
        f.copy_(x)
    got = attn.qk_norm_rope(far[0], far[1], pos, q_out=far[4], k_out=far[5])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = attn.qk_norm_rope_backward(far[0], far[1], pos, None, None, far[2], far[3],
                                     dq_out=far[4], dk_out=far[5])
    assert all(torch.equal(a, b) for a, b in zip(got, back))


# Size and kind of the kernels' paths: 16-byte pieces in either type, and any
# head size (80).
@pytest.mark.parametrize("size", [1e13, 1e14, 1e15, 1e16, 1e17, 1e18])
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float32),
                                     (128, torch.float32), (80, torch.float32)])
def test_large_heads_keep_the_gradients_projection(d, dtype, size):
    """Heads of root mean square `size`, whose squares' sum is just inside fp32:
    the gradient is of size |dy| / size, both terms of it."""
    attn, w = layer(6, 2, d, dtype)
    q, k, pos, dq, dk = case(2, 9, 6, 2, d, dtype, "dense", 7)
    q, k = (size * x.double() / x.double().square().mean(-1, keepdim=True).sqrt() for x in (q, k))
    q, k = q.to(dtype), k.to(dtype)
    # along x, so that the projection takes most of the gradient away
    dq = (dq.double() + 3 * q.double() / size).to(dtype)
    res = attn.qk_norm_rope_backward(q, k, pos.cuda(), None, None, dq, dk)
    y = attn.qk_norm_rope(q, k, pos.cuda())
    f = lambda t: t.double().cpu()  # noqa: E731
    for x, gain, dy, out, dx, dg, name in ((q, w["q_norm"], dq, y[0], res[0], res[2], "q"),
                                           (k, w["k_norm"], dk, y[1], res[1], res[3], "k")):
        want, z = R.qk_rope(f(x), f(gain), pos, THETA, EPS)
        close(out, want, z, dtype, 20, name)
        want, wdg, z, gz = R.qk_rope_backward(f(x), f(gain), pos, THETA, EPS, f(dy))
        close(dx, want, z, dtype, 40, "d" + name)
        close(dg, wdg, gz, torch.float32, 128, "gain of " + name)


# More work than the backward's persistent warps (152 SMs: 1824, 3648 of the
# kernel for any head size) take at once, of both kinds: rings that are filled
# again, gains summed over several items, CTAs shared between the kinds.
MANY = [(2, 4099, 21, 3, 128, torch.bfloat16),  # items of 16 heads, the second one of 5
        (1, 10007, 4, 2, 64, torch.float32), (3, 1301, 9, 3, 128, torch.float32),
        (2, 2003, 6, 3, 80, torch.float32), (2, 2003, 9, 3, 64, torch.float32)]


@pytest.mark.parametrize("B,rows,nq,nkv,d,dtype", MANY)
def test_more_items_than_warps(B, rows, nq, nkv, d, dtype):
    """A gain's gradient: a thread adds up to 14 items of 4 heads (fp32 heads of
    80: 10 of one), then 2 to 5 exchanges, 4 or 8 warps, 8 slices of CTAs and
    the 8 + 3 of their sum: below 88 additions, and 40 for the terms: 128."""
    attn, w = layer(nq, nkv, d, dtype)
    q, k, pos, dq, dk = case(B, rows, nq, nkv, d, dtype, "slices", rows)
    copy = torch.clone
    if (nq, d) == (9, 64):  # rows that are not on 16-byte boundaries
        def copy(t):
            wide = torch.zeros(B, rows, t.shape[2] * d + 1, device="cuda")
            wide[:, :, 1:] = t.flatten(2)
            return wide[:, :, 1:].unflatten(-1, t.shape[2:])
        q, k = copy(q), copy(k)
    p = pos.cuda()
    y = attn.qk_norm_rope(q, k, p)
    res = attn.qk_norm_rope_backward(q, k, p, None, None, dq, dk)
    alone = (attn.qk_norm_rope_backward(q, None, p, None, None, dq, None),
             attn.qk_norm_rope_backward(None, k, p, None, None, None, dk))
    assert torch.equal(res[0], alone[0][0]) and torch.equal(res[1], alone[1][1])
    f = lambda t: t.double().cpu()  # noqa: E731
    for x, gain, dy, out, dx, dg, name in ((q, w["q_norm"], dq, y[0], res[0], res[2], "q"),
                                           (k, w["k_norm"], dk, y[1], res[1], res[3], "k")):
        want, size = R.qk_rope(f(x), f(gain), pos, THETA, EPS)
        close(out, want, size, dtype, 20, name)
        want, wdg, size, gsize = R.qk_rope_backward(f(x), f(gain), pos, THETA, EPS, f(dy))
        close(dx, want, size, dtype, 40, "d" + name)
        close(dg, wdg, gsize, torch.float32, 128, "gain of " + name)
    # in place: no piece may be copied ahead after it was overwritten
    for over in (0, 1):
        a, b = (copy(q), dq) if over == 0 else (q, copy(dq))
        got = attn.qk_norm_rope_backward(a, None, p, None, None, b, None,
                                         dq_out=a if over == 0 else b)
        assert torch.equal(got[0], alone[0][0]) and torch.equal(got[2], alone[0][2])


def test_addresses_that_are_not_aligned_are_refused():
    """On the host, before anything is launched: odd addresses of the 32-bit
    tensors, and of bf16 heads and gains off their 16-byte boundaries."""
    from ctypes import c_int64, c_void_p, cast
    from block_diffusion_draft_gb300 import lib
    attn, _ = layer(4, 2, 128, torch.bfloat16)
    q = torch.randn(1, 3, 4, 128, device="cuda").bfloat16()
    out, pos = torch.zeros_like(q), torch.arange(3, device="cuda", dtype=torch.int32)
    dg, ws = torch.zeros(132, device="cuda"), torch.zeros(1 << 20, device="cuda")
    gain = torch.ones(136, device="cuda", dtype=torch.bfloat16)

    def call(pos_off=0, dg_off=0, x_off=0, out_off=0, gain_off=0, back=True):
        head = lambda t, o: cast((c_int64 * 4)(t.data_ptr() + o, 0, 512, 128),  # noqa: E731
                                 c_void_p)
        x, y, p = head(q, x_off), head(out, out_off), pos.data_ptr() + pos_off
        g = gain.data_ptr() + gain_off
        stream = torch.cuda.current_stream().cuda_stream
        if not back:
            return lib().dflash_qk_norm_rope(attn.handle, 1, 3, x, None, g, None, p, y, None, stream)
        return lib().dflash_qk_norm_rope_backward(
            attn.handle, 1, 3, x, None, g, None, p, x, None, y, None, dg.data_ptr() + dg_off, None,
            ws.data_ptr(), 4 * ws.numel(), stream)

    for back in (False, True):
        for kw in (dict(pos_off=1), dict(pos_off=2), dict(x_off=8), dict(out_off=2),
                   dict(gain_off=4)) + ((dict(dg_off=2),) if back else ()):
            assert call(back=back, **kw) == -1 and b"align" in lib().dflash_last_error(), kw
    torch.cuda.synchronize()
    assert (out == 0).all() and (dg == 0).all()
    assert call(back=False) == 0 and call() == 0
    assert torch.isfinite(dg[:128]).all() and (dg[128:] == 0).all()
