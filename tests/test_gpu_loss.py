"""Cross entropy of a linear head and its gradients on the GPU, against the
definition in 64 bits.

Tolerances (u = 2^-24).  A logit: products of bf16 numbers are exact, their sum
over H goes in steps of 16 whose roundings (cut off, 2u) follow the sum of
sizes: e_z = (H / 16 + 32) * 2u * sum |x||w|.  An exponential is off by e_z, by
the rounding of its exponent (2u |z|) and by 4u, against a reference off by as
much; sums of up to 256 columns and of the tiles: below 256u.  So nll and each
p / (sum of p) are off by
    e = 2 e_z + 4u |z| + 264u  (relative to p, absolute for nll, of which and of
lse 4u each are rounded off).  A gradient rounds the factor p once to bf16
(half a step: 2^-8), sums its terms in steps of 16 again, and rounds the result
to bf16.  For dw the factor of a column's own row is rounded without loss, at
the price of a factor of 1 +- 2^-8 for the column's others: 2^-8 once more.
Below 2^-126, the smallest normal number of fp32 and bf16, numbers may
be lost: each of a sum's terms (factors p, relative to a reference of at least
the target's p, times |d w| or |x|) and the result, 2^-126 * (1 + sum of the
other factors) in all."""
import math

import pytest
import torch

from block_diffusion_draft_gb300 import (DFlashError, linear_cross_entropy,
                                         linear_cross_entropy_grad)
import train_reference as R

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8


def inputs(N, V, H, seed, ignored=0.0, pull=6.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w = torch.zeros(V, H + pad, device="cuda", dtype=torch.bfloat16)
    w[:, :H] = rand(V, H) / math.sqrt(H)
    w = w[:, :H]
    t = torch.randint(0, V, (N,), device="cuda", generator=g)
    x = torch.zeros(N, H + pad, device="cuda", dtype=torch.bfloat16)
    x[:, :H] = 1.5 * rand(N, H) + pull * torch.rand(N, 1, device="cuda",
                                                    generator=g) * w[t].float()
    x = x[:, :H]
    drop = torch.rand(N, device="cuda", generator=g) < ignored
    t = torch.where(drop, torch.where(torch.arange(N, device="cuda") % 2 == 0, -100, V), t)
    d = (rand(N) / N).float()
    return x, w, t.int(), d


def within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = ((got - want).abs() / tol.clamp(min=1e-300)).max() if got.numel() else 0.0
    assert over <= 1.0, f"{what}: {float(over):.3g} of the tolerance"


def check(x, w, t, d, grads=("none", "x", "xw")):
    N, V, H = x.shape[0], w.shape[0], x.shape[1]
    nll, lse, dx, dw, z_size, z_top, dx_size, dw_size = R.linear_cross_entropy_sizes(
        x.double(), w.double(), t, d.double())
    e = 2 * (H / 16 + 32) * 2 * U * z_size + 4 * U * z_top + 264 * U
    held = ((t >= 0) & (t < V)).double()
    for grad in grads:
        if grad == "none":
            got = linear_cross_entropy(x, w, t) + (None, None)
        else:
            got = linear_cross_entropy_grad(x, w, t, d, need_dw=grad == "xw")
        torch.cuda.synchronize()
        within(got[0], nll, (e + 4 * U * nll.abs()) * held, f"nll ({grad})")
        within(got[1], lse, (e + 4 * U * lse.abs()) * held, f"lse ({grad})")
        if got[2] is not None:
            rel = HALF + e[:, None] + (V / 16 + 32) * 2 * U
            lost = 2.0 ** -126 * (1 + d.double().abs()[:, None] * w.double().abs().sum(0))
            within(got[2], dx, HALF * 1.01 * dx.abs() + rel * dx_size + lost, f"dx ({grad})")
        assert (got[3] is not None) == (grad == "xw")
        if got[3] is not None:
            rel = 2 * HALF + float(e.max() if N else 0) + (N / 16 + 32) * 2 * U
            at = x[held > 0].double()
            lost = 2.0 ** -126 * (1 + at.abs().sum(0))
            within(got[3], dw, HALF * 1.01 * dw.abs() + rel * dw_size + lost, "dw")


SIZES = [(1, 1, 8), (1, 2, 8), (3, 5, 16), (16, 300, 64), (17, 257, 72), (127, 256, 128),
         (128, 1000, 256), (129, 999, 200), (255, 2048, 64), (257, 513, 1000), (300, 5000, 320),
         (1000, 300, 8), (2, 40001, 104), (384, 700, 128), (385, 700, 128), (383, 1300, 72),
         (320, 600, 64), (640, 513, 64)]


@pytest.mark.parametrize("ignored", [0.0, 0.4])
@pytest.mark.parametrize("N,V,H", SIZES)
def test_equal_to_the_definition(N, V, H, ignored):
    check(*inputs(N, V, H, N + V, ignored))


@pytest.mark.parametrize("N,V,H", [(20, 700, 64), (200, 700, 136)])
def test_row_strides(N, V, H):
    check(*inputs(N, V, H, 1, 0.2, pad=24))


@pytest.mark.parametrize("N", [40, 300])
def test_sure_rows_keep_their_small_losses(N):
    x, w, t, d = inputs(N, 900, 128, 5, pull=0.0)
    x = (20.0 * w[t.long()].float()).bfloat16()
    nll, _, _, _ = linear_cross_entropy_grad(x, w, t, d, need_dw=False)
    assert float(nll.min()) < 1e-4
    check(x, w, t, d)


def far_rows(x, w, t, rows, column, size):
    """Rows whose logit of `column` lies `size` above the others'."""
    for r in rows:
        u = w[column].float()
        x[r] = (x[r].float() + size * u / u.square().sum()).bfloat16()
        if int(t[r]) == column:
            t[r] = (column + 1) % w.shape[0]


@pytest.mark.parametrize("size", [50.0, 70.0, 120.0, 400.0])
@pytest.mark.parametrize("N", [30, 300])
def test_targets_far_below_the_largest_logit(N, size):
    x, w, t, d = inputs(N, 1500, 256, 9)
    far_rows(x, w, t, range(3, N, 7), 700, size)
    check(x, w, t, d)


@pytest.mark.parametrize("N,V", [(30, 1500), (300, 1500), (19000, 30000)])
def test_tiny_weights_of_rows_far_below_their_largest_logit(N, V):
    """Weights of 2^-77 of rows whose target is up to 2^-79 as likely as the
    largest one (one more would have the row done again): gradients of 2^-77,
    both terms of them.  In one piece and in two."""
    x, w, t, d = inputs(N, V, 256 if N < 1000 else 64, 9)
    for i, size in enumerate((20.0, 40.0, 45.0, 50.0)):
        far_rows(x, w, t, range(3 + i, N, 7 if N < 1000 else 700), 700, size)
    d = torch.sign(d) * 2.0 ** -77
    check(x, w, t, d, ("x", "xw"))


def test_every_row_far_apart():
    x, w, t, d = inputs(200, 1500, 256, 10)
    check((x.float() * 60.0).bfloat16(), w, t, d)


def test_several_pieces():
    """The exponentials of 20000 rows and 30000 columns (1.2 GB) come in
    two pieces; rows with a far logit in either."""
    x, w, t, d = inputs(20000, 30000, 64, 11, 0.01)
    for i, column in enumerate((5, 12000, 20000, 29999)):
        far_rows(x, w, t, range(100 + i, 20000, 4999), column, 90.0 + 30.0 * i)
    far_rows(x, w, t, range(300, 400, 13), 100, 100.0)    # far in the first piece
    far_rows(x, w, t, range(300, 400, 13), 29000, 210.0)  # and further in the last
    check(x, w, t, d)


@pytest.mark.parametrize("N,V,H", [(12011, 45007, 520), (12011, 100003, 520)])
def test_several_pieces_of_a_wide_head(N, V, H):
    """Two and three pieces, 9 k-blocks of which the last is an eighth, three
    tiles of hidden channels; rows that are done again in one piece, in each of
    the others, and in several of them; the same in every run."""
    x, w, t, d = inputs(N, V, H, 13, 0.01)
    for i, column in enumerate((5, V // 3, V // 2 + 300, V - 1)):
        far_rows(x, w, t, range(100 + i, N, 3001), column, 90.0 + 30.0 * i)
    far_rows(x, w, t, range(300, 400, 13), 100, 100.0)
    far_rows(x, w, t, range(300, 400, 13), V // 2 + 700, 210.0)
    far_rows(x, w, t, range(300, 400, 26), V - 900, 330.0)
    check(x, w, t, d, ("x", "xw"))
    a, b = (linear_cross_entropy_grad(x, w, t, d) for _ in range(2))
    assert all(torch.equal(m, n) for m, n in zip(a, b))


def test_several_pieces_of_tiles_of_one_cta():
    """Up to 128 rows a piece is 2^21 columns."""
    N, V = 100, 2200003
    x, w, t, d = inputs(N, V, 72, 14, 0.1)
    far_rows(x, w, t, range(3, N, 17), 5, 90.0)
    far_rows(x, w, t, range(4, N, 17), V - 700, 120.0)
    far_rows(x, w, t, range(3, N, 34), V - 900, 210.0)
    check(x, w, t, d, ("x", "xw"))


def test_a_head_whose_rows_lie_far_apart():
    x, w, t, d = inputs(20, 260, 64, 15)
    space = torch.zeros(260 * ((1 << 23) + 8), device="cuda", dtype=torch.bfloat16)
    far = space.as_strided((260, 64), ((1 << 23) + 8, 1))
    far.copy_(w)
    want = linear_cross_entropy_grad(x, w, t, d)
    assert all(torch.equal(a, b) for a, b in zip(linear_cross_entropy_grad(x, far, t, d), want))


def test_a_head_of_more_than_2_31_values():
    """Zero but for its last 64 columns, which hold the targets: the other
    columns' logits are 0 and their dw the same everywhere.  Tolerances as
    above, with z of the last columns alone."""
    N, V, H, last = 8, 530000, 4096, 64
    x, tail, t, d = inputs(N, last, H, 16)
    w = torch.zeros(V, H, device="cuda", dtype=torch.bfloat16)
    w[-last:] = tail
    nll, lse, dx, dw = linear_cross_entropy_grad(x, w, t + (V - last), d)
    z = x.double() @ tail.double().t()
    want = torch.log(z.exp().sum(1) + (V - last))
    z_size = (x.double().abs() @ tail.double().abs().t()).amax(1)
    e = 2 * (H / 16 + 32) * 2 * U * z_size + 4 * U * z.abs().amax(1) + 264 * U
    within(lse, want, e + 4 * U * want.abs(), "lse")
    within(nll, want - z.gather(1, t.long()[:, None])[:, 0], e + 4 * U * nll.double().abs(), "nll")
    p = torch.cat([torch.zeros(N, last, device="cuda", dtype=torch.float64), z], 1)
    p = (p - want[:, None]).exp()
    hit = torch.nn.functional.one_hot(t.long() + last, 2 * last)
    f = d.double()[:, None] * (p - hit)
    rows = torch.cat([dw[:last], dw[-last:]])
    rel = 2 * HALF + float(e.max()) + (N / 16 + 32) * 2 * U
    size = (d.double()[:, None] * (p + hit)).abs().t() @ x.double().abs()
    ref = f.t() @ x.double()
    within(rows, ref, HALF * 1.01 * ref.abs() + rel * size, "dw")
    assert torch.equal(dw[:last], dw[:1].expand(last, H))
    assert torch.equal(dw[V // 2:V // 2 + last], dw[:last])
    assert torch.equal(dw[V - 2 * last:V - last], dw[:last])
    ref = f[:, last:] @ tail.double()
    size = (d.double()[:, None] * (p + hit)).abs()[:, last:] @ tail.double().abs()
    within(dx, ref, HALF * 1.01 * ref.abs() + (HALF + e[:, None] + (V / 16 + 32) * 2 * U) * size,
           "dx")


def test_nothing_counts():
    x, w, t, d = inputs(50, 400, 64, 2)
    t.fill_(-1)
    nll, lse, dx, dw = linear_cross_entropy_grad(x, w, t, d)
    for z in (nll, lse, dx, dw):
        assert (z == 0).all()
    e = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16)
    nll, lse, dx, dw = linear_cross_entropy_grad(e, w, t[:0], d[:0])
    assert nll.shape == (0,) and dx.shape == (0, 64) and (dw == 0).all()
    assert linear_cross_entropy(e, w, t[:0])[0].shape == (0,)


def test_rows_that_do_not_count_may_hold_anything():
    x, w, t, d = inputs(150, 400, 64, 3)
    x, d = x.clone(), d.clone()
    t[::3] = -100
    clean = linear_cross_entropy_grad(x, w, t, d)
    x[::3] = float("nan")
    d[::3] = float("inf")
    got = linear_cross_entropy_grad(x, w, t, d)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))


def test_non_finite_rows_stay_by_themselves():
    x, w, t, d = inputs(150, 400, 64, 4)
    clean = linear_cross_entropy_grad(x, w, t, d, need_dw=False)
    x = x.clone()
    x[7, 3], x[140, 0] = float("nan"), float("inf")
    got = linear_cross_entropy_grad(x, w, t, d, need_dw=False)
    keep = torch.ones(150, dtype=torch.bool, device="cuda")
    keep[[7, 140]] = False
    for a, b in zip(got[:3], clean[:3]):
        assert torch.equal(a[keep], b[keep])
        assert not torch.isfinite(a[~keep]).reshape(2, -1).all(-1).any()


@pytest.mark.parametrize("N", [60, 400])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_logit_that_is_not_finite_leaves_no_finite_loss(N, value):
    """Column 11 is `value` times the first channel: infinite for every row
    whose first channel has the sign for it; it is the target of some rows."""
    x, w, t, _ = inputs(N, 700, 64, 14)
    x, w = x.clone(), w.clone()
    x[:, 0] = torch.where(torch.arange(N, device="cuda") % 3 == 0, 0.0, 1.0)
    w[:, 0] = 0.0
    w[11, 0] = value
    t[t == 11] = 12
    t[1::9] = 11
    d = torch.ones(N, device="cuda")
    # 0 * value: not a number; -inf is a probability of zero where it is no target
    bad = torch.ones(N, dtype=torch.bool, device="cuda")
    if value == -math.inf:
        bad = (x[:, 0] == 0) | (t == 11)
    for nll in (linear_cross_entropy(x, w, t)[0],
                linear_cross_entropy_grad(x, w, t, d, need_dw=False)[0],
                linear_cross_entropy_grad(x, w, t, d)[0]):
        assert not torch.isfinite(nll[bad]).any()
        assert torch.isfinite(nll[~bad]).all()


@pytest.mark.parametrize("N", [60, 400])
def test_the_same_in_every_run_on_streams_and_in_graphs(N):
    x, w, t, d = inputs(N, 3001, 200, 6, 0.1)
    want = linear_cross_entropy_grad(x, w, t, d) + linear_cross_entropy(x, w, t)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = []
    for s in (side, other):
        with torch.cuda.stream(s):
            runs.append(linear_cross_entropy_grad(x, w, t, d) + linear_cross_entropy(x, w, t))
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = linear_cross_entropy_grad(x, w, t, d) + linear_cross_entropy(x, w, t)
        graphs.append((graph, out))
    for _ in range(5):
        for _, out in graphs:
            for z in out:
                z.zero_()
        torch.cuda.synchronize()
        for (graph, _), s in zip(graphs, (side, other)):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for out in runs + [o for _, o in graphs]:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_gradient_equals_differences():
    """Central differences of the loss along random directions.  nll is off by
    at most e (about 1e-4 here), the step is 2^-4 of exact bf16 changes."""
    x, w, t, d = inputs(9, 60, 16, 8)
    x, w = (x.float() * 64).round().div(64).bfloat16(), (w.float() * 64).round().div(64).bfloat16()
    _, _, dx, dw = linear_cross_entropy_grad(x, w, t, d)
    loss = lambda a, b: float((linear_cross_entropy(a, b, t)[0].double()  # noqa: E731
                               * d.double()).sum())
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(5):
        for v, grad in ((x, dx), (w, dw)):
            step = torch.where(torch.rand(v.shape, device="cuda", generator=g) < 0.5, -1.0,
                               1.0) / 64
            lo, hi = (v.float() - step).bfloat16(), (v.float() + step).bfloat16()
            a, b = ((lo, w), (hi, w)) if v is x else ((x, lo), (x, hi))
            slope = float((grad.double() * (hi.double() - lo.double())).sum())
            size = float((grad.double().abs() * (hi.double() - lo.double()).abs()).sum())
            # third derivative: below size * (sum of |step| over a row)^2
            spread = float((hi.double() - lo.double()).abs().sum(1).max())
            assert abs(loss(*b) - loss(*a) - slope) <= size * (0.02 + spread ** 2) + 1e-5


@pytest.mark.parametrize("N,V", [(96, 4000), (500, 20000)])
def test_own_factors_of_dw_lose_nothing(N, V):
    """Rows with targets of their own: what is left of dw's error is its last
    rounding (relative to the 2-norm 2^-8 / sqrt(3) at most for numbers of one
    binade's lower end) and the other factors', which are below 2^-4 of the
    targets' here: together below 2^-8 * (0.58 + 2^-4 * 2)."""
    x, w, t, d = inputs(N, V, 128, 12, pull=1.0)
    t = torch.randperm(V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)
                       )[:N].int()
    d = d.abs() + 1e-3
    _, _, _, dw = linear_cross_entropy_grad(x, w, t, d)
    want = R.linear_cross_entropy(x.double(), w.double(), t, d.double())[3]
    own = torch.zeros(V, dtype=torch.bool, device="cuda")
    own[t.long()] = True
    assert float(want[~own].norm()) < 2 ** -4 * float(want[own].norm())
    assert float((dw.double() - want).norm() / want.norm()) <= HALF * (0.58 + 2 ** -3)


def test_refusals():
    x, w, t, d = inputs(8, 40, 64, 1)
    for f in (lambda: linear_cross_entropy(x.float(), w, t),
              lambda: linear_cross_entropy(x, w.half(), t),
              lambda: linear_cross_entropy(x, w[:, :32], t),
              lambda: linear_cross_entropy(x, w, t.long()),
              lambda: linear_cross_entropy(x, w, t[:5]),
              lambda: linear_cross_entropy(x.cpu(), w, t),
              lambda: linear_cross_entropy(x.t().contiguous().t(), w, t),
              lambda: linear_cross_entropy_grad(x, w, t, d.double()),
              lambda: linear_cross_entropy_grad(x, w, t, d[:3])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(DFlashError, match="SHAPE"):
        linear_cross_entropy(x[:, :60].contiguous(), w[:, :60].contiguous(), t)
    wide = torch.zeros(8, 68, device="cuda", dtype=torch.bfloat16)
    for a, b in ((wide[:, :64], w), (x, torch.zeros(40, 68, device="cuda",
                                                   dtype=torch.bfloat16)[:, 4:])):
        with pytest.raises(DFlashError, match="ARG"):
            linear_cross_entropy(a, b, t)
