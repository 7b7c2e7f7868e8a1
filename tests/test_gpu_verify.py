"""Verification of drafted tokens on the GPU: equal, token by token, to the
definition in exact arithmetic."""
import math

import numpy as np
import pytest
import torch

from block_diffusion_draft_gb300 import verify_draft

import q8_reference as R

pytestmark = pytest.mark.gpu


def inputs(B, D, V, dtype, greedy, seed, pad=0, sharp=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(B, D + 1, V, generator=g)
    guess = logits[:, :D] + 0.3 * sharp * torch.randn(B, D, V, generator=g)
    t = torch.zeros(B, D + 1, V + pad, dtype=dtype)
    t[..., :V] = torch.softmax(logits, -1).to(dtype)
    q = torch.zeros(B, D, V + pad, dtype=dtype)
    q[..., :V] = torch.softmax(guess, -1).to(dtype)
    if greedy or D == 0:
        x = guess.argmax(-1).int() if D else torch.zeros(B, 0, dtype=torch.int32)
    else:
        x = torch.multinomial(torch.softmax(guess, -1).view(-1, V), 1, generator=g).view(B, D).int()
    ua, us = torch.rand(B, D, generator=g), torch.rand(B, generator=g)
    return x, None if greedy else q, t, ua, us


def check(x, q, t, ua, us, n=None, V=None):
    V = V or t.shape[2]
    dev = lambda z: None if z is None else z.cuda()  # noqa: E731
    tq, tt = dev(q), dev(t)
    acc, tok = verify_draft(dev(x), None if tq is None else tq[..., :V], tt[..., :V], dev(ua),
                            dev(us), dev(n))
    acc, tok = acc.cpu(), tok.cpu()
    for b in range(x.shape[0]):
        want = R.verify(x[b].tolist(), None if q is None else q[b, :, :V].double().numpy(),
                        t[b, :, :V].double().numpy(), ua[b].tolist(), float(us[b]),
                        x.shape[1] if n is None else int(n[b]))
        assert int(acc[b]) == want[0], b
        assert tok[b].tolist() == want[1], b


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("B,D,V", [(1, 1, 1), (2, 3, 2), (3, 1, 31), (1, 7, 128), (5, 2, 129),
                                   (2, 15, 1000), (40, 4, 513), (1, 2, 40001), (3, 0, 77)])
def test_equal_to_the_definition(dtype, greedy, B, D, V):
    for seed in range(3):
        check(*inputs(B, D, V, dtype, greedy, seed))


@pytest.mark.parametrize("pad", [1, 3, 4, 8])
def test_row_strides_and_alignment(pad):
    for dtype in (torch.float32, torch.bfloat16):
        check(*inputs(3, 4, 1001, dtype, False, 5, pad), V=1001)
        check(*inputs(3, 4, 1000, dtype, True, 6, pad), V=1000)
    # one row of probabilities for every place and sequence (stride 0)
    x, q, t, ua, us = inputs(2, 3, 300, torch.float32, False, 7)
    q1, t1 = q[:1, :1].expand(2, 3, 300), t[:1, :1].expand(2, 4, 300)
    acc, tok = verify_draft(x.cuda(), q[:1, :1].cuda().expand(2, 3, 300),
                            t[:1, :1].cuda().expand(2, 4, 300), ua.cuda(), us.cuda())
    for b in range(2):
        want = R.verify(x[b].tolist(), q1[b].double().numpy(), t1[b].double().numpy(),
                        ua[b].tolist(), float(us[b]), 3)
        assert (int(acc[b]), tok[b].tolist()) == want


def test_drafts_of_different_numbers():
    x, q, t, ua, us = inputs(9, 6, 400, torch.float32, False, 8, sharp=0.5)
    check(x, q, t, ua, us, torch.tensor([0, 1, 2, 3, 4, 5, 6, 99, -4], dtype=torch.int32))
    x, q, t, ua, us = inputs(9, 6, 400, torch.float32, True, 9, sharp=0.1)
    check(x, q, t, ua * 1e-3, us, torch.tensor([6, 0, 1, 2, 3, 4, 5, 6, 6], dtype=torch.int32))


def test_many_drafts_of_one_sequence():
    x, q, t, ua, us = inputs(1, 700, 16, torch.float32, False, 10, sharp=0.05)
    check(x, q, t, ua * 0.3, us)   # more drafts than a CTA has threads
    check(x, q, t, ua * 0.0, us)   # all accepted


def test_uniform_numbers_at_their_ends():
    x, q, t, ua, us = inputs(6, 3, 333, torch.float32, False, 11)
    t[:, :, :5] = 0
    t[:, :, 300:] = 0
    for u in (0.0, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, math.nan, 2.0 ** -60, math.inf):
        us.fill_(u)
        check(x, q, t, ua, us)
    for u in (0.0, 1 - 2.0 ** -24):
        check(x, q, t, torch.full_like(ua, u), us * 0 + 0.5)


def test_acceptance_is_exact_at_its_border():
    """u q against p where their rounded fp32 product would decide otherwise."""
    q0, u0 = np.float32(0.7), np.float32(0.3)
    prod = float(q0) * float(u0)
    near = np.float32(prod)
    around = [near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(1))]
    B = len(around)
    t = torch.full((B, 2, 8), 0.01)
    q = torch.full((B, 1, 8), 0.01)
    for b, p in enumerate(around):
        t[b, 0, 3] = float(p)
        q[b, 0, 3] = float(q0)
    x = torch.full((B, 1), 3, dtype=torch.int32)
    check(x, q, t, torch.full((B, 1), float(u0)), torch.full((B,), 0.4))
    assert len({R.verify([3], q[b].double().numpy(), t[b].double().numpy(), [float(u0)], .4, 1)[0]
                for b in range(B)}) == 2


@pytest.mark.parametrize("greedy", [False, True])
def test_rows_without_weight_and_values_that_are_no_probabilities(greedy):
    V = 200
    x, q, t, ua, us = inputs(8, 2, V, torch.float32, greedy, 12)
    ua.fill_(1 - 2.0 ** -24)
    t[0] = 0                                  # nothing anywhere: token -1
    if not greedy:
        q[1] = 1.0                            # difference empty: drawn from the target
        q[2] = math.nan
    t[3, :, ::2] = math.nan
    t[4, :, 1::3] = -0.5
    t[5, :, 7] = math.inf
    t[6] = 1.0                                # unnormalised: sums far above 1
    t[7] = 2.0 ** -60                         # below the resolution
    check(x, q, t, ua, us)
    only = torch.zeros(1, 3, V)
    only[0, :, 4] = 1.0
    x1 = torch.full((1, 2), 4, dtype=torch.int32)
    x1[0, 0] = 5
    check(x1, None, only, ua[:1], us[:1])      # the draft is rejected, 4 follows
    x1[0, 0] = 4
    check(x1, None, only, ua[:1], us[:1])      # all accepted


def test_tokens_outside_the_vocabulary_are_rejected():
    for greedy in (False, True):
        x, q, t, ua, us = inputs(4, 3, 64, torch.float32, greedy, 13, sharp=0.1)
        x[0, 0], x[1, 1], x[2, 2], x[3, 0] = -1, 64, 2 ** 31 - 1, -2 ** 31
        check(x, q, t, ua * 0.1, us)


def test_largest_rows_sum_without_overflow():
    V = (1 << 19) - 1
    t = torch.ones(1, 1, V)
    x, ua = torch.zeros(1, 0, dtype=torch.int32), torch.zeros(1, 0)
    for u in (0.0, 0.37, 1 - 2.0 ** -24):
        us = torch.tensor([u])
        _, tok = verify_draft(x.cuda(), torch.zeros(1, 0, V).cuda(), t.cuda(), ua.cuda(), us.cuda())
        total = V << 44
        want = min(math.floor(float(us[0]) * float(total)), total - 1) >> 44
        assert int(tok[0, 0]) == want


def test_output_tokens_follow_the_target():
    """100000 sequences of one draft over 6 tokens: the first output token's
    frequencies against the target's probabilities, within six standard
    deviations of a binomial."""
    B = 100_000
    g = torch.Generator(device="cuda").manual_seed(2)
    p = torch.tensor([0.4, 0.05, 0.2, 0.1, 0.05, 0.2], device="cuda")
    q = torch.tensor([0.1, 0.3, 0.2, 0.3, 0.1, 0.0], device="cuda")
    x = torch.multinomial(q.expand(B, 6), 1, generator=g).int()
    acc, tok = verify_draft(x, q.expand(B, 1, 6), p.expand(B, 2, 6),
                            torch.rand(B, 1, device="cuda", generator=g),
                            torch.rand(B, device="cuda", generator=g))
    n = torch.bincount(tok[:, 0].long(), minlength=6).double().cpu().numpy()
    want = p.double().cpu().numpy()
    assert np.all(np.abs(n - B * want) <= 6 * np.sqrt(B * want * (1 - want)))
    want_acc = float(torch.minimum(p, q).sum())
    assert abs(float(acc.double().sum()) - B * want_acc) <= 6 * math.sqrt(B * want_acc)


def test_other_stream_and_captured_call():
    x, q, t, ua, us = (z.cuda() for z in inputs(4, 5, 3001, torch.float32, False, 14))
    want = verify_draft(x, q, t, ua, us)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = verify_draft(x, q, t, ua, us)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = verify_draft(x, q, t, ua, us)
    us.copy_(torch.rand_like(us))
    ua.copy_(torch.rand_like(ua))
    g.replay()
    torch.cuda.synchronize()
    want = verify_draft(x, q, t, ua, us)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_empty_batch_and_refusals():
    x, q, t, ua, us = (z.cuda() for z in inputs(2, 3, 50, torch.float32, False, 15))
    acc, tok = verify_draft(x[:0], q[:0], t[:0], ua[:0], us[:0])
    assert acc.shape == (0,) and tok.shape == (0, 4)
    for bad in (dict(target_probs=t[:, :3]), dict(draft_probs=q[:, :2]), dict(u_accept=ua[:, :2]),
                dict(u_sample=us[:1]), dict(draft_tokens=x.long()), dict(draft_probs=q.bfloat16()),
                dict(u_sample=us.double()), dict(n_draft=torch.zeros(3, dtype=torch.int32).cuda()),
                dict(target_probs=t.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(u_sample=us.cpu()), dict(draft_probs=q.cpu())):
        args = dict(draft_tokens=x, draft_probs=q, target_probs=t, u_accept=ua, u_sample=us)
        args.update(bad)
        with pytest.raises(ValueError):
            verify_draft(**args)
