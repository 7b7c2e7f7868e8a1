"""Attention over the 8-bit cache at the sizes of serving: segments of many
tiles, CTAs that go from one pair to the next, references that move in the
middle of a segment, and the same call over and over."""
import math
import random

import pytest
import torch

from block_diffusion_draft_gb300 import Q8Cache

from test_gpu_q8 import layer

pytestmark = pytest.mark.gpu
TK = 128        # keys of a tile
PAIR_COST = 4   # places of a pair without a tile


def plan_share(counts, n_kv, n_q_tiles, sms):
    """Places of the line of key tiles that a CTA takes (no window)."""
    tiles = [max(1, -(-n // TK)) for n in counts]
    total = sum(t + PAIR_COST for t in tiles) * n_kv * n_q_tiles
    return max(-(-total // sms), (max(tiles) + 29) // 30)


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


def reference(q, k, v, window=0, causal=False):
    """One sequence in 64 bits on the GPU: q [T, nq, d], k and v [n, nkv, d] ->
    out [T, nq, d], lse [T, nq], A = sum p |v| / sum p, and Q, the row's
    largest sum_c |q_c k_c| / sqrt(d)."""
    T, nq, d = q.shape
    n, nkv = k.shape[:2]
    g = nq // nkv
    qh = q.double().view(T, nkv, g, d).permute(1, 0, 2, 3).reshape(nkv, T * g, d)
    kh, vh = k.double().transpose(0, 1), v.double().transpose(0, 1)  # [nkv, n, d]
    at = (n - T + torch.arange(T, device=q.device)).view(T, 1)
    key = torch.arange(n, device=q.device).view(1, n)
    seen = torch.ones(T, n, dtype=torch.bool, device=q.device)
    if window:
        seen &= (at - key).abs() < window
    if causal:
        seen &= key <= at
    seen = seen.repeat_interleave(g, 0)
    s = (qh @ kh.transpose(1, 2) / math.sqrt(d)).masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    big = (qh.abs() @ kh.abs().transpose(1, 2) / math.sqrt(d)).masked_fill(~seen, 0.0).amax(-1)
    back = lambda x: x.view(nkv, T, g, -1).permute(1, 0, 2, 3).reshape(T, nq, -1)  # noqa: E731
    return (back(p @ vh), back(top + torch.log(total)).squeeze(-1), back(p @ vh.abs()),
            back(big.unsqueeze(-1)).squeeze(-1))


def check(a, q, out, lse, k, v, counts, half, window=0, causal=False):
    """Every sequence against 64 bits.  A score's fp32 sum of 128 products is
    off by at most 128 * 2^-24 of the sum of their magnitudes (Q), which moves a
    probability by that much relatively, twice with the row's sum; the row's
    sum of n terms by n * 2^-24; exp2's 2 ulp and the rescalings are covered by
    2^-18 in all.  P is rounded once, 2^-11 relative in fp16 (and below 2^-14,
    where the largest is 2^7 or more, by 2^-25: n * 2^-32 of the largest |v|) or
    2^-8 in bf16, the output once more to bf16."""
    unit = 2.0 ** -11 if half else 2.0 ** -8
    begin = 0
    for b, n in enumerate(counts):
        kb, vb = k[begin:begin + n], v[begin:begin + n]
        begin += n
        if n == 0:
            assert not out[b].any() and bool((lse[b] == -math.inf).all())
            continue
        ref, rl, A, Q = reference(q[b], kb, vb, window, causal)
        noise = 2 * (2.0 ** -17 * Q + n * 2.0 ** -24 + 2.0 ** -18)
        tol = 1.01 * (unit * A + 2.0 ** -8 * ref.abs()) + noise[..., None] * A
        tol += n * 2.0 ** -32 * vb.double().abs().max()
        off = (out[b].double() - ref).abs() - tol
        assert bool((off <= 0).all()), (b, n, float(off.max()), int((off > 0).sum()))
        none = rl == -math.inf
        assert torch.equal(lse[b] == -math.inf, none)
        far = torch.where(none, 0.0, (lse[b].double() - rl).abs() - noise - 2.0 ** -21 * rl.abs())
        assert bool((far <= 0).all()), (b, n, float(far.max()))
    assert a.device_error() == 0


def uneven_rows(n, heads, gen):
    """K rows with uneven channels, V rows of one size."""
    gain = torch.exp(0.5 * torch.randn(heads, 128, device="cuda", generator=gen))
    k = torch.randn(n, heads, 128, device="cuda", generator=gen) * gain
    return k.bfloat16(), torch.randn(n, heads, 128, device="cuda", generator=gen).bfloat16()


def one_case(a, counts, q_len, fmt, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k, v = uneven_rows(sum(counts), a.n_kv_heads, gen)
    cache = Q8Cache(a, len(counts), max(counts), fmt)
    cache.append(k, v, counts)
    q = torch.randn(len(counts), q_len, a.n_heads, 128, device="cuda", generator=gen).bfloat16()
    return cache, q


@pytest.mark.parametrize("fmt,n_heads,n_kv,q_len,counts", [
    ("int8", 32, 8, 16, [random.Random(6).randint(512, 8192) for _ in range(32)]),
    ("e4m3", 32, 8, 16, [32800] * 4),
    ("int8", 8, 2, 40, [700, 0, 5000, 129, 3000] * 6)])
def test_every_pass_gives_the_same_bits(fmt, n_heads, n_kv, q_len, counts):
    """Two caches in turn, ten passes at a time with nothing between them: each
    pass is the first one's, and that one is right."""
    a = layer(n_heads, n_kv)
    for seed in range(3):
        two = [one_case(a, counts, q_len, fmt, 10 * seed + i) for i in range(2)]
        want = []
        for cache, q in two:
            out, lse = a.q8_core(cache, q)
            k, v = cache.read()
            check(a, q, out, lse, k, v, counts, True)
            want.append((out, lse))
        for _ in range(20):
            got = [(i & 1, a.q8_core(*two[i & 1])) for i in range(10)]
            same = torch.stack([(x == y).all() for i, r in got for x, y in zip(r, want[i])])
            assert bool(same.all()), same.tolist()
    assert a.device_error() == 0


def make_wide(v):
    """Groups of V 2^40 apart: the head's codes are then decoded to bf16."""
    v[len(v) // 2, :, 32:64] *= 2.0 ** -40
    return v


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("wide", [False, True])
def test_references_rise_within_long_segments(fmt, wide):
    """Every CTA has one whole pair of 13 tiles, whose scores rise by more
    than 2^8 at the 2nd, the 5th and the last tile for some rows, fall or stay
    for others."""
    sms, tiles = sm_count(), 13
    a = layer(4, 1)
    n = tiles * TK - 37
    counts = [n] * sms
    assert plan_share(counts, 1, 1, sms) == tiles + PAIR_COST
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = uneven_rows(sum(counts), 1, gen)
    tile = torch.arange(n, device="cuda") // TK
    level = 9.4 * ((tile >= 1).float() + (tile >= 4).float() + (tile >= tiles - 1).float())
    k[:, 0, 0] = level.repeat(sms).bfloat16()
    v = v.view(sms, n, 1, 128)
    if wide:
        for b in range(sms):
            make_wide(v[b])
    v = v.view(-1, 1, 128)
    q = 0.3 * torch.randn(sms, 16, 4, 128, device="cuda", generator=gen)
    lead = torch.tensor([8.0, -8.0, 4.0, 0.0, 12.0, -3.0, 9.0], device="cuda")
    q[..., 0] = lead[torch.arange(sms * 64, device="cuda") % 7].view(sms, 16, 4)
    q = q.bfloat16()
    cache = Q8Cache(a, sms, n, fmt)
    cache.append(k, v, counts)
    out, lse = a.q8_core(cache, q)
    ck, cv = cache.read()
    # the rises, in log2 units, of a row whose first channel is 8
    s = (ck[:n, 0].double() @ q[0, 0, 0].double()) / math.sqrt(128) / math.log(2)
    top = torch.stack([s[tile == t].max() for t in range(tiles)]).tolist()
    assert q[0, 0, 0, 0] == 8 and all(top[t] - max(top[:t]) > 8 for t in (1, 4, tiles - 1))
    check(a, q, out, lse, ck, cv, counts, not wide)


@pytest.mark.parametrize("fmt,wide,window,causal", [
    ("int8", False, 0, False), ("e4m3", False, 0, False), ("int8", True, 0, False),
    ("e4m3", True, 0, True), ("int8", False, 2100, True), ("e4m3", False, 1900, False),
    ("int8", True, 2000, False)])
def test_levels_that_wander_and_ctas_that_go_from_pair_to_pair(fmt, wide, window, causal):
    """Pairs of 13 to 20 tiles, about two to a CTA, the level of the scores
    another one in every tile."""
    sms = sm_count()
    r = random.Random(3)
    counts = [r.randint(1600, 2500) for _ in range(sms // 4 + 1)]
    a = layer(32, 8, window, causal)
    assert plan_share(counts, 8, 1, sms) >= 2 * (13 + PAIR_COST)
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = uneven_rows(sum(counts), 8, gen)
    begin = 0
    for n in counts:
        step = torch.tensor([r.choice([-6.0, 0.0, 0.0, 9.0]) for _ in range(-(-n // TK))])
        level = step.cumsum(0).repeat_interleave(TK)[:n].cuda()
        k[begin:begin + n, :, 64] = level.bfloat16()[:, None]
        if wide:
            make_wide(v[begin:begin + n])
        begin += n
    q = 0.3 * torch.randn(len(counts), 16, 32, 128, device="cuda", generator=gen)
    q[..., 64] = torch.linspace(-10, 10, 32, device="cuda")
    q = q.bfloat16()
    cache = Q8Cache(a, len(counts), max(counts), fmt)
    cache.append(k, v, counts)
    out, lse = a.q8_core(cache, q)
    ck, cv = cache.read()
    check(a, q, out, lse, ck, cv, counts, not wide, window, causal)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("why", ["wide", "hidden nan"])
def test_large_scores_of_a_head_decoded_to_bf16(fmt, why):
    """Queries 2^-60 to 2^100 apart, and keys 2^60 apart, on a head whose
    codes are decoded to bf16: rows whose scores are far apart read their one
    key, none loses its result."""
    a = layer(4, 1, 0, True)
    n, T = 900, 16
    gen = torch.Generator(device="cuda").manual_seed(4)
    k, v = uneven_rows(n, 1, gen)
    q = 0.3 * torch.randn(1, T, 4, 128, device="cuda", generator=gen)
    for i, e in enumerate((-60, -11, 0, 5, 20, 26, 30, 31, 33, 40, 64, 100)):
        q[0, i, i % 4] *= 2.0 ** e
    q = q.bfloat16()
    if why == "wide":
        make_wide(v)
        k[n // 3] *= 2.0 ** 20
    else:
        v[n - 1, 0, 5] = math.nan  # seen by the last block row only
    cache = Q8Cache(a, 1, n, fmt)
    cache.append(k, v, [n])
    out, lse = a.q8_core(cache, q)
    ck, cv = cache.read()
    rows = T - 1
    if why != "wide":
        assert bool(out[0, rows, :, :32].isnan().all())
    ref, rl, A, Q = reference(q[0], torch.nan_to_num(ck), torch.nan_to_num(cv), 0, True)
    out, lse = out[0, :rows], lse[0, :rows]
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    noise = 2 * (2.0 ** -17 * Q + n * 2.0 ** -24 + 2.0 ** -18)[:rows]
    far = (lse.double() - rl[:rows]).abs() - noise - 2.0 ** -21 * rl[:rows].abs()
    assert bool((far <= 0).all()), float(far.max())
    sure = 0
    for t in range(rows):
        seen = n - T + t + 1
        s = ck[:seen, 0].double() @ q[0, t].double().T / math.sqrt(128)  # [keys, heads]
        first, at = s.max(0)
        second = s.scatter(0, at[None], -math.inf).max(0).values
        for h in range(4):
            tol = 1.01 * 2.0 ** -8 * (A[t, h] + ref[t, h].abs()) + noise[t, h] * A[t, h]
            assert bool(((out[t, h].double() - ref[t, h]).abs() <= tol).all()), (t, h)
            if first[h] - second[h] > 200 + 2 * noise[t, h]:  # exp(-200) of the others
                assert torch.equal(out[t, h], cv[at[h], 0]), (t, h)
                sure += 1
    assert sure >= 6
