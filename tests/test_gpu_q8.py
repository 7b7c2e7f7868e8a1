"""The 8-bit draft cache on the GPU: rows written and read back, attention
over it, the layer step, against 64-bit references."""
import ctypes
import math

import numpy as np
import pytest
import torch

from block_diffusion_draft_gb300 import DFlashError, Q8Cache, verify_draft
from block_diffusion_draft_gb300 import workloads as W
from block_diffusion_draft_gb300.dflash_attn import DFlashAttention, check, lib
from oracle import dflash_oracle as O

import helpers as T
import q8_reference as R

pytestmark = pytest.mark.gpu
FMTS = ["int8", "e4m3"]


def layer(n_heads, n_kv, window=0, causal=False):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    d = 128
    return DFlashAttention(
        dict(wq=z(n_heads * d, d), wk=z(n_kv * d, d), wv=z(n_kv * d, d), wo=z(d, n_heads * d),
             q_norm=z(d), k_norm=z(d)),
        hidden=d, n_heads=n_heads, n_kv_heads=n_kv, head_dim=d, max_position=64,
        sliding_window=window, causal=causal)


def rows(n, heads, seed, spread=0.5):
    g = np.random.default_rng(seed)
    gain = np.exp(spread * g.standard_normal((heads, 128)))
    x = g.standard_normal((n, heads, 128)) * gain
    return torch.from_numpy(x).to(torch.bfloat16)


def same(got, want):
    return np.array_equal(T.f64(got), want, equal_nan=True)


# ------------------------------------------------------------ write and read
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n_kv,counts", [(1, [1]), (2, [3, 0, 17]), (8, [33]), (3, [129, 5]),
                                         (8, [0, 0, 1, 2])])
def test_rows_read_back_as_defined(fmt, n_kv, counts):
    cache = Q8Cache(layer(n_kv, n_kv), len(counts), 140, fmt)
    k, v = rows(sum(counts), n_kv, 1), rows(sum(counts), n_kv, 2, 2.0)
    cache.append(k.cuda(), v.cuda(), counts)
    assert cache.lengths() == counts
    gk, gv = cache.read()
    assert same(gk, R.stored_values(T.f64(k), fmt))
    assert same(gv, R.stored_values(T.f64(v), fmt))


@pytest.mark.parametrize("fmt", FMTS)
def test_edge_values(fmt):
    """Zeros, the smallest and largest numbers, values at and next to a
    scale's border, ties, infinities and NaN, one group each."""
    inf, nan = math.inf, math.nan
    top = R.QMAX[fmt]
    groups = [[0.0], [-0.0], [2.0 ** -133], [2.0 ** -126, -2.0 ** -120], [3e38], [-2.0 ** 127, 1.0],
              [2.0 ** 126, -2.0 ** 110], [inf], [-inf, 1.0], [nan], [1.0, nan, inf], [1e-30, 5e-31],
              [2.0 ** -109, 2.0 ** -118], [2.0 ** 120 * 1.5, 2.0 ** 115]]
    for e in (-60, 0, 40, 90):
        b = math.ldexp(top, e)
        groups += [[b], [-b, b / 3], [b * (1 + 2.0 ** -7)], [b * (1 - 2.0 ** -7)],
                   [b] + [math.ldexp(i + 0.5, e) for i in range(8, 39)],  # ties
                   [b] + [-math.ldexp(1.0625 + i / 8, e) for i in range(31)],
                   [b] + [math.ldexp(i / 4, e - 9) for i in range(31)]]
    n = (len(groups) + 3) // 4
    x = torch.zeros(n * 4, 32, dtype=torch.float64)
    for i, g in enumerate(groups):
        x[i, :len(g)] = torch.tensor(g, dtype=torch.float64)
    x = x.bfloat16().view(n, 1, 128)
    cache = Q8Cache(layer(1, 1), 1, n, fmt)
    cache.append(x.cuda(), x.flip(0).cuda(), [n])
    gk, gv = cache.read()
    assert same(gk, R.stored_values(T.f64(x), fmt))
    assert same(gv, R.stored_values(T.f64(x.flip(0)), fmt))


@pytest.mark.parametrize("fmt", FMTS)
def test_slices_of_a_projection_crops_and_neighbours(fmt):
    """Rows that are slices of a wider tensor; a crop and a new append replace
    rows; other sequences and rows behind stay as they were."""
    n_kv, counts = 4, [5, 9, 2]
    a = layer(8, n_kv)
    cache = Q8Cache(a, 3, 40, fmt)
    fused = rows(16, 16, 3)
    k, v = fused[:, 8:12], fused[:, 12:]
    f = fused.cuda()
    cache.append(f[:, 8:12], f[:, 12:], counts)
    gk, gv = cache.read()
    assert same(gk, R.stored_values(T.f64(k), fmt)) and same(gv, R.stored_values(T.f64(v), fmt))
    cache.crop([5, 3, 2])
    new = rows(3, n_kv, 4).cuda()
    cache.append(new, new, [0, 3, 0])
    assert cache.lengths() == [5, 6, 2]
    k2, v2 = cache.read()
    keep = list(range(8)) + [14, 15]  # rows 0-4 of 0, 0-2 of 1, 0-1 of 2
    at = list(range(8)) + [11, 12]
    assert torch.equal(k2[at], gk[keep]) and torch.equal(v2[at], gv[keep])
    assert same(k2[8:11], R.stored_values(T.f64(new), fmt))
    part, _ = cache.read([1, 6, 0], [2, 0, 1])
    assert torch.equal(part, torch.cat([k2[1:3], k2[11:12]]))


class _Memory:
    """Device memory of the library as a tensor (no copy)."""

    def __init__(self, ptr, shape):
        self.__cuda_array_interface__ = dict(shape=shape, typestr="|u1", data=(ptr.value, False),
                                             version=3)


def storage(cache):
    """The cache's code and scale bytes [batch, n_kv, rows, 128 | 4]."""
    ptr = [ctypes.c_void_p() for _ in range(4)]
    geo = [ctypes.c_int32() for _ in range(4)]
    check(lib().dflash_q8_cache_data(cache.handle, *map(ctypes.byref, ptr + geo)))
    b, h, n, d = (g.value for g in geo)
    torch.cuda.synchronize()
    return [torch.as_tensor(_Memory(p, (b, h, n, w)), device="cuda")
            for p, w in zip(ptr, (d, d, d // 32, d // 32))]


@pytest.mark.parametrize("fmt", FMTS)
def test_storage_outside_the_appended_rows_is_untouched(fmt):
    cache = Q8Cache(layer(2, 2), 2, 200, fmt)
    x = rows(100, 2, 8).cuda()
    cache.append(x, x, [60, 40])
    before = [t.clone() for t in storage(cache)]
    assert before[0].shape == (2, 2, 256, 128)
    cache.crop([60, 30])
    y = rows(9, 2, 9).cuda()
    cache.append(y, y, [5, 4])
    for b, a in zip(before, storage(cache)):
        new = torch.zeros(2, 256, dtype=torch.bool, device="cuda")
        new[0, 60:65] = True
        new[1, 30:34] = True
        keep = ~new[:, None, :, None].expand(b.shape)
        assert torch.equal(a[keep], b[keep])
        assert not torch.equal(a, b)


def test_refusals():
    a = layer(4, 2)
    with pytest.raises(ValueError):
        Q8Cache(a, 1, 16, "fp6")
    for bad in (dict(batch=0, capacity=4), dict(batch=1, capacity=0), dict(batch=513, capacity=4)):
        with pytest.raises(DFlashError):
            Q8Cache(a, **bad)
    sp = W.SPECS["tiny_fp32"]
    with pytest.raises(DFlashError, match="UNSUPPORTED"):
        Q8Cache(T.gpu_layer(sp, W.weights(sp, 0)), 1, 16)
    cache = Q8Cache(a, 2, 20)
    x = rows(12, 2, 1).cuda()
    cache.append(x, x, [8, 4])
    before = cache.read()[0]
    with pytest.raises(DFlashError, match="CAPACITY"):
        cache.append(rows(14, 2, 1).cuda(), rows(14, 2, 1).cuda(), [13, 1])
    for n in ([12], [6, 6, 0], [5, 5]):
        with pytest.raises(ValueError):
            cache.append(x, x, n)
    with pytest.raises(DFlashError, match="ARG"):
        cache.append(x, x, [13, -1])
    with pytest.raises(ValueError):
        cache.append(x.float(), x, [6, 6])
    with pytest.raises(ValueError):
        cache.append(x.cpu(), x, [6, 6])
    with pytest.raises(ValueError, match="dense"):
        cache.append(x.transpose(1, 2).contiguous().transpose(1, 2), x, [6, 6])
    odd = torch.zeros(12 * 256 + 8, device="cuda", dtype=torch.bfloat16)[1:1 + 12 * 256]
    with pytest.raises(DFlashError, match="16-byte"):
        cache.append(odd.view(12, 2, 128), x, [6, 6])
    for first, n in (([0, 0], [9, 0]), ([-1, 0], [1, 0]), ([0, 4], [0, 1])):
        with pytest.raises(DFlashError, match="RANGE"):
            cache.read(first, n)
    with pytest.raises(DFlashError, match="RANGE"):
        cache.crop([9, 0])
    assert cache.lengths() == [8, 4] and torch.equal(cache.read()[0], before)
    q = torch.zeros(2, 3, 4, 128, device="cuda", dtype=torch.bfloat16)
    for bad in (q[:1], q[:, :, :2], q[..., :64], q.float(), q.cpu(), q.transpose(0, 1)):
        with pytest.raises(ValueError):
            a.q8_core(cache, bad)
    with pytest.raises(DFlashError, match="ARG"):
        a.q8_core(cache, q[:, :0])
    with pytest.raises(DFlashError, match="SHAPE"):
        layer(4, 4).q8_core(cache, q)
    with pytest.raises(DFlashError, match="UNSUPPORTED"):
        wide = layer(129, 1)
        c1 = Q8Cache(wide, 1, 8)
        wide.q8_core(c1, torch.zeros(1, 1, 129, 128, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        a.forward_q8(cache, torch.zeros(2, 3, 64, device="cuda", dtype=torch.bfloat16), None,
                     [0, 0], torch.zeros(6, device="cuda", dtype=torch.int32))
    with pytest.raises(DFlashError, match="ARG"):
        cache.reserve(21)


# ---------------------------------------------------------------- attention
def bounds(q, k, v, window, causal):
    """One sequence's reference (out, lse) and how far an evaluation may be
    off, elementwise.  P is rounded once to bf16 (2^-8 relative; fp16 where the
    scales allow it, which is finer), the output once more; a score's fp32 sum
    of 128 products is off by at most 128 * 2^-24 of the sum of their
    magnitudes (Q), which moves a probability by that much relatively, twice
    with the row's sum; the row's sum of n terms by n * 2^-24; exp2's 2 ulp and
    the rescalings are covered by 2^-18 in all."""
    ref, rl, A, Q = R.attend(q, k, v, window, causal)
    noise = 2 * (2.0 ** -17 * Q + k.shape[0] * 2.0 ** -24 + 2.0 ** -18)
    return ref, rl, 2.0 ** -8 * (A + np.abs(ref)) * 1.01 + noise[..., None] * A, noise


def check_attention(a, cache, q, out, lse, k, v, counts, window, causal):
    at = 0
    for b, n in enumerate(counts):
        kb, vb = T.f64(k[at:at + n]), T.f64(v[at:at + n])
        at += n
        ref, rl, tol, noise = bounds(T.f64(q[b]), kb, vb, window, causal)
        got, gl = T.f64(out[b]), T.f64(lse[b])
        bad = np.abs(got - ref) > tol
        assert not bad.any(), (b, np.argwhere(bad)[:5], np.abs(got - ref).max())
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(gl), empty)
        assert np.all(got[empty] == 0)
        diff = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, rl))
        assert np.all(diff <= noise + 2.0 ** -21 * np.abs(np.where(empty, 0, rl))), diff.max()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n_heads,n_kv,q_len,counts", [
    (1, 1, 1, [1]), (4, 1, 1, [127, 128, 129]), (8, 8, 1, [5, 0, 300]),
    (8, 2, 16, [16, 17, 255, 400]), (7, 1, 5, [64, 1000]), (16, 2, 8, [3, 700]),
    (14, 2, 13, [0, 5, 333]), (8, 1, 16, [128, 384]), (16, 1, 17, [200]), (4, 4, 40, [41, 130]),
    (2, 1, 150, [160]), (128, 1, 1, [70]), (100, 1, 3, [90])])
def test_attention_over_the_cache(fmt, n_heads, n_kv, q_len, counts):
    a = layer(n_heads, n_kv)
    cache = Q8Cache(a, len(counts), max(max(counts), 1), fmt)
    k, v = rows(sum(counts), n_kv, 1).cuda(), rows(sum(counts), n_kv, 2).cuda()
    cache.append(k, v, counts)
    q = rows(len(counts) * q_len, n_heads, 3, 0.2).view(len(counts), q_len, n_heads, 128).cuda()
    out, lse = a.q8_core(cache, q)
    ck, cv = cache.read()
    check_attention(a, cache, q, out, lse, ck, cv, counts, 0, False)
    out2, lse2 = a.q8_core(cache, q)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert a.device_error() == 0


@pytest.mark.parametrize("window,causal", [(0, True), (1, False), (1, True), (7, False),
                                           (130, True), (200, False), (5000, True),
                                           (2 ** 31 - 1, False)])
@pytest.mark.parametrize("q_len,counts", [(1, [300, 1]), (16, [16, 8, 400, 0, 129]),
                                          (37, [20, 140, 500])])
def test_windows_and_causal_layers(window, causal, q_len, counts):
    a = layer(8, 2, window, causal)
    cache = Q8Cache(a, len(counts), 512, "int8")
    k, v = rows(sum(counts), 2, 4).cuda(), rows(sum(counts), 2, 5).cuda()
    cache.append(k, v, counts)
    q = rows(len(counts) * q_len, 8, 6, 0.2).view(len(counts), q_len, 8, 128).cuda()
    out, lse = a.q8_core(cache, q)
    ck, cv = cache.read()
    check_attention(a, cache, q, out, lse, ck, cv, counts, window, causal)


@pytest.mark.parametrize("fmt", FMTS)
def test_split_keys_long_contexts_and_many_sequences(fmt):
    # one long sequence (units split and merged), then a ragged batch
    for n_heads, n_kv, q_len, counts in ((8, 2, 4, [5000]), (2, 1, 16, [9000, 40]),
                                         (4, 2, 2, list(range(1, 400, 17)))):
        a = layer(n_heads, n_kv)
        cache = Q8Cache(a, len(counts), max(counts), fmt)
        k, v = rows(sum(counts), n_kv, 7).cuda(), rows(sum(counts), n_kv, 8).cuda()
        cache.append(k, v, counts)
        q = rows(len(counts) * q_len, n_heads, 9, 0.2).view(-1, q_len, n_heads, 128).cuda()
        out, lse = a.q8_core(cache, q)
        ck, cv = cache.read()
        check_attention(a, cache, q, out, lse, ck, cv, counts, 0, False)


def test_rising_scores_rescale():
    """Scores that grow along the keys by far more than the lazy rescale's
    threshold, and fall again."""
    a = layer(2, 1)
    n = 600
    cache = Q8Cache(a, 1, n, "e4m3")
    k = torch.zeros(n, 1, 128, dtype=torch.bfloat16)
    k[:, 0, 0] = torch.linspace(-300, 300, n).bfloat16()
    k[500:, 0, 0] = -100
    v = rows(n, 1, 1)
    cache.append(k.cuda(), v.cuda(), [n])
    q = torch.zeros(1, 3, 2, 128, dtype=torch.bfloat16)
    q[0, :, 0, 0] = torch.tensor([1.0, -2.0, 0.5])
    q[0, :, 1, 0] = torch.tensor([5.0, 0.0, -7.0])
    out, lse = a.q8_core(cache, q.cuda())
    ck, cv = cache.read()
    check_attention(a, cache, q, out, lse, ck, cv, [n], 0, False)


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_reaches_only_what_sees_it(fmt):
    """A NaN in V reaches the rows that see its key, in its group's channels;
    one in K the rows that see it, whole; rows whose mask hides them (and
    anything behind the sequence's end) not at all."""
    a = layer(2, 1, 0, True)
    T_, n = 8, 150
    k, v = rows(n, 1, 1), rows(n, 1, 2)
    q = rows(T_, 2, 3, 0.2).view(1, T_, 2, 128).cuda()
    # the rows that see neither NaN are held to the same bounds as without it
    want, wl, tol, noise = bounds(T.f64(q[0]), R.stored_values(T.f64(k), fmt),
                                  R.stored_values(T.f64(v), fmt), 0, True)
    v2, k2 = v.clone(), k.clone()
    v2[n - 3, 0, 40] = math.nan   # key 147: seen by rows 5, 6, 7; channels 32..63
    k2[n - 2, 0, 7] = math.inf    # key 148: seen by rows 6, 7
    cache = Q8Cache(a, 1, 256, fmt)
    cache.append(k2.cuda(), v2.cuda(), [n])
    # and rows that were NaN before a crop, behind the end
    bad = torch.full((60, 1, 128), math.nan, device="cuda", dtype=torch.bfloat16)
    cache.append(bad, bad, [60])
    cache.crop([n])
    out, lse = a.q8_core(cache, q)
    got, gl = T.f64(out[0]), T.f64(lse[0])
    diff = np.abs(got - want) - tol
    assert np.all(diff[:5] <= 0) and np.all(diff[5, :, :32] <= 0) and np.all(diff[5, :, 64:] <= 0)
    assert np.all(np.isnan(got[5, :, 32:64]))
    assert np.all(np.abs(gl[:6] - wl[:6]) <= noise[:6] + 2.0 ** -21 * np.abs(wl[:6]))
    assert np.all(np.isnan(got[6:])) and np.all(np.isnan(gl[6:]))


@pytest.mark.parametrize("fmt", FMTS)
def test_scales_far_apart(fmt):
    """Groups whose scales lie 2^19, 2^20 and up to 2^200 apart, zero rows and
    groups, and the largest numbers in keys that the mask hides: the others
    keep their precision."""
    a = layer(2, 1, 0, True)
    T_ = 4
    for n, small, hide in ((140, 2.0 ** -19, 1.0), (140, 2.0 ** -20, 1.0), (300, 2.0 ** -40, 1.0),
                           (300, 1.0, 2.0 ** 100), (130, 2.0 ** -100, 2.0 ** 90)):
        k, v = rows(n, 1, 1, 0.0), rows(n, 1, 2, 0.0)
        v[:, :, 32:64] *= small      # a group of small channels
        v[n // 2] *= small           # a key of small values
        v[5], k[9] = 0, 0            # zero rows
        v[3, :, 64:96] = 0
        k[7, :, :32] = 0
        v[n - 2:] *= hide            # seen by the last two block rows only
        cache = Q8Cache(a, 1, 512, fmt)
        cache.append(k.cuda(), v.cuda(), [n])
        q = rows(T_, 2, 3, 0.2).view(1, T_, 2, 128).cuda()
        out, lse = a.q8_core(cache, q)
        ck, cv = cache.read()
        check_attention(a, cache, q, out, lse, ck, cv, [n], 0, True)


@pytest.mark.parametrize("fmt", FMTS)
def test_query_rows_far_apart(fmt):
    """Queries of one tile whose magnitudes lie 2^-60 to 2^100 apart, zero rows
    and rows with infinities and NaN among them: no row's result depends on
    another's."""
    for n_heads, q_len in ((4, 16), (7, 5)):
        a = layer(n_heads, 1)
        n = 300
        cache = Q8Cache(a, 1, n, fmt)
        k, v = rows(n, 1, 1).cuda(), rows(n, 1, 2).cuda()
        cache.append(k, v, [n])
        q = rows(q_len, n_heads, 3, 0.2)
        for i, e in enumerate((-60, -30, -11, -10, -9, 0, 5, 30, 100)):
            q[i % q_len, i % n_heads] *= 2.0 ** e
        q[1, 2] = 0
        q[2, 0, 5], q[3, 1, 127], q[4, 2, 0] = math.nan, math.inf, -math.inf
        out, lse = a.q8_core(cache, q[None].cuda())
        ck, cv = cache.read()
        for t, h in ((2, 0), (3, 1), (4, 2)):
            assert bool(out[0, t, h].isnan().all()) and bool(lse[0, t, h].isnan())
            q[t, h], out[0, t, h], lse[0, t, h] = 0, 0, 0
        whole = torch.ones(q_len, n_heads, dtype=torch.bool)
        for t, h in ((2, 0), (3, 1), (4, 2)):
            whole[t, h] = False
        assert bool(out[0][whole.cuda()].isfinite().all())
        ref, rl, tol, noise = bounds(T.f64(q), T.f64(ck), T.f64(cv), 0, False)
        assert np.all((np.abs(T.f64(out[0]) - ref) <= tol)[whole.numpy()])
        diff = np.abs(T.f64(lse[0]) - rl)[whole.numpy()]
        assert np.all(diff <= (noise + 2.0 ** -21 * np.abs(rl))[whole.numpy()])


@pytest.mark.parametrize("n_heads,n_kv,q_len,counts", [
    (2, 1, 1, [0] * 300), (8, 8, 3, [0, 0, 0, 1] * 40), (2, 2, 2, [i % 3 for i in range(512)]),
    (4, 2, 1, [0, 0, 0, 130, 0, 0, 0, 0, 257, 1] * 12), (4, 1, 40, [0, 5, 0, 0, 129] * 9)])
def test_many_short_and_empty_sequences(n_heads, n_kv, q_len, counts):
    """Many segments to a block, runs of them without a key."""
    a = layer(n_heads, n_kv)
    cache = Q8Cache(a, len(counts), 300, "int8")
    k, v = rows(sum(counts), n_kv, 1).cuda(), rows(sum(counts), n_kv, 2).cuda()
    cache.append(k, v, counts)
    q = rows(len(counts) * q_len, n_heads, 3, 0.2).view(-1, q_len, n_heads, 128).cuda()
    out, lse = a.q8_core(cache, q)
    ck, cv = cache.read()
    check_attention(a, cache, q, out, lse, ck, cv, counts, 0, False)
    assert a.device_error() == 0


@pytest.mark.parametrize("n_heads,n_kv,n", [(8, 8, 16000), (3, 3, 45000)])
def test_a_large_append_is_many_small_ones(n_heads, n_kv, n):
    """Codes, scales and what the attention makes of them."""
    a = layer(n_heads, n_kv)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(n, n_kv, 128, device="cuda", generator=g).bfloat16()
    v = torch.randn(n, n_kv, 128, device="cuda", generator=g).bfloat16()
    k[n - 3, 1] *= 2.0 ** 6  # the largest scale, met once
    v[777, 0] *= 2.0 ** -9
    k[5000:5100] = 0
    once, often = Q8Cache(a, 2, n, "int8"), Q8Cache(a, 2, n, "int8")
    m = n // 3
    once.append(k, v, [n - m, m])
    for i in range(0, m, 1000):
        j = min(i + 1000, m)
        at = torch.cat([torch.arange(i, j), n - m + torch.arange(i, j)]).cuda()
        often.append(k[at], v[at], [j - i, j - i])
    for i in range(m, n - m, 1000):
        j = min(i + 1000, n - m)
        often.append(k[i:j], v[i:j], [j - i, 0])
    assert once.lengths() == often.lengths()
    for x, y in zip(storage(once), storage(often)):
        assert torch.equal(x, y)
    q = torch.randn(2, 2, n_heads, 128, device="cuda", generator=g).bfloat16()
    for x, y in zip(a.q8_core(once, q), a.q8_core(often, q)):
        assert torch.equal(x, y) and bool(x.isfinite().all())


def test_nan_through_split_units():
    a = layer(2, 1)
    n = 6000
    k, v = rows(n, 1, 1), rows(n, 1, 2)
    v[3000, 0, 100] = math.nan
    cache = Q8Cache(a, 1, n, "int8")
    cache.append(k.cuda(), v.cuda(), [n])
    q = rows(4, 2, 3, 0.2).view(1, 4, 2, 128).cuda()
    out, lse = a.q8_core(cache, q)
    assert bool(out[..., 96:].isnan().all()) and bool(out[..., :96].isfinite().all())
    assert bool(lse.isfinite().all())


def test_offsets_past_32_bits():
    """A cache whose second sequence starts past 2^31 bytes of codes."""
    a = layer(8, 8)
    cap, n = 2_200_000, 300
    cache = Q8Cache(a, 2, cap, "int8")
    k, v = rows(n, 8, 1).cuda(), rows(n, 8, 2).cuda()
    cache.append(k, v, [0, n])
    ck, cv = cache.read()
    assert same(ck, R.stored_values(T.f64(k), "int8"))
    q = rows(2 * 4, 8, 3, 0.2).view(2, 4, 8, 128).cuda()
    out, lse = a.q8_core(cache, q)
    check_attention(a, cache, q, out, lse, ck, cv, [0, n], 0, False)


# ------------------------------------------------------- streams and graphs
def test_other_stream_and_captured_calls():
    a = layer(8, 2)
    cache = Q8Cache(a, 2, 700, "int8")
    k, v = rows(900, 2, 1).cuda(), rows(900, 2, 2).cuda()
    q = rows(32, 8, 3, 0.2).view(2, 16, 8, 128).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        cache.append(k, v, [600, 300])
        want = a.q8_core(cache, q)
    s.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        cache.crop([600, 300])
        cache.append(k[:20], v[:20], [10, 10])
        out1 = a.q8_core(cache, q)
    with torch.cuda.graph(g2):
        cache.crop([600, 300])
        out2 = a.q8_core(cache, q)
    for _ in range(2):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2[0], want[0]) and torch.equal(out2[1], want[1])
    cache.append(k[:20], v[:20], [10, 10])
    now = a.q8_core(cache, q)
    assert torch.equal(out1[0], now[0]) and torch.equal(out1[1], now[1])


def test_two_caches_on_two_streams():
    """Calls on different caches may run at the same time, also of one layer."""
    a = layer(8, 2)
    sizes = ([3000, 0, 70], [900] * 5)
    caches, queries, want = [], [], []
    for i, counts in enumerate(sizes):
        c = Q8Cache(a, len(counts), max(counts), FMTS[i])
        c.append(rows(sum(counts), 2, i).cuda(), rows(sum(counts), 2, i + 5).cuda(), counts)
        q = rows(len(counts) * 16, 8, i + 9, 0.2).view(len(counts), 16, 8, 128).cuda()
        caches.append(c)
        queries.append(q)
        want.append(a.q8_core(c, q))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(a.q8_core(caches[i], queries[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    assert a.device_error() == 0


# ---------------------------------------------------------------- the layer
def _layer_step(sp, w, cfg, lw, attn, cache, step, n_ctx, L, q_len):
    th = [W.hidden_rows(sp, 5, "hidden", step, b, n) for b, n in enumerate(n_ctx)]
    nz = [W.hidden_rows(sp, 5, "noise", step, b, q_len) for b in range(len(n_ctx))]
    pos = [W.window_positions(L[b], n, q_len) for b, n in enumerate(n_ctx)]
    out = attn.forward_q8(cache, torch.stack(nz).cuda(),
                          torch.cat(th).cuda() if sum(n_ctx) else None, n_ctx,
                          torch.cat(pos).cuda())
    # K and V as defined, before they are encoded
    new = []
    for b, n in enumerate(n_ctx):
        kc, vc = O.project_kv(cfg, lw, T.f64(th[b]), pos[b].numpy()[:n])
        kn, vn = O.project_kv(cfg, lw, T.f64(nz[b]), pos[b].numpy()[n:])
        new.append((np.concatenate([kc, kn], 1), np.concatenate([vc, vn], 1)))
    q = [O.project_q(cfg, lw, T.f64(nz[b]), pos[b].numpy()[n_ctx[b]:])
         for b in range(len(n_ctx))]
    return out, new, q


@pytest.mark.parametrize("fmt,window,causal,q_len", [("int8", 0, False, 16), ("e4m3", 0, False, 16),
                                                     ("int8", 24, True, 5),
                                                     ("e4m3", 40, False, 70)])
def test_layer_step_over_the_cache(fmt, window, causal, q_len):
    """Three steps with crops.  The cached rows stand for the oracle's K and V
    within half a code step (of the group's scale) and the bf16 rounding
    before it; the output is the oracle's attention over the rows the cache
    holds, within the library's bf16 tolerances."""
    sp = W.spec("qwen3_8b_single", hidden=512, n_heads=8, n_kv_heads=2, n_target_layers=1,
                max_position=4096, sliding_window=window, causal=causal)
    w = W.weights(sp, 3, random_gains=True, with_fc=False)
    cfg, lw = T.oracle_layer(sp, w)
    attn = T.gpu_layer(sp, w)
    cache = Q8Cache(attn, 3, 400, fmt)
    for step, n_ctx in enumerate(([150, 3, 0], [1, 16, 7], [0, 0, 0])):
        L = cache.lengths()
        out, new, q = _layer_step(sp, w, cfg, lw, attn, cache, step, n_ctx, L, q_len)
        now = [a + n + q_len for a, n in zip(L, n_ctx)]
        assert cache.lengths() == now
        k, v = cache.read()
        at, ref = 0, []
        for b, n in enumerate(now):
            kb, vb = (T.f64(x[at:at + n]).transpose(1, 0, 2) for x in (k, v))
            at += n
            for got, want in ((kb[:, L[b]:], new[b][0]), (vb[:, L[b]:], new[b][1])):
                shape = want.shape[:2] + (4, 32)
                amax = np.abs(want).reshape(shape).max(-1, keepdims=True) * np.ones(32)
                half = (amax.reshape(want.shape) / 127 if fmt == "int8" else
                        np.maximum(np.abs(want) * 2.0 ** -4, amax.reshape(want.shape) * 2.0 ** -17))
                assert np.all(np.abs(got - want) <= half + T.BF16_MAX_ABS)
            allowed = np.ones((q_len, n), dtype=bool)
            if window:
                allowed &= O.band_mask(q_len, n, window)
            if causal:
                allowed &= O.causal_mask(q_len, n)
            ref.append(O.linear(O.attention(cfg, q[b], kb, vb, allowed), lw.wo))
        T.assert_close(T.f64(out), np.stack(ref), "bf16", f"step {step}")
        cache.crop([a + n for a, n in zip(L, n_ctx)])
    assert attn.device_error() == 0


def test_draft_verify_crop_run():
    """The pieces together as a serving loop uses them: a block over the 8-bit
    cache, logits from its output, verification, crop to the accepted rows,
    the next step."""
    sp = W.spec("qwen3_8b_single", hidden=256, n_heads=4, n_kv_heads=2, n_target_layers=1,
                max_position=4096)
    w = W.weights(sp, 4, with_fc=False)
    attn = T.gpu_layer(sp, w)
    B, D, V = 3, 8, 1000
    cache = Q8Cache(attn, B, 300, "int8")
    cache.reserve(64)
    g = torch.Generator(device="cuda").manual_seed(1)
    head = torch.randn(V, sp.hidden, device="cuda", generator=g) * 0.5
    n_ctx, L = [40, 17, 2], [0, 0, 0]
    for step in range(4):
        th = torch.cat([W.hidden_rows(sp, 6, "hidden", step, b, n)
                        for b, n in enumerate(n_ctx)]).cuda()
        nz = torch.stack([W.hidden_rows(sp, 6, "noise", step, b, D) for b in range(B)]).cuda()
        pos = torch.cat([W.window_positions(L[b], n_ctx[b], D) for b in range(B)]).cuda()
        out = attn.forward_q8(cache, nz, th, n_ctx, pos)
        draft = torch.softmax(out.float() @ head.T * 8, -1)
        target = torch.softmax(torch.log(draft + 1e-6) + 0.3 * torch.randn(
            B, D, V, device="cuda", generator=g), -1)
        target = torch.cat([target, target[:, :1]], 1)
        drafts = torch.multinomial(draft.view(-1, V), 1, generator=g).view(B, D).int()
        ua = torch.rand(B, D, device="cuda", generator=g)
        us = torch.rand(B, device="cuda", generator=g)
        acc, tok = verify_draft(drafts, draft, target, ua, us)
        for b in range(B):
            want = R.verify(drafts[b].tolist(), draft[b].cpu().numpy(), target[b].cpu().numpy(),
                            ua[b].tolist(), float(us[b]), D)
            assert int(acc[b]) == want[0] and tok[b].tolist() == want[1]
        L = [a + n for a, n in zip(L, n_ctx)]
        cache.crop(L)  # the block's rows are dropped; its accepted tokens come as context
        n_ctx = [int(x) + 1 for x in acc]
    assert attn.device_error() == 0
