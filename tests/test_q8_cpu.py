"""8-bit cache and draft verification: what is refused on the host (no GPU),
and the references' own pins."""
import ctypes
import math

import numpy as np
import pytest
import torch

from block_diffusion_draft_gb300 import build
from block_diffusion_draft_gb300 import dflash_attn as D

import q8_reference as R


@pytest.fixture(scope="module")
def L():
    build.build()
    return D.lib()


def test_calls_reject_null_handles_and_arguments(L):
    out = ctypes.c_void_p(7)
    assert L.dflash_q8_cache_create(None, 1, 16, 1, ctypes.byref(out)) == -1
    assert out.value is None
    assert L.dflash_q8_cache_create(None, 1, 16, 1, None) == -1
    assert L.dflash_q8_cache_destroy(None) == 0
    assert L.dflash_q8_cache_lengths(None, None) == -1
    assert L.dflash_q8_cache_crop(None, None) == -1
    assert L.dflash_q8_cache_data(None, None, None, None, None, None, None, None, None) == -1
    assert L.dflash_q8_cache_reserve(None, 1) == -1
    assert L.dflash_q8_cache_append(None, None, None, 128, 128, None, None) == -1
    assert L.dflash_q8_cache_read(None, None, None, None, None, None) == -1
    assert L.dflash_q8_attn_core(None, None, 1, 1, None, None, None, None) == -1
    assert L.dflash_attn_forward_q8(None, None, 1, 1, None, None, None, None, None, None) == -1


def _verify(L, **kw):
    fake = ctypes.c_void_p(0x1000)
    a = dict(batch=1, n_draft=2, vocab=8, dtype=1, draft_tokens=fake, draft_probs=fake, db=16,
             dr=8, target_probs=fake, tb=24, tr=8, u_accept=fake, u_sample=fake, seq=None,
             accepted=fake, tokens=fake, stream=None)
    a.update(kw)
    return L.dflash_verify(*a.values())


@pytest.mark.parametrize("kw,rc", [
    (dict(dtype=2), -1), (dict(batch=-1), -1), (dict(n_draft=-1), -1), (dict(vocab=0), -1),
    (dict(vocab=1 << 19), -2), (dict(batch=1 << 25), -2), (dict(n_draft=1 << 21), -2),
    (dict(target_probs=None), -1), (dict(u_sample=None), -1), (dict(accepted=None), -1),
    (dict(tokens=None), -1), (dict(draft_tokens=None), -1), (dict(u_accept=None), -1),
    (dict(tr=-8), -1), (dict(tb=-1), -1), (dict(dr=-8), -1), (dict(db=-1), -1),
    (dict(target_probs=ctypes.c_void_p(0x1002)), -1),
    (dict(draft_probs=ctypes.c_void_p(0x1001), dtype=0), -1), (dict(batch=0), 0)])
def test_verify_checks_its_arguments_on_the_host(L, kw, rc):
    assert _verify(L, **kw) == rc


def test_verify_draft_checks_tensors():
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        D.verify_draft(i(1, 2), f(1, 2, 8), f(1, 3, 8), f(1, 2), f(1))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        D.verify_draft(i(1, 2), f(1, 2, 8), f(1, 3, 8).double(), f(1, 2), f(1))
    with pytest.raises(ValueError, match=r"\[B, D"):
        D.verify_draft(i(2), f(1, 2, 8), f(1, 3, 8), f(1, 2), f(1))


# ------------------------------------------------------- the references' pins
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_scale_is_the_smallest_that_holds_the_largest_magnitude(fmt):
    top = R.QMAX[fmt]
    for k in (-100, -3, 0, 5, 100):
        assert R.scale_exponent(math.ldexp(top, k), fmt) == k
        assert R.scale_exponent(math.ldexp(top, k) * (1 + 2.0 ** -20), fmt) == k + 1
        assert R.scale_exponent(math.ldexp(top, k) * 0.75, fmt) == k
    assert R.scale_exponent(0.0, fmt) == -117
    assert R.scale_exponent(2.0 ** -130, fmt) == -117


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_stored_values_stay_within_half_a_step_and_are_idempotent(fmt):
    x = np.random.default_rng(1).standard_normal((40, 128)) * np.exp(
        np.random.default_rng(2).standard_normal(128))
    y = R.stored_values(x, fmt)
    amax = np.repeat(np.abs(x).reshape(40, 4, 32).max(-1), 32).reshape(40, 128)
    bound = amax / 127 if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, amax * 2.0 ** -17)
    assert np.all(np.abs(x - y) <= bound)
    assert np.array_equal(R.stored_values(y, fmt), y)
    # and they are bf16 numbers
    assert np.array_equal(torch.from_numpy(y).bfloat16().double().numpy(), y)


def test_e4m3_codes_are_torch_float8_values():
    y = np.linspace(-448, 448, 20011)
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round_code(np.float32(y).astype(np.float64), "e4m3"), want)


def test_reference_attention_equals_softmax_by_torch():
    g = torch.Generator().manual_seed(3)
    q = torch.randn(3, 4, 128, generator=g, dtype=torch.float64)
    k = torch.randn(9, 2, 128, generator=g, dtype=torch.float64)
    v = torch.randn(9, 2, 128, generator=g, dtype=torch.float64)
    out, lse, _, _ = R.attend(q.numpy(), k.numpy(), v.numpy())
    s = torch.einsum("thd,khd->thk", q, k.repeat_interleave(2, 1)) / math.sqrt(128)
    want = torch.einsum("thk,khd->thd", s.softmax(-1), v.repeat_interleave(2, 1))
    assert np.allclose(out, want.numpy(), atol=1e-13)
    assert np.allclose(lse, s.logsumexp(-1).numpy(), atol=1e-13)
    # causal rows before the first key see nothing
    out, lse, _, _ = R.attend(q.numpy(), k[:2].numpy(), v[:2].numpy(), causal=True)
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0])) and np.all(np.isfinite(lse[1:]))


def test_verification_yields_the_targets_distribution():
    """Over a grid of n x n uniform numbers the first output token of a single
    draft follows the target's distribution, whatever the draft's.  The grid
    misplaces a border by at most 1 / (2 n), once at the acceptance and once
    at the draw."""
    p = np.array([0.5, 0.125, 0.25, 0.0625, 0.0625])
    q = np.array([0.125, 0.5, 0.25, 0.0, 0.125])
    target = np.stack([p, p])
    n, got = 64, np.zeros(5)
    for x in range(5):
        if q[x] == 0:
            continue
        for i in range(n):
            for j in range(n):
                a, tok = R.verify([x], q[None], target, [(i + 0.5) / n], (j + 0.5) / n, 1)
                got[tok[0]] += q[x] / n / n
    assert np.all(np.abs(got - p) <= 1 / n) and abs(got.sum() - 1) < 1e-12
