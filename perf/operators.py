"""Cases of the 8-bit draft KV cache, the attention over it and the
verification of drafted tokens, for measurement.

``run`` computes one pass of a case: with ``own`` false in plain torch, with
``own`` true through the library.  The operators:

store   K/V rows quantised into a cache of 8-bit codes with one power-of-two
        scale per 32 channels, then read back as bf16.
attend  the attention of a block of query rows over such a cache.
verify  acceptance of drafted tokens against the target's probabilities, and
        the token that follows the accepted ones.
"""
import math
import random

import numpy as np
import torch

own = False

HEAD = 128          # channels of a head
GROUP = 32          # channels that share a scale
FIX = 44            # probabilities are read as multiples of 2^-44
QMAX = {"int8": 127.0, "e4m3": 448.0}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one new row of one sequence: the smallest append, latency alone
        dict(name="store one row", op="store", batch=1, n_lo=1, n_hi=1, held=4096, kv_heads=8,
             fmt="int8", fused=False, lens=1),
        # a serving step of 32 sequences: 1..16 context rows and a block of 16
        # each, K and V taken as slices of a fused projection's output
        dict(name="store serving step", op="store", batch=32, n_lo=17, n_hi=32, held=8192,
             kv_heads=8, fmt="int8", fused=True, lens=2),
        # the prefill of four long prompts
        dict(name="store prefill", op="store", batch=4, n_lo=8192, n_hi=8192, held=0, kv_heads=8,
             fmt="e4m3", fused=False, lens=3),
        # one token of one sequence over 4096 cached rows
        dict(name="attend one token", op="attend", batch=1, q_len=1, heads=32, kv_heads=8,
             len_lo=4096, len_hi=4096, window=0, causal=False, fmt="int8", lens=4),
        # a block of 16 of one sequence over 4096 cached rows
        dict(name="attend one block", op="attend", batch=1, q_len=16, heads=32, kv_heads=8,
             len_lo=4128, len_hi=4128, window=0, causal=False, fmt="e4m3", lens=5),
        # a serving batch, ragged lengths, a block of 16 per sequence
        dict(name="attend serving", op="attend", batch=32, q_len=16, heads=32, kv_heads=8,
             len_lo=512, len_hi=8192, window=0, causal=False, fmt="int8", lens=6),
        # four long contexts, a block of 16 each
        dict(name="attend long", op="attend", batch=4, q_len=16, heads=32, kv_heads=8,
             len_lo=32800, len_hi=32800, window=0, causal=False, fmt="e4m3", lens=7),
        # a causal band layer: odd block and head counts, short ragged lengths
        # (some rows see nothing)
        dict(name="attend band", op="attend", batch=7, q_len=13, heads=14, kv_heads=2, len_lo=0,
             len_hi=1500, window=257, causal=True, fmt="int8", lens=8),
        # a block of one sequence, the draft's distributions given
        dict(name="verify one block", op="verify", batch=1, drafted=15, vocab=150000,
             dtype="float32", greedy=False, ragged=False, pad=0, lens=9),
        # the serving batch's blocks
        dict(name="verify serving", op="verify", batch=32, drafted=15, vocab=150000,
             dtype="float32", greedy=False, ragged=True, pad=0, lens=10),
        # short drafts of many sequences in bf16, rows padded to an even stride
        dict(name="verify many bf16", op="verify", batch=128, drafted=7, vocab=50001,
             dtype="bfloat16", greedy=False, ragged=True, pad=7, lens=11),
        # drafts that were chosen without sampling (no distribution), odd sizes
        dict(name="verify greedy", op="verify", batch=5, drafted=16, vocab=32003,
             dtype="float32", greedy=True, ragged=False, pad=0, lens=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    lens = rng.randrange(1, 1 << 30)
    op = rng.choice(["store", "attend", "attend", "verify"])
    if op == "store":
        batch = _log_int(rng, 1, 64)
        n_hi = _log_int(rng, 1, 32768 // batch)
        return dict(op=op, batch=batch, n_lo=rng.choice([0, n_hi // 2, n_hi]), n_hi=n_hi,
                    held=_log_int(rng, 1, 2048) - 1, kv_heads=rng.choice([1, 2, 4, 8]),
                    fmt=rng.choice(["int8", "e4m3"]), fused=rng.random() < 0.5, lens=lens)
    if op == "attend":
        batch = _log_int(rng, 1, 64)
        len_hi = _log_int(rng, 1, min(32768, 131072 // batch))
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 7, 8] if kv_heads <= 2 else [1, 2, 4])
        window = _log_int(rng, 16, 4096) if rng.random() < 0.25 else 0
        return dict(op=op, batch=batch, q_len=rng.choice([1, 2, 5, 8, 16, 16, 17]),
                    heads=group * kv_heads, kv_heads=kv_heads,
                    len_lo=rng.choice([0, len_hi // 2, len_hi]), len_hi=len_hi, window=window,
                    causal=rng.random() < 0.3, fmt=rng.choice(["int8", "e4m3"]), lens=lens)
    batch = _log_int(rng, 1, 128)
    drafted = rng.randrange(1, 17)
    vocab = _log_int(rng, 1000, min(150000, 72_000_000 // (batch * (drafted + 1))))
    return dict(op=op, batch=batch, drafted=drafted, vocab=vocab,
                dtype=rng.choice(["float32", "bfloat16"]), greedy=rng.random() < 0.3,
                ragged=rng.random() < 0.5, pad=rng.choice([0, 0, rng.randrange(1, 64)]),
                lens=lens)


def _counts(case, lo, hi):
    """Rows of each sequence: they belong to the case, not to the seed."""
    r = random.Random(case["lens"])
    n = [r.randint(case[lo], case[hi]) for _ in range(case["batch"])]
    return n if any(n) else n[:-1] + [case[hi]]


# -------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _kv_rows(rows, heads, gen):
    """K rows with the uneven channels that norm gains leave, V rows N(0, 1)."""
    gain = torch.exp(0.5 * torch.randn(heads, HEAD, device="cuda", generator=gen))
    k = torch.randn(rows, heads, HEAD, device="cuda", generator=gen) * gain
    v = torch.randn(rows, heads, HEAD, device="cuda", generator=gen)
    return k.bfloat16(), v.bfloat16()


def _layer(heads, kv_heads, window=0, causal=False):
    from block_diffusion_draft_gb300 import DFlashAttention
    z = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    w = dict(wq=z(heads * HEAD, HEAD), wk=z(kv_heads * HEAD, HEAD), wv=z(kv_heads * HEAD, HEAD),
             wo=z(HEAD, heads * HEAD), q_norm=z(HEAD), k_norm=z(HEAD))
    return DFlashAttention(w, hidden=HEAD, n_heads=heads, n_kv_heads=kv_heads, head_dim=HEAD,
                           max_position=64, sliding_window=window, causal=causal)


def _places(counts, first):
    """(sequence, row) of every new row."""
    seq = np.repeat(np.arange(len(counts)), counts)
    row = np.concatenate([np.arange(f, f + n) for f, n in zip(first, counts)])
    to = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int64)).cuda()  # noqa: E731
    return to(seq), to(row)


def _store_rows(case, seed):
    n = _counts(case, "n_lo", "n_hi")
    rows, heads = sum(n), case["kv_heads"]
    k, v = _kv_rows(rows, heads, _generator(seed))
    if case["fused"]:  # [Q heads | K heads | V heads] of one projection
        fused = torch.empty(rows, 6 * heads, HEAD, device="cuda", dtype=torch.bfloat16).zero_()
        fused[:, 4 * heads:5 * heads] = k
        fused[:, 5 * heads:] = v
        k, v = fused[:, 4 * heads:5 * heads], fused[:, 5 * heads:]
    return n, k, v


def _attend_inputs(case, seed):
    n = _counts(case, "len_lo", "len_hi")
    gen = _generator(seed)
    k, v = _kv_rows(sum(n), case["kv_heads"], gen)
    q = torch.randn(case["batch"], case["q_len"], case["heads"], HEAD, device="cuda",
                    generator=gen).bfloat16()
    return n, k, v, q


def _verify_inputs(case, seed):
    B, D, V, pad = case["batch"], case["drafted"], case["vocab"], case["pad"]
    gen = _generator(seed)
    dt = getattr(torch, case["dtype"])
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    target = torch.empty(B, D + 1, V + pad, device="cuda", dtype=dt)[..., :V]
    draft = None if case["greedy"] else torch.empty(B, D, V + pad, device="cuda",
                                                    dtype=dt)[..., :V]
    tokens = torch.empty(B, D, device="cuda", dtype=torch.int32)
    for b in range(B):  # one sequence at a time: the logits are not kept
        logits = 4.0 * rand(D + 1, V)
        target[b] = torch.softmax(logits, -1).to(dt)
        guess = logits[:D] + 1.5 * rand(D, V)
        if draft is None:
            tokens[b] = guess.argmax(-1).int()
        else:
            draft[b] = torch.softmax(guess, -1).to(dt)
            u = torch.rand(D, V, device="cuda", generator=gen).clamp_(1e-7, 1 - 1e-7)
            tokens[b] = (guess - torch.log(-torch.log(u))).argmax(-1).int()
    u_accept = torch.rand(B, D, device="cuda", generator=gen)
    u_sample = torch.rand(B, device="cuda", generator=gen)
    count = None
    if case["ragged"]:
        r = random.Random(case["lens"])
        count = torch.tensor([r.randint(0, D) for _ in range(B)], dtype=torch.int32).cuda()
    return dict(draft_tokens=tokens, draft_probs=draft, target_probs=target, u_accept=u_accept,
                u_sample=u_sample, n_draft=count)


def prepare(case, seed):
    op, s = case["op"], {"case": case}
    if op == "verify":
        s["in"] = _verify_inputs(case, seed)
        return s
    if op == "store":
        n, s["k"], s["v"] = _store_rows(case, seed)
        held = [case["held"]] * case["batch"]
        cap = case["held"] + case["n_hi"]
        if own:
            s["attn"] = _layer(case["kv_heads"], case["kv_heads"])
            from block_diffusion_draft_gb300 import Q8Cache
            s["cache"] = Q8Cache(s["attn"], case["batch"], max(cap, 1), case["fmt"])
            if case["held"]:
                z = torch.zeros(sum(held), case["kv_heads"], HEAD, device="cuda",
                                dtype=torch.bfloat16)
                s["cache"].append(z, z, held)
        else:
            s["store"] = _plain_storage(case, max(cap, 1))
            s["at"] = _places(n, held)
        s["held"], s["n"] = held, n
        return s
    n, k, v, s["q"] = _attend_inputs(case, seed)
    cap = max(max(n), 1)
    if own:
        s["attn"] = _layer(case["heads"], case["kv_heads"], case["window"], case["causal"])
        from block_diffusion_draft_gb300 import Q8Cache
        s["cache"] = Q8Cache(s["attn"], case["batch"], cap, case["fmt"])
        s["cache"].append(k, v, n)
    else:
        s["store"] = _plain_storage(case, cap)
        _plain_append(s["store"], k, v, _places(n, [0] * len(n)), case["fmt"])
        s["len"] = torch.tensor(n).cuda()
    return s


# --------------------------------------------------------------- plain forms
def _power(e):
    """2^e as float32, for whole e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_storage(case, cap):
    dt = torch.int8 if case["fmt"] == "int8" else torch.float8_e4m3fn
    shape = (case["batch"], cap, case["kv_heads"], HEAD // GROUP)
    return [(torch.zeros(*shape, GROUP, device="cuda", dtype=torch.uint8).view(dt),
             torch.zeros(*shape, device="cuda", dtype=torch.int32)) for _ in range(2)]


def _plain_quantise(x, fmt):
    """Codes and exponents of x: the smallest power of two that brings a
    group's largest magnitude to the format's range, at least 2^-117."""
    x = x.float().unflatten(-1, (HEAD // GROUP, GROUP)).clamp(-2.0 ** 126, 2.0 ** 126)
    mant, ex = torch.frexp(x.abs().amax(-1))
    top, width = (127 / 128, 7) if fmt == "int8" else (448 / 512, 9)
    e = (ex - width + (mant > top)).clamp(min=-117)
    y = x * _power(-e).unsqueeze(-1)
    code = torch.round(y).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)
    return code, e.to(torch.int32)


def _plain_values(code, e):
    return (code.float() * _power(e).unsqueeze(-1)).flatten(-2)


def _plain_append(store, k, v, at, fmt):
    for (codes, exps), x in zip(store, (k, v)):
        c, e = _plain_quantise(x, fmt)
        codes.view(torch.uint8)[at[0], at[1]] = c.view(torch.uint8)
        exps[at[0], at[1]] = e


def _plain_read(store, at):
    out = []
    for codes, exps in store:
        c = codes.view(torch.uint8)[at[0], at[1]].view(codes.dtype)
        out.append(_plain_values(c, exps[at[0], at[1]]).bfloat16())
    return out


def _plain_attend(s):
    case, q = s["case"], s["q"].float()
    B, T, nq, _ = q.shape
    nkv = case["kv_heads"]
    k, v = (_plain_values(c, e).transpose(1, 2) for c, e in s["store"])  # [B, nkv, cap, d]
    cap = k.shape[2]
    q = q.view(B, T, nkv, nq // nkv, HEAD).permute(0, 2, 3, 1, 4).reshape(B, nkv, -1, HEAD)
    score = (q @ k.transpose(-1, -2)).view(B, nkv, nq // nkv, T, cap) * HEAD ** -0.5
    key = torch.arange(cap, device=q.device)
    length = s["len"].view(B, 1, 1)
    at = length - T + torch.arange(T, device=q.device).view(1, T, 1)
    seen = (key < length).expand(B, T, cap)
    if case["window"]:
        seen = seen & ((at - key).abs() < case["window"])
    if case["causal"]:
        seen = seen & (key <= at)
    score = score.masked_fill(~seen.view(B, 1, 1, T, cap), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, nkv, -1, cap) @ v).view(B, nkv, nq // nkv, T, HEAD)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return (out.permute(0, 3, 1, 2, 4).reshape(B, T, nq, HEAD).bfloat16(),
            lse.permute(0, 3, 1, 2).reshape(B, T, nq))


def _fixed(p):
    """Probabilities as whole multiples of 2^-44, cut off below."""
    return torch.floor(p.double().clamp(0.0, 1.0) * 2.0 ** FIX).to(torch.int64)


def _plain_verify(draft_tokens, draft_probs, target_probs, u_accept, u_sample, n_draft):
    B, D = draft_tokens.shape
    V, dev = target_probs.shape[-1], target_probs.device
    x = draft_tokens.long().unsqueeze(-1)
    p = target_probs[:, :D].gather(-1, x).squeeze(-1).double()
    q = 1.0 if draft_probs is None else draft_probs.gather(-1, x).squeeze(-1).double()
    count = torch.full((B,), D, device=dev) if n_draft is None else n_draft.long()
    place = torch.arange(D + 1, device=dev)
    ok = (u_accept.double() * q < p) & (place[:D] < count[:, None])
    a = ok.long().cumprod(1).sum(1)
    one = torch.arange(B, device=dev)
    last = (a - (a == D).long()).clamp(min=0)
    rejected = (a < count).long()[:, None]
    wp = _fixed(target_probs[one, a])
    if draft_probs is None:
        wq = torch.zeros_like(wp).scatter_(1, x[one, last], 1 << FIX)
    else:
        wq = _fixed(draft_probs[one, last])
    w = (wp - wq * rejected).clamp(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, wp)
    c = w.cumsum(1)
    total = c[:, -1:]
    t = torch.floor(u_sample.double()[:, None] * total.double()).to(torch.int64)
    token = torch.where(total > 0, (c <= t).sum(1, keepdim=True), -1)
    kept = torch.cat([draft_tokens.long(), draft_tokens.new_zeros(B, 1).long()], 1)
    tokens = torch.where(place < a[:, None], kept, torch.where(place == a[:, None], token, -1))
    return a.int(), tokens.int()


# ----------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if op == "store":
        if own:
            s["cache"].crop(s["held"])
            s["cache"].append(s["k"], s["v"], s["n"])
            k, v = s["cache"].read(s["held"], s["n"])
        else:
            _plain_append(s["store"], s["k"], s["v"], s["at"], s["case"]["fmt"])
            k, v = _plain_read(s["store"], s["at"])
        return {"k": k, "v": v}
    if op == "attend":
        out, lse = s["attn"].q8_core(s["cache"], s["q"]) if own else _plain_attend(s)
        return {"out": out, "lse": lse}
    if own:
        from block_diffusion_draft_gb300 import verify_draft
        accepted, tokens = verify_draft(**s["in"])
    else:
        accepted, tokens = _plain_verify(**s["in"])
    return {"accepted": accepted, "tokens": tokens}


def work(case):
    if case["op"] == "store":
        # bf16 rows in, codes and scales out; then the same the other way
        values = 2 * sum(_counts(case, "n_lo", "n_hi")) * case["kv_heads"] * HEAD
        return {"bytes": 2 * values * (2 + 1 + 1 / GROUP) + 1, "flops": 0}
    if case["op"] == "attend":
        T, nq, nkv = case["q_len"], case["heads"], case["kv_heads"]
        keys = pairs = 0
        for n in _counts(case, "len_lo", "len_hi"):
            first = n
            for t in range(T):
                at = n - T + t
                lo, hi = 0, n
                if case["window"]:
                    lo, hi = max(lo, at - case["window"] + 1), min(hi, at + case["window"])
                if case["causal"]:
                    hi = min(hi, at + 1)
                pairs += max(0, hi - lo)
                first = min(first, lo) if hi > lo else first
            keys += n - first
        rows = case["batch"] * T * nq
        return {"bytes": keys * nkv * 2 * (HEAD + HEAD // GROUP) + rows * (4 * HEAD + 4),
                "flops": 4 * HEAD * nq * pairs}
    # what decides: a probability per drafted token, then the target's row and
    # (unless the draft has no distribution) the draft's row at one place
    size = 4 if case["dtype"] == "float32" else 2
    rows = 1 if case["greedy"] else 2
    return {"bytes": case["batch"] * (rows * case["vocab"] * size +
                                      case["drafted"] * (4 + 4 + 4 + rows * size) + 8),
            "flops": 0}


# --------------------------------------------------------------------- exact
def _exact_values(x, fmt):
    """What the stored codes of x stand for, from the formats' definitions."""
    x = x.double().unflatten(-1, (HEAD // GROUP, GROUP))
    f, e = torch.frexp(x.abs().amax(-1, keepdim=True) / QMAX[fmt])
    e = torch.where(f > 0.5, e, e - 1).clamp(min=-117).double()
    y = x / torch.exp2(e)
    if fmt == "int8":
        step = torch.ones_like(y)
    else:  # 3 fraction bits, smallest exponent -6
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    if case["op"] == "store":
        _, k, v = _store_rows(case, seed)
        return {"k": _exact_values(k, case["fmt"]), "v": _exact_values(v, case["fmt"])}
    if case["op"] == "attend":
        n, k, v, q = _attend_inputs(case, seed)
        T, nq, nkv = case["q_len"], case["heads"], case["kv_heads"]
        out = torch.zeros(case["batch"], T, nq, HEAD, device="cuda", dtype=torch.float64)
        lse = torch.full((case["batch"], T, nq), -math.inf, device="cuda", dtype=torch.float64)
        begin = 0
        for b, length in enumerate(n):
            kb = _exact_values(k[begin:begin + length], case["fmt"])
            vb = _exact_values(v[begin:begin + length], case["fmt"])
            begin += length
            for t in range(T):
                at = length - T + t
                lo, hi = 0, length
                if case["window"]:
                    lo, hi = max(lo, at - case["window"] + 1), min(hi, at + case["window"])
                if case["causal"]:
                    hi = min(hi, at + 1)
                if hi <= lo:
                    continue
                qh = q[b, t].double().view(nkv, nq // nkv, HEAD)
                z = torch.einsum("hgd,khd->hgk", qh, kb[lo:hi]) / math.sqrt(HEAD)
                out[b, t] = torch.einsum("hgk,khd->hgd", torch.softmax(z, -1),
                                         vb[lo:hi]).reshape(nq, HEAD)
                lse[b, t] = torch.logsumexp(z, -1).reshape(nq)
        return {"out": out, "lse": lse}
    d = _verify_inputs(case, seed)
    accepted, tokens = [], []
    whole = lambda r: np.floor(np.minimum(r.double().cpu().numpy(), 1.0) * 2.0 ** FIX  # noqa: E731
                               ).astype(np.int64)
    for b in range(case["batch"]):
        D = case["drafted"] if d["n_draft"] is None else int(d["n_draft"][b])
        a = 0
        while a < D:
            x = int(d["draft_tokens"][b, a])
            q = 1.0 if d["draft_probs"] is None else float(d["draft_probs"][b, a, x])
            if not float(d["u_accept"][b, a]) * q < float(d["target_probs"][b, a, x]):
                break
            a += 1
        w = whole(d["target_probs"][b, a])
        if a < D:
            r = w.copy()
            if d["draft_probs"] is None:
                r[int(d["draft_tokens"][b, a])] = 0
            else:
                r = np.maximum(r - whole(d["draft_probs"][b, a]), 0)
            w = r if r.any() else w
        c = np.cumsum(w)
        x = int(np.searchsorted(c, math.floor(float(d["u_sample"][b]) * float(c[-1])), "right"))
        row = d["draft_tokens"][b, :a].tolist() + [x if c[-1] else -1]
        accepted.append(a)
        tokens.append(row + [-1] * (case["drafted"] + 1 - len(row)))
    return {"accepted": torch.tensor(accepted, dtype=torch.int32),
            "tokens": torch.tensor(tokens, dtype=torch.int32)}
