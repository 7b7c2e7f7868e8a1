"""The draw of dflash_verify at borders where u * (sum of the weights), rounded
to 53 bits, would decide otherwise than the product itself."""
import math
import random
from fractions import Fraction

import numpy as np
import pytest
import torch

from block_diffusion_draft_gb300 import verify_draft

pytestmark = pytest.mark.gpu
ONE = 1 << 44


def pieces(w):
    """fp32 probabilities whose weights sum to w, the last one not zero."""
    p = [1.0] * (w // ONE)
    rest = w % ONE
    cut = max(0, rest.bit_length() - 24)
    for part in (rest >> cut << cut, rest & ((1 << cut) - 1)):
        if part:
            p.append(part / ONE)
    assert sum(int(Fraction(float(np.float32(x))) * ONE) for x in p) == w
    return p


def border_case(r, top):
    """u, and a row whose border between two tokens lies between the product's
    floor and that of its rounded form; the index of the token drawn."""
    while True:
        total, u = r.randrange(top // 2, top), float(np.float32(r.random()))
        exact = math.floor(Fraction(u) * total)
        rounded = math.floor(u * float(total))
        if rounded != exact and 0 < exact < total - 1:
            border = max(exact, rounded)
            first = pieces(border)
            row = first + pieces(total - border)
            return u, row, len(first) - 1 if exact < border else len(first)


@pytest.mark.parametrize("top", [1 << 44, 1 << 50, 1 << 54])
def test_borders_between_the_product_and_its_rounded_form(top):
    r = random.Random(5)
    cases = [border_case(r, top) for _ in range(12)]
    V = max(len(row) for _, row, _ in cases)
    p = torch.zeros(len(cases), 1, V)
    for b, (_, row, _) in enumerate(cases):
        p[b, 0, :len(row)] = torch.tensor(row)
    u = torch.tensor([c[0] for c in cases])
    x = torch.zeros(len(cases), 0, dtype=torch.int32)
    acc, tok = verify_draft(x.cuda(), None, p.cuda(), torch.zeros(len(cases), 0).cuda(), u.cuda())
    assert tok[:, 0].tolist() == [c[2] for c in cases]
    assert not acc.any()


def test_small_and_largest_uniform_numbers():
    """Every magnitude of u, subnormal numbers among them, on a row of equal
    weights."""
    V = 4096
    us = [float(np.float32(m * 2.0 ** -e)) for e in range(0, 150, 3) for m in (1.0, 0.75, 0.999)]
    us += [float(np.nextafter(np.float32(1), np.float32(0))), 2.0 ** -149]
    p = torch.full((len(us), 1, V), 1.0 / 1024)
    x = torch.zeros(len(us), 0, dtype=torch.int32)
    _, tok = verify_draft(x.cuda(), None, p.cuda(), torch.zeros(len(us), 0).cuda(),
                          torch.tensor(us).cuda())
    w, total = ONE >> 10, V * (ONE >> 10)
    want = [min(math.floor(Fraction(u) * total), total - 1) // w for u in us]
    assert tok[:, 0].tolist() == want
