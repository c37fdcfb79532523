"""The place u S of the drawn token next to a border: rows of ones, where S is the vocabulary's size and the answer is the
whole part of an exact product."""
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V,B", [(1009, 200), (32003, 19), (100003, 40), (131071, 150)])
def test_products_next_to_whole_numbers(V, B, dt):
    import decode_batches_gb300 as p
    k = np.random.RandomState(V + B).randint(1, V, B)
    u = (k / V).astype(np.float32)                                   # u V is within V 2^-25 of k, on either side
    u[1::3] = np.nextafter(u[1::3], np.float32(0))
    u[2::3] = np.nextafter(u[2::3], np.float32(1))
    want = [int(Fraction(float(v)) * V) for v in u]
    ones = torch.ones((B, V), dtype=dt, device="cuda")
    off = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    us = torch.from_numpy(u).cuda()
    tokens, accepted = p.verify_drafts(ones, torch.zeros(B, dtype=torch.int32, device="cuda"), off, us, us)
    assert tokens.tolist() == want and not accepted.any()
    assert {w - int(i) for w, i in zip(want, k)} == {-1, 0}          # both sides of the borders are met
