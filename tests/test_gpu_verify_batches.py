"""Batches of 20 to 110 requests, whose requests have fewer threads each than those of small calls:
the same answers as in calls of a few requests, and the exact ones.  (A sum is off by some 2^-40 of itself at most, so two
right kernels differ where u falls that near to a border: no number here does, or the exact form would show it.)"""
import pytest
import torch

from test_gpu_verify import TYPES, inputs, place, pkg
from verify_helpers import verify_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,V,dt,pad,shift", [(20, 24576, "fp32", 0, 0), (57, 24575, "fp32", 0, 1), (58, 24576, "fp32", 0, 0),
                                              (33, 32003, "fp32", 0, 0), (57, 49153, "bf16", 7, 0), (40, 65536, "fp16", 0, 0),
                                              (24, 131072, "bf16", 0, 0), (100, 12289, "fp32", 0, 3), (110, 12288, "bf16", 0, 0),
                                              (90, 6151, "fp16", 1, 0)])
def test_batches_as_in_small_calls(B, V, dt, pad, shift):
    counts = [(3 * b) % 4 for b in range(B)]                        # (a request without rows among them)
    p, q, d, off, u, us = inputs(counts, V, TYPES[dt], B + V, sharp=2.0)
    rows = [place(p, pad, shift), place(q, pad, shift)]
    dd, ud, usd = d.cuda(), u.cuda(), us.cuda()
    for probs in (rows[1], None):
        ofs = torch.tensor(off, dtype=torch.int32, device="cuda")
        tokens, accepted = pkg().verify_drafts(rows[0], dd, ofs, ud, usd, probs)
        for b in range(0, B, 7):
            last = min(b + 7, B)
            lo, hi = off[b], off[last]
            few = torch.tensor([o - lo for o in off[b:last + 1]], dtype=torch.int32, device="cuda")
            t, a = pkg().verify_drafts(rows[0][lo:hi], dd[lo:hi], few, ud[lo:hi], usd[b:last],
                                       None if probs is None else probs[lo:hi])
            assert torch.equal(t, tokens[lo:hi]) and torch.equal(a, accepted[b:last])
        lo, hi = off[1], off[3]
        ref, racc = verify_ref(p[lo:hi], d[lo:hi].tolist(), [o - lo for o in off[1:4]], u[lo:hi].tolist(), us[1:3].tolist(),
                               None if probs is None else q[lo:hi])
        assert accepted[1:3].tolist() == racc and tokens[lo:hi].tolist() == ref
