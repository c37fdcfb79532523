"""Softmax scores of continuous logits with a wide spread, weights not renormalised, against fp64."""
import math

import pytest
import torch

from test_gpu_scored_routing import make_plan

pytestmark = pytest.mark.gpu

# In units of 2^-24, relative.  A term exp(v - m): the rounded difference moves the exponent by |v - m|,
# expf is good to 2 ulp (4).  The sum: its terms' errors, weighted by the scores themselves (4, and the mean of
# |v - m| under a softmax, at most ln E), E / 32 additions a lane and 5 across them.  Reciprocal, product and
# the scale 1 each.  Where a score is below the normal numbers: a few steps of 2^-149.
def weight_tol(E, dist):
    return (dist + 4 + 4 + math.log(E) + E / 32 + 5 + 3) * 2.0 ** -24


@pytest.mark.parametrize("spread", [2.0, 30.0, 80.0])
@pytest.mark.parametrize("T,E,k", [(64, 32, 32), (40, 12, 12), (33, 384, 32), (16, 1024, 32), (9, 512, 8)])
def test_softmax_weights_of_a_wide_spread(T, E, k, spread):
    g = torch.Generator().manual_seed(E + int(spread))
    # every expert its own level, no two closer than half a level: the order is that of any precision
    gap = spread / E
    level = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).double()
    logits = ((level + 0.5 * torch.rand((T, E), generator=g).double()) * gap + 3 * torch.randn((T, 1), generator=g)).float()
    plan = make_plan(E, k)
    plan.set_routing("softmax", renormalize=False, scale=2.5)
    ids, w = plan.route_logits(logits.cuda())
    l = logits.double()
    top = l.sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids.cpu().long(), top.indices[:, :k])
    ref = 2.5 * torch.softmax(l, 1).gather(1, top.indices[:, :k])
    dist = top.values[:, :1] - top.values[:, :k]
    err = (w.double().cpu() - ref).abs()
    assert (err <= weight_tol(E, dist) * ref + 16 * 2.0 ** -149).all(), float((err / (weight_tol(E, dist) * ref)).max())
    assert plan.device_error() == 0
