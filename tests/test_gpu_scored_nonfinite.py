"""Softmax scores with logits that are NaN or +inf: the other experts keep their scores, nothing masked is
chosen in their place, and the error bit is set whether or not the logit's expert is chosen."""
import math

import pytest
import torch

from test_gpu_scored_routing import exact_logits, make_plan, weight_tol

pytestmark = pytest.mark.gpu


def limit_scores(l):
    """fp64 softmax of a row in the limit: NaN logits are left out (score NaN), the +inf ones share 1."""
    l = l.double()
    odd, top = l.isnan(), l == math.inf
    if top.any():
        s = top.double() / top.sum()
    else:
        e = torch.where(odd, 0.0, torch.exp(l - torch.where(odd, -math.inf, l).amax()))
        s = e / e.sum()
    return torch.where(odd, math.nan, s)


def best(l, bias, k, groups, keep, top):
    """ids of the k largest keys: (value desc, index asc), masked experts next, NaN last."""
    s = limit_scores(l)
    key = s if bias is None else s + bias.double()
    key = [-math.inf if float(v) == -math.inf else float(c) for v, c in zip(l, key)]
    order = lambda v: sorted(range(len(v)), key=lambda i: (1, 0, i) if math.isnan(v[i]) else (0, -v[i], i))
    per = len(key) // groups
    if groups > 1:
        rank = []
        for g in range(groups):
            part = key[g * per:(g + 1) * per]
            rank.append(sum(part[i] for i in order(part)[:top]))
        kept = order(rank)[:keep]
        key = [c if i // per in kept else -math.inf for i, c in enumerate(key)]
    ids = order(key)[:k]
    return ids, torch.stack([s[i] if key[i] != -math.inf else s.new_zeros(()) for i in ids])


def row(seed, E):
    return exact_logits(1, E, seed, "softmax")[0]


def cases():
    E = 16
    out = {}
    l = row(1, E); l[10] = math.nan
    out["nan, not chosen"] = (l, None, 1, 1, 1)
    l = row(2, E); l[10] = math.nan; l[:9] = -math.inf
    out["nan beside masked experts"] = (l, None, 1, 1, 1)
    l = row(3, E); l[12] = math.inf
    out["infinite, chosen"] = (l, None, 1, 1, 1)
    l = row(4, E); l[12] = l[3] = math.inf; l[5] = math.nan
    out["two infinite and a nan"] = (l, None, 1, 1, 1)
    l = row(5, E); l[12] = math.inf
    bias = torch.zeros(E); bias[12] = -8.0; bias[:4] = 1.0
    out["infinite, kept out by its bias"] = (l, bias, 1, 1, 1)
    l = row(6, E); l[0] = math.nan
    out["nan in a group, best two"] = (l, None, 4, 2, 2)
    l = row(7, E); l[0:4] = math.nan; l[5] = -math.inf
    out["a group of nan"] = (l, None, 4, 2, 1)
    l = row(8, E); l[15] = math.inf
    bias = torch.zeros(E); bias[:8] = 4.0
    out["infinite in a dropped group"] = (l, bias, 2, 1, 2)
    return out


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("name", list(cases()))
def test_softmax_with_odd_logits(name, renorm):
    from decode_batches_gb300 import DEVERR_NONFINITE
    l, bias, groups, keep, top = cases()[name]
    E, k = len(l), 3
    plan = make_plan(E, k)
    plan.set_routing("softmax", bias=None if bias is None else bias.cuda(), n_groups=groups, topk_groups=keep,
                     group_top=top, renormalize=renorm, scale=2.5)
    clean = row(99, E)
    ids, w = plan.route_logits(torch.stack([clean, l]).cuda())
    assert plan.device_error() == DEVERR_NONFINITE
    rid, rw = best(l, bias, k, groups, keep, top)
    assert ids[1].tolist() == rid and not rw.isnan().any()
    if renorm:
        rw = rw / (rw.sum() + 1e-20)
    assert ((w[1].double().cpu() - 2.5 * rw).abs() <= weight_tol(E) * 2.5 * rw + 1e-44).all()
    # the token beside it is as if alone
    ids0, w0 = plan.route_logits(clean[None].cuda())
    assert torch.equal(ids[0], ids0[0]) and torch.equal(w[0], w0[0]) and plan.device_error() == 0


def test_softmax_of_nothing_but_nan():
    from decode_batches_gb300 import DEVERR_NONFINITE
    plan = make_plan(40, 3)
    plan.set_routing("softmax")
    l = torch.full((1, 40), math.nan)
    ids, w = plan.route_logits(l.cuda())
    assert ids.tolist() == [[0, 1, 2]] and w.isnan().all() and plan.device_error() == DEVERR_NONFINITE
    l[0, 7] = -math.inf                           # a masked expert is a number below all others, NaN below it
    ids, w = plan.route_logits(l.cuda())
    assert ids.tolist() == [[7, 0, 1]] and plan.device_error() == DEVERR_NONFINITE


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_layer_reports_a_nan_router_row(T):
    """A router row of NaN: every front end of the layer flags it and the other experts serve the step."""
    from decode_batches_gb300 import DEVERR_NONFINITE, MoePlan
    E, k, d, f = 64, 4, 256, 128
    g = torch.Generator().manual_seed(3)
    bf = lambda *s: (torch.randn(s, generator=g) * s[-1] ** -0.5).to(torch.bfloat16).cuda()
    w_router = torch.randn((E, d), generator=g) * 0.05
    w_router[E - 1] = math.nan
    plan = MoePlan(E, k, d, f, 0, "bf16")
    plan.set_weights(w_router.cuda(), None, bf(E, f, d), bf(E, f, d), bf(E, d, f))
    plan.allocate_workspace(T)
    plan.set_routing("softmax", renormalize=False)
    x = torch.randn((T, d), generator=g).to(torch.bfloat16).cuda()
    out = plan.forward(x)
    assert plan.device_error() == DEVERR_NONFINITE
    logits, ids, gates = plan.route(x)
    assert plan.device_error() == DEVERR_NONFINITE
    assert logits[:, -1].isnan().all() and int(ids.max()) < E - 1 and gates.isfinite().all()
    assert out.isfinite().all() and torch.equal(out, plan.forward_routed(x, ids, gates))
