"""Scored routing (softmax or sigmoid scores, selection bias, groups, renormalised weights) against a
plain 64-bit form, at ties, masks, NaN and every front end that routes."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

# A weight's relative error: expf (2 ulp), 1 + e and its reciprocal (1.5 ulp) or the sum of E terms and
# its reciprocal, then the renormalising sum and quotient and the scale: under 16 + E / 32 ulp of 2^-24.
def weight_tol(E):
    return (16 + E / 32) * 2.0 ** -24


def reference(logits, k, score, bias=None, groups=1, keep=1, top=1, renorm=True, scale=1.0):
    """ids and weights of the formula in fp64; orders are (value desc, index asc, NaN lowest)."""
    l = logits.double()
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        m = torch.where(l.isnan(), -math.inf, l).amax(1, keepdim=True)
        e = torch.exp(l - torch.where(m == -math.inf, 0.0, m))
        z = e.sum(1, keepdim=True)
        s = torch.where(z > 0, e / z, torch.where(z.isnan(), z, torch.zeros_like(z)))
    s = s.float().double()                        # scores are fp32 numbers: the smallest ones vanish
    key = s + (0 if bias is None else bias.double())
    key = torch.where(l == -math.inf, -math.inf, key)
    T, E = l.shape
    ids = torch.empty((T, k), dtype=torch.int32)
    w = torch.zeros((T, k), dtype=torch.float64)
    order = lambda v: sorted(range(len(v)), key=lambda i: (1, 0, i) if math.isnan(v[i]) else (0, -v[i], i))
    for t in range(T):
        kt = key[t].tolist()
        if groups > 1:
            per = E // groups
            gs = []
            for g in range(groups):
                part = kt[g * per:(g + 1) * per]
                gs.append(sum(part[i] for i in order(part)[:top]))
            kept = set(order(gs)[:keep])
            kt = [v if i // per in kept else -math.inf for i, v in enumerate(kt)]
        pick = order(kt)[:k]
        ids[t] = torch.tensor(pick)
        w[t] = torch.tensor([0.0 if kt[i] == -math.inf else float(s[t, i]) for i in pick])
        if renorm:
            w[t] = w[t] / (w[t].sum() + 1e-20)
    return ids, w * scale


def make_plan(E, k, d=128, f=128, **kw):
    from decode_batches_gb300 import MoePlan
    plan = MoePlan(E, k, d, f, **kw)
    return plan


def exact_logits(T, E, seed, score):
    """Logits whose scores differ by far more than a few ulp wherever they differ: a coarse grid with
    many exact ties (equal logits have equal scores in any precision)."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-12, 13, (T, E), generator=g).float() / 4


def check(plan, logits, k, **cfg):
    bias = cfg.get("bias")
    plan.set_routing(cfg["score"], bias=None if bias is None else bias.cuda(), n_groups=cfg.get("groups", 1),
                     topk_groups=cfg.get("keep", 1), group_top=cfg.get("top", 1), renormalize=cfg.get("renorm", True),
                     scale=cfg.get("scale", 1.0))
    ids, w = plan.route_logits(logits.cuda())
    rid, rw = reference(logits, k, **cfg)
    assert torch.equal(ids.cpu(), rid)
    got = w.double().cpu()
    assert torch.equal(got.isnan(), rw.isnan())
    ok = ~rw.isnan()
    assert ((got - rw).abs()[ok] <= weight_tol(logits.shape[1]) * rw.abs()[ok] + 1e-44).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,keep,top", [
    (1, 1, 1, 1, 1, 1), (3, 8, 8, 1, 1, 1), (5, 33, 4, 1, 1, 1), (40, 256, 8, 8, 4, 2), (17, 384, 6, 12, 5, 1),
    (9, 64, 6, 8, 3, 2), (130, 160, 6, 8, 3, 1), (4, 512, 32, 32, 7, 2), (2, 1024, 8, 4, 1, 2), (33, 60, 5, 3, 2, 2),
    (6, 96, 3, 32, 1, 1), (7, 40, 10, 4, 4, 2), (2, 31, 31, 31, 31, 1)])
def test_selection_and_weights(score, T, E, k, groups, keep, top):
    plan = make_plan(E, k)
    logits = exact_logits(T, E, 1, score)
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        check(plan, logits, k, score=score, groups=groups, keep=keep, top=top, renorm=renorm, scale=scale)
    assert plan.device_error() == 0


@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (8, 4, 2), (4, 1, 1)])
def test_bias_selects_and_does_not_weigh(groups, keep, top):
    T, E, k = 50, 64, 6
    plan = make_plan(E, k)
    # scores that are exact in fp32 (1/2 from logits of 0, 0 from -200) and biases on a coarse grid
    g = torch.Generator().manual_seed(2)
    logits = torch.where(torch.rand((T, E), generator=g) < 0.7, 0.0, -200.0)
    bias = torch.randint(-64, 65, (E,), generator=g).float() / 64
    check(plan, logits, k, score="sigmoid", bias=bias, groups=groups, keep=keep, top=top, scale=2.5)
    check(plan, logits, k, score="sigmoid", bias=-bias, groups=groups, keep=keep, top=top, renorm=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(score):
    T, E, k = 24, 48, 4
    plan = make_plan(E, k)
    logits = exact_logits(T, E, 3, score)
    logits[:, 5:20] = -math.inf                   # switched off for every token
    logits[3] = -math.inf                         # nothing left: ids 0..k-1, weights 0
    logits[4, 2:] = -math.inf                     # fewer than k left
    logits[5] = torch.finfo(torch.float32).min    # the type's lowest value is a value, not a mask
    logits[6, 1:] = torch.finfo(torch.float32).min
    bias = torch.full((E,), 0.5)
    bias[5:20] = 100.0                            # a bias does not bring a masked expert back
    for b in (None, bias):
        for groups, keep, top in ((1, 1, 1), (6, 2, 2), (6, 2, 1)):
            check(plan, logits, k, score=score, bias=b, groups=groups, keep=keep, top=top)
    ids, w = plan.route_logits(logits.cuda())
    assert not w[3].any() and plan.device_error() == 0


def test_nan_and_infinite_logits():
    from decode_batches_gb300 import DEVERR_NONFINITE
    plan = make_plan(16, 3)
    logits = exact_logits(4, 16, 4, "sigmoid")
    logits[0, 3] = math.nan                       # ranks below everything: never chosen here
    logits[2, :14] = math.nan                     # two left: a NaN has to be chosen
    check(plan, logits[:2], 3, score="sigmoid")
    assert plan.device_error() == 0
    check(plan, logits, 3, score="sigmoid", renorm=False)
    assert plan.device_error() == DEVERR_NONFINITE
    logits = exact_logits(4, 16, 4, "sigmoid")
    logits[1, 7] = math.inf                       # sigmoid 1: chosen, and flagged
    check(plan, logits, 3, score="sigmoid")
    assert plan.device_error() == DEVERR_NONFINITE


def test_extreme_scores_keep_their_order_and_ties():
    plan = make_plan(12, 4)
    # sigmoid saturates to 1 (ties go to the lowest index) and underflows to 0
    logits = torch.tensor([[100.0, 90.0, 200.0, 3.0, 88.0, -300.0, -200.0, 0.0, 1.0, 2.0, -1.0, 95.0],
                           [-300.0] * 12])
    check(plan, logits, 4, score="sigmoid")
    check(plan, logits, 4, score="softmax")
    big = torch.tensor([[3e38, -3e38, 1e38, 0.0] + [-1e38] * 8])
    check(plan, big, 4, score="softmax")


@pytest.mark.parametrize("T", [1, 7, 40, 64, 65, 300])
@pytest.mark.parametrize("E", [64, 256])
def test_every_front_end_routes_alike(T, E):
    """The layer's own routing (tiny, small and large steps) and moe_route select as moe_route_logits
    does on the same logits: the routed call with those ids gives the layer's output bit for bit."""
    from fp8_helpers import random_experts, random_rows
    from decode_batches_gb300 import MoePlan
    k, d, f = 4, 256, 128
    gate, up, down = random_experts(8, f, d, 0)
    rep = lambda t: t.repeat(E // 8, *[1] * (t.dim() - 1)).cuda()
    plan = MoePlan(E, k, d, f, 0, "fp8")
    g = torch.Generator().manual_seed(1)
    plan.set_weights((torch.randn((E, d), generator=g) * 0.05).cuda(), None, rep(gate[0]), rep(up[0]), rep(down[0]),
                     rep(gate[1]), rep(up[1]), rep(down[1]))
    plan.allocate_workspace(T)
    x = random_rows(T, d, 2).cuda()
    bias = (torch.randint(-20, 21, (E,), generator=g).float() / 100).cuda()
    plain = plan.forward(x)
    plan.set_routing("sigmoid", bias=bias, n_groups=8, topk_groups=3, group_top=2, scale=2.5)
    out = plan.forward(x)
    logits, ids, gates = plan.route(x)
    ids2, gates2 = plan.route_logits(logits)
    assert torch.equal(ids, ids2) and torch.equal(gates, gates2)
    assert torch.equal(out, plan.forward_routed(x, ids, gates))
    assert not torch.equal(out, plain)
    plan.set_routing(None)
    assert torch.equal(plan.forward(x), plain)


def test_softmax_scores_renormalised_weigh_like_the_default():
    T, E, k = 100, 128, 8
    plan = make_plan(E, k)
    g = torch.Generator().manual_seed(6)
    logits = torch.randn((T, E), generator=g).cuda()
    ids0, w0 = plan.route_logits(logits)
    plan.set_routing("softmax")
    ids, w = plan.route_logits(logits)
    assert torch.equal(ids, ids0)
    assert ((w - w0).abs() <= 2 * weight_tol(E) * w0).all()


def test_empty_step_other_stream_graph_and_new_bias():
    T, E, k = 90, 64, 4
    plan = make_plan(E, k)
    g = torch.Generator().manual_seed(7)
    logits = exact_logits(T, E, 8, "sigmoid")
    plan.set_routing("sigmoid")
    ids, w = plan.route_logits(logits[:0].cuda())
    assert ids.shape == (0, k) and w.shape == (0, k)
    lc = logits.cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ids, w = plan.route_logits(lc, stream=st)
    st.synchronize()
    rid, _ = reference(logits, k, "sigmoid")
    assert torch.equal(ids.cpu(), rid)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gi, gw = plan.route_logits(lc)
    l2 = exact_logits(T, E, 9, "sigmoid")
    lc.copy_(l2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(gi.cpu(), reference(l2, k, "sigmoid")[0])
    for sign in (1.0, -1.0):                      # a bias given again replaces the plan's copy
        bias = sign * torch.arange(E).float() * 8
        plan.set_routing("sigmoid", bias=bias.cuda())
        ids, _ = plan.route_logits(lc)
        assert torch.equal(ids.cpu(), reference(l2, k, "sigmoid", bias=bias)[0])


def test_refusals():
    from decode_batches_gb300 import MoeError
    plan = make_plan(64, 8)
    for bad in (dict(n_groups=0), dict(n_groups=7), dict(n_groups=64), dict(n_groups=8, topk_groups=0),
                dict(n_groups=8, topk_groups=9), dict(n_groups=16, topk_groups=1), dict(group_top=3), dict(group_top=0),
                dict(scale=math.inf), dict(scale=math.nan)):
        with pytest.raises(MoeError):
            plan.set_routing("sigmoid", **bad)
    with pytest.raises(KeyError):
        plan.set_routing("tanh")
    for bias in (torch.zeros(63, device="cuda"), torch.zeros(64), torch.zeros(64, device="cuda").double()):
        with pytest.raises(ValueError):
            plan.set_routing("sigmoid", bias=bias)
    with pytest.raises(MoeError):                 # group_top larger than a group
        make_plan(8, 2).set_routing("softmax", n_groups=8, topk_groups=2, group_top=2)
