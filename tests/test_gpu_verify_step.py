"""The example's verify step and its training step: adapters, expert layer, logits and verification together, and the
gradients through sorted rows."""
import importlib.util
import os

import pytest
import torch

from verify_helpers import verify_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("B", [1, 5, 80])
def test_verify_step(example, B):
    x, ids, offsets, u, us = example.requests(B, seed=B)
    step = example.Step(x.shape[0])
    p = step.probabilities(x, ids)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.softmax(p.log() + 0.3 * torch.randn(p.shape, device="cuda", generator=g), 1)
    drafts = torch.multinomial(q, 1, generator=g)[:, 0].int()
    tokens, accepted = step(x, ids, drafts, offsets, u, us, q)
    ref, racc = verify_ref(p.cpu(), drafts.tolist(), offsets.tolist(), u.tolist(), us.tolist(), q.cpu())
    assert tokens.tolist() == ref and accepted.tolist() == racc
    assert step.device_error() == 0
    # the adapters are part of it: without them a row of an adapter gets other probabilities, one of none the same
    plain = torch.softmax(step.head.forward(step.plan.forward(step.proj.forward(x)), out_dtype=torch.float32), 1)
    same = (plain == p).all(1)
    assert same[ids < 0].all() and not same[ids >= 0].any()
    # the whole step in one graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, ids, drafts, offsets, u, us, q)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], tokens) and torch.equal(got[1], accepted)


def test_example_runs(example):
    tokens, accepted = example.main(3)
    assert accepted.shape == (3,) and tokens.dtype == torch.int32


def test_gradients_of_own_experts(example):
    T, E, k, D = 37, example.E, example.K_TOP, 24
    g = torch.Generator().manual_seed(5)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    x, w = torch.randn((T, D), generator=g), torch.randn((E, D, D), generator=g) * D ** -0.5
    gates, out_grad = torch.softmax(torch.randn((T, k), generator=g), 1), torch.randn((T, D), generator=g)
    plan = example.MoePlan(E, k, D, 8)
    plan.allocate_workspace(T)
    leaf = lambda t: t.clone().cuda().requires_grad_()
    a = [leaf(x), leaf(gates), leaf(w)]
    out = example.own_experts(plan, a[0], ids.cuda(), a[1], a[2])
    out.backward(out_grad.cuda())
    b = [t.double().requires_grad_() for t in (x, gates, w)]
    ref = (b[1][:, :, None] * torch.tanh(torch.einsum("td,tkde->tke", b[0], b[2][ids.long()]))).sum(1)
    ref.backward(out_grad.double())
    # fp32 throughout: sums of up to D or T terms of order one, the products in fp32 (no TF32 by default)
    for got, want in [(out, ref)] + [(s.grad, t.grad) for s, t in zip(a, b)]:
        scale = float(want.detach().abs().max())
        assert float((got.detach().double().cpu() - want.detach()).abs().max()) <= 64 * (T + D) * 2.0 ** -24 * max(scale, 1.0)
    # against differences, in 64 bits for the formula's own part: d loss / d gates along a direction
    loss = lambda gt: float((example.own_experts(plan, x.cuda(), ids.cuda(), gt.cuda(), w.cuda()).double().cpu()
                             * out_grad.double()).sum())
    v = torch.randn((T, k), generator=g)
    difference = (loss(gates + v) - loss(gates - v)) / 2              # the output is linear in the gates
    along = float((a[1].grad.double().cpu() * v.double()).sum())
    size = float(((gates.abs() + v.abs()).sum(1, keepdim=True) * out_grad.abs()).double().sum())
    assert abs(difference - along) <= (k + D + 32) * 2.0 ** -22 * size
