"""The example's training step with assignments that permute drops: they add nothing to the output or to any gradient,
whatever lay in the memory that new tensors get."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step_example_dropped", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def leave_nan_behind():
    """The memory of tensors that are made from now on held NaN last."""
    held = [torch.full((n,), float("nan"), device="cuda") for n in (64, 256, 1024, 4096, 16384, 65536, 1 << 20) for _ in range(24)]
    del held


@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_gradients_with_dropped_assignments(example, share):
    T, E, k, D = 37, example.E, example.K_TOP, 24
    g = torch.Generator().manual_seed(7)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    lost = torch.rand((T, k), generator=g) < share
    ids = torch.where(lost, torch.where(torch.rand((T, k), generator=g) < 0.5, -1, E), ids)
    ids[3], ids[4, 1:] = torch.tensor([2, 2, 5, 2])[:k], ids[4, 0]                # ids that a token has already
    valid = (ids >= 0) & (ids < E)
    used = valid & ~torch.stack([(ids[:, j:j + 1] == ids[:, :j]).any(1) for j in range(k)], 1)
    x, w = torch.randn((T, D), generator=g), torch.randn((E, D, D), generator=g) * D ** -0.5
    gates, out_grad = torch.softmax(torch.randn((T, k), generator=g), 1), torch.randn((T, D), generator=g)
    plan = example.MoePlan(E, k, D, 8)
    plan.allocate_workspace(T)
    leaf = lambda t: t.clone().cuda().requires_grad_()
    a = [leaf(x), leaf(gates), leaf(w)]
    b = [t.double().requires_grad_() for t in (x, gates, w)]
    ids_gpu, grad_gpu = ids.int().cuda(), out_grad.cuda()
    leave_nan_behind()
    out = example.own_experts(plan, a[0], ids_gpu, a[1], a[2])
    leave_nan_behind()
    out.backward(grad_gpu)
    y = torch.tanh(torch.einsum("td,tkde->tke", b[0], b[2][ids.clamp(0, E - 1)]))
    ref = (torch.where(used, b[1], 0.0)[:, :, None] * y).sum(1)
    ref.backward(out_grad.double())
    # fp32 throughout: sums of up to D or T terms of order one
    for got, want in [(out, ref)] + [(s.grad, t.grad) for s, t in zip(a, b)]:
        got, want = got.detach().double().cpu(), want.detach()
        assert torch.isfinite(got).all()
        assert float((got - want).abs().max()) <= 64 * (T + D) * 2.0 ** -24 * max(float(want.abs().max()), 1.0)
