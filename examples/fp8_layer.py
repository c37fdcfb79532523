"""A serving step with 8-bit weights: an input projection (Fp8Linear), then an MoE layer whose router
scores with a sigmoid, a balance bias and expert groups (MoePlan.set_routing) and whose experts run on
e4m3 weights (weight_dtype="fp8").

    python examples/fp8_layer.py [T]

Needs a GB300 and the built library.  Prints how far the step is from the same step on the
dequantised weights in fp32 torch, and its time.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from decode_batches_gb300 import Fp8Linear, MoePlan, quantize_fp8_weight  # noqa: E402

E, K_TOP, D, F = 64, 8, 1024, 256            # experts, experts a token, model width, hidden width
GROUPS, KEEP = 8, 4


def dequantise(q, s):
    """Codes [..., rows, K] and scales of 128 x 128 blocks as fp32 values."""
    s = s.repeat_interleave(128, -2)[..., : q.shape[-2], :].repeat_interleave(128, -1)[..., : q.shape[-1]]
    return q.float() * s


def build(T_max, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, device="cuda", generator=g) * shape[-1] ** -0.5
    w = {name: quantize_fp8_weight(rnd(*shape).to(torch.bfloat16))
         for name, shape in (("in", (D, D)), ("gate", (E, F, D)), ("up", (E, F, D)), ("down", (E, D, F)))}
    w["router"] = rnd(E, D)
    w["bias"] = 0.01 * torch.randint(-5, 6, (E,), device="cuda", generator=g).float()
    proj = Fp8Linear(D, D)
    proj.set_weights(*w["in"])
    proj.allocate_workspace(T_max)
    plan = MoePlan(E, K_TOP, D, F, weight_dtype="fp8")
    plan.set_weights(w["router"], None, w["gate"][0], w["up"][0], w["down"][0], w["gate"][1], w["up"][1], w["down"][1])
    plan.set_routing("sigmoid", bias=w["bias"], n_groups=GROUPS, topk_groups=KEEP, group_top=2, scale=2.5)
    plan.allocate_workspace(T_max)
    return proj, plan, w


def step(proj, plan, x):
    return plan.forward(proj.forward(x), n_prefill=x.shape[0])


def step_plain(w, x, ids, gates):
    """The step in fp32 without activation quantisation, for the same routing."""
    y = x.float() @ dequantise(*w["in"]).T
    out = torch.zeros_like(y)
    gate, up, down = (dequantise(*w[n]) for n in ("gate", "up", "down"))
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = torch.nn.functional.silu(y[t] @ gate[e].T) * (y[t] @ up[e].T)
        out.index_add_(0, t, gates[t, j][:, None] * (h @ down[e].T))
    return out


def main(T=256):
    proj, plan, w = build(T)
    x = torch.randn((T, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
    out = step(proj, plan, x)
    _, ids, gates = plan.route(proj.forward(x))
    ref = step_plain(w, x, ids, gates)
    err = float((out.float() - ref).norm() / ref.norm())
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        step(proj, plan, x)
    stop.record()
    torch.cuda.synchronize()
    print(f"T={T}: relative distance from the fp32 step {err:.4f}, {start.elapsed_time(stop) / 20 * 1e3:.1f} us a step")
    return err, plan.device_error() | proj.device_error()


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 256)
