"""A verify step of several requests, each with an adapter of its own, and a training step of own experts.

step:   hidden rows -> 8-bit projection with each request's low-rank adapter (Fp8Linear, LowRankAdapters) -> expert
        layer (MoePlan) -> vocabulary logits (Fp8Linear) -> probabilities -> drafted tokens checked (verify_drafts)
train:  tokens sorted by expert, experts in torch, back with the gates' weights (sort_rows, combine_rows), and the
        gradients of x, the experts' weights and the gates

    python examples/verify_step.py

Needs a GB300 and the built library.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from decode_batches_gb300 import (Fp8Linear, LowRankAdapters, MoePlan, combine_rows, combine_rows_backward,  # noqa: E402
                                  quantize_fp8_weight, sort_rows, sort_rows_backward, verify_drafts)

E, K_TOP, D, F, V = 16, 4, 512, 128, 1000    # experts, experts a token, model width, hidden width, vocabulary
ADAPTERS, RANK = 6, 16


class Step:
    def __init__(self, T_max, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *shape: torch.randn(shape, device="cuda", generator=g) * shape[-1] ** -0.5
        bf = lambda *shape: rnd(*shape).to(torch.bfloat16)
        self.w = {"in": bf(D, D), "head": 4 * bf(V, D), "A": [bf(RANK, D) for _ in range(ADAPTERS)],
                  "B": [bf(D, RANK) for _ in range(ADAPTERS)], "gate": bf(E, F, D), "up": bf(E, F, D), "down": bf(E, D, F),
                  "router": rnd(E, D)}
        self.proj, self.head = Fp8Linear(D, D), Fp8Linear(V, D)
        self.proj.set_weights(*quantize_fp8_weight(self.w["in"]))
        self.head.set_weights(*quantize_fp8_weight(self.w["head"]))
        self.adapters = LowRankAdapters(ADAPTERS, D, D, RANK)
        for i in range(ADAPTERS):
            self.adapters.set(i, self.w["A"][i], self.w["B"][i], 0.5)
        self.plan = MoePlan(E, K_TOP, D, F)
        self.plan.set_weights(self.w["router"], None, self.w["gate"], self.w["up"], self.w["down"])
        for part in (self.proj, self.head, self.adapters, self.plan):
            part.allocate_workspace(T_max)

    def probabilities(self, x, adapter_ids):
        y = self.plan.forward(self.proj.forward(x, adapters=self.adapters, adapter_ids=adapter_ids))
        return torch.softmax(self.head.forward(y, out_dtype=torch.float32), 1)

    def __call__(self, x, adapter_ids, drafts, offsets, u, u_sample, draft_probs=None):
        return verify_drafts(self.probabilities(x, adapter_ids), drafts, offsets, u, u_sample, draft_probs)

    def device_error(self):
        return self.proj.device_error() | self.head.device_error() | self.adapters.device_error() | self.plan.device_error()


class SortRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, inv):
        ctx.save_for_backward(inv)
        return sort_rows(x, inv)

    @staticmethod
    def backward(ctx, grad):
        return sort_rows_backward(grad.contiguous(), *ctx.saved_tensors), None


class CombineRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, inv, gates):
        ctx.save_for_backward(y, inv, gates)
        return combine_rows(y, inv, gates)

    @staticmethod
    def backward(ctx, grad):
        y, inv, gates = ctx.saved_tensors
        # (rows that no entry names, those of dropped assignments, have no gradient)
        dy, dgates = combine_rows_backward(grad.contiguous(), inv, gates, y, out=torch.zeros_like(y))
        return dy, None, dgates


def own_experts(plan, x, ids, gates, weights):
    """out[t] = sum_j gates[t, j] tanh(x[t] weights[e]), e = ids[t, j]: any expert function may stand in its place.  An id
    outside [0, E) and one that a token has already contribute nothing; their rows lie behind the last expert's."""
    _, offsets, _, inv = plan.permute(ids)
    inv = inv.view(ids.shape)
    rows = SortRows.apply(x, inv)
    *parts, dropped = torch.tensor_split(rows, offsets[1:].tolist())
    y = torch.cat([torch.tanh(p @ w) for p, w in zip(parts, weights)] + [torch.zeros_like(dropped)])
    return CombineRows.apply(y, inv, gates)


def requests(B, seed=1):
    """Hidden rows, adapters, drafts and random numbers of B requests with up to five drafts each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = torch.randint(1, 7, (B,), device="cuda", generator=g)
    offsets = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = n.cumsum(0)
    T = int(offsets[-1])
    ids = torch.repeat_interleave(torch.randint(-1, ADAPTERS, (B,), device="cuda", generator=g), n, output_size=T).int()
    x = torch.randn((T, D), device="cuda", generator=g).to(torch.bfloat16)
    return x, ids, offsets, torch.rand(T, device="cuda", generator=g), torch.rand(B, device="cuda", generator=g)


def main(B=12):
    x, ids, offsets, u, u_sample = requests(B)
    step = Step(x.shape[0])
    p = step.probabilities(x, ids)
    q = torch.softmax(p.log() + 0.3 * torch.randn_like(p), 1)           # a draft model near the target
    drafts = torch.multinomial(q, 1)[:, 0].int()
    tokens, accepted = step(x, ids, drafts, offsets, u, u_sample, q)
    drafted = offsets.diff() - 1
    print(f"{B} requests, {x.shape[0]} rows: {int(accepted.sum())} of {int(drafted.sum())} drafts accepted, "
          f"error bits {step.device_error():#x}")
    return tokens, accepted


if __name__ == "__main__":
    main()
