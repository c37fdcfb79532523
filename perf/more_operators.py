"""Measured cases of the operators that move and adapt the rows of a step and check its drafts.

    sort      S[inv[t,j]] = w[t,j] x[t]: token rows to the expert order, and the gradients of it
    combine   out[t] = sum_j w[t,j] y[inv[t,j]] + shared[t]: back again, and the gradients of it
    adapters  out[t] = base[t] + s_a B_a (A_a x[t]), a = ids[t]: low-rank adapters of many requests
              beside a shared projection's output (ids[t] = -1: none)
    verify    drafted tokens against the target's probabilities: row i of a request is accepted while
              u_i q_i < p_i, then one token is drawn from max(p - q, 0) of the first refused row (from
              p of the row behind the last draft) at a given uniform number

`own` false: elementary torch operations in fp32 (fp64 for the cumulative sums of probabilities).
`own` true: the calls of this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a verify batch's rows to their experts
        dict(name="sort_verify", op="sort", back=False, T=48, E=384, k=8, d=4096, dt="bf16", out="bf16", w=False, lost=0.0),
        # a mixed step of 2048 prefill rows and three decode rows, weights applied before the experts
        dict(name="sort_mixed", op="sort", back=False, T=2051, E=256, k=8, d=2048, dt="bf16", out="bf16", w=True, lost=0.0),
        # the gradient of the rows of the largest step
        dict(name="sort_back_large", op="sort", back=True, T=8195, E=256, k=8, d=2048, dt="bf16", out="bf16", w=False, lost=0.0),
        # experts' outputs in fp16 back to the tokens of one decode step, with the shared experts' term
        dict(name="combine_decode", op="combine", back=False, T=4, E=256, k=8, d=2048, dt="fp16", out="bf16", w=True, lost=0.0),
        # the gradient at sizes that divide into nothing, fp32, a tenth of the assignments dropped
        dict(name="combine_back_ragged", op="combine", back=True, T=517, E=40, k=3, d=1337, dt="fp32", out="fp32", w=True, lost=0.1),
        # a training step of wide rows: gradients of the experts' outputs and of the gates
        dict(name="combine_back_large", op="combine", back=True, T=8195, E=384, k=6, d=4096, dt="bf16", out="bf16", w=True, lost=0.0),
        # one request's token
        dict(name="adapters_token", op="adapters", T=1, n=8, r=16, K=4096, N=4096, dt="bf16", out="bf16", rows="mixed", none=0.0),
        # a verify batch of many requests, nearly each with an adapter of its own, fp32 out
        dict(name="adapters_verify", op="adapters", T=48, n=64, r=32, K=2048, N=4096, dt="fp16", out="fp32", rows="mixed", none=0.1),
        # a mixed step: one prompt's prefill rows with one adapter, three decode rows with others
        dict(name="adapters_mixed", op="adapters", T=2051, n=64, r=16, K=2048, N=2048, dt="bf16", out="bf16", rows="runs", none=0.0),
        # the largest step, rows of 32 requests interleaved, a fifth of them without an adapter
        dict(name="adapters_large", op="adapters", T=8195, n=32, r=64, K=4096, N=4096, dt="bf16", out="bf16", rows="mixed", none=0.2),
        # four requests of five drafts each, odd vocabulary
        dict(name="verify_few", op="verify", B=4, most=5, V=32003, dt="fp32", draft=True, sharp=2.0),
        # a full decode batch over a large vocabulary
        dict(name="verify_many", op="verify", B=192, most=7, V=131072, dt="fp32", draft=True, sharp=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "combine", "adapters", "verify"])
    if op in ("sort", "combine"):
        E, k = _log(rng, 8, 384), rng.randint(1, 8)
        d = _log(rng, 64, 4096)
        d = d | 1 if rng.random() < 0.3 else -(-d // 8) * 8
        dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        out = rng.choice([dt, "bf16", "fp32"]) if op == "combine" else dt
        return dict(op=op, back=rng.random() < 0.5, T=_log(rng, 1, 8195 if dt != "fp32" else 4096), E=E, k=k, d=d, dt=dt,
                    out=out, w=op == "combine" or rng.random() < 0.5, lost=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "adapters":
        K, N = _log(rng, 64, 4096), _log(rng, 64, 4096)
        if rng.random() < 0.7:
            K, N = -(-K // 8) * 8, -(-N // 8) * 8
        return dict(op=op, T=_log(rng, 1, 8195), n=_log(rng, 1, 128), r=rng.choice([4, 8, 16, 16, 24, 32, 64]), K=K, N=N,
                    dt=rng.choice(["bf16", "bf16", "fp16"]), out=rng.choice(["bf16", "fp32", "fp16"]),
                    rows=rng.choice(["mixed", "runs"]), none=rng.choice([0.0, 0.2, 0.9]))
    V = _log(rng, 1000, 131072)
    return dict(op=op, B=_log(rng, 1, 192), most=rng.randint(0, 7), V=V | 1 if rng.random() < 0.5 else -(-V // 8) * 8,
                dt=rng.choice(["fp32", "fp32", "bf16", "fp16"]), draft=rng.random() < 0.7, sharp=rng.choice([0.5, 2.0, 4.0]))


# ------------------------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    return g


def _normal(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _hidden(g, T, d, dt):
    """Rows with a token's own magnitude and a few loud channels, as hidden states have."""
    x = _normal(g, T, d) * torch.exp(0.3 * _normal(g, T, 1))
    x *= torch.where(torch.rand((d,), device="cuda", generator=g) < 0.01, 8.0, 1.0)
    return x.to(DTYPES[dt])


def _moe_inputs(case, seed):
    """inv [T][k] (-1 where an assignment was dropped), weights or None, and the operands."""
    g = _gen(seed, 11)
    T, E, k, d = case["T"], case["E"], min(case["k"], case["E"]), case["d"]
    top = _normal(g, T, E).topk(k, dim=1)
    ids = torch.where(torch.rand((T, k), device="cuda", generator=g) < case["lost"], E, top.indices).reshape(-1)
    order = ids.sort(stable=True).indices
    inv = torch.empty_like(order)
    inv[order] = torch.arange(T * k, device="cuda")
    inv = torch.where(ids == E, -1, inv).view(T, k).int()
    w = torch.softmax(top.values, 1) if case["w"] else None
    tok, rows = _hidden(g, T, d, case["out" if case["op"] == "combine" else "dt"]), None
    if (case["op"] == "sort") == case["back"] or case["w"]:  # a tensor in the expert order goes in
        rows = torch.cat([_hidden(g, min(8192, T * k - i), d, case["dt"]) for i in range(0, T * k, 8192)])
    return inv, w, tok, rows


def _adapter_inputs(case, seed):
    g = _gen(seed, 12)
    T, n, r, K, N, dt = (case[c] for c in ("T", "n", "r", "K", "N", "dt"))
    x = _hidden(g, T, K, dt)
    A = (_normal(g, n, r, K) * K ** -0.5).to(DTYPES[dt])
    B = (_normal(g, n, N, r) * r ** -0.5).to(DTYPES[dt])
    scale = torch.exp2(torch.randint(-1, 3, (n,), device="cuda", generator=g).float()).tolist()
    base = _normal(g, T, N).to(DTYPES[case["out"]])
    ids = torch.randint(0, n, (T,), device="cuda", generator=g)
    if case["rows"] == "runs":  # prompts' chunks, then decode rows
        tail = min(T - 1, 3)
        runs = (torch.arange(T - tail, device="cuda") * max(1, min(3, T // 1024))) // (T - tail)
        ids[: T - tail] = ids[runs]
    ids = torch.where(torch.rand((T,), device="cuda", generator=g) < case["none"], -1, ids)
    return x, A, B, scale, base, ids.int()


def _verify_inputs(case, seed):
    """Rows of B requests with 0 to `most` drafts each (how many goes by the case alone): probabilities,
    drafts drawn from the draft's (without draft probabilities: the likeliest token of a model near the
    target), uniform numbers."""
    g = _gen(seed, 13)
    B, V, dt = case["B"], case["V"], DTYPES[case["dt"]]
    n = torch.randint(0, case["most"] + 1, (B,), device="cuda", generator=_gen(B, 14))
    n[0] = case["most"]
    offsets = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = (n + 1).cumsum(0)
    R = int(offsets[-1])
    target = torch.empty((R, V), dtype=dt, device="cuda")
    probs = torch.empty((R, V), dtype=dt, device="cuda") if case["draft"] else None
    drafts = torch.empty((R,), dtype=torch.int64, device="cuda")
    for i in range(0, R, 64):
        m = min(64, R - i)
        l = case["sharp"] * _normal(g, m, V)
        near = l + 0.5 * _normal(g, m, V)
        target[i:i + m] = torch.softmax(l, 1).to(dt)
        q = torch.softmax(near, 1).to(dt)
        if case["draft"]:
            probs[i:i + m] = q
            drafts[i:i + m] = torch.multinomial(q.float(), 1, generator=g)[:, 0]
        else:
            drafts[i:i + m] = near.argmax(1)
    u = torch.rand((R,), device="cuda", generator=g)
    u_sample = torch.rand((B,), device="cuda", generator=g)
    return target, probs, drafts.int(), offsets, u, u_sample


def prepare(case, seed):
    st = dict(case)
    if case["op"] in ("sort", "combine"):
        st["inv"], st["weights"], st["tok"], st["rows"] = _moe_inputs(case, seed)
        if (case["op"] == "sort") != case["back"]:  # the caller's rows in expert order
            st["buffer"] = torch.zeros((st["inv"].numel(), case["d"]), dtype=DTYPES[case["dt"]], device="cuda")
    elif case["op"] == "adapters":
        st["x"], A, B, scale, st["base"], st["ids"] = _adapter_inputs(case, seed)
        if own:
            from decode_batches_gb300 import LowRankAdapters
            ad = LowRankAdapters(case["n"], case["N"], case["K"], case["r"], dtype=DTYPES[case["dt"]])
            for i in range(case["n"]):
                ad.set(i, A[i], B[i], scale[i])
            ad.allocate_workspace(case["T"])
            st["adapters"] = ad
        else:
            st["A"], st["B"], st["scale"] = A, B, scale
    else:
        (st["target"], st["probs"], st["drafts"], st["offsets"], st["u"], st["u_sample"]) = _verify_inputs(case, seed)
    return st


# ------------------------------------------------------------------------------------ plain forms
def _plain_spread(tok, inv, w, rows, out):
    """rows[inv[t,j]] = w[t,j] tok[t] and, where `rows` are given, <tok[t], rows[inv[t,j]]>."""
    x, used = tok.float(), inv >= 0
    v = x[:, None, :] * (1.0 if w is None else w[:, :, None])
    out[inv[used].long()] = v.expand(*inv.shape, x.shape[1])[used].to(out.dtype)
    if rows is None:
        return out
    z = rows[inv.clamp_min(0).long()].float()
    return out, (x[:, None, :] * z).sum(2).masked_fill(~used, 0.0)


def _plain_gather(rows, inv, w, tok, out_dtype, shared=None):
    """sum_j w[t,j] rows[inv[t,j]] and, where `tok` is given, <tok[t], rows[inv[t,j]]>."""
    z = rows[inv.clamp_min(0).long()].float().masked_fill((inv < 0)[:, :, None], 0.0)
    out = (z if w is None else z * w[:, :, None]).sum(1)
    if shared is not None:
        out = out + shared.float()
    out = out.to(out_dtype)
    return out if tok is None else (out, (tok.float()[:, None, :] * z).sum(2))


def _plain_adapters(st):
    x, ids, out = st["x"].float(), st["ids"], st["base"].float()
    if st["T"] <= 128:  # few rows: each with its own copy of its adapter
        a = ids.clamp_min(0).long()
        scale = torch.tensor(st["scale"], device=x.device)[a].masked_fill(ids < 0, 0.0)
        low = (st["A"][a].float() @ x[:, :, None]) * scale[:, None, None]
        return (out + (st["B"][a].float() @ low)[:, :, 0]).to(st["base"].dtype)
    for a in range(st["n"]):
        t = torch.nonzero(ids == a)[:, 0]
        out[t] += st["scale"][a] * ((x[t] @ st["A"][a].float().t()) @ st["B"][a].float().t())
    return out.to(st["base"].dtype)


def _plain_verify(st):
    p, q, drafts, offsets, u = st["target"], st["probs"], st["drafts"].long(), st["offsets"].long(), st["u"]
    R, V = p.shape
    first, n = offsets[:-1], offsets[1:] - offsets[:-1] - 1
    pd = p.gather(1, drafts[:, None])[:, 0].double()
    qd = q.gather(1, drafts[:, None])[:, 0].double() if q is not None else torch.ones_like(pd)
    ok = u.double() * qd < pd
    step = torch.arange(int(st["most"]), device=p.device)
    live = step[None] < n[:, None]
    passed = (ok[(first[:, None] + step).clamp_max(R - 1)] & live).long().cumprod(1).sum(1)
    row = first + passed
    at = p[row].double()
    if q is not None:
        rest = (at - q[row].double()).clamp_min(0.0)
    else:
        rest = at.scatter(1, drafts[row][:, None], 0.0)
    left = torch.where((passed < n)[:, None], rest, at)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, at)
    c = left.cumsum(1)
    token = (c <= st["u_sample"].double()[:, None] * c[:, -1:]).sum(1).clamp_max(V - 1)
    tokens = torch.full((R,), -1, dtype=torch.int32, device=p.device)
    request = torch.repeat_interleave(torch.arange(len(n), device=p.device), n + 1, output_size=R)
    keep = torch.arange(R, device=p.device) < row[request]
    tokens = torch.where(keep, drafts.int(), tokens)
    tokens[row] = token.int()
    return tokens, passed.int()


def run(st):
    op = st["op"]
    if own:
        import decode_batches_gb300 as lib
        if op == "sort":
            if st["back"]:
                return lib.sort_rows_backward(st["rows"], st["inv"], st["weights"], st["tok"] if st["w"] else None)
            return lib.sort_rows(st["tok"], st["inv"], st["weights"], out=st["buffer"])
        if op == "combine":
            if st["back"]:
                return lib.combine_rows_backward(st["tok"], st["inv"], st["weights"], st["rows"], out=st["buffer"])
            return lib.combine_rows(st["rows"], st["inv"], st["weights"], shared=st["tok"], out_dtype=DTYPES[st["out"]])
        if op == "adapters":
            return st["adapters"].forward(st["x"], st["ids"], st["base"])
        return lib.verify_drafts(st["target"], st["drafts"], st["offsets"], st["u"], st["u_sample"],
                                 draft_probs=st["probs"])
    if op == "sort":
        if st["back"]:
            return _plain_gather(st["rows"], st["inv"], st["weights"], st["tok"] if st["w"] else None, st["rows"].dtype)
        return _plain_spread(st["tok"], st["inv"], st["weights"], None, st["buffer"])
    if op == "combine":
        if st["back"]:
            return _plain_spread(st["tok"], st["inv"], st["weights"], st["rows"], st["buffer"])
        return _plain_gather(st["rows"], st["inv"], st["weights"], None, DTYPES[st["out"]], st["tok"])
    return _plain_adapters(st) if op == "adapters" else _plain_verify(st)


# ------------------------------------------------------------------------------------ bounds
def work(case):
    op = case["op"]
    if op in ("sort", "combine"):
        T, k, d = case["T"], min(case["k"], case["E"]), case["d"]
        rows = T * k * (1 - case["lost"])
        spread = (op == "sort") != case["back"]
        dots = case["w"] and case["back"]
        token = SIZE[case["out" if op == "combine" else "dt"]]
        moved = rows * SIZE[case["dt"]] * (2 if spread and dots else 1)      # rows in expert order, in and out
        moved += T * token * (1 if spread else 2 if dots or op == "combine" else 1)  # token rows, in and out
        idx = T * k * (4 + (4 if case["w"] else 0) + (4 if dots else 0))
        return {"bytes": moved * d + idx, "flops": rows * d * ((2 if case["w"] or not spread else 0) + (2 if dots else 0))}
    if op == "adapters":
        T, n, r, K, N = (case[c] for c in ("T", "n", "r", "K", "N"))
        rows = T * (1 - case["none"])
        touched = n * (1 - (1 - 1 / n) ** rows) if case["rows"] == "mixed" else min(n, rows, 6)
        return {"bytes": rows * K * 2 + 2 * T * N * SIZE[case["out"]] + T * 4 + touched * r * (K + N) * 2,
                "flops": 2 * rows * r * (K + N)}
    B, V, size = case["B"], case["V"], SIZE[case["dt"]]
    rows = B * (1 + case["most"] / 2)
    read = B * V * (2 if case["draft"] and case["most"] else 1)  # the target's row and, nearly always, the draft's
    return {"bytes": read * size + rows * (4 * 3 + 2 * 32) + B * 12, "flops": 3 * read}


# ------------------------------------------------------------------------------------ 64 bits
def _exact_moe(case, seed):
    inv, w, tok, rows = _moe_inputs(case, seed)
    T, k = inv.shape
    x, z = tok.double(), None if rows is None else rows.double()
    w64 = torch.ones((T, k), dtype=torch.float64, device="cuda") if w is None else w.double()
    dots = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    if (case["op"] == "sort") != case["back"]:
        out = torch.zeros((T * k, case["d"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            at = inv[t, j].long()
            out[at] = w64[t, j, None] * x[t]
            if case["back"] and case["w"]:
                dots[t, j] = torch.einsum("td,td->t", x[t], z[at])
    else:
        out = torch.zeros((T, case["d"]), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            at = inv[t, j].long()
            out[t] += w64[t, j, None] * z[at]
            if case["back"] and case["w"]:
                dots[t, j] = torch.einsum("td,td->t", x[t], z[at])
        if case["op"] == "combine":
            out += x
    return (out, dots) if case["back"] and case["w"] else out


def _exact_verify(case, seed):
    target, probs, drafts, offsets, u, u_sample = _verify_inputs(case, seed)
    drafts, offsets, u, u_sample = (v.tolist() for v in (drafts, offsets, u, u_sample))
    tokens, accepted = [-1] * len(drafts), []
    pd = target.double().gather(1, torch.tensor(drafts, device="cuda")[:, None])[:, 0].tolist()
    qd = probs.double().gather(1, torch.tensor(drafts, device="cuda")[:, None])[:, 0].tolist() if probs is not None else [1.0] * len(pd)
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        r = lo
        while r < hi - 1 and u[r] * qd[r] < pd[r]:
            tokens[r] = drafts[r]
            r += 1
        p = target[r].double()
        if r < hi - 1:
            q = torch.zeros_like(p)
            if probs is None:
                q[drafts[r]] = p[drafts[r]]
            else:
                q = probs[r].double()
            rest = torch.maximum(p - q, torch.zeros_like(p))
            p = rest if float(rest.sum()) > 0 else p
        c = torch.cumsum(p, 0)
        tokens[r] = min(int(torch.searchsorted(c, u_sample[b] * c[-1], right=True)), len(p) - 1)
        accepted.append(r - lo)
    whole = lambda v: torch.tensor(v, dtype=torch.float64, device="cuda")
    return whole(tokens), whole(accepted)


def exact(case, seed):
    if case["op"] in ("sort", "combine"):
        return _exact_moe(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, seed)
    x, A, B, scale, base, ids = _adapter_inputs(case, seed)
    out = base.double()
    for t0 in range(0, len(ids), 1024):
        for a in set(ids[t0:t0 + 1024].tolist()) - {-1}:
            t = t0 + torch.nonzero(ids[t0:t0 + 1024] == a)[:, 0]
            low = torch.einsum("tk,rk->tr", x[t].double(), A[a].double())
            out[t] += scale[a] * torch.einsum("tr,nr->tn", low, B[a].double())
    return out
