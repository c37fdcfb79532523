"""Measured cases of the operators around 8-bit experts: scored expert routing, the block-scaled
8-bit matrix product, and the expert FFN on 8-bit weights.

    route    logits -> expert ids and weights: softmax or sigmoid scores, a balance bias that only
             selects, expert groups, top-k, renormalised and scaled weights
    linear   out = x W^T with both operands in e4m3: x quantised in blocks of 1 x 128, W given in
             blocks of 128 x 128 with an fp32 scale each
    experts  out[t] = sum_j gate[t,j] W_d,e (silu(W_g,e x_t) * (W_u,e x_t)), e = ids[t,j], the same
             8-bit product for all three matrices, the hidden vector quantised like x

`own` false: elementary torch operations in fp32.  `own` true: the calls of this package.
"""
import math

import torch

own = False

BLOCK = 128          # elements that share a scale
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of four sequences: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="route_decode", op="route", T=4, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2,
             renorm=True, scale=2.5, masked=0),
        # a verify batch over a large expert count, plain softmax scores, some experts switched off
        dict(name="route_verify", op="route", T=48, E=384, k=8, score="softmax", bias=False, groups=1, keep=1, top=1,
             renorm=True, scale=1.0, masked=5),
        # a mixed step: 2048 prefill rows and three decode rows
        dict(name="route_mixed", op="route", T=2051, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2,
             renorm=True, scale=2.5, masked=0),
        # the largest mixed step, groups ranked by their best expert, weights not renormalised
        dict(name="route_large", op="route", T=8195, E=384, k=6, score="softmax", bias=False, groups=12, keep=5, top=1,
             renorm=False, scale=16.0, masked=0),
        # one token through a projection: the weights' bytes are all there is
        dict(name="linear_token", op="linear", T=1, K=4096, N=4096, x="bf16", out="bf16", pad=0),
        # a verify batch, fp32 out (logits or a residual kept in 32 bits), x a slice of a wider tensor
        dict(name="linear_verify", op="linear", T=48, K=2048, N=4096, x="bf16", out="fp32", pad=64),
        # sizes that divide into nothing: ragged rows, a last block of K and of N that is partial
        dict(name="linear_ragged", op="linear", T=517, K=1000, N=1337, x="fp16", out="bf16", pad=0),
        # a prefill step of 8192 rows: the tensor cores' rate is the bound
        dict(name="linear_prefill", op="linear", T=8192, K=4096, N=4096, x="bf16", out="bf16", pad=0),
        # one decode step of four sequences
        dict(name="experts_decode", op="experts", T=4, E=256, k=8, d=2048, f=512, zipf=0.0),
        # a verify batch over many wide experts
        dict(name="experts_verify", op="experts", T=48, E=384, k=8, d=4096, f=1024, zipf=0.0),
        # a mixed step, near-uniform load, about 64 rows an expert
        dict(name="experts_mixed", op="experts", T=2051, E=256, k=8, d=2048, f=512, zipf=0.0),
        # a mixed step with skewed expert popularity
        dict(name="experts_skewed", op="experts", T=2051, E=384, k=8, d=4096, f=1024, zipf=1.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "linear", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8, 12])
        E = groups * rng.randrange(8, 49) if groups > 1 else rng.randrange(16, 513)
        keep = rng.randint(max(1, groups // 3), groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op="route", T=_log(rng, 1, 8195 * 384 // max(E, 384)), E=E, k=k, score=score,
                    bias=score == "sigmoid" and rng.random() < 0.7, groups=groups, keep=keep,
                    top=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]),
                    masked=rng.choice([0, 0, 3]) if groups == 1 and E >= k + 3 else 0)
    if op == "linear":
        K, N = _log(rng, 128, 4096), _log(rng, 64, 4096)
        if rng.random() < 0.5:
            K, N = -(-K // 128) * 128, -(-N // 128) * 128
        else:
            K, N = -(-K // 8) * 8, N | 1
        K, N = K - 8 * (K == 3072), N - 1 * (N == 3072)
        T = _log(rng, 1, 8192)
        return dict(op="linear", T=T - (T == 3072), K=K, N=N, x=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    out=rng.choice(["bf16", "bf16", "fp32"]), pad=rng.choice([0, 0, 64]))
    d = rng.choice([512, 1024, 1000, 2048, 2048, 4096])
    f = rng.choice([128, 256, 264, 512, 512, 1024])
    E = _log(rng, 8, 384)
    T = _log(rng, 1, 2051)
    return dict(op="experts", T=T, E=E, k=rng.randint(1, 8), d=d, f=f, zipf=rng.choice([0.0, 0.0, 1.1]))


# ------------------------------------------------------------------------------------ inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    return g


def _weights(n, rows, K, g):
    """n matrices [rows][K] ~ N(0, 1/K) as e4m3 codes and fp32 scales of 128 x 128 blocks."""
    rb, kb = -(-rows // BLOCK), -(-K // BLOCK)
    q = torch.empty((n, rows, K), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((n, rb, kb), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 28) // (rows * K))
    for i in range(0, n, step):
        m = min(step, n - i)
        w = torch.zeros((m, rb * BLOCK, kb * BLOCK), device="cuda")
        w[:, :rows, :K] = torch.randn((m, rows, K), device="cuda", generator=g) * K ** -0.5
        b = w.view(m, rb, BLOCK, kb, BLOCK)
        sc = (b.abs().amax(dim=(2, 4)) / E4M3_MAX).clamp_min(SCALE_MIN)
        b = b * (1.0 / sc)[:, :, None, :, None]
        q[i:i + m] = b.reshape(w.shape)[:, :rows, :K].to(torch.float8_e4m3fn)
        s[i:i + m] = sc
    return q, s


def _activations(T, K, dtype, pad, g):
    """Rows with a token's own magnitude and a few loud channels, as hidden states have."""
    x = torch.randn((T, K + pad), device="cuda", generator=g)
    x *= torch.exp(0.3 * torch.randn((T, 1), device="cuda", generator=g))
    x *= torch.where(torch.rand((K + pad,), device="cuda", generator=g) < 0.01, 8.0, 1.0)
    return x.to(dtype)[:, :K]


def _route_inputs(case, seed):
    g = _gen(seed, 1)
    T, E = case["T"], case["E"]
    bias = 0.001 * torch.randint(-50, 51, (E,), device="cuda", generator=g).float() if case["bias"] else None
    off = torch.randperm(E, device="cuda", generator=g)[: case["masked"]]
    logits = torch.empty((T, E), device="cuda")
    redo = torch.ones(T, dtype=torch.bool, device="cuda")
    # Rows in which two candidates (or two groups) are too close for 32 bits to tell apart are
    # drawn again, so that the ids are those of the formula in any precision.
    for _ in range(8):
        fresh = torch.randn((T, E), device="cuda", generator=g)
        fresh[:, off] = -math.inf
        logits = torch.where(redo[:, None], fresh, logits)
        key, gs = _route_keys64(logits, bias, case)
        near = 4e-6 * torch.where(key.isfinite(), key.abs(), 0.0).amax(1, keepdim=True)
        top = key.sort(dim=1, descending=True).values[:, : case["k"] + 1]
        redo = ((top[:, :-1] - top[:, 1:]).abs() < near).any(1)
        if gs is not None and case["keep"] < case["groups"]:
            o = gs.sort(dim=1, descending=True).values
            redo |= (o[:, case["keep"] - 1] - o[:, case["keep"]]) < 2 * near[:, 0]
    return logits, bias


def _route_keys64(logits, bias, case):
    l = logits.double()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    key = s if bias is None else s + bias.double()
    key = key.masked_fill(l == -math.inf, -math.inf)
    if case["groups"] == 1:
        return key, None
    per = key.view(key.shape[0], case["groups"], -1)
    gs = per.sort(dim=2, descending=True).values[:, :, : case["top"]].sum(2)
    kept = gs.sort(dim=1, descending=True, stable=True).indices[:, : case["keep"]]
    dead = torch.ones_like(gs, dtype=torch.bool).scatter(1, kept, False)
    return per.masked_fill(dead[:, :, None], -math.inf).reshape(key.shape), gs


def _linear_inputs(case, seed):
    g = _gen(seed, 2)
    q, s = _weights(1, case["N"], case["K"], g)
    return _activations(case["T"], case["K"], DTYPES[case["x"]], case["pad"], g), q[0], s[0]


def _experts_inputs(case, seed):
    g = _gen(seed, 3)
    T, E, k, d, f = case["T"], case["E"], min(case["k"], case["E"]), case["d"], case["f"]
    ws = _weights(E, f, d, g) + _weights(E, f, d, g) + _weights(E, d, f, g)
    logits = torch.randn((T, E), device="cuda", generator=g)
    logits -= case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda").float())
    top = logits.topk(k, dim=1)
    return _activations(T, d, torch.bfloat16, 0, g), top.indices.int(), torch.softmax(top.values, 1), ws


def prepare(case, seed):
    state = dict(case)
    if case["op"] == "route":
        state["logits"], state["balance"] = _route_inputs(case, seed)
        if own:
            from decode_batches_gb300 import MoePlan
            plan = MoePlan(case["E"], case["k"], 2048, 512)
            plan.set_routing(case["score"], bias=state["balance"], n_groups=case["groups"], topk_groups=case["keep"],
                             group_top=case["top"], renormalize=case["renorm"], scale=case["scale"])
            state["plan"] = plan
    elif case["op"] == "linear":
        state["act"], state["q"], state["s"] = _linear_inputs(case, seed)
        if own:
            from decode_batches_gb300 import Fp8Linear
            lin = Fp8Linear(case["N"], case["K"])
            lin.set_weights(state["q"], state["s"])
            lin.allocate_workspace(case["T"])
            state["linear"] = lin
    else:
        state["act"], state["ids"], state["gates"], state["ws"] = _experts_inputs(case, seed)
        if own:
            from decode_batches_gb300 import MoePlan
            (qg, sg, qu, su, qd, sd) = state.pop("ws")
            plan = MoePlan(case["E"], state["ids"].shape[1], case["d"], case["f"], weight_dtype="fp8")
            plan.set_weights(torch.zeros((case["E"], case["d"]), device="cuda"), None, qg, qu, qd, sg, su, sd)
            plan.allocate_workspace(case["T"])
            state["plan"] = plan
    return state


# ------------------------------------------------------------------------------------ plain forms
def _dequantised(q, s):
    """[n][rows][K] codes and [n][rows/128][K/128] scales -> fp32."""
    s = s.repeat_interleave(BLOCK, 1)[:, : q.shape[1]].repeat_interleave(BLOCK, 2)[:, :, : q.shape[2]]
    return q.float() * s


def _quantised(x):
    """fp32 values of x after the e4m3 rounding in blocks of 1 x 128."""
    K = x.shape[-1]
    b = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    s = (b.abs().amax(-1, keepdim=True) / E4M3_MAX).clamp_min(SCALE_MIN)
    return ((b * (1.0 / s)).to(torch.float8_e4m3fn).float() * s).flatten(-2)[..., :K]


def _plain_route(st):
    l = st["logits"]
    if st["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    key = s if st["balance"] is None else s + st["balance"]
    key = key.masked_fill(l == -math.inf, -math.inf)
    if st["groups"] > 1:
        per = key.view(key.shape[0], st["groups"], -1)
        gs = per.sort(dim=2, descending=True).values[:, :, : st["top"]].sum(2)
        kept = gs.sort(dim=1, descending=True, stable=True).indices[:, : st["keep"]]
        dead = torch.ones_like(gs, dtype=torch.bool).scatter(1, kept, False)
        key = per.masked_fill(dead[:, :, None], -math.inf).reshape(key.shape)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, : st["k"]]
    w = s.gather(1, ids).masked_fill(key.gather(1, ids) == -math.inf, 0.0)
    if st["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return ids.int(), w * st["scale"]


def _plain_experts(st):
    x, ids, gates = st["act"], st["ids"].long(), st["gates"]
    qg, sg, qu, su, qd, sd = st["ws"]
    E, (T, k) = st["E"], ids.shape
    flat = ids.reshape(-1)
    order = flat.sort(stable=True).indices
    counts = torch.zeros(E, dtype=torch.long, device=x.device).scatter_add_(0, flat, torch.ones_like(flat))
    first = counts.cumsum(0) - counts
    e = flat[order]
    slot = torch.arange(T * k, device=x.device) - first[e]
    rows = torch.zeros((E, int(counts.max()), x.shape[1]), device=x.device)
    rows[e, slot] = _quantised(x)[order // k]
    gate = rows @ _dequantised(qg, sg).transpose(1, 2)
    h = gate / (1.0 + torch.exp(-gate)) * (rows @ _dequantised(qu, su).transpose(1, 2))
    y = _quantised(h) @ _dequantised(qd, sd).transpose(1, 2)
    back = torch.empty((T * k, x.shape[1]), device=x.device)
    back[order] = y[e, slot]
    return (back.view(T, k, -1) * gates[:, :, None]).sum(1).to(torch.bfloat16)


def run(state):
    op = state["op"]
    if own:
        if op == "route":
            return state["plan"].route_logits(state["logits"])
        if op == "linear":
            return state["linear"].forward(state["act"], out_dtype=DTYPES[state["out"]])
        return state["plan"].forward_routed(state["act"], state["ids"], state["gates"])
    if op == "route":
        return _plain_route(state)
    if op == "linear":
        w = _dequantised(state["q"][None], state["s"][None])[0]
        return (_quantised(state["act"]) @ w.t()).to(DTYPES[state["out"]])
    return _plain_experts(state)


# ------------------------------------------------------------------------------------ bounds
def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        return {"bytes": T * E * 4 + T * k * 8 + (E * 4 if case["bias"] else 0), "flops": T * E * 4}
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        scales = -(-K // BLOCK) * -(-N // BLOCK) * 4
        return {"bytes": T * K * size[case["x"]] + N * K + scales + T * N * size[case["out"]], "flops": 2 * T * K * N}
    E, k, d, f = case["E"], min(case["k"], case["E"]), case["d"], case["f"]
    if case["zipf"]:  # the expected number of experts that get a row
        p = [(e + 1) ** -case["zipf"] for e in range(E)]
        touched = sum(1 - (1 - min(1.0, k * q / sum(p))) ** T for q in p)
    else:
        touched = E * (1 - (1 - k / E) ** T)
    expert = 3 * d * f * (1 + 4 / BLOCK ** 2)
    return {"bytes": touched * expert + 2 * T * d * 2 + T * k * 8, "flops": T * k * 6 * d * f}


# ------------------------------------------------------------------------------------ 64 bits
def _exact_rows(x):
    """The values of x after quantisation, in fp64: the scale is an fp32 number by definition (so
    are the products with its reciprocal); the rounding to e4m3 is written out."""
    T, K = x.shape
    b = torch.zeros((T, -(-K // BLOCK) * BLOCK), dtype=torch.float32, device=x.device)
    b[:, :K] = x
    b = b.view(T, -1, BLOCK)
    s = torch.clamp(b.abs().max(2, keepdim=True).values / E4M3_MAX, min=SCALE_MIN)
    v = (b * (1.0 / s)).double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)  # spacing of e4m3 at |v|
    v = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)                 # ties to even
    return (v * s.double()).view(T, -1)[:, :K]


def _exact_matrix(q, s):
    out = q.double()
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            out[BLOCK * i:BLOCK * i + BLOCK, BLOCK * j:BLOCK * j + BLOCK] *= s[i, j].double()
    return out


def exact(case, seed):
    if case["op"] == "route":
        logits, bias = _route_inputs(case, seed)
        key, _ = _route_keys64(logits, bias, case)
        ids = torch.topk(key, case["k"], dim=1, sorted=True).indices
        l = logits.double()
        s = 1 / (1 + torch.exp(-l)) if case["score"] == "sigmoid" else torch.softmax(l, 1)
        w = torch.gather(s, 1, ids)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return None, w * case["scale"]
    if case["op"] == "linear":
        x, q, s = _linear_inputs(case, seed)
        return _exact_rows(x) @ _exact_matrix(q, s).T
    x, ids, gates, ws = _experts_inputs(case, seed)
    xr = _exact_rows(x.float())
    out = torch.zeros((case["T"], case["d"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        g = xr[t] @ _exact_matrix(ws[0][e], ws[1][e]).T
        u = xr[t] @ _exact_matrix(ws[2][e], ws[3][e]).T
        h = g * torch.sigmoid(g) * u
        y = _exact_rows(h.float()) @ _exact_matrix(ws[4][e], ws[5][e]).T
        out[t] += gates[t, j].double()[:, None] * y
    return out
