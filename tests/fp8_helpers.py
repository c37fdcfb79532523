"""Plain 64-bit forms of the 8-bit operators, for the tests.  The quantisation rule is fp32 by
definition (scale, reciprocal and product each rounded once), so the codes are reproduced exactly;
everything after the codes is fp64."""
import torch

BLOCK = 128
R448 = torch.tensor(1.0) / 448.0            # fp32


def blocks(n):
    return -(-n // BLOCK)


def quantize_rows_ref(x):
    """x [T][K] (any float type, CPU) -> codes fp64 [T][K], scales fp64 [T][nb]."""
    T, K = x.shape
    b = torch.zeros((T, blocks(K) * BLOCK), dtype=torch.float32)
    b[:, :K] = x.float()
    b = b.view(T, -1, BLOCK)
    s = torch.maximum(b.abs().amax(2) * R448, torch.tensor(2.0 ** -126))
    q = (b * (1.0 / s)[:, :, None]).to(torch.float8_e4m3fn).double()
    return q.view(T, -1)[:, :K], s.double()


def quantize_weight_ref(w):
    rows, K = w.shape
    rb, kb = blocks(rows), blocks(K)
    b = torch.zeros((rb * BLOCK, kb * BLOCK), dtype=torch.float32)
    b[:rows, :K] = w.float()
    v = b.view(rb, BLOCK, kb, BLOCK)
    s = torch.maximum(v.abs().amax(dim=(1, 3)) * R448, torch.tensor(2.0 ** -126))
    q = (v * (1.0 / s)[:, None, :, None]).reshape(b.shape)[:rows, :K].to(torch.float8_e4m3fn)
    return q, s


def expand(s, rows, K):
    return s.double().repeat_interleave(BLOCK, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :K]


def product_ref(xq, xs, wq, ws):
    """fp64 product of quantised operands and the sum of its terms' magnitudes."""
    N, K = wq.shape
    a = xq.double() * xs.double().repeat_interleave(BLOCK, 1)[:, :K]
    w = wq.double() * expand(ws, N, K)
    return a @ w.T, a.abs() @ w.abs().T


def sum_tolerance(K):
    """Of the product relative to the sum of its terms' magnitudes.  The products of two e4m3 codes
    are exact in fp32.  A block's 128 of them are added by the tensor core in fp32, each step off
    by at most one unit in the last place (2^-23, truncation included); then each block is scaled
    (the scale itself is a rounded product: 2^-24) and added with one rounding (2^-24 each)."""
    return 128 * 2.0 ** -23 + (blocks(K) + 2) * 2.0 ** -24


def random_weight(N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((N, K), generator=g) * K ** -0.5
    return quantize_weight_ref(w)


def random_rows(T, K, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    return x.to(dtype)


# ---- the expert FFN ---------------------------------------------------------------------------
SWIGLU_REL = 2.0 ** -18   # fast exp and division of the fp32 SwiGLU, with room for large |gate|


def e4m3_near(v, dv):
    """Of fp64 values v (|v| <= 448) that are known to dv: the e4m3 spacing where an error of dv can
    change the rounding, else 0."""
    step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    pos = v.abs() / step
    to_tie = (pos - torch.floor(pos) - 0.5).abs() * step     # distance to the nearest rounding boundary
    return torch.where(to_tie <= dv, step, torch.zeros_like(step))


def quantize_known_to(h, dh):
    """fp64 h known to dh -> dequantised values, and how far they may be off: one step where the
    rounding is open, and the scale's own error."""
    rows, K = h.shape
    pad = (blocks(K) * BLOCK - K)
    hp = torch.nn.functional.pad(h, (0, pad)).view(rows, -1, BLOCK)
    dp = torch.nn.functional.pad(dh, (0, pad)).view(rows, -1, BLOCK)
    q, s = quantize_rows_ref(h)                     # codes of the fp32-rounded h
    rel = 2.0 ** -22 + (dp.amax(2) / hp.abs().amax(2).clamp_min(1e-300)).clamp_max(1.0)
    v = hp / s[:, :, None]
    dv = dp / s[:, :, None] + v.abs() * rel[:, :, None]
    off = e4m3_near(v.clamp(-448, 448), dv) * s[:, :, None]
    deq = (torch.nn.functional.pad(q, (0, pad)).view(rows, -1, BLOCK) * s[:, :, None])
    off = off + deq.abs() * rel[:, :, None]
    return deq.view(rows, -1)[:, :K], off.view(rows, -1)[:, :K]


def ffn_ref(x, g, u, dn):
    """One expert on rows x: (y fp64, tolerance of an fp32 evaluation before y's own rounding).
    g, u, dn: (codes, scales) of gate [f][d], up [f][d], down [d][f]."""
    (gq, gs), (uq, us), (dq, ds) = g, u, dn
    xq, xs = quantize_rows_ref(x)
    gv, gm = product_ref(xq, xs, gq, gs)
    uv, um = product_ref(xq, xs, uq, us)
    e = sum_tolerance(gq.shape[1])
    dg, du = e * gm, e * um
    sig = torch.sigmoid(gv)
    h = gv * sig * uv
    slope = sig * (1 + gv.abs() * (1 - sig))        # bounds |d silu| with room for dg's own size
    dh = (slope * dg * 1.1 + dg * dg) * (uv.abs() + du) + (gv * sig).abs() * du + SWIGLU_REL * (1 + gv.abs()) * h.abs()
    hq, hoff = quantize_known_to(h, dh)
    w = dq.double() * expand(ds, *dq.shape)
    y = hq @ w.T
    tol = hoff @ w.abs().T + sum_tolerance(dq.shape[1]) * (hq.abs() @ w.abs().T)
    return y, tol


def layer_ref(x, ids, gates, gate, up, down, shared=None):
    """out[t] = sum_j gates[t, j] FFN_ids[t, j](x[t]) (+ shared) in fp64, and its tolerance: the
    experts', fp16 y (2^-11), the fp32 sum over slots, bf16 out (2^-8).  Invalid or repeated ids
    contribute nothing."""
    T, k = ids.shape
    E = gate[0].shape[0]
    out = torch.zeros((T, x.shape[1]), dtype=torch.float64)
    tol = torch.zeros_like(out)
    for e in range(E):
        sel = [(t, j) for t in range(T) for j in range(k) if int(ids[t, j]) == e and e not in ids[t, :j].tolist()]
        if not sel:
            continue
        t = torch.tensor([a for a, _ in sel])
        w = gates[t, torch.tensor([b for _, b in sel])].double()[:, None]
        y, dy = ffn_ref(x[t], (gate[0][e], gate[1][e]), (up[0][e], up[1][e]), (down[0][e], down[1][e]))
        out[t] += w * y
        tol[t] += w.abs() * (dy + (y.abs() + dy) * 2.0 ** -11 + 2.0 ** -24) + (k + 1) * 2.0 ** -24 * (w * y).abs()
    if shared is not None:
        out, tol = out + shared[0], tol + shared[1]
    return out, tol + 2.0 ** -8 * (out.abs() + tol)


def random_experts(E, f, d, seed):
    def many(rows, K, s0):
        qs = [random_weight(rows, K, s0 + e) for e in range(E)]
        return torch.stack([q for q, _ in qs]), torch.stack([s for _, s in qs])
    return many(f, d, seed), many(f, d, seed + 1000), many(d, f, seed + 2000)
