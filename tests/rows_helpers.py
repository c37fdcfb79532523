"""Plain 64-bit forms of the row moves, and how far a kernel's rounded result may be from them."""
import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24                                        # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    """Half the spacing of the type's smallest values."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def assignments(T, k, seed, lost=0.0, spare=0):
    """inv [T][k]: a random order of the kept assignments over T * k + spare rows, -1 for dropped ones."""
    g = torch.Generator().manual_seed(seed)
    rows = torch.randperm(T * k + spare, generator=g)[: T * k].view(T, k).int()
    return torch.where(torch.rand((T, k), generator=g) < lost, torch.tensor(-1, dtype=torch.int32), rows)


def tensor(rows, d, dtype, seed, pad=0, shift=0):
    """(the tensor on the GPU with a row pitch of d + pad that starts `shift` elements into its memory)"""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((rows, d), generator=g) * torch.exp(torch.randn((rows, 1), generator=g))).to(dtype)
    buf = torch.full((rows * (d + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    out = buf[shift:].view(rows, d + pad)[:, :d]
    out.copy_(x)
    return out


def spread_ref(x, inv, w, n_rows):
    """(fp64 rows, which rows are named)"""
    x = x.double().cpu()
    out, named = torch.zeros((n_rows, x.shape[1]), dtype=torch.float64), torch.zeros(n_rows, dtype=torch.bool)
    for t in range(inv.shape[0]):
        for j in range(inv.shape[1]):
            r = int(inv[t, j])
            if 0 <= r < n_rows:
                out[r] = x[t] * (1.0 if w is None else float(w[t, j]))
                named[r] = True
    return out, named


def gather_ref(rows, inv, w, T):
    """(fp64 sums, sums of the magnitudes) of the named rows"""
    rows = rows.double().cpu()
    n_rows = rows.shape[0]
    used = (inv >= 0) & (inv < n_rows)
    z = torch.zeros((*inv.shape, rows.shape[1]), dtype=torch.float64)
    z[used] = rows[inv[used].long()]
    if w is not None:
        z = z * w.double()[:, :, None]
    return z.sum(1), z.abs().sum(1)


def dots_ref(x, rows, inv):
    x, rows = x.double().cpu(), rows.double().cpu()
    used = (inv >= 0) & (inv < rows.shape[0])
    out, mag = torch.zeros(inv.shape, dtype=torch.float64), torch.zeros(inv.shape, dtype=torch.float64)
    for t, j in torch.nonzero(used).tolist():
        p = x[t] * rows[int(inv[t, j])]
        out[t, j], mag[t, j] = p.sum(), p.abs().sum()
    return out, mag


def close(got, ref, slack, dtype):
    """|got - ref| <= slack (of the fp32 arithmetic) and the final rounding of a value that far off."""
    got = got.double().cpu()
    room = slack + half_step(dtype) * (ref.abs() + slack) + floor_of(dtype)
    worst = float(((got - ref).abs() - room).max()) if got.numel() else 0.0
    assert torch.isfinite(got).all() and worst <= 0, worst


def dot_slack(d, mag):
    """Sums of d products: a lane adds up at most 8 ceil(d / 2048) + 8 of them (8 columns a span of 256, spans
    shared by up to 8 warps), five steps join the lanes and eight the warps; every step rounds once."""
    return (8 * -(-d // 256) + 13) * U32 * (1 + 2.0 ** -10) * mag
