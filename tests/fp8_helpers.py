"""Plain 64-bit forms of the 8-bit operators, for the tests.  The quantisation rule is fp32 by
definition (scale, reciprocal and product each rounded once), so the codes are reproduced exactly;
everything after the codes is fp64."""
import torch

BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def quantize_rows_ref(x):
    """x [T][K] (any float type, CPU) -> codes fp64 [T][K], scales fp64 [T][nb]."""
    T, K = x.shape
    b = torch.zeros((T, blocks(K) * BLOCK), dtype=torch.float32)
    b[:, :K] = x.float()
    b = b.view(T, -1, BLOCK)
    s = torch.maximum(b.abs().amax(2) / 448.0, torch.tensor(2.0 ** -126))
    q = (b * (1.0 / s)[:, :, None]).to(torch.float8_e4m3fn).double()
    return q.view(T, -1)[:, :K], s.double()


def quantize_weight_ref(w):
    rows, K = w.shape
    rb, kb = blocks(rows), blocks(K)
    b = torch.zeros((rb * BLOCK, kb * BLOCK), dtype=torch.float32)
    b[:rows, :K] = w.float()
    v = b.view(rb, BLOCK, kb, BLOCK)
    s = torch.maximum(v.abs().amax(dim=(1, 3)) / 448.0, torch.tensor(2.0 ** -126))
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
