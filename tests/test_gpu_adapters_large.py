"""Low-rank adapters at the sizes where the larger steps' kernels change: all slots in use, tiles of every size, one CTA of
sixteen warps an SM; against the formula in 64 bits (on the GPU)."""
import pytest
import torch

from rows_helpers import TYPES, U32, floor_of, half_step

pytestmark = pytest.mark.gpu


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


def run(T, n, r, K, N, dtype, out_dtype, ids, seed, used=None, base=True, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=g)
    used = range(n) if used is None else used
    ad = pkg().LowRankAdapters(n, N, K, r, dtype)
    A, B = (rnd(n, r, K) * K ** -0.5).to(dtype), rnd(n, N, r).to(dtype)
    for i in used:
        ad.set(i, A[i], B[i], 0.5)
    ad.allocate_workspace(T)
    x = torch.empty((T, K + pad), dtype=dtype, device="cuda")[:, :K]
    x.copy_(rnd(T, K))
    b = rnd(T, N).to(out_dtype) if base else None
    ids = ids.cuda().int()
    got = ad.forward(x, ids, b, out_dtype=out_dtype)
    again = ad.forward(x, ids, b, out_dtype=out_dtype)
    assert torch.equal(got, again)
    ref = torch.zeros((T, N), dtype=torch.float64, device="cuda") if b is None else b.double()
    plain, slack = ref.clone(), torch.zeros_like(ref)
    live = torch.zeros(T, dtype=torch.bool, device="cuda")
    for a in used:
        t = torch.nonzero(ids == a)[:, 0]
        if not len(t):
            continue
        live[t] = True
        u, mag = 0.5 * x[t].double() @ A[a].double().T, 0.5 * x[t].double().abs() @ A[a].double().abs().T
        du = (K + 64) * 2 * U32 * mag + 2.0 ** -16 * u.abs().amax(1, keepdim=True)
        ref[t] += u @ B[a].double().T
        slack[t] += (du + (2 * r + 64) * 2 * U32 * u.abs()) @ B[a].double().abs().T
    slack = (slack + U32 * ref.abs()) * (1 + 2.0 ** -8)
    room = slack + half_step(out_dtype) * (ref.abs() + slack) + floor_of(out_dtype)
    assert torch.isfinite(got).all() and float(((got.double() - ref).abs() - room).max()) <= 0
    assert torch.equal(got[~live].double(), plain[~live])
    if b is not None:
        inplace = b.clone()
        ad.forward(x, ids, inplace, out=inplace)
        assert torch.equal(inplace, got)
    assert ad.device_error() == 0


@pytest.mark.parametrize("T", [60, 300, 1024, 1025, 1500])
def test_all_1024_slots(T):
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-1, 1024, (T,), generator=g)
    ids[: T // 3] = 1023
    ids[T // 3: T // 2] = -1
    run(T, 1024, 4, 40, 48, torch.bfloat16, torch.float32, ids, T, used=range(0, 1024, 3))


@pytest.mark.parametrize("ot", sorted(TYPES))
@pytest.mark.parametrize("r", [16, 24, 64, 128])
@pytest.mark.parametrize("T", [3500, 3501, 9000])
def test_both_cuts_of_large_steps(T, r, ot):
    g = torch.Generator().manual_seed(T + r)
    shares = torch.tensor([0.02, 0.5, 0.01, 0.2, 0.07, 0.1, 0.1])
    ids = torch.multinomial(shares, T, replacement=True, generator=g) - 1
    run(T, 6, r, 200, 264, torch.float16 if r == 24 else torch.bfloat16, TYPES[ot], ids, r)


@pytest.mark.parametrize("T,N,K,pad", [(4000, 131, 65, 1), (4000, 1025, 32, 0), (2000, 33, 1000, 3), (700, 259, 129, 0)])
def test_odd_widths(T, N, K, pad):
    ids = torch.randint(-1, 9, (T,), generator=torch.Generator().manual_seed(1))
    run(T, 9, 32, K, N, torch.bfloat16, torch.bfloat16, ids, 2, pad=pad)
    run(T, 9, 32, K, N, torch.float16, torch.float32, ids, 3, base=False, pad=pad)


@pytest.mark.parametrize("count", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 385])
def test_tiles_of_every_size(count):
    """One slot with `count` rows among others that fill the step."""
    T = 1200
    ids = torch.full((T,), -1)
    ids[torch.randperm(T, generator=torch.Generator().manual_seed(count))[:count]] = 3
    ids[ids < 0] = torch.where(torch.rand(int((ids < 0).sum()), generator=torch.Generator().manual_seed(5)) < 0.3, 7, -1)
    run(T, 8, 16, 64, 136, torch.bfloat16, torch.float32, ids, count)
    run(600, 8, 16, 64, 136, torch.bfloat16, torch.float32, ids[:600], count)


def test_one_slot_and_wide_products():
    ids = torch.zeros(5000, dtype=torch.int64)
    run(5000, 1, 64, 2048, 2048, torch.bfloat16, torch.bfloat16, ids, 1)
    run(300, 1, 8, 64, 40000, torch.bfloat16, torch.bfloat16, ids[:300], 2)
    run(9, 1, 8, 40000, 64, torch.float16, torch.float16, ids[:9], 3)
    run(300, 1, 8, 40000, 64, torch.float16, torch.float16, ids[:300], 4)
