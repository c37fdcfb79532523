"""How many bits of u = s A x an fp32 result of the adapters has, read off directly: B is the identity, so a feature is one
element of u."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


@pytest.mark.parametrize("rank,pad_to", [(1, 16), (16, 16), (7, 32), (32, 32), (64, 64), (3, 128), (128, 128)])
@pytest.mark.parametrize("T", [1, 40, 256, 300, 1000, 2100, 4000])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_u_keeps_its_bits(T, rank, pad_to, dt):
    """u[j] = a0 x0 + a1 x1 with 8-bit factors whose products lie 2^-9 apart: 24 bits or so.  Sums with two terms that are
    not zero, then one product a term of u (in bf16 three, together all 24 bits; in fp16 two, half a step of the second of
    which is 2^-23 of the row's largest u): each of these steps keeps 24 bits of the larger operand, 2^-23 of it is lost at
    most; u itself is exact in 64 bits."""
    K, N = 2, 128
    g = torch.Generator().manual_seed(T + rank)
    draw = lambda *s: (torch.randint(128, 256, s, generator=g) / 128 * torch.where(torch.rand(s, generator=g) < 0.5, -1.0, 1.0))
    A, x = draw(rank, K), draw(T, K)
    A[:, 1] *= 2.0 ** -9
    B = torch.zeros(N, rank)
    B[torch.arange(rank), torch.arange(rank)] = 1.0
    ad = pkg().LowRankAdapters(2, N, K, pad_to, dt)
    ad.set(1, A.to(dt).cuda(), B.to(dt).cuda(), 2.0)
    ad.allocate_workspace(T)
    ids = torch.ones(T, dtype=torch.int32)
    ids[1::7] = 0
    u = 2.0 * (x.double() @ A.double().T)
    u[ids == 0] = 0.0
    got = ad.forward(x.to(dt).cuda(), ids.cuda(), out_dtype=torch.float32).double().cpu()
    size = u.abs() if dt == torch.bfloat16 else u.abs().amax(1, keepdim=True)
    steps = 5                                             # the shrink's sum, three products' sums, the last term's rounding
    assert ((got[:, :rank] - u).abs() <= steps * 2.0 ** -23 * size).all()
    assert not got[:, rank:].any()
    assert ad.device_error() == 0


@pytest.mark.parametrize("T,n,rank", [(20000, 1, 64), (20000, 1, 128), (4000, 160, 16), (2000, 160, 16)])
def test_long_sums_of_u(T, n, rank):
    """u = A x over K = 16384 in one CTA: 1024 steps of 16 products, of which an accumulator of the tensor core takes an
    eighth (rank 128: a quarter).  A step cuts 2^-23 of its sum at most, towards zero, and the sum after i of m steps of
    random signs is sqrt(i / m) of the last: 2/3 m 2^-23 of u's norm in all.  The sums of the accumulators, and of
    u's three terms with the identity, round some 16 times more."""
    K, N, m = 16384, 128, 256 if rank == 128 else 128
    g = torch.Generator(device="cuda").manual_seed(T + rank)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=g)
    ad = pkg().LowRankAdapters(n, N, K, rank)
    A, B = rnd(rank, K).bfloat16(), torch.zeros((N, rank), device="cuda", dtype=torch.bfloat16)
    B[torch.arange(rank), torch.arange(rank)] = 1.0
    ad.set(n - 1, A, B)
    ad.allocate_workspace(T)
    x = rnd(T, K).bfloat16()
    ids = torch.full((T,), n - 1, dtype=torch.int32, device="cuda")
    got = ad.forward(x, ids, out_dtype=torch.float32)[:, :rank].double()
    for rows in (slice(0, 200), slice(T - 200, T)):
        u = x[rows].double() @ A.double().T
        assert float((got[rows] - u).norm() / u.norm()) <= (2 * m / 3 + 16) * 2.0 ** -23


@pytest.mark.parametrize("rank,T", [(16, 1), (16, 300), (64, 40), (64, 2100), (128, 600), (32, 4000)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_small_u_beside_large_ones(T, rank, dt):
    """The u of a row lie up to 2^15 apart: each keeps its own bits, as many steps as above from exact."""
    K, N = 2, 128
    g = torch.Generator().manual_seed(T + rank)
    draw = lambda *s: (torch.randint(128, 256, s, generator=g) / 128 * torch.where(torch.rand(s, generator=g) < 0.5, -1.0, 1.0))
    A, x = draw(rank, K), draw(T, K)
    A *= 2.0 ** (8 - torch.arange(rank) % 16)[:, None]
    A[:, 1] *= 2.0 ** -9
    assert torch.equal(A.to(dt).float(), A) and torch.equal(x.to(dt).float(), x)
    B = torch.zeros(N, rank)
    B[torch.arange(rank), torch.arange(rank)] = 1.0
    for scale in (1.0, 2.0 ** 40, 2.0 ** -60):
        ad = pkg().LowRankAdapters(1, N, K, rank, dt)
        ad.set(0, A.to(dt).cuda(), B.to(dt).cuda(), scale)
        ad.allocate_workspace(T)
        u = scale * (x.double() @ A.double().T)
        got = ad.forward(x.to(dt).cuda(), torch.zeros(T, dtype=torch.int32).cuda(), out_dtype=torch.float32).double().cpu()
        assert ((got[:, :rank] - u).abs() <= 5 * 2.0 ** -23 * u.abs()).all()
        assert not got[:, rank:].any()
