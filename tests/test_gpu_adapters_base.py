"""Rows without an adapter, or of an empty slot: out is base, bit for bit, whatever the step's size."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BITS = {torch.bfloat16: torch.int16, torch.float16: torch.int16, torch.float32: torch.int32}


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


@pytest.mark.parametrize("out", sorted(BITS, key=str))
@pytest.mark.parametrize("N,pad", [(264, 0), (1337, 0), (2048, 8), (96, 1), (1, 0)])
@pytest.mark.parametrize("T", [1, 20, 33, 256, 257, 1024, 1025, 3600])
def test_bits_of_the_base(T, N, pad, out):
    K = 64
    g = torch.Generator(device="cuda").manual_seed(T + N)
    ad = pkg().LowRankAdapters(3, N, K, 16)
    A = torch.randn((16, K), device="cuda", generator=g).bfloat16()
    B = torch.randn((N, 16), device="cuda", generator=g).bfloat16()
    ad.set(0, A, B)
    ad.set(2, A, B)
    ad.clear(2)
    ad.allocate_workspace(T)
    x = torch.randn((T, K), device="cuda", generator=g).bfloat16()
    # every bit pattern may lie there: zeros of both signs, NaN with payloads, subnormals
    info = torch.iinfo(BITS[out])
    bits = torch.randint(info.min, info.max, (T, N + pad), device="cuda", generator=g).to(BITS[out])
    some = torch.tensor([0.0, -0.0, float("nan"), float("inf")], dtype=out).view(BITS[out]).tolist()
    for i, v in enumerate(some + [some[2] + 1, -1, 1]):
        bits.view(-1)[i::13] = v
    base = bits.view(out)[:, :N]
    for ids in (torch.full((T,), -1), torch.full((T,), 2), torch.randint(-1, 3, (T,), generator=torch.Generator().manual_seed(T))):
        plain = (ids != 0).cuda()
        got = ad.forward(x, ids.int().cuda(), base)
        assert torch.equal(got.view(BITS[out])[plain], bits[:, :N][plain])
        zero = ad.forward(x, ids.int().cuda(), out_dtype=out)
        assert not zero.view(BITS[out])[plain].any()
        wide = torch.full((T, N + 24), 3.0, dtype=out, device="cuda")
        ad.forward(x, ids.int().cuda(), base, out=wide[:, 8:N + 8])
        assert torch.equal(wide[:, 8:N + 8].contiguous().view(BITS[out])[plain], bits[:, :N][plain])
        assert (wide[:, :8] == 3.0).all() and (wide[:, N + 8:] == 3.0).all()
    assert ad.device_error() == 0
