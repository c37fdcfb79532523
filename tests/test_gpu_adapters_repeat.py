"""Adapter calls one behind the other with nothing waiting between them: two handles in turn, each with its own base.
The base is read, never written, and a call's answer does not depend on what ran before it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def state(T, K, N, n, r, dtype, out, seed):
    from decode_batches_gb300 import LowRankAdapters
    g = torch.Generator().manual_seed(seed)
    ad = LowRankAdapters(n, N, K, r, dtype=dtype)
    for i in range(n):
        ad.set(i, (torch.randn((r, K), generator=g) * K ** -0.5).to(dtype).cuda(),
               (torch.randn((N, r), generator=g) * r ** -0.5).to(dtype).cuda(), 0.5 + i)
    ad.allocate_workspace(T)
    x = torch.randn((T, K), generator=g).to(dtype).cuda()
    base = torch.randn((T, N), generator=g).to(out).cuda()
    return ad, x, torch.randint(-1, n, (T,), generator=g).int().cuda(), base


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,K,N,n,r", [(1, 264, 136, 3, 8), (40, 520, 264, 7, 24), (200, 1032, 2048, 7, 16),
                                       (700, 333, 261, 7, 24), (1500, 512, 1024, 5, 64), (4001, 256, 384, 9, 32)])
def test_three_passes_with_another_handle_between(T, K, N, n, r, dtype, out):
    one, two = state(T, K, N, n, r, dtype, out, 1), state(T, K, N, n, r, dtype, out, 2)
    before = one[3].clone()
    want = one[0].forward(one[1], one[2], base=one[3])
    torch.cuda.synchronize()
    assert torch.equal(want[one[2] < 0], before[one[2] < 0])
    for _ in range(4):
        first = one[0].forward(one[1], one[2], base=one[3])
        other = two[0].forward(two[1], two[2], base=two[3])
        last = one[0].forward(one[1], one[2], base=one[3])
        del other                      # (its memory may serve the next turn's calls)
        assert torch.equal(first, want) and torch.equal(last, want)
    assert torch.equal(one[3], before)
    assert one[0].device_error() == 0 and two[0].device_error() == 0
