"""Low-rank adapters on tiles that end inside a warp's rows: lanes without a row skip the stores and have to be back for the
next load of the whole warp (tensor memory, fragments).  Every row against the same row in a step without gaps."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


# rows of the slot that ends raggedly: within 8, 16 and 32 rows of a tile of 64 and of 128, in steps of every kernel
@pytest.mark.parametrize("rows", [1, 3, 9, 17, 27, 41, 63, 77, 93, 125])
@pytest.mark.parametrize("T,rank", [(200, 16), (200, 128), (300, 64), (300, 128), (1000, 64), (1000, 128), (2500, 64),
                                    (2500, 100), (5000, 64)])
def test_rows_of_ragged_tiles(T, rank, rows):
    K, N = 192, 328
    g = torch.Generator(device="cuda").manual_seed(T + rank + rows)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=g)
    ad = pkg().LowRankAdapters(2, N, K, rank)
    A, B = (rnd(2, rank, K) * K ** -0.5).bfloat16(), rnd(2, N, rank).bfloat16()
    for i in range(2):
        ad.set(i, A[i], B[i], 0.5)
    ad.allocate_workspace(T)
    x, base = rnd(T, K).bfloat16(), rnd(T, N)
    ids = torch.full((T,), 1, dtype=torch.int32, device="cuda")
    few = torch.randperm(T, device="cuda", generator=g)[:rows]
    ids[few] = 0
    for out in (torch.float32, torch.bfloat16, torch.float16):
        b = base.to(out)
        first = ad.forward(x, ids, b)
        for _ in range(3):
            assert torch.equal(ad.forward(x, ids, b), first)
        # a slot of T rows: its tiles but the last are whole
        whole = ad.forward(x, torch.zeros_like(ids), b)
        assert torch.equal(first[few], whole[few])
        whole = ad.forward(x, torch.ones_like(ids), b)
        rest = ids == 1
        assert torch.equal(first[rest], whole[rest])
    assert ad.device_error() == 0
