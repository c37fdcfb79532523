"""Adapters of rank 65 to 128 in steps of 257 to 1024 rows: tiles found in the ids by CTAs of sixteen warps, with less and more
than one slot a counting thread."""
import pytest
import torch

from rows_helpers import TYPES
from test_gpu_adapters_large import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [6, 600])
@pytest.mark.parametrize("r", [65, 128])
@pytest.mark.parametrize("T", [257, 511, 513, 700, 1024])
def test_tiles_from_the_ids(T, r, n, dt):
    g = torch.Generator().manual_seed(T + r + n)
    ids = torch.randint(-1, n, (T,), generator=g)
    ids = torch.where(torch.rand(T, generator=g) < 0.2, -1, ids)
    ids[T // 2: T // 2 + 150] = n - 1                          # a slot of more than one tile
    used = range(n) if n == 6 else sorted({int(i) for i in ids.unique()} - {-1} | {0})[::2] + [n - 1]
    for ot in sorted(TYPES):
        run(T, n, r, 72, 136, dt, TYPES[ot], ids, T, used=sorted(set(used)))
    run(T, n, r, 72, 137, dt, torch.float32, ids, T, used=sorted(set(used)), base=False)
