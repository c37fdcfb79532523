"""The weights' gradients of the row moves within the rounding of their reduction."""
import pytest
import torch

from rows_helpers import TYPES, U32, assignments, close, dots_ref, tensor

pytestmark = pytest.mark.gpu


def slack(d, mag):
    """A lane adds up 8 products of each of its warp's spans of 256 columns, which 8 warps share (8 ceil(d / 2048) steps);
    five steps join the lanes, eight the warps; every step rounds once, by half a step of at most all the magnitudes."""
    return (8 * -(-d // 2048) + 13) * U32 * (1 + 2.0 ** -10) * mag


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("T,k,d,pad,shift", [(40, 8, 2048, 0, 0), (40, 3, 2056, 0, 0), (9, 11, 2049, 1, 1), (30, 4, 4096, 0, 0),
                                             (20, 2, 4104, 0, 0), (12, 9, 5000, 0, 3), (7, 32, 8191, 0, 0), (5, 1, 256, 0, 0)])
def test_weight_gradients(T, k, d, pad, shift, dt):
    import decode_batches_gb300 as p
    dtype = TYPES[dt]
    inv = assignments(T, k, 1, 0.1)
    w = torch.softmax(torch.randn((T, k), generator=torch.Generator().manual_seed(2)), 1).cuda()
    x, rows = tensor(T, d, dtype, 3, pad, shift), tensor(T * k, d, dtype, 4, pad, shift)
    ref, mag = dots_ref(x, rows, inv)
    for got in (p.sort_rows_backward(rows, inv.cuda(), w, x)[1], p.combine_rows_backward(x, inv.cuda(), w, rows)[1]):
        close(got, ref, slack(d, mag), torch.float32)
        assert (got.cpu()[inv < 0] == 0).all()
