"""8-bit blocks and the 8-bit projection at the edges of their arguments: tensors that end with their last
value, empty matrices, other streams."""
import pytest
import torch

from fp8_helpers import blocks, quantize_rows_ref, random_rows
from test_gpu_fp8_linear import check, make_linear, pkg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1, 128, 129, 640, 700, 1152])
def test_one_row_whose_scales_end_with_the_last_block(K):
    """One row needs no padding behind its scales; nothing of the memory behind them is read."""
    N = 300
    lin, wq, ws = make_linear(N, K, 1)
    x = random_rows(1, K, 21)
    q, s = pkg().quantize_fp8(x.cuda())
    flat = s.reshape(-1).clone().view(1, -1)
    assert flat.shape == (1, blocks(K)) and flat.untyped_storage().nbytes() == 4 * blocks(K)
    out = lin.forward_quantized(q, flat, out_dtype=torch.float32)
    check(out, *quantize_rows_ref(x), wq, ws)
    assert torch.equal(out, lin.forward(x.cuda(), out_dtype=torch.float32)) and lin.device_error() == 0


def test_last_row_of_the_scales_may_be_unpadded():
    """Rows at a pitch of four scales whose last row's storage ends with its last scale."""
    T, N, K = 37, 260, 640                        # 5 blocks, pitch 8
    lin, wq, ws = make_linear(N, K, T)
    x = random_rows(T, K, 22)
    q, s = pkg().quantize_fp8(x.cuda())
    store = torch.full((8 * (T - 1) + 5,), float("nan"), device="cuda")
    cut = store.as_strided((T, 5), (8, 1))
    cut.copy_(s)
    check(lin.forward_quantized(q, cut, out_dtype=torch.float32), *quantize_rows_ref(x), wq, ws)


@pytest.mark.parametrize("shape", [(0, 128), (0, 5), (3, 0, 130), (0, 64, 130), (0, 0, 7), (2, 0, 3, 9)])
def test_a_weight_without_rows_has_no_codes(shape):
    q, s = pkg().quantize_fp8_weight(torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
    assert q.shape == shape and q.dtype == torch.float8_e4m3fn
    assert s.shape == (*shape[:-2], blocks(shape[-2]), blocks(shape[-1])) and s.dtype == torch.float32
