"""Host-side checks of the 8-bit calls (no GPU): bad arguments are refused before any launch."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from decode_batches_gb300 import build, load_library
    build.build()
    return load_library()


def test_linear_entry_points_refuse_bad_arguments(lib):
    from decode_batches_gb300 import MOE_ERR_INVALID_ARG, MOE_ERR_NOT_READY, MOE_ERR_WORKSPACE
    assert lib.moe_linear_create(0, 4) is None and lib.moe_linear_create(4, 0) is None
    assert lib.moe_last_error()
    h = lib.moe_linear_create(300, 200)
    assert h
    try:
        assert lib.moe_linear_set_weights(h, None, None) == MOE_ERR_INVALID_ARG
        assert lib.moe_linear_forward(h, None, 0, 200, 4, None, 0, 300, None) == MOE_ERR_NOT_READY
        assert lib.moe_linear_forward(None, None, 0, 200, 4, None, 0, 300, None) == MOE_ERR_INVALID_ARG
        assert lib.moe_linear_forward_quantized(h, None, 256, None, 4, -1, None, 0, 300, None) == MOE_ERR_INVALID_ARG
        assert lib.moe_linear_set_workspace(h, None, 0, 4) == MOE_ERR_INVALID_ARG
        assert lib.moe_linear_set_workspace(h, 128, 1 << 20, 4) == MOE_ERR_WORKSPACE      # misaligned
        assert lib.moe_linear_set_workspace(h, 256, 64, 4) == MOE_ERR_WORKSPACE           # too small
        b1, b2 = lib.moe_linear_workspace_bytes(h, 1), lib.moe_linear_workspace_bytes(h, 1000)
        assert 0 < b1 < b2 and b2 >= 1000 * (256 + 4 * 2)
    finally:
        lib.moe_linear_destroy(h)
    lib.moe_linear_destroy(None)


def test_quantise_entry_points_refuse_bad_arguments(lib):
    from decode_batches_gb300 import MOE_ERR_INVALID_ARG
    q = 4096  # never dereferenced: every call here is refused (or empty) on the host
    assert lib.moe_quantize_rows(q, 0, 128, 0, 128, q, 128, q, 1, None) == 0
    for args in ((q, 0, 128, -1, 128, q, 128, q, 1), (q, 0, 128, 4, 0, q, 128, q, 1), (q, 5, 128, 4, 128, q, 128, q, 1),
                 (None, 0, 128, 4, 128, q, 128, q, 1), (q, 0, 127, 4, 128, q, 128, q, 1), (q, 0, 129, 4, 129, q, 129, q, 2),
                 (q, 0, 128, 4, 128, q + 4, 128, q, 1), (q, 0, 128, 4, 128, q, 128, q, 0), (q + 1, 0, 128, 4, 128, q, 128, q, 1)):
        assert lib.moe_quantize_rows(*args, None) == MOE_ERR_INVALID_ARG, args
    assert lib.moe_quantize_blocks(q, 0, 0, 128, q, q, None) == 0
    for args in ((q, 0, -1, 128, q, q), (q, 0, 4, 0, q, q), (q, 9, 4, 4, q, q), (None, 0, 4, 4, q, q)):
        assert lib.moe_quantize_blocks(*args, None) == MOE_ERR_INVALID_ARG, args


def test_reference_quantisation_is_the_rule():
    """The tests' own 64-bit form of the rule, on numbers worked out by hand."""
    from fp8_helpers import quantize_rows_ref
    x = torch.zeros((1, 130))
    x[0, 0], x[0, 1], x[0, 2], x[0, 128] = 448.0, 17.0, -27.0, 7.0
    q, s = quantize_rows_ref(x)
    assert s.tolist() == [[1.0, float(torch.tensor(7.0) * (torch.tensor(1.0) / 448.0))]]
    assert q[0, 0] == 448 and q[0, 1] == 16 and q[0, 2] == -28 and q[0, 128] == 448   # 17, 27 tie to even
    z, sz = quantize_rows_ref(torch.zeros((1, 3)))
    assert not z.any() and float(sz) == 2.0 ** -126
