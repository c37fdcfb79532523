"""Host-side checks of the 8-bit calls (no GPU): lengths near 2^31, where a partial block's end would pass it,
are refused before any launch."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from decode_batches_gb300 import build, load_library
    build.build()
    return load_library()


LONG = [2**31 - 1, 2**31 - 128, 2**31 - 1024]


@pytest.mark.parametrize("K", LONG)
def test_quantise_refuses_rows_whose_blocks_pass_2_31(lib, K):
    from decode_batches_gb300 import MOE_ERR_UNSUPPORTED
    q = 4096  # never dereferenced
    assert lib.moe_quantize_rows(q, 0, 1 << 31, 2, K, q, 1 << 31, q, 1 << 24, None) == MOE_ERR_UNSUPPORTED
    assert lib.moe_quantize_blocks(q, 0, 2, K, q, q, None) == MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("T", LONG)
def test_workspace_for_rows_whose_parts_pass_2_31_is_refused(lib, T):
    from decode_batches_gb300 import MOE_ERR_UNSUPPORTED
    h = lib.moe_linear_create(4, 4)
    try:
        assert lib.moe_linear_set_workspace(h, 256, 1 << 40, T) == MOE_ERR_UNSUPPORTED
    finally:
        lib.moe_linear_destroy(h)
