"""Host-side checks of the low-rank adapters (no GPU): bad arguments are refused before any launch."""
import pytest

P = 4096  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from decode_batches_gb300 import build, load_library
    build.build()
    return load_library()


def test_adapter_entry_points_refuse_bad_arguments(lib):
    from decode_batches_gb300 import MOE_ERR_INVALID_ARG, MOE_ERR_NOT_READY, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE
    for args in ((0, 8, 8, 8, 0), (1025, 8, 8, 8, 0), (4, 0, 8, 8, 0), (4, 8, 0, 8, 0), (4, 2**20 + 1, 8, 8, 0),
                 (4, 8, 2**20 + 1, 8, 0), (4, 8, 8, 0, 0), (4, 8, 8, 129, 0), (4, 8, 8, 8, 2), (4, 8, 8, 8, 7)):
        assert lib.moe_adapters_create(*args) is None, args
        assert lib.moe_last_error()
    h = lib.moe_adapters_create(4, 64, 96, 16, 0)
    assert h
    try:
        for args in ((-1, P, P, 4, 1.0), (4, P, P, 4, 1.0), (0, P, P, 17, 1.0), (0, P, P, -1, 1.0), (0, None, P, 4, 1.0),
                     (0, P, None, 4, 1.0), (0, P + 1, P, 4, 1.0), (0, P, P, 4, float("nan")), (0, P, P, 4, float("inf"))):
            assert lib.moe_adapters_set(h, *args) == MOE_ERR_INVALID_ARG, args
        assert lib.moe_adapters_set(None, 0, P, P, 4, 1.0) == MOE_ERR_INVALID_ARG
        fwd = lambda x=P, ldx=96, T=4, ids=P, base=P, ldb=64, out=2 * P, dt=0, ldo=64: lib.moe_adapters_forward(
            h, x, ldx, T, ids, base, ldb, out, dt, ldo, None)
        assert fwd() == MOE_ERR_NOT_READY
        assert fwd(T=-1) == MOE_ERR_INVALID_ARG and fwd(dt=3) == MOE_ERR_INVALID_ARG
        assert lib.moe_adapters_forward(None, P, 96, 4, P, P, 64, P, 0, 64, None) == MOE_ERR_INVALID_ARG
        b1, b2 = lib.moe_adapters_workspace_bytes(h, 1), lib.moe_adapters_workspace_bytes(h, 10000)
        assert 0 < b1 < b2 and b2 >= 40000
        assert lib.moe_adapters_set_workspace(h, None, b2, 10000) == MOE_ERR_INVALID_ARG
        assert lib.moe_adapters_set_workspace(h, 256, b2, 0) == MOE_ERR_INVALID_ARG
        assert lib.moe_adapters_set_workspace(h, 128, b2, 10000) == MOE_ERR_WORKSPACE
        assert lib.moe_adapters_set_workspace(h, 256, b1, 10000) == MOE_ERR_WORKSPACE
        assert lib.moe_adapters_set_workspace(h, 256, 1 << 40, 2**27) == MOE_ERR_UNSUPPORTED
        assert lib.moe_adapters_get_device_error(h, None) == MOE_ERR_INVALID_ARG
    finally:
        lib.moe_adapters_destroy(h)
    lib.moe_adapters_destroy(None)
