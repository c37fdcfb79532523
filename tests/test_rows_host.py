"""Host-side checks of the row moves (no GPU): bad arguments are refused before any launch."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from decode_batches_gb300 import build, load_library
    build.build()
    return load_library()


P = 4096  # a pointer that is never dereferenced: every call here is refused (or empty) on the host
BF16, FP32 = 0, 2

GOOD = {
    "moe_sort_rows": dict(x=P, dt=BF16, ldx=64, T=4, k=2, d=64, inv=P, w=None, out=P, ldo=64, n=8),
    "moe_sort_rows_backward": dict(g=P, dt=BF16, ldg=64, n=8, T=4, k=2, d=64, inv=P, w=None, x=P, ldx=64, dx=P, lddx=64,
                                   dw=P),
    "moe_combine_rows": dict(y=P, ydt=BF16, ldy=64, n=8, T=4, k=2, d=64, inv=P, w=P, sh=P, sdt=FP32, lds=64, out=P,
                             odt=FP32, ldo=64),
    "moe_combine_rows_backward": dict(g=P, gdt=FP32, ldg=64, T=4, k=2, d=64, inv=P, w=P, y=P, ldy=64, dy=P, ydt=BF16,
                                      lddy=64, n=8, dw=P),
}
BAD = {
    "moe_sort_rows": [dict(T=-1), dict(k=0), dict(k=33), dict(d=0), dict(n=-1), dict(dt=7), dict(x=None), dict(x=P + 1),
                      dict(ldx=63), dict(inv=None), dict(out=None), dict(ldo=63), dict(out=P + 1)],
    "moe_sort_rows_backward": [dict(T=-1), dict(k=0), dict(d=0), dict(dt=-1), dict(g=None), dict(ldg=1), dict(inv=None),
                               dict(x=None), dict(ldx=63), dict(dx=None), dict(lddx=0)],
    "moe_combine_rows": [dict(T=-2), dict(k=40), dict(ydt=3), dict(odt=3), dict(sdt=9), dict(y=None), dict(ldy=8),
                         dict(inv=None), dict(lds=4), dict(out=None), dict(out=P + 2), dict(sh=P + 1), dict(n=0, ydt=9)],
    "moe_combine_rows_backward": [dict(T=-1), dict(gdt=5), dict(ydt=5), dict(g=None), dict(y=None), dict(ldy=1),
                                  dict(dy=None), dict(lddy=2), dict(inv=None), dict(g=P + 2)],
}


@pytest.mark.parametrize("name", sorted(GOOD))
def test_row_moves_refuse_bad_arguments(lib, name):
    from decode_batches_gb300 import MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED
    fn = getattr(lib, name)
    call = lambda **kw: fn(*{**GOOD[name], **kw}.values(), None)
    assert call(T=0) == 0
    for kw in BAD[name]:
        assert call(**kw) == MOE_ERR_INVALID_ARG, (name, kw)
        assert lib.moe_last_error()
    assert call(T=2**30, k=2) == MOE_ERR_UNSUPPORTED
    assert call(n=2**31) == MOE_ERR_UNSUPPORTED
    assert call(d=2**24 + 8, **{k: 2**25 for k in GOOD[name] if k.startswith("ld")}) == MOE_ERR_UNSUPPORTED


def test_row_moves_refuse_tensors_of_the_host():
    import decode_batches_gb300 as pkg
    x, inv = torch.zeros(2, 8), torch.zeros((2, 1), dtype=torch.int32)
    if torch.cuda.is_available():
        pytest.skip("needs no GPU, and a context on one changes the message")
    for call in (pkg.sort_rows, pkg.sort_rows_backward, pkg.combine_rows, pkg.combine_rows_backward):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call(x, inv)
