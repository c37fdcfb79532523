"""Gathering rows of so many tokens that a block takes several of them in turn: the same bits as in calls of few
tokens, where every token has a block of its own (what a token sums, and in which order, does not depend on T)."""
import pytest
import torch

from rows_helpers import TYPES, assignments, dot_slack, dots_ref, gather_ref, tensor, close, U32

pytestmark = pytest.mark.gpu


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


# (tokens, slots, columns, elements between rows)
SHAPES = [(2503, 8, 2048, 0), (2503, 11, 2040, 8), (2503, 3, 2047, 0), (20011, 2, 64, 0), (20011, 9, 37, 3)]


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_sort_rows_backward_in_turns(shape, dt):
    T, k, d, pad = shape
    p, dtype = pkg(), TYPES[dt]
    inv = assignments(T, k, 71, 0.1)
    w = torch.randn((T, k), generator=torch.Generator().manual_seed(72))
    grad, x = tensor(T * k, d, dtype, 73, pad), tensor(T, d, dtype, 74, pad)
    inv_d, w_d = inv.cuda(), w.cuda()
    plain = p.sort_rows_backward(grad, inv_d)
    dx, dw = p.sort_rows_backward(grad, inv_d, weights=w_d, x=x)
    for i in range(0, T, 250):
        part = inv_d[i:i + 250].contiguous()
        assert torch.equal(p.sort_rows_backward(grad, part), plain[i:i + 250])
        px, pw = p.sort_rows_backward(grad, part, weights=w_d[i:i + 250].contiguous(), x=x[i:i + 250])
        assert torch.equal(px, dx[i:i + 250]) and torch.equal(pw, dw[i:i + 250])
    last = slice(T - 40, T)
    ref, mag = gather_ref(grad, inv[last], w[last], 40)
    close(dx[last], ref, (k + 1) * U32 * (1 + 2.0 ** -10) * mag, dtype)
    ref, mag = dots_ref(x[last], grad, inv[last])
    close(dw[last], ref, dot_slack(d, mag), torch.float32)


@pytest.mark.parametrize("st", ["none", *sorted(TYPES)])
@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_combine_rows_in_turns(shape, dt, st):
    T, k, d, pad = shape
    p = pkg()
    inv = assignments(T, k, 75, 0.1)
    w = torch.randn((T, k), generator=torch.Generator().manual_seed(76))
    y, inv_d, w_d = tensor(T * k, d, TYPES[dt], 77, pad), inv.cuda(), w.cuda()
    shared = None if st == "none" else tensor(T, d, TYPES[st], 78, pad)
    out = p.combine_rows(y, inv_d, w_d, shared=shared, out_dtype=torch.float32)
    for i in range(0, T, 250):
        few = None if shared is None else shared[i:i + 250]
        got = p.combine_rows(y, inv_d[i:i + 250].contiguous(), w_d[i:i + 250].contiguous(), shared=few, out_dtype=torch.float32)
        assert torch.equal(got, out[i:i + 250])
    last = slice(T - 40, T)
    ref, mag = gather_ref(y, inv[last], w[last], 40)
    if shared is not None:
        ref, mag = ref + shared[last].double().cpu(), mag + shared[last].double().cpu().abs()
    close(out[last], ref, (k + 2) * U32 * (1 + 2.0 ** -10) * mag, torch.float32)
