"""sort_rows and combine_rows on tensors that require a gradient: refused, since their results would be detached (no GPU: the
refusal comes before any look at the tensors' device)."""
import pytest
import torch


def cases():
    import decode_batches_gb300 as p
    x, y = torch.zeros(4, 8), torch.zeros(8, 8)
    inv, w, s = torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 8)
    g = lambda t: t.clone().requires_grad_()
    return [("sort_rows", lambda: p.sort_rows(g(x), inv)), ("sort_rows", lambda: p.sort_rows(x, inv, g(w))),
            ("combine_rows", lambda: p.combine_rows(g(y), inv, w)), ("combine_rows", lambda: p.combine_rows(y, inv, g(w))),
            ("combine_rows", lambda: p.combine_rows(y, inv, w, g(s)))]


@pytest.mark.parametrize("i", range(5))
def test_a_lost_gradient_is_refused(i):
    name, call = cases()[i]
    with pytest.raises(ValueError, match=f"{name}_backward"):
        call()
    with torch.no_grad(), pytest.raises(Exception) as e:      # what is refused now is the host's memory
        call()
    assert "_backward" not in str(e.value)


@pytest.mark.gpu
def test_calls_without_recording_work():
    import decode_batches_gb300 as p
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    inv = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    with pytest.raises(ValueError, match="sort_rows_backward"):
        p.sort_rows(x, inv)
    with torch.no_grad():
        rows = p.sort_rows(x, inv)
    assert torch.equal(rows, x.detach().repeat_interleave(2, 0)) and torch.equal(p.sort_rows(x.detach(), inv), rows)
    assert torch.equal(p.sort_rows_backward(rows, inv), 2 * x.detach())
    y = rows.clone().requires_grad_()
    dy, dw = p.combine_rows_backward(x.detach(), inv, torch.ones(4, 2, device="cuda"), y)
    assert dy.shape == y.shape and dw.shape == (4, 2)
