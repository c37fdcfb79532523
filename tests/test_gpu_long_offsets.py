"""Rows whose element offsets pass 2^31, and steps larger than the other tests': the last rows against the formulas."""
import pytest
import torch

from rows_helpers import U32, close
from verify_helpers import verify_ref

pytestmark = pytest.mark.gpu


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


def test_sorted_rows_beyond_2_31_elements():
    n, d, T = 540000, 4096, 5                              # 2.2e9 elements of expert rows
    y = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    inv = torch.tensor([[n - 1 - 2 * t, 7 * t] for t in range(T)], dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, d), generator=g).bfloat16()
    w = torch.rand((T, 2), generator=g)
    pkg().sort_rows(x.cuda(), inv.cuda(), out=y)
    assert torch.equal(y[inv[:, 0].long().cuda()].cpu(), x) and torch.equal(y[inv[:, 1].long().cuda()].cpu(), x)
    out = pkg().combine_rows(y, inv.cuda(), w.cuda(), out_dtype=torch.float32)
    ref = x.double() * w.double().sum(1, keepdim=True)
    close(out, ref, 3 * U32 * ref.abs(), torch.float32)
    dy, dw = pkg().combine_rows_backward(x.cuda(), inv.cuda(), w.cuda(), y, out=torch.empty_like(y))
    assert torch.equal(dy[n - 1].cpu(), (x[0].float() * w[0, 0]).bfloat16())
    dref = (x.double() ** 2).sum(1)
    close(dw[:, 0], dref, 200 * U32 * dref, torch.float32)


def test_verified_rows_beyond_2_31_elements():
    R, V = 17000, 131072                                   # 2.2e9 probabilities
    p = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((R, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(2)
    rows = 6
    p[-rows:] = torch.softmax(2 * torch.randn((rows, V), generator=g), 1).bfloat16().cuda()
    q[-rows:] = torch.softmax(2 * torch.randn((rows, V), generator=g), 1).bfloat16().cuda()
    drafts = torch.zeros(R, dtype=torch.int32)
    drafts[-rows:] = p[-rows:].argmax(1).int().cpu()
    offsets = torch.tensor([R - 6, R - 3, R], dtype=torch.int32)
    u, us = torch.rand(R, generator=g), torch.rand(2, generator=g)
    tokens, accepted = pkg().verify_drafts(p, drafts.cuda(), offsets.cuda(), u.cuda(), us.cuda(), q)
    ref, acc = verify_ref(p[-rows:].cpu(), drafts[-rows:].tolist(), [0, 3, 6], u[-rows:].tolist(), us.tolist(), q[-rows:].cpu())
    assert tokens[-rows:].tolist() == ref and accepted.tolist() == acc


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_adapters_of_a_large_step(dtype):
    """33000 rows that begin 2^31 elements into their memory's pitch, many tiles a cluster's grid."""
    T, K, N, n, r = 33000, 96, 136, 5, 16
    pitch = 65600                                          # 33000 rows of it: 2.16e9 elements
    g = torch.Generator().manual_seed(3)
    x = torch.empty((T, pitch), dtype=dtype, device="cuda")[:, :K]
    x.copy_(torch.randn((T, K), generator=g).to(dtype))
    base = torch.randn((T, N), generator=g)
    A, B = torch.randn((n, r, K), generator=g).to(dtype), torch.randn((n, N, r), generator=g).to(dtype)
    ad = pkg().LowRankAdapters(n, N, K, r, dtype)
    for i in range(n):
        ad.set(i, A[i].cuda(), B[i].cuda(), 0.25)
    ad.allocate_workspace(T)
    ids = torch.randint(-1, n, (T,), generator=g).int()
    ids[:9000] = 2
    got = ad.forward(x, ids.cuda(), base.cuda()).double().cpu()
    u = 0.25 * torch.einsum("tk,trk->tr", x.double().cpu(), A.double()[ids.clamp_min(0).long()])
    u[ids < 0] = 0.0
    mag = 0.25 * torch.einsum("tk,trk->tr", x.double().abs().cpu(), A.double().abs()[ids.clamp_min(0).long()])
    Bt = B.double()[ids.clamp_min(0).long()]
    ref = base.double() + torch.einsum("tr,tnr->tn", u, Bt)
    du = (K + 64) * 2 * U32 * mag + 2.0 ** -16 * u.abs().amax(1, keepdim=True)
    slack = torch.einsum("tr,tnr->tn", du + (2 * r + 64) * 2 * U32 * u.abs(), Bt.abs()) + U32 * ref.abs()
    close(got, ref, slack * (1 + 2.0 ** -8), torch.float32)
    assert torch.equal(got[ids < 0], base.double()[ids < 0]) and ad.device_error() == 0
