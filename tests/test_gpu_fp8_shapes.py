"""The 8-bit kernels at served widths and at stores that end inside vectors, against their 64-bit forms."""
import pytest
import torch

from fp8_helpers import ffn_ref, quantize_rows_ref, random_experts, random_rows
from test_gpu_fp8_experts import routing
from test_gpu_fp8_linear import DT, check, make_linear

pytestmark = pytest.mark.gpu


# More units than half the SMs: no split along K, so whole and partial sets of 32 rows leave element by
# element where N is odd or the columns start off a 16-byte boundary.
@pytest.mark.parametrize("N,col", [(1321, 16), (1337, 0), (1320, 5), (1344, 1)])
@pytest.mark.parametrize("T", [2048, 2100])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_linear_many_rows_by_element(T, N, col, out):
    K = 384
    lin, wq, ws = make_linear(N, K, T)
    x = random_rows(T, K, 8)
    wide = torch.full((T + 3, N + 24), 7.0, dtype=DT[out], device="cuda")
    got = wide[2:2 + T, col:col + N]
    lin.forward(x.cuda(), out=got, out_dtype=DT[out])
    check(got, *quantize_rows_ref(x), wq, ws)
    assert (wide[:2] == 7).all() and (wide[2 + T:] == 7).all()
    assert (wide[:, :col] == 7).all() and (wide[:, col + N:] == 7).all()
    assert lin.device_error() == 0


@pytest.mark.parametrize("T", [1, 6, 40])
def test_wide_layer_of_384_experts(T):
    """d_model 4096, d_ff 1024, 384 experts (eight distinct ones, 48 times over), top 8."""
    from decode_batches_gb300 import MoePlan
    E, k, d, f, distinct = 384, 8, 4096, 1024, 8
    gate, up, down = random_experts(distinct, f, d, 0)
    rep = lambda t: t.cuda().repeat(E // distinct, *[1] * (t.dim() - 1))
    plan = MoePlan(E, k, d, f, 0, "fp8")
    plan.set_weights(torch.zeros((E, d), device="cuda"), None, rep(gate[0]), rep(up[0]), rep(down[0]), rep(gate[1]),
                     rep(up[1]), rep(down[1]))
    plan.allocate_workspace(T)
    x = random_rows(T, d, 3)
    ids, gates = routing(T, E, k, 4)
    out = plan.forward_routed(x.cuda(), ids.cuda(), gates.cuda())
    ref = torch.zeros((T, d), dtype=torch.float64)
    tol = torch.zeros_like(ref)
    for e in range(distinct):
        t, j = torch.nonzero(ids % distinct == e, as_tuple=True)
        if not len(t):
            continue
        y, dy = ffn_ref(x[t], *((m[0][e], m[1][e]) for m in (gate, up, down)))
        w = gates[t, j].double()[:, None]
        ref.index_add_(0, t, w * y)               # fp16 y 2^-11, the fp32 sum over slots
        tol.index_add_(0, t, w * (dy + (y.abs() + dy) * 2.0 ** -11 + 2.0 ** -24) + (k + 1) * 2.0 ** -24 * (w * y).abs())
    got = out.double().cpu()
    assert ((got - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all()
    # That bound adds up the worst of every term, 4096 of them, and is wide here.  The roundings are
    # independent, so a row's mean square is known better: bf16 out at most 2^-8 / sqrt(3) of its size,
    # fp16 y 2^-11 / sqrt(3), and an open rounding of h (one in 10^5, by 2^-4) 2e-4: 2.3e-3 together.
    assert ((got - ref).pow(2).mean(1).sqrt() <= 2.5e-3 * ref.pow(2).mean(1).sqrt()).all()
    assert plan.device_error() == 0
