"""The layer with 8-bit experts against its 64-bit form (tests/fp8_helpers.py)."""
import pytest
import torch

from fp8_helpers import ffn_ref, layer_ref, random_experts, random_rows

pytestmark = pytest.mark.gpu


def make_plan(E, k, d, f, T_max, seed=0, w_router=None, n_shared=0, f_s=0):
    from decode_batches_gb300 import MoePlan
    gate, up, down = random_experts(E, f, d, seed)
    plan = MoePlan(E, k, d, f, n_shared, "fp8")
    if w_router is None:
        g = torch.Generator().manual_seed(seed + 5)
        w_router = torch.randn((E, d), generator=g) * 0.02
    plan.set_weights(w_router.cuda(), None, gate[0].cuda(), up[0].cuda(), down[0].cuda(), gate[1].cuda(), up[1].cuda(),
                     down[1].cuda())
    shared = None
    if n_shared:
        g = torch.Generator().manual_seed(seed + 6)
        shared = [(torch.randn(s, generator=g) * s[-1] ** -0.5).to(torch.bfloat16)
                  for s in ((n_shared, f_s, d), (n_shared, f_s, d), (n_shared, d, f_s))]
        plan.set_shared(f_s, *[w.cuda() for w in shared])
    plan.allocate_workspace(T_max)
    return plan, gate, up, down, shared


def routing(T, E, k, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=g) - skew * torch.log(torch.arange(1, E + 1).float())
    v, i = l.topk(k, dim=1)
    return i.int(), torch.softmax(v, 1)


def close(out, ref, tol):
    got = out.double().cpu()
    bad = (got - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}: worst {float(((got - ref).abs() / tol.clamp_min(1e-300)).max()):.2f} x"
    # the tolerance must not be what makes it pass
    assert float(tol.pow(2).mean().sqrt()) < 0.05 * float(ref.pow(2).mean().sqrt()) + 1e-30


@pytest.mark.parametrize("T,E,k,d,f,skew", [
    (1, 1, 1, 128, 128, 0), (1, 8, 2, 256, 256, 0), (4, 16, 8, 512, 128, 0), (8, 8, 8, 256, 384, 0),
    (5, 8, 2, 200, 136, 0), (64, 12, 3, 264, 264, 0), (65, 8, 2, 256, 128, 0), (33, 5, 1, 1000, 8, 0),
    (300, 4, 2, 256, 256, 2.0), (700, 6, 2, 384, 128, 1.1), (129, 1, 1, 256, 256, 0), (2, 40, 4, 8, 8, 0)])
def test_routed_layer_against_64_bits(T, E, k, d, f, skew):
    plan, gate, up, down, _ = make_plan(E, k, d, f, T)
    x = random_rows(T, d, 3)
    ids, gates = routing(T, E, k, 4, skew)
    out = plan.forward_routed(x.cuda(), ids.cuda(), gates.cuda())
    close(out, *layer_ref(x, ids, gates, gate, up, down))
    assert plan.device_error() == 0


def test_many_units_per_cta():
    """More (segment, tile) units than CTAs in both GEMMs: stages, TMEM buffers and the exchange of
    row maxima wrap around many times."""
    T, E, k, d, f = 260, 48, 4, 256, 640
    plan, gate, up, down, _ = make_plan(E, k, d, f, T, seed=7)
    x = random_rows(T, d, 8)
    ids, gates = routing(T, E, k, 9)
    close(plan.forward_routed(x.cuda(), ids.cuda(), gates.cuda()), *layer_ref(x, ids, gates, gate, up, down))


@pytest.mark.parametrize("T", [3, 40, 100])
def test_forward_is_route_then_forward_routed(T):
    E, k, d, f = 128, 4, 256, 128
    plan, *_ = make_plan(E, k, d, f, T, seed=2)
    x = random_rows(T, d, 5).cuda()
    a = plan.forward(x, n_prefill=T // 2)
    _, ids, gates = plan.route(x)
    assert torch.equal(a, plan.forward_routed(x, ids, gates))
    counts, offsets, perm, inv = plan.permute(ids)
    y, _ = plan.experts(x, offsets, perm)
    assert torch.equal(a, plan.combine(y.float(), gates, inv))


@pytest.mark.parametrize("T", [2, 100])
def test_shared_experts_beside_8_bit_ones(T):
    E, k, d, f = 8, 2, 256, 128
    plan, gate, up, down, (sg, su, sd) = make_plan(E, k, d, f, T, n_shared=2, f_s=64)
    x = random_rows(T, d, 3)
    ids, gates = routing(T, E, k, 4)
    xf = x.double()
    ref = torch.zeros((T, d), dtype=torch.float64)
    mag = torch.zeros_like(ref)
    for i in range(2):
        g, u = xf @ sg[i].double().T, xf @ su[i].double().T
        h = g * torch.sigmoid(g) * u
        ref += h @ sd[i].double().T
        mag += h.abs() @ sd[i].double().abs().T
    # fp16 h and fp16 y (2^-11 each), fp32 sums
    tol = mag * (2.0 ** -11 + 2.0 ** -16) + ref.abs() * 2.0 ** -11 + 2.0 ** -20
    close(plan.forward_routed(x.cuda(), ids.cuda(), gates.cuda()), *layer_ref(x, ids, gates, gate, up, down, (ref, tol)))
    _, ids2, gates2 = plan.route(x.cuda())
    assert torch.equal(plan.forward(x.cuda()), plan.forward_routed(x.cuda(), ids2, gates2))


def test_experts_entry_gives_each_row_its_experts_output():
    T, E, k, d, f = 30, 6, 2, 256, 128
    plan, gate, up, down, _ = make_plan(E, k, d, f, T)
    x = random_rows(T, d, 3)
    ids, _ = routing(T, E, k, 4)
    counts, offsets, perm, inv = plan.permute(ids.cuda())
    y, ys = plan.experts(x.cuda(), offsets, perm)
    assert ys is None
    off, pm = offsets.cpu().tolist(), perm.cpu()
    for e in range(E):
        rows = pm[off[e]:off[e + 1]] // k
        if len(rows):
            ref, tol = ffn_ref(x[rows.long()], (gate[0][e], gate[1][e]), (up[0][e], up[1][e]), (down[0][e], down[1][e]))
            got = y[off[e]:off[e + 1]].double().cpu()
            assert ((got - ref).abs() <= tol + 2.0 ** -11 * (ref.abs() + tol) + 2.0 ** -24).all()


@pytest.mark.parametrize("T", [6, 90])
def test_invalid_and_repeated_ids_contribute_nothing(T):
    from decode_batches_gb300 import DEVERR_EXPERT_RANGE
    E, k, d, f = 8, 3, 128, 128
    plan, gate, up, down, _ = make_plan(E, k, d, f, T)
    x = random_rows(T, d, 3)
    ids, gates = routing(T, E, k, 4)
    ids[0] = torch.tensor([-1, E, 1 << 30])      # a token with no expert at all
    ids[1, 2] = ids[1, 0]
    out = plan.forward_routed(x.cuda(), ids.cuda(), gates.cuda())
    close(out, *layer_ref(x, ids, gates, gate, up, down))
    assert not out[0].any()
    assert plan.device_error() == DEVERR_EXPERT_RANGE
    ids[:] = -5                                   # nothing routed: every segment list is empty
    assert not plan.forward_routed(x.cuda(), ids.cuda(), gates.cuda()).any()


def test_rows_are_independent_and_runs_identical():
    T, E, k, d, f = 150, 8, 2, 256, 256
    plan, *_ = make_plan(E, k, d, f, T)
    x = random_rows(T, d, 3).cuda()
    ids, gates = (a.cuda() for a in routing(T, E, k, 4, 1.0))
    a = plan.forward_routed(x, ids, gates)
    for _ in range(3):
        assert torch.equal(a, plan.forward_routed(x, ids, gates))
    y = x.clone()
    y[7] = float("nan")
    y[100, 3] = float("inf")
    b = plan.forward_routed(y, ids, gates)
    keep = torch.ones(T, dtype=torch.bool)
    keep[[7, 100]] = False
    assert torch.equal(a[keep], b[keep]) and b[7].isnan().all() and b[100].isnan().all()


def test_zero_rows_zero_x_and_overflow():
    from decode_batches_gb300 import DEVERR_RANGE
    E, k, d, f = 4, 2, 128, 128
    plan, *_ = make_plan(E, k, d, f, 8)
    ids, gates = (a.cuda() for a in routing(8, E, k, 4))
    assert plan.forward_routed(torch.empty((0, d), dtype=torch.bfloat16, device="cuda"), ids[:0], gates[:0]).shape == (0, d)
    assert not plan.forward_routed(torch.zeros((8, d), dtype=torch.bfloat16, device="cuda"), ids, gates).any()
    assert plan.device_error() == 0
    big = (random_rows(8, d, 1).float() * 1e4).to(torch.bfloat16).cuda()   # y leaves the fp16 range
    out = plan.forward_routed(big, ids, gates)
    assert out.isfinite().all() and plan.device_error() == DEVERR_RANGE


@pytest.mark.parametrize("T", [4, 80])
def test_another_stream_and_a_graph(T):
    E, k, d, f = 16, 4, 256, 128
    plan, gate, up, down, _ = make_plan(E, k, d, f, T)
    ids, gates = routing(T, E, k, 4)
    x = random_rows(T, d, 3)
    xc, ic, gc = x.cuda(), ids.cuda(), gates.cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = plan.forward_routed(xc, ic, gc, stream=st)
    st.synchronize()
    close(out, *layer_ref(x, ids, gates, gate, up, down))
    buf = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.forward_routed(xc, ic, gc, out=buf)
    x2 = random_rows(T, d, 30)
    ids2, gates2 = routing(T, E, k, 40)
    xc.copy_(x2), ic.copy_(ids2), gc.copy_(gates2)
    g.replay()
    torch.cuda.synchronize()
    close(buf, *layer_ref(x2, ids2, gates2, gate, up, down))


@pytest.mark.parametrize("dtype", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [6, 70])
def test_forward_routed_serves_the_other_weight_types(dtype, T):
    import numpy as np

    import synth
    from moe_helpers import make_plan as make_synth
    w = synth.workload("tiny") if dtype == "bf16" else None
    if w is not None:
        plan = make_synth(w, T_max=T)
        d = w.spec.d
    else:
        from decode_batches_gb300 import MoePlan
        E, k, d, f = 8, 2, 256, 128
        rng = np.random.default_rng(1)
        cu = lambda a: torch.from_numpy(a).cuda()
        plan = MoePlan(E, k, d, f, 0, "mxfp4")
        plan.set_weights(cu(rng.standard_normal((E, d)).astype(np.float32)), None,
                         cu(rng.integers(0, 256, (E, f, d // 2), dtype=np.uint8)),
                         cu(rng.integers(0, 256, (E, f, d // 2), dtype=np.uint8)),
                         cu(rng.integers(0, 256, (E, d, f // 2), dtype=np.uint8)),
                         cu(rng.integers(118, 122, (E, f, d // 32), dtype=np.uint8)),
                         cu(rng.integers(118, 122, (E, f, d // 32), dtype=np.uint8)),
                         cu(rng.integers(118, 122, (E, d, f // 32), dtype=np.uint8)))
        plan.allocate_workspace(T)
    x = random_rows(T, d, 3).cuda()
    _, ids, gates = plan.route(x)
    assert torch.equal(plan.forward(x), plan.forward_routed(x, ids, gates))


def test_refusals():
    from decode_batches_gb300 import MoeError, MoePlan
    with pytest.raises(KeyError):
        MoePlan(8, 2, 256, 256, 0, "fp9")
    with pytest.raises(MoeError):
        MoePlan(8, 2, 255, 256, 0, "fp8")
    plan, gate, up, down, _ = make_plan(8, 2, 256, 128, 4)
    with pytest.raises(MoeError):
        plan.set_path("simt")
    assert plan.resolved_path()[0] == "tc"
    x = random_rows(4, 256, 1).cuda()
    ids, gates = (a.cuda() for a in routing(4, 8, 2, 1))
    for bad in ((x, ids.long(), gates), (x, ids, gates.double()), (x, ids[:3], gates), (x.float(), ids, gates),
                (x[:, :128], ids, gates), (x, ids, gates.t())):
        with pytest.raises(ValueError):
            plan.forward_routed(*bad)
    with pytest.raises(MoeError):                 # more rows than the workspace holds
        plan.forward_routed(torch.cat([x, x]), torch.cat([ids, ids]), torch.cat([gates, gates]))
    p2 = MoePlan(8, 2, 256, 128, 0, "fp8")
    wr = torch.zeros((8, 256), device="cuda")
    with pytest.raises(ValueError):               # scales of another shape
        p2.set_weights(wr, None, gate[0].cuda(), up[0].cuda(), down[0].cuda(), gate[1].cuda(), up[1].cuda(), gate[1].cuda())
    with pytest.raises(MoeError):                 # no scales
        p2.set_weights(wr, None, gate[0].cuda(), up[0].cuda(), down[0].cuda())
    with pytest.raises(MoeError):                 # weights not set
        p2.allocate_workspace(4), p2.forward_routed(x, ids, gates)
    p3 = MoePlan(8, 2, 200, 128, 1, "fp8")
    z = torch.zeros
    with pytest.raises(MoeError):                 # shared experts that the 16-bit kernels cannot tile
        p3.set_shared(64, *(z(s, dtype=torch.bfloat16, device="cuda") for s in ((1, 64, 200), (1, 64, 200), (1, 200, 64))))


@pytest.mark.parametrize("T", [5, 90])
def test_forward_routed_on_the_cuda_core_path(T):
    """A shape without tensor-core tiles (bf16, d not a multiple of 128): the same call on the CUDA cores."""
    from decode_batches_gb300 import MoePlan
    E, k, d, f = 6, 2, 72, 40
    g = torch.Generator().manual_seed(0)
    bf = lambda *s: (torch.randn(s, generator=g) * s[-1] ** -0.5).to(torch.bfloat16).cuda()
    plan = MoePlan(E, k, d, f, 0, "bf16")
    plan.set_weights(torch.randn((E, d), generator=g).cuda(), None, bf(E, f, d), bf(E, f, d), bf(E, d, f))
    plan.allocate_workspace(T)
    assert plan.resolved_path()[0] == "simt"
    x = random_rows(T, d, 3).cuda()
    _, ids, gates = plan.route(x)
    assert torch.equal(plan.forward(x), plan.forward_routed(x, ids, gates))
