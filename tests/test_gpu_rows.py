"""sort_rows, combine_rows and their gradients against the formulas in 64 bits."""
import pytest
import torch

from rows_helpers import (TYPES, U32, assignments, close, dot_slack, dots_ref, floor_of, gather_ref, half_step, spread_ref,
                          tensor)

pytestmark = pytest.mark.gpu


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


def weights(T, k, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.softmax(torch.randn((T, k), generator=g), 1) * 2.5


# (T, k, d, share dropped, spare rows, pad, shift): one row, one column, widths around a span and a vector, more
# slots than are in flight together, rows that start on any element
SHAPES = [(1, 1, 1, 0.0, 0, 0, 0), (1, 8, 256, 0.0, 0, 0, 0), (5, 3, 7, 0.3, 2, 0, 0), (33, 8, 264, 0.0, 5, 8, 8),
          (17, 2, 1337, 0.2, 1, 3, 1), (9, 11, 512, 0.3, 0, 0, 0), (4, 32, 2056, 0.1, 0, 0, 0), (64, 4, 248, 1.0, 0, 0, 0),
          (3, 9, 5000, 0.0, 0, 0, 3), (257, 6, 96, 0.1, 0, 4, 4), (2, 8, 4104, 0.0, 3, 0, 0)]


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_sort_rows(shape, dt):
    T, k, d, lost, spare, pad, shift = shape
    dtype = TYPES[dt]
    inv = assignments(T, k, 1, lost, spare)
    x = tensor(T, d, dtype, 2, pad, shift)
    n = T * k + spare
    for w in (None, weights(T, k, 3)):
        out = tensor(n, d, dtype, 4, pad, shift)
        before = out.clone()
        got = pkg().sort_rows(x, inv.cuda(), None if w is None else w.cuda(), out=out)
        assert got is out
        ref, named = spread_ref(x, inv, w, n)
        if w is None:
            assert torch.equal(got.cpu()[named].double(), ref[named])
        else:
            close(got[named.cuda()], ref[named], U32 * ref[named].abs() + floor_of(torch.float32), dtype)
        assert torch.equal(got[~named.cuda()], before[~named.cuda()])        # rows that nothing names stay


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_sort_rows_backward(shape, dt):
    T, k, d, lost, spare, pad, shift = shape
    dtype = TYPES[dt]
    inv = assignments(T, k, 5, lost, spare)
    x, grad = tensor(T, d, dtype, 6, pad, shift), tensor(T * k + spare, d, dtype, 7, pad, shift)
    free = torch.ones(T * k + spare, dtype=torch.bool)
    free[inv[inv >= 0].long()] = False
    grad[free.cuda()] = float("nan")                                         # rows that nothing names are not read
    clean = torch.where(free[:, None], 0.0, grad.double().cpu())
    for w in (None, weights(T, k, 8)):
        ref, mag = gather_ref(clean, inv, w, T)
        wc = None if w is None else w.cuda()
        close(pkg().sort_rows_backward(grad, inv.cuda(), wc), ref, k * U32 * (1 + 2.0 ** -10) * mag, dtype)
        dx, dw = pkg().sort_rows_backward(grad, inv.cuda(), wc, x)
        close(dx, ref, k * U32 * (1 + 2.0 ** -10) * mag, dtype)
        dref, dmag = dots_ref(x, clean, inv)
        close(dw, dref, dot_slack(d, dmag), torch.float32)
        assert (dw.cpu()[inv < 0] == 0).all()


@pytest.mark.parametrize("yt", sorted(TYPES))
@pytest.mark.parametrize("ot", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_combine_rows(shape, yt, ot):
    T, k, d, lost, spare, pad, shift = shape
    inv, w = assignments(T, k, 9, lost, spare), weights(T, k, 10)
    y = tensor(T * k + spare, d, TYPES[yt], 11, pad, shift)
    ref, mag = gather_ref(y, inv, w, T)
    slack = k * U32 * (1 + 2.0 ** -10) * mag
    close(pkg().combine_rows(y, inv.cuda(), w.cuda(), out_dtype=TYPES[ot]), ref, slack, TYPES[ot])
    for st in TYPES:
        s = tensor(T, d, TYPES[st], 12, pad, shift)
        out = tensor(T, d, TYPES[ot], 13, pad, shift)
        got = pkg().combine_rows(y, inv.cuda(), w.cuda(), shared=s, out=out)
        total = ref + s.double().cpu()
        close(got, total, slack + U32 * (total.abs() + slack), TYPES[ot])


@pytest.mark.parametrize("gt", sorted(TYPES))
@pytest.mark.parametrize("yt", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_combine_rows_backward(shape, gt, yt):
    T, k, d, lost, spare, pad, shift = shape
    inv, w = assignments(T, k, 14, lost, spare), weights(T, k, 15)
    n = T * k + spare
    grad, y = tensor(T, d, TYPES[gt], 16, pad, shift), tensor(n, d, TYPES[yt], 17, pad, shift)
    ref, named = spread_ref(grad, inv, w, n)
    out = tensor(n, d, TYPES[yt], 18, pad, shift)
    before = out.clone()
    dy, dw = pkg().combine_rows_backward(grad, inv.cuda(), w.cuda(), y, out=out)
    close(dy[named.cuda()], ref[named], U32 * ref[named].abs() + floor_of(torch.float32), TYPES[yt])
    assert torch.equal(dy[~named.cuda()], before[~named.cuda()])
    dref, dmag = dots_ref(grad, y, inv)
    close(dw, dref, dot_slack(d, dmag), torch.float32)
    assert (dw.cpu()[inv < 0] == 0).all()
    plain = pkg().combine_rows_backward(grad, inv.cuda(), w.cuda(), out=tensor(n, d, TYPES[yt], 18, pad, shift))
    assert torch.equal(plain[named.cuda()], dy[named.cuda()])


def test_entries_behind_the_rows_are_dropped():
    T, k, d, n = 6, 2, 40, 7
    inv = assignments(T, k, 20)
    inv[0, 0], inv[1, 1] = 2**31 - 1, -2**31
    x, y = tensor(T, d, torch.float32, 21), tensor(n, d, torch.float32, 22)
    ref, named = spread_ref(x, inv, None, n)
    guard = torch.full((n + 4, d), 7.0, device="cuda")
    pkg().sort_rows(x, inv.cuda(), out=guard[:n])
    assert torch.equal(guard[:n][named.cuda()].double().cpu(), ref[named]) and (guard[n:] == 7.0).all()
    ref, mag = gather_ref(y, inv, None, T)
    close(pkg().combine_rows(y, inv.cuda()), ref, k * U32 * mag, torch.float32)


def test_no_tokens_and_no_rows():
    p, e = pkg(), torch.empty((0, 2), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    assert p.sort_rows(x, e).shape == (0, 16) and p.combine_rows(x, e).shape == (0, 16)
    assert p.sort_rows_backward(x, e, None, x)[1].shape == (0, 2)
    inv = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    s = tensor(3, 16, torch.bfloat16, 23)
    assert torch.equal(p.combine_rows(x, inv, shared=s), s)                  # all dropped: the shared term alone
    assert not p.combine_rows(x, inv).any()
    dy, dw = p.combine_rows_backward(s, inv, None, x)
    assert dy.shape == (0, 16) and not dw.any()


def test_special_values_stay_in_their_token():
    T, k, d = 8, 2, 64
    inv = assignments(T, k, 24)
    y = tensor(T * k, d, torch.bfloat16, 25)
    y[int(inv[2, 1]), 5], y[int(inv[4, 0]), 6] = float("nan"), float("inf")
    out = pkg().combine_rows(y, inv.cuda(), weights(T, k, 26).cuda())
    bad = ~torch.isfinite(out.float()).cpu()
    assert bad.sum() == 2 and bad[2, 5] and bad[4, 6]
    x = tensor(T, d, torch.bfloat16, 27)
    x.view(torch.int16)[0, 0] = 0x7FA5                                       # a NaN with a payload: bits are moved
    assert torch.equal(pkg().sort_rows(x, inv.cuda()).view(torch.int16)[inv.long().cuda()][:, 1], x.view(torch.int16))
    big = pkg().combine_rows(torch.full((2, 8), 6e4, device="cuda"), torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"),
                             out_dtype=torch.float16)
    assert torch.isinf(big).all()                                            # beyond fp16: infinity


def test_gradients_against_differences():
    """<G, sort(x, w)> and <g, combine(y, w)> are linear in each argument, so a central difference of any width has
    no truncation error; what remains are the fp32 roundings of the results."""
    T, k, d = 23, 4, 136
    p, inv = pkg(), assignments(T, k, 30, 0.2).cuda()
    r = lambda n, c, s: tensor(n, c, torch.float32, s)
    x, y, G, g, w = r(T, d, 31), r(T * k, d, 32), r(T * k, d, 33), r(T, d, 34), weights(T, k, 35).cuda()
    u, v, s = r(T, d, 36), r(T * k, d, 37), weights(T, k, 38).cuda()
    named = torch.zeros(T * k, 1, device="cuda", dtype=torch.float64)
    named[inv[inv >= 0].long()] = 1.0
    f = lambda x_, w_: (G.double() * named * p.sort_rows(x_, inv, w_, out=torch.zeros_like(y)).double())
    plus, minus = f(x + u, w + s), f(x - u, w - s)
    dx, dw = p.sort_rows_backward(G, inv, w, x)
    want = (dx.double() * u.double()).sum() + (dw.double() * s.double()).sum()
    # each of a, b = x +- u, w +- s, their product, and each gradient's sum rounds: fewer than 32 + d/32 steps a term
    room = (32 + d) * U32 * (plus.abs().sum() + minus.abs().sum() + (dx * u).abs().double().sum() * k
                             + (x.abs().double().sum(1, keepdim=True) * s.abs()).sum() * G.abs().max())
    assert abs(float((plus - minus).sum() / 2 - want)) <= float(room)
    h = lambda y_, w_: g.double() * p.combine_rows(y_, inv, w_).double()
    plus, minus = h(y + v, w + s), h(y - v, w - s)
    dy, dw = p.combine_rows_backward(g, inv, w, y, out=torch.zeros_like(y))
    want = (dy.double() * v.double()).sum() + (dw.double() * s.double()).sum()
    scale = p.combine_rows((y.abs() + v.abs()), inv, w + s.abs()).double()
    room = (32 + d) * U32 * 4 * (g.abs().double() * scale).sum()
    assert abs(float((plus - minus).sum() / 2 - want)) <= float(room)


def test_the_plan_path_and_own_experts_agree():
    """permute -> sort_rows -> experts -> combine_rows, as a user with experts of their own runs it, against
    forward_routed's formula: here each expert multiplies by a number of its own."""
    E, k, d, T = 16, 4, 128, 50
    p = pkg()
    plan = p.MoePlan(E, k, d, 64)
    plan.allocate_workspace(T)
    g = torch.Generator().manual_seed(40)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    gates, x = weights(T, k, 41).cuda(), tensor(T, d, torch.bfloat16, 42)
    _, offsets, perm, inv = plan.permute(ids)
    rows = p.sort_rows(x, inv.view(T, k))
    assert torch.equal(rows, x[(perm // k).long()])
    factor = torch.repeat_interleave(torch.arange(1, E + 1, device="cuda"), offsets.diff(), output_size=T * k).float()
    y = rows.float() * factor[:, None]
    out = p.combine_rows(y, inv.view(T, k), gates, out_dtype=torch.bfloat16)
    assert torch.equal(out, plan.combine(y, gates, inv))
    ref = x.double() * (gates.double() * (ids + 1)).sum(1, keepdim=True)
    mag = (x.double().abs() * (gates.double() * (ids + 1)).sum(1, keepdim=True)).cpu()
    close(out, ref.cpu(), (k + 1) * U32 * (1 + 2.0 ** -10) * mag, torch.bfloat16)


def test_graph_replay_and_another_stream():
    T, k, d = 70, 8, 512
    p, inv, w = pkg(), assignments(T, k, 50, 0.1).cuda(), weights(T, k, 51).cuda()
    x, y = tensor(T, d, torch.bfloat16, 52), tensor(T * k, d, torch.bfloat16, 53)
    def step():
        return (*p.combine_rows_backward(x, inv, w, y, out=bufs[0]), p.combine_rows(y, inv, w, out=bufs[1]),
                *p.sort_rows_backward(y, inv, w, x, out=bufs[2]), p.sort_rows(x, inv, out=bufs[3]))
    bufs = [torch.zeros_like(y), torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(y)]
    want = [t.clone() for t in step()]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = p.combine_rows(y, inv, w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(other, want[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for b in bufs:
        b.zero_()
    x2, y2 = x.clone(), y.clone()
    for scale in (2.0, 1.0):
        x.copy_(x2 * scale), y.copy_(y2 * scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[2], (want[2].float() * scale).to(torch.bfloat16))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    p = pkg()
    x, inv = tensor(4, 16, torch.bfloat16, 60), assignments(4, 2, 61).cuda()
    y, w = tensor(8, 16, torch.bfloat16, 62), weights(4, 2, 63).cuda()
    for call in (lambda: p.sort_rows(x, inv.view(-1)), lambda: p.sort_rows(x, inv.long()), lambda: p.sort_rows(x[:3], inv),
                 lambda: p.sort_rows(x, inv, w.double()), lambda: p.sort_rows(x, inv, w[:, :1]),
                 lambda: p.sort_rows(x.double(), inv), lambda: p.sort_rows(x, inv, out=y.float()),
                 lambda: p.sort_rows(x, inv, out=y[:, :8]), lambda: p.sort_rows(x.t(), inv), lambda: p.sort_rows(x, inv.cpu()),
                 lambda: p.sort_rows(y[:4], inv, out=y), lambda: p.combine_rows(y, inv, out=y[:4]),
                 lambda: p.combine_rows(y, inv, w, shared=x[:2]), lambda: p.combine_rows(y, inv, out_dtype=torch.float64),
                 lambda: p.combine_rows(y, inv, out=x[:3]), lambda: p.sort_rows_backward(y, inv, w, x.float()),
                 lambda: p.sort_rows_backward(y, inv, out=x[:1]), lambda: p.combine_rows_backward(x, inv, w, y, out=y),
                 lambda: p.combine_rows_backward(x, inv, w, y, out=y[:6].clone()),
                 lambda: p.combine_rows_backward(x[:2], inv, w, y)):
        with pytest.raises((ValueError, p.MoeError)):
            call()
