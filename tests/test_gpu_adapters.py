"""Low-rank adapters against the formula in 64 bits."""
import pytest
import torch

from rows_helpers import TYPES, U32, close, tensor

pytestmark = pytest.mark.gpu
HALF = {"bf16": torch.bfloat16, "fp16": torch.float16}


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


def make(n, N, K, rank, dtype, seed, ranks=None, T_max=1100):
    """(handle, per-slot (A, B, scale) in fp64); ranks[i] == 0 leaves a slot empty"""
    g = torch.Generator().manual_seed(seed)
    ad, slots = pkg().LowRankAdapters(n, N, K, rank, dtype), []
    for i in range(n):
        r = rank if ranks is None else ranks[i % len(ranks)]
        A = (torch.randn((r, K), generator=g) * K ** -0.5).to(dtype)
        B = torch.randn((N, r), generator=g).to(dtype)
        scale = 2.0 ** float(torch.randint(-2, 3, (1,), generator=g)) * 0.75
        if r:
            ad.set(i, A.cuda(), B.cuda(), scale)
        slots.append((A.double(), B.double(), scale))
    ad.allocate_workspace(T_max)
    return ad, slots


def reference(x, ids, base, slots, dtype):
    """(fp64 result, slack of the arithmetic).  u = s A x: sums of K products in the tensor core (each step of 16 may
    lose 2^-20 of the magnitudes so far, K 2^-24 in all; 2^-23 here), joined over warps and CTAs (64 steps at most); two
    16-bit terms of u (2^-16 of u in bf16, 2^-22 of the row's largest in fp16); sums of 2 r products; the base added."""
    x = x.double().cpu()
    T, N = x.shape[0], slots[0][1].shape[0]
    out = torch.zeros((T, N), dtype=torch.float64) if base is None else base.double().cpu()
    slack = torch.zeros((T, N), dtype=torch.float64)
    for a in sorted(set(ids.tolist())):
        if not 0 <= a < len(slots) or not slots[a][0].shape[0]:
            continue
        t = torch.nonzero(ids == a)[:, 0]
        A, B, s = slots[a]
        u, mag = s * x[t] @ A.T, abs(s) * x[t].abs() @ A.abs().T
        held = 2.0 ** -16 * u.abs() if dtype == torch.bfloat16 else 2.0 ** -22 * u.abs().amax(1, keepdim=True)
        du = (x.shape[1] + 64) * 2 * U32 * mag + held
        out[t] += u @ B.T
        slack[t] += (du + (2 * A.shape[0] + 64) * 2 * U32 * u.abs()) @ B.abs().T
    return out, (slack + U32 * out.abs()) * (1 + 2.0 ** -8)


def ids_of(kind, T, n, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, n, (T,), generator=g)
    if kind == "one":
        ids[:] = n - 1
    elif kind == "none":
        ids[:] = -1
    elif kind == "runs":
        ids = torch.arange(T) * min(n, 3) // T
        ids[-3:] = torch.arange(len(ids[-3:])) % n
    elif kind == "holes":
        ids = torch.where(torch.rand(T, generator=g) < 0.4, -1, ids)
    return ids.int()


# (T, n, rank, K, N, pad, shift)
SHAPES = [(1, 1, 1, 1, 1, 0, 0), (1, 3, 16, 256, 256, 0, 0), (5, 3, 4, 8, 40, 0, 0), (17, 2, 8, 33, 31, 1, 1),
          (48, 40, 32, 200, 264, 8, 8), (33, 5, 17, 1000, 72, 0, 0), (70, 7, 64, 512, 320, 0, 0), (40, 3, 100, 264, 96, 0, 0),
          (256, 3, 16, 128, 1337, 0, 0), (257, 5, 16, 264, 136, 0, 0), (300, 4, 33, 96, 200, 8, 0), (700, 40, 64, 160, 64, 0, 0),
          (1030, 6, 128, 72, 48, 0, 8), (1100, 300, 8, 40, 32, 3, 1)]


@pytest.mark.parametrize("ot", sorted(TYPES))
@pytest.mark.parametrize("dt", sorted(HALF))
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dt, ot):
    T, n, rank, K, N, pad, shift = shape
    ranks = [rank, max(1, rank // 2), rank, 0] if n > 2 else [rank]
    ad, slots = make(n, N, K, rank, HALF[dt], T + n, ranks)
    x = tensor(T, K, HALF[dt], 1, pad, shift)
    for kind in ("mixed", "one", "none", "runs", "holes"):
        ids = ids_of(kind, T, n, 2)
        base = tensor(T, N, TYPES[ot], 3, pad, shift)
        ref, slack = reference(x, ids, base, slots, HALF[dt])
        got = ad.forward(x, ids.cuda(), base)
        close(got, ref, slack, TYPES[ot])
        same = ad.forward(x, ids.cuda(), base.clone())
        assert torch.equal(same, got)                                # a row's result does not depend on its place
        inplace = base.clone()
        wide = tensor(T, N, TYPES[ot], 4, pad, shift)
        wide.copy_(base)
        ad.forward(x, ids.cuda(), wide, out=wide)
        ad.forward(x, ids.cuda(), inplace, out=inplace)
        assert torch.equal(wide, got) and torch.equal(inplace, got)
        if kind == "none":
            assert torch.equal(got, base)
    ref, slack = reference(x, ids, None, slots, HALF[dt])
    close(ad.forward(x, ids.cuda(), out_dtype=TYPES[ot]), ref, slack, TYPES[ot])
    assert ad.device_error() == 0


@pytest.mark.parametrize("T", [1, 40, 300])
def test_result_does_not_depend_on_the_other_rows(T):
    ad, _ = make(4, 128, 256, 32, torch.bfloat16, 11)
    x, base = tensor(T, 256, torch.bfloat16, 12), tensor(T, 128, torch.float32, 13)
    ids = ids_of("mixed", T, 4, 14)
    got = ad.forward(x, ids.cuda(), base)
    order = torch.randperm(T, generator=torch.Generator().manual_seed(15)).cuda()
    again = ad.forward(x[order].contiguous(), ids.cuda()[order].contiguous(), base[order].contiguous())
    assert torch.equal(again, got[order])


def test_slots_come_and_go():
    ad, slots = make(3, 96, 64, 16, torch.bfloat16, 21)
    x, base, ids = tensor(9, 64, torch.bfloat16, 22), tensor(9, 96, torch.bfloat16, 23), ids_of("mixed", 9, 3, 24)
    before = ad.forward(x, ids.cuda(), base)
    g = torch.Generator().manual_seed(25)
    A, B = torch.randn((5, 64), generator=g).bfloat16(), torch.randn((96, 5), generator=g).bfloat16()
    ad.set(1, A.cuda(), B.cuda(), -0.5)
    slots[1] = (A.double(), B.double(), -0.5)
    got = ad.forward(x, ids.cuda(), base)
    ref, slack = reference(x, ids, base, slots, torch.bfloat16)
    close(got, ref, slack, torch.bfloat16)
    others = (ids != 1).cuda()
    assert torch.equal(got[others], before[others])
    ad.clear(1)
    assert torch.equal(ad.forward(x, ids.cuda(), base)[~others], base[~others])


@pytest.mark.parametrize("T", [6, 400])
def test_ids_outside_the_slots_set_the_error_bit(T):
    ad, slots = make(2, 64, 64, 8, torch.float16, 31)
    x, base = tensor(T, 64, torch.float16, 32), tensor(T, 64, torch.float32, 33)
    ids = ids_of("mixed", T, 2, 34)
    ids[1], ids[3], ids[4] = 2, -2, 2**31 - 1
    got = ad.forward(x, ids.cuda(), base)
    ref, slack = reference(x, ids, base, slots, torch.float16)
    close(got, ref, slack, torch.float32)
    assert ad.device_error() == pkg().DEVERR_EXPERT_RANGE and ad.device_error() == 0


@pytest.mark.parametrize("dt", sorted(HALF))
@pytest.mark.parametrize("T", [20, 300])
def test_wide_ranges_and_special_values(T, dt):
    """u beyond fp16's range and far below it; NaN and infinite rows stay by themselves."""
    dtype = HALF[dt]
    ad, N = pkg().LowRankAdapters(2, 64, 64, 8, dtype), 64
    A, B = torch.full((8, 64), 100.0), torch.eye(64, 8) * 2.0 ** -10
    A[1] *= 2.0 ** -12
    ad.set(0, A.to(dtype).cuda(), B.to(dtype).cuda(), 16.0)
    ad.allocate_workspace(T)
    x = torch.zeros((T, 64), dtype=dtype)
    x[:] = 64.0
    x[1] = 2.0 ** -14
    x[2, 5], x[3, 6] = float("nan"), float("inf")
    ids = torch.zeros(T, dtype=torch.int32)
    got = ad.forward(x.cuda(), ids.cuda(), out_dtype=torch.float32).cpu()
    ref, slack = reference(x, ids, None, [(A.to(dtype).double(), B.to(dtype).double(), 16.0)], dtype)
    keep = torch.ones(T, dtype=torch.bool)
    keep[2:4] = False
    close(got[keep], ref[keep], slack[keep], torch.float32)
    assert torch.isnan(got[2]).any() and not torch.isfinite(got[3]).all()
    empty = torch.ones(T, dtype=torch.int32)                          # slot 1 holds nothing: x is not looked at
    assert not ad.forward(x.cuda(), empty.cuda(), out_dtype=torch.float32).any()


def test_beside_an_8_bit_projection():
    p = pkg()
    N, K, T = 200, 264, 37
    w = tensor(N, K, torch.bfloat16, 41)
    lin = p.Fp8Linear(N, K)
    lin.set_weights(*p.quantize_fp8_weight(w))
    lin.allocate_workspace(512)
    ad, slots = make(5, N, K, 16, torch.bfloat16, 42, T_max=512)
    for T in (1, 37, 500):
        x, ids = tensor(T, K, torch.bfloat16, 43), ids_of("holes", T, 5, 44)
        for dtype in (torch.bfloat16, torch.float32):
            base = lin.forward(x, out_dtype=dtype)
            got = lin.forward(x, out_dtype=dtype, adapters=ad, adapter_ids=ids.cuda())
            assert torch.equal(got, ad.forward(x, ids.cuda(), base))
            ref, slack = reference(x, ids, base, slots, torch.bfloat16)
            close(got, ref, slack, dtype)
            out = torch.empty_like(base)
            assert lin.forward(x, out, adapters=ad, adapter_ids=ids.cuda()) is out and torch.equal(out, got)
    for bad in (dict(adapters=ad), dict(adapter_ids=ids.cuda()), dict(adapters=ad, adapter_ids=ids[:-1].cuda()),
                dict(adapters=make(1, N, 8, 4, torch.bfloat16, 45)[0], adapter_ids=ids.cuda()),
                dict(adapters=make(1, N, K, 4, torch.bfloat16, 45, T_max=8)[0], adapter_ids=ids.cuda()),
                dict(adapters=make(1, N, K, 4, torch.float16, 45)[0], adapter_ids=ids.cuda())):
        with pytest.raises(ValueError):
            lin.forward(x, **bad)


@pytest.mark.parametrize("T", [24, 300])
def test_graph_replay_and_another_stream(T):
    ad, slots = make(6, 160, 192, 16, torch.bfloat16, 51)
    x, base = tensor(T, 192, torch.bfloat16, 52), tensor(T, 160, torch.bfloat16, 53)
    ids = ids_of("holes", T, 6, 54).cuda()
    want = ad.forward(x, ids, base)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = ad.forward(x, ids, base, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ad.forward(x, ids, base)
    ids2 = ids_of("mixed", T, 6, 55)
    ids.copy_(ids2)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    ref, slack = reference(x, ids2, base, slots, torch.bfloat16)
    close(got, ref, slack, torch.bfloat16)
    assert ad.device_error() == 0


def test_no_rows_and_refusals():
    p = pkg()
    ad, _ = make(2, 64, 32, 8, torch.bfloat16, 61, T_max=8)
    x, ids, base = tensor(4, 32, torch.bfloat16, 62), ids_of("mixed", 4, 2, 63).cuda(), tensor(4, 64, torch.float32, 64)
    assert ad.forward(x[:0], ids[:0], base[:0]).shape == (0, 64)
    big = tensor(9, 32, torch.bfloat16, 65)
    for call in (lambda: ad.forward(x.half(), ids, base), lambda: ad.forward(x.float(), ids, base),
                 lambda: ad.forward(x[:, :31], ids, base), lambda: ad.forward(x, ids.long(), base),
                 lambda: ad.forward(x, ids[:3], base), lambda: ad.forward(x, ids, base[:3]),
                 lambda: ad.forward(x, ids, base[:, :63]), lambda: ad.forward(x, ids, base.double()),
                 lambda: ad.forward(x, ids, base, out=base.bfloat16()), lambda: ad.forward(x, ids, base, out_dtype=torch.bfloat16),
                 lambda: ad.forward(x, ids, out_dtype=torch.float64), lambda: ad.forward(x, ids.cpu(), base),
                 lambda: ad.forward(x, ids, base[:1].expand(4, 64)), lambda: ad.forward(x, ids, base[:3], out=base[1:]),
                 lambda: ad.forward(big, torch.zeros(9, dtype=torch.int32, device="cuda")),
                 lambda: ad.set(2, x[:, :32], base[:, :4].bfloat16()), lambda: ad.set(2**32, x[:2], x[:2].t().contiguous()),
                 lambda: ad.clear(-1), lambda: ad.clear(2), lambda: ad.set(0, x, base.bfloat16()),
                 lambda: ad.set(0, x.half(), base[:, :4].half()), lambda: p.LowRankAdapters(2, 8, 8, 8, torch.float32),
                 lambda: p.LowRankAdapters(2, 8, 8, 200), lambda: p.LowRankAdapters(2, 8, 8, 8).forward(x[:, :8], ids)):
        with pytest.raises((ValueError, p.MoeError)):
            call()
    # one row's tensors overlap with the output of another: refused; the same rows: in place
    buf = torch.zeros((5, 64), device="cuda")
    with pytest.raises(ValueError):
        ad.forward(x, ids, buf[:4], out=buf[1:])
    ad.forward(x, ids, buf[:4], out=buf[:4])
    # parts of one wide buffer: other columns of the same rows are no overlap, shared ones are
    wide = torch.zeros((4, 160), dtype=torch.float32, device="cuda")
    wide[:, :64] = base
    assert torch.equal(ad.forward(x, ids, wide[:, :64], out=wide[:, 64:128]), ad.forward(x, ids, base))
    with pytest.raises(ValueError):
        ad.forward(x, ids, wide[:, :64], out=wide[:, 60:124])


def test_two_handles_on_two_streams():
    """Calls of two handles, and of verify_drafts, at the same time: nothing of a call is shared."""
    a, b = make(4, 256, 512, 16, torch.bfloat16, 71)[0], make(7, 192, 384, 40, torch.float16, 72)[0]
    xa, xb = tensor(700, 512, torch.bfloat16, 73), tensor(1100, 384, torch.float16, 74)
    ia, ib = ids_of("mixed", 700, 4, 75).cuda(), ids_of("holes", 1100, 7, 76).cuda()
    p = torch.softmax(tensor(96, 5000, torch.float32, 77), 1)
    off = torch.arange(0, 97, 4, dtype=torch.int32, device="cuda")
    d = torch.zeros(96, dtype=torch.int32, device="cuda")
    u, us = torch.rand(96, device="cuda"), torch.rand(24, device="cuda")
    calls = [lambda: a.forward(xa, ia), lambda: b.forward(xb, ib, out_dtype=torch.float32),
             lambda: pkg().verify_drafts(p, d, off, u, us)[0]]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(20):
        for i, (c, st) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(st):
                got[i].append(c())
    torch.cuda.synchronize()
    for w, results in zip(want, got):
        assert all(torch.equal(w, r) for r in results)
    assert a.device_error() == b.device_error() == 0
