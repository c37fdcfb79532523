"""8-bit blocks and the 8-bit projection against their 64-bit forms (tests/fp8_helpers.py)."""
import pytest
import torch

from fp8_helpers import blocks, product_ref, quantize_rows_ref, quantize_weight_ref, random_rows, random_weight, sum_tolerance

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def pkg():
    import decode_batches_gb300 as m
    return m


def make_linear(N, K, T_max, seed=1):
    wq, ws = random_weight(N, K, seed)
    lin = pkg().Fp8Linear(N, K)
    lin.set_weights(wq.cuda(), ws.cuda())
    lin.allocate_workspace(max(1, T_max))
    return lin, wq, ws


def check(out, xq, xs, wq, ws):
    ref, mag = product_ref(xq, xs, wq, ws)
    got = out.double().cpu()
    tol = sum_tolerance(wq.shape[1]) * mag
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    bad = (got - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}: worst {float(((got - ref).abs() / tol.clamp_min(1e-300)).max()):.2f} x"


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K", [(1, 1), (3, 127), (5, 128), (7, 129), (33, 1000), (130, 2048)])
def test_rows_quantise_bit_for_bit(T, K, dtype):
    x = random_rows(T, K, 3, DT[dtype])
    if T > 2:
        x[1] = 0                                  # an empty block: smallest scale, codes zero
        x[2] = x[2] * 1e-6
    q, s = pkg().quantize_fp8(x.cuda())
    rq, rs = quantize_rows_ref(x)
    assert q.shape == (T, K) and s.shape == (T, blocks(K))
    assert torch.equal(s.double().cpu(), rs)
    assert torch.equal(q.float().double().cpu(), rq)


def test_rows_quantise_strided_unaligned_and_tiny():
    g = torch.Generator().manual_seed(9)
    big = torch.randn((9, 700), generator=g).to(torch.bfloat16)
    for view in (big[:, 1:301], big[::2, 8:520], big[:, 3:4]):
        q, s = pkg().quantize_fp8(big.cuda().as_strided(view.shape, view.stride(), view.storage_offset()))
        rq, rs = quantize_rows_ref(view)
        assert torch.equal(s.double().cpu(), rs) and torch.equal(q.float().double().cpu(), rq)
    tiny = torch.tensor([[2.0 ** -140, -2.0 ** -149, 0.0, 2.0 ** -133]])   # below the smallest scale's grid
    q, s = pkg().quantize_fp8(tiny.cuda())
    rq, rs = quantize_rows_ref(tiny)
    assert torch.equal(s.double().cpu(), rs) and torch.equal(q.float().double().cpu(), rq)
    q, s = pkg().quantize_fp8(torch.empty((0, 64), device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0, 1)


def test_rows_quantise_nan_and_infinity():
    x = torch.ones((3, 256))
    x[0, 5] = float("nan")
    x[1, 200] = float("inf")
    q, s = pkg().quantize_fp8(x.cuda())
    q, s = q.float().cpu(), s.cpu()
    assert q[0, 5].isnan() and not q[0, 6].isnan() and float(q[0, 6]) == 448.0
    assert s[1, 1] == float("inf") and q[1, 200].isnan() and float(q[1, 5]) == 448.0
    assert torch.equal(q[2], torch.full((256,), 448.0))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (130, 257), (300, 1000), (2, 64, 96)])
def test_weights_quantise_bit_for_bit(shape, dtype):
    g = torch.Generator().manual_seed(4)
    w = torch.randn(shape, generator=g).to(DT[dtype])
    q, s = pkg().quantize_fp8_weight(w.cuda())
    assert q.shape == shape
    for i, m in enumerate(w.view(-1, *shape[-2:])):
        rq, rs = quantize_weight_ref(m)
        assert torch.equal(q.view(-1, *shape[-2:])[i].float().cpu(), rq.float())
        assert torch.equal(s.view(-1, *s.shape[-2:])[i].cpu(), rs)


@pytest.mark.parametrize("T,N,K", [
    (1, 1, 1), (1, 128, 128), (1, 256, 4096), (2, 129, 127), (3, 257, 130), (16, 512, 640), (31, 1000, 1000),
    (32, 384, 256), (33, 383, 513), (64, 2048, 2048), (127, 256, 384), (128, 256, 512), (129, 300, 777),
    (257, 1337, 1000), (700, 640, 2048), (1300, 2048, 512)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_linear_against_64_bits(T, N, K, out):
    lin, wq, ws = make_linear(N, K, T)
    x = random_rows(T, K, 5)
    got = lin.forward(x.cuda(), out_dtype=DT[out])
    assert got.shape == (T, N) and got.dtype == DT[out]
    check(got, *quantize_rows_ref(x), wq, ws)
    assert lin.device_error() == 0


# More units than half the SMs (no split): whole sets of 32 rows leave as boxes of 64 columns, the rest of
# a part as row pieces; N ends before, at and behind a box's last column, and nothing outside is written.
@pytest.mark.parametrize("N", [1320, 1344, 1352, 1536])
@pytest.mark.parametrize("T", [2048, 2100])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_linear_many_rows_into_a_wider_output(T, N, out):
    K = 384
    lin, wq, ws = make_linear(N, K, T)
    x = random_rows(T, K, 8)
    wide = torch.full((T + 40, N + 24), 7.0, dtype=DT[out], device="cuda")
    got = wide[16:16 + T, 16:16 + N]
    lin.forward(x.cuda(), out=got, out_dtype=DT[out])
    check(got, *quantize_rows_ref(x), wq, ws)
    assert (wide[:16] == 7).all() and (wide[16 + T:] == 7).all()
    assert (wide[:, :16] == 7).all() and (wide[:, 16 + N:] == 7).all()
    assert lin.device_error() == 0


@pytest.mark.parametrize("dtype", list(DT))
def test_linear_strided_rows_and_output(dtype):
    T, N, K = 50, 264, 200
    lin, wq, ws = make_linear(N, K, T)
    big = random_rows(T, K + 40, 6, DT[dtype])
    for off in (0, 8, 3):                         # aligned, vector-aligned and odd starts
        x = big.cuda()[:, off:off + K]
        out = torch.full((T, N + 24), 7.0, dtype=torch.float32, device="cuda")
        for col in (0, 8, 5):
            lin.forward(x, out=out[:, col:col + N])
            check(out[:, col:col + N], *quantize_rows_ref(big[:, off:off + K]), wq, ws)
            rest = torch.ones(N + 24, dtype=torch.bool)
            rest[col:col + N] = False
            assert (out[:, rest] == 7.0).all()    # nothing beyond the row's N columns is written
            out.fill_(7.0)


def test_linear_quantised_rows_are_the_same_call():
    T, N, K = 70, 500, 1100
    lin, wq, ws = make_linear(N, K, T)
    x = random_rows(T, K, 8).cuda()
    q, s = pkg().quantize_fp8(x)
    assert torch.equal(lin.forward_quantized(q, s, out_dtype=torch.float32), lin.forward(x, out_dtype=torch.float32))
    assert torch.equal(lin.forward_quantized(q[:1], s[:1]), lin.forward(x[:1]))
    # columns beyond K are not read, whatever they hold
    wide = torch.full((T, 1280), float("nan"), device="cuda").to(torch.float8_e4m3fn)
    wide[:, :K] = q
    assert torch.equal(lin.forward_quantized(wide[:, :K], s), lin.forward(x))


def test_linear_is_run_to_run_identical_and_row_independent():
    T, N, K = 300, 512, 1536
    lin, _, _ = make_linear(N, K, T)
    x = random_rows(T, K, 11).cuda()
    a = lin.forward(x, out_dtype=torch.float32)
    assert torch.equal(a, lin.forward(x, out_dtype=torch.float32))
    y = x.clone()
    y[17] = float("nan")
    y[200, 3] = float("inf")
    b = lin.forward(y, out_dtype=torch.float32)
    keep = torch.ones(T, dtype=torch.bool)
    keep[[17, 200]] = False
    assert torch.equal(a[keep], b[keep]) and b[17].isnan().all() and b[200].isnan().all()


def test_linear_nan_weight_reaches_its_column_only():
    N, K, T = 200, 300, 20
    wq, ws = random_weight(N, K, 2)
    wq[150, 299] = float("nan")
    lin = pkg().Fp8Linear(N, K)
    lin.set_weights(wq.cuda(), ws.cuda())
    lin.allocate_workspace(T)
    out = lin.forward(random_rows(T, K, 1).cuda(), out_dtype=torch.float32).cpu()
    assert out[:, 150].isnan().all() and not out[:, torch.arange(N) != 150].isnan().any()


def test_linear_on_another_stream_in_a_graph_and_with_zero_rows():
    T, N, K = 40, 256, 512
    lin, wq, ws = make_linear(N, K, T)
    x = random_rows(T, K, 12)
    xc = x.cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = lin.forward(xc, stream=st)
    st.synchronize()
    check(out, *quantize_rows_ref(x), wq, ws)
    assert lin.forward(xc[:0]).shape == (0, N)
    g = torch.cuda.CUDAGraph()
    buf = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    with torch.cuda.graph(g):
        lin.forward(xc, out=buf)
    xc.copy_(random_rows(T, K, 13).cuda())
    g.replay()
    torch.cuda.synchronize()
    check(buf, *quantize_rows_ref(random_rows(T, K, 13)), wq, ws)


def test_linear_large_grid_and_reused_weights():
    """More units than CTAs (several units a CTA, both TMEM buffers and all stages reused), and new
    weights in the same handle."""
    T, N, K = 2100, 4224, 384
    lin, wq, ws = make_linear(N, K, T)
    x = random_rows(T, K, 14)
    check(lin.forward(x.cuda(), out_dtype=torch.float32), *quantize_rows_ref(x), wq, ws)
    wq, ws = random_weight(N, K, 77)
    lin.set_weights(wq.cuda(), ws.cuda())
    check(lin.forward(x.cuda()), *quantize_rows_ref(x), wq, ws)


def test_linear_refusals():
    m = pkg()
    for n, k in ((0, 5), (5, 0), (1 << 21, 5), (-1, 5)):
        with pytest.raises(m.MoeError):
            m.Fp8Linear(n, k)
    lin = m.Fp8Linear(64, 96)
    x = torch.zeros((4, 96), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(m.MoeError):               # no weights yet
        lin.forward(x)
    wq, ws = random_weight(64, 96, 0)
    with pytest.raises(ValueError):
        lin.set_weights(wq.cuda()[:, :64].contiguous(), ws.cuda())
    with pytest.raises(ValueError):
        lin.set_weights(wq.cuda(), ws.cuda().double())
    lin.set_weights(wq.cuda(), ws.cuda())
    with pytest.raises(m.MoeError):               # no workspace yet
        lin.forward(x)
    with pytest.raises(m.MoeError):
        lin.set_workspace(torch.empty(64, dtype=torch.uint8, device="cuda"), 4)
    lin.allocate_workspace(3)
    with pytest.raises(m.MoeError):               # more rows than the workspace holds
        lin.forward(x)
    x = x[:3]
    for bad in (x.int(), x.cpu(), x[:, :95], x.t(), x[None]):
        with pytest.raises(ValueError):
            lin.forward(bad)
    with pytest.raises(ValueError):
        lin.forward(x, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        lin.forward(x, out=torch.empty((2, 64), dtype=torch.bfloat16, device="cuda"))
    q, s = m.quantize_fp8(x)
    with pytest.raises(ValueError):
        lin.forward_quantized(q, s[:2])
    with pytest.raises(m.MoeError):               # scale rows of an odd pitch
        lin.forward_quantized(q, s.contiguous())
    with pytest.raises(ValueError):
        m.quantize_fp8(x.int())
    with pytest.raises(ValueError):
        m.quantize_fp8(x[0])
