"""Calls on a stream of their own while the current stream is busy: their results, and the copies that they
make, must not lie in memory that queued work of the current stream still uses, nor wait for it."""
import pytest
import torch

from fp8_helpers import quantize_rows_ref, quantize_weight_ref, random_rows
from test_gpu_fp8_experts import make_plan, routing
from test_gpu_fp8_linear import make_linear, pkg

pytestmark = pytest.mark.gpu
BUSY = 50_000_000                                 # cycles: some 25 ms


def beside_busy_work(shape, dtype, call):
    """call(stream) while the current stream is about to read a freed tensor like call's result; the copy
    that it makes of that tensor must be whole."""
    st = torch.cuda.Stream()
    call(None), call(st)                          # lazy set-up, and memory in both streams' pools
    torch.cuda.synchronize()
    old = torch.full(shape, 3, device="cuda").to(dtype)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    copy = old.clone()
    del old                                       # free for the current stream, in whose order the copy was queued
    got = call(st)
    st.synchronize()
    torch.cuda.synchronize()
    assert (copy.float() == 3).all()
    return got


@pytest.mark.parametrize("T", [3, 200])
def test_layer_results_on_another_stream(T):
    E, k, d, f = 16, 4, 256, 128
    plan, *_ = make_plan(E, k, d, f, T)
    x = random_rows(T, d, 3).cuda()
    ids, gates = (a.cuda() for a in routing(T, E, k, 4))
    logits, rids, rgates = plan.route(x)
    want, routed = plan.forward(x), plan.forward_routed(x, ids, gates)
    _, offsets, perm, inv = plan.permute(ids)
    y, _ = plan.experts(x, offsets, perm)
    bf = torch.bfloat16
    assert torch.equal(want, beside_busy_work((T, d), bf, lambda s: plan.forward(x, stream=s)))
    assert torch.equal(routed, beside_busy_work((T, d), bf, lambda s: plan.forward_routed(x, ids, gates, stream=s)))
    assert torch.equal(logits, beside_busy_work((T, E), torch.float32, lambda s: plan.route(x, stream=s)[0]))
    assert torch.equal(rids, beside_busy_work((T, k), torch.int32, lambda s: plan.route_logits(logits, stream=s)[0]))
    assert torch.equal(perm, beside_busy_work((T * k,), torch.int32, lambda s: plan.permute(ids, stream=s)[2]))
    assert torch.equal(y, beside_busy_work((T * k, d), torch.float16, lambda s: plan.experts(x, offsets, perm, stream=s)[0]))
    yf = y.float()
    assert torch.equal(routed, beside_busy_work((T, d), bf, lambda s: plan.combine(yf, gates, inv, stream=s)))


def test_8_bit_results_on_another_stream():
    T, N, K = 90, 256, 384
    lin, _, _ = make_linear(N, K, T)
    x = random_rows(T, K, 5)
    xc = x.cuda()
    assert torch.equal(lin.forward(xc), beside_busy_work((T, N), torch.bfloat16, lambda s: lin.forward(xc, stream=s)))
    q, s = pkg().quantize_fp8(xc)
    got = beside_busy_work((T, N), torch.float32, lambda st: lin.forward_quantized(q, s, out_dtype=torch.float32, stream=st))
    assert torch.equal(got, lin.forward(xc, out_dtype=torch.float32))
    codes = beside_busy_work((T, K), torch.float8_e4m3fn, lambda st: pkg().quantize_fp8(xc, stream=st)[0])
    assert torch.equal(codes.float().double().cpu(), quantize_rows_ref(x)[0])


def test_transposed_weight_on_another_stream():
    """A weight that is not contiguous is copied on the stream that quantises it."""
    w = torch.randn((300, 260), generator=torch.Generator().manual_seed(1))
    wc = w.t().contiguous().cuda().t()
    assert not wc.is_contiguous()
    q, s = beside_busy_work((300, 260), torch.float32, lambda st: pkg().quantize_fp8_weight(wc, stream=st))
    rq, rs = quantize_weight_ref(w)
    assert torch.equal(q.float().cpu(), rq.float()) and torch.equal(s.cpu(), rs)


def test_an_error_right_after_the_word_was_read_is_kept():
    """Reading the error word clears it before the call returns, so a fault on another stream just after it
    is not cleared away."""
    from decode_batches_gb300 import DEVERR_EXPERT_RANGE
    T, E, k, d = 4, 8, 2, 128
    plan, *_ = make_plan(E, k, d, 128, T)
    x, gates = random_rows(T, d, 3).cuda(), torch.ones((T, k), device="cuda")
    bad = torch.full((T, k), E, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(200):
            plan.forward_routed(x, bad, gates)
            assert plan.device_error() == DEVERR_EXPERT_RANGE
