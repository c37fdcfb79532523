"""verify_drafts against exact rational arithmetic.  Tokens are whole numbers and have to be equal."""
import pytest
import torch

from verify_helpers import verify_ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def pkg():
    import decode_batches_gb300
    return decode_batches_gb300


def place(x, pad=0, shift=0):
    """x on the GPU with a row pitch of V + pad, starting `shift` elements into its memory."""
    R, V = x.shape
    buf = torch.full((R * (V + pad) + shift,), float("nan"), dtype=x.dtype, device="cuda")
    out = buf[shift:].view(R, V + pad)[:, :V]
    out.copy_(x)
    return out


def inputs(counts, V, dtype, seed, sharp=1.0):
    g = torch.Generator().manual_seed(seed)
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    R = offsets[-1]
    l = sharp * torch.randn((R, V), generator=g)
    p = torch.softmax(l, 1).to(dtype)
    q = torch.softmax(l + 0.5 * torch.randn((R, V), generator=g), 1).to(dtype)
    d = torch.multinomial(q.float(), 1, generator=g)[:, 0].int() if R else torch.empty(0, dtype=torch.int32)
    return p, q, d, offsets, torch.rand(R, generator=g), torch.rand(len(counts), generator=g)


def check(p, q, d, offsets, u, us, pad=0, shift=0, qshift=None):
    ref, racc = verify_ref(p, d.tolist(), offsets, u.tolist(), us.tolist(), q)
    tokens = torch.full((p.shape[0],), -7, dtype=torch.int32, device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got, acc = pkg().verify_drafts(place(p, pad, shift), d.cuda(), off, u.cuda(), us.cuda(),
                                   None if q is None else place(q, pad, shift if qshift is None else qshift), tokens=tokens)
    assert got is tokens
    assert acc.tolist() == racc
    assert got.tolist() == [-7 if t is None else t for t in ref]


COUNTS = [[1], [6], [6, 6, 6, 6], [1, 3, 1, 8, 2, 0, 5], [40], [0, 0], [300]]


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("V", [1, 2, 7, 32, 129, 1000, 4097])
@pytest.mark.parametrize("counts", COUNTS)
def test_against_exact_arithmetic(counts, V, dt):
    if sum(counts) * V > 200000:
        counts = counts[:1] if counts != [300] else [20]
    p, q, d, off, u, us = inputs(counts, V, TYPES[dt], V + len(counts))
    check(p, q, d, off, u, us)
    check(p, None, d, off, u, us)
    check(p, q, d, off, u, us, pad=5, shift=3)
    check(p, q, d, off, u, us, pad=8, shift=8, qshift=5)          # p and q aligned differently


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("V,pad", [(32003, 0), (131072, 0), (151553, 7)])
def test_large_vocabularies(V, pad, dt):
    p, q, d, off, u, us = inputs([3, 1, 2], V, TYPES[dt], V, sharp=2.0)
    check(p, q, d, off, u, us, pad=pad)
    u[0], us[0] = 1.0, 1.0                                          # out of [0, 1): a refusal, the last index with r > 0
    check(p, q, d, off, u, us, pad=pad)


def test_numbers_on_the_borders():
    """Probabilities that are sums of powers of two: u S falls on a cumulative sum exactly."""
    V = 300
    for i in range(8):
        p = torch.zeros((2, V))
        p[:, [3, 70, 71, 299]] = torch.tensor([.5, .25, .125, .125])
        q = torch.zeros((2, V))
        q[:, 3], q[:, 5] = .5, .5
        for u0 in (0.0, 1.0 - 2.0 ** -24):
            check(p, q, torch.tensor([5, 0], dtype=torch.int32), [0, 2], torch.tensor([u0, 0.]), torch.tensor([i / 8]))
            check(p, q, torch.tensor([3, 0], dtype=torch.int32), [0, 2], torch.tensor([u0, 0.]), torch.tensor([i / 8]))
            check(p, None, torch.tensor([3, 0], dtype=torch.int32), [0, 2], torch.tensor([u0, 0.]), torch.tensor([i / 8]))


def test_rows_that_leave_nothing():
    V = 777
    p, q, d, off, u, us = inputs([2, 2, 2, 1, 3], V, torch.float32, 5)
    q[0] = p[0]                                                      # p - q is 0 everywhere, the draft refused by u = 1
    u[0] = 1.0
    p[2] = 0.0                                                       # an empty target row under a draft
    p[6] = 0.0                                                       # an empty row behind the last draft
    d[7] = -1                                                        # drafts outside the vocabulary
    d[8] = V
    check(p, q, d, off, u, us)
    check(p, None, d, off, u, us)
    p[7] = 0.0
    p[7, int(d[8]) % V] = 1.0
    check(p, None, d, off, u, us)


def test_values_that_count_as_nothing():
    V = 1030
    p, q, d, off, u, us = inputs([4, 4], V, torch.float32, 6)
    bad = [float("nan"), float("inf"), -float("inf"), -1.0, 2.0 ** 65, torch.finfo(torch.float32).max, -0.0]
    for r in range(8):
        for i, v in enumerate(bad):
            p[r, 11 * i + r] = v
            q[r, 13 * i + 3 + r] = v
    d[0], d[4] = 0, 11                                               # drafts that are NaN and infinite in p
    check(p, q, d, off, u, us)
    p[1, :] = float("nan")
    check(p, q, d, off, u, us)
    p[:, 0], q[:, 1] = 2.0 ** 64, 1e-45                              # the largest that counts; a subnormal
    check(p, q, d, off, u, us)


def test_residuals_far_below_the_probabilities():
    """p - q of the order of p's last bit: every bit of the differences counts."""
    V = 5000
    g = torch.Generator().manual_seed(8)
    p = torch.softmax(torch.randn((3, V), generator=g), 1)
    q = p * (1 + 2.0 ** -22 * (torch.randint(-2, 3, (3, V), generator=g)))
    d = torch.tensor([5, 6, 7], dtype=torch.int32)
    for us in torch.linspace(0, 0.999, 23):
        check(p, q, d, [0, 3], torch.ones(3), us.view(1))


def test_offsets_outside_the_rows_are_refused():
    p, q, d, off, u, us = inputs([2, 2, 2], 64, torch.bfloat16, 9)
    us = torch.rand(5)
    check(p, q, d, [-1, 1, 0, 3, 7, 9], u, us)
    check(p, q, d, [2**31 - 1, -2**31, 0, 3, 6, 6], u, us)
    check(p, q, d, [1, 2, 4, 4, 5, 5], u, us)                        # rows 0 and 5 belong to nobody
    empty = pkg().verify_drafts(p[:0].cuda(), d[:0].cuda(), torch.zeros(3, dtype=torch.int32, device="cuda"),
                                u[:0].cuda(), us[:2].cuda())
    assert empty[0].numel() == 0 and empty[1].tolist() == [0, 0]
    none = pkg().verify_drafts(p.cuda(), d.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), u.cuda(), us[:0].cuda())
    assert none[1].numel() == 0


def test_the_drawn_tokens_follow_the_target():
    """Over the uniform numbers, accepted and drawn tokens together have the target's distribution: u and u_sample on
    a grid give frequencies that differ from p by the grid's spacing alone."""
    V, n = 5, 256
    p, q = torch.tensor([.1, .2, .3, .25, .15]), torch.tensor([.3, .1, .2, .1, .3])
    freq = torch.zeros(V, dtype=torch.float64)
    B = n * n
    grid = (torch.arange(n) + .5) / n
    u, us = grid.repeat_interleave(n), grid.repeat(n)
    R = 2 * B
    both = torch.zeros(R)
    both[0::2] = u
    pr, qr = p.expand(R, V).contiguous().cuda(), q.expand(R, V).contiguous().cuda()
    for tok in range(V):
        d = torch.full((R,), tok, dtype=torch.int32, device="cuda")
        for part in range(0, B, 32768):
            rows = slice(2 * part, 2 * part + 65536)
            off = (2 * torch.arange(32769)).int().cuda()
            t, _ = pkg().verify_drafts(pr[rows], d[rows], off, both[rows].cuda(), us[part:part + 32768].cuda(), qr[rows])
            freq += float(q[tok]) * torch.bincount(t[0::2].cpu(), minlength=V).double() / B
    # each drafted token: the accepted share and every drawn token's share are off by at most one grid step each
    assert (freq - p.double()).abs().max() <= 2.0 / n


def test_graph_replay_another_stream_and_repeats():
    p, q, d, off, u, us = inputs([6, 1, 4, 6] * 8, 4099, torch.float32, 10, sharp=2.0)
    args = [t.cuda() for t in (p, d, torch.tensor(off, dtype=torch.int32), u, us)]
    qc = q.cuda()
    want = pkg().verify_drafts(*args, qc)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = pkg().verify_drafts(*args, qc, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pkg().verify_drafts(*args, qc)
    u2 = torch.rand(u.shape, generator=torch.Generator().manual_seed(11))
    args[3].copy_(u2)
    graph.replay()
    torch.cuda.synchronize()
    ref, acc = verify_ref(p, d.tolist(), off, u2.tolist(), us.tolist(), q)
    assert got[0].tolist() == ref and got[1].tolist() == acc


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("V,B", [(2000003, 2), (2000003, 60), (300000, 40)])
def test_vocabularies_of_many_groups(V, B, dt):
    """Ranges too long for the ring and for one part of the search; against 64-bit cumulative sums (whose own rounding is
    1e-10 of a probability here)."""
    g = torch.Generator(device="cuda").manual_seed(V + B)
    p = torch.rand((B, V), device="cuda", generator=g).to(TYPES[dt])
    p[0, : V // 2] = 0.0
    us = torch.rand(B, device="cuda", generator=g)
    off = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    tokens, accepted = pkg().verify_drafts(p, torch.zeros(B, dtype=torch.int32, device="cuda"), off, us, us)
    c = p.double().cumsum(1)
    want = torch.searchsorted(c, us.double()[:, None] * c[:, -1:], right=True)[:, 0]
    assert torch.equal(tokens.long(), want) and not accepted.any()


def test_refusals():
    p, q, d, off, u, us = inputs([3, 2], 40, torch.float32, 12)
    off = torch.tensor(off, dtype=torch.int32)
    good = dict(target=p, drafts=d, offsets=off, u=u, u_sample=us, draft_probs=q)
    dev = {k: v.cuda() for k, v in good.items()}
    pkg().verify_drafts(**dev)
    for k, v in dict(target=dev["target"].double(), drafts=dev["drafts"].long(), offsets=dev["offsets"][:-1], u=dev["u"][:-1],
                     u_sample=dev["u_sample"].double(), draft_probs=dev["draft_probs"].half()).items():
        with pytest.raises(ValueError):
            pkg().verify_drafts(**{**dev, k: v})
    for bad in (dict(target=p), dict(target=dev["target"].t()), dict(draft_probs=dev["draft_probs"][:, :-1]),
                dict(draft_probs=dev["draft_probs"][:-1]), dict(tokens=dev["drafts"]), dict(tokens=dev["drafts"][:-1].clone()),
                dict(accepted=torch.empty(2, device="cuda")), dict(target=dev["target"][0])):
        with pytest.raises(ValueError):
            pkg().verify_drafts(**{**dev, **bad})
