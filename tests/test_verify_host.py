"""Host-side checks of the draft verification (no GPU), and the tests' plain form on cases worked out by hand."""
import pytest
import torch

from verify_helpers import verify_ref

P = 4096  # never dereferenced: every call here is refused (or empty) on the host


@pytest.fixture(scope="module")
def lib():
    from decode_batches_gb300 import build, load_library
    build.build()
    return load_library()


GOOD = dict(target=P, dt=0, ldt=64, draft=P, ldd=64, R=6, V=64, drafts=P, offsets=P, B=2, u=P, us=P, tokens=P, acc=P)


def test_bad_arguments_are_refused(lib):
    from decode_batches_gb300 import MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED
    call = lambda **kw: lib.moe_verify_drafts(*{**GOOD, **kw}.values(), None)
    assert call(B=0) == 0
    for kw in (dict(R=-1), dict(V=0), dict(B=-1), dict(dt=3), dict(target=None), dict(ldt=63), dict(ldd=63), dict(drafts=None),
               dict(offsets=None), dict(u=None), dict(us=None), dict(tokens=None), dict(acc=None), dict(target=P + 1),
               dict(draft=P + 1), dict(dt=2, target=P + 2)):
        assert call(**kw) == MOE_ERR_INVALID_ARG, kw
    assert call(V=2**30 + 1, ldt=2**31, ldd=2**31) == MOE_ERR_UNSUPPORTED
    assert call(B=65536) == MOE_ERR_UNSUPPORTED


def test_the_plain_form_by_hand():
    p = torch.tensor([[.5, .25, .25, 0.], [.25, .25, .25, .25], [0., 0., 1., 0.]])
    q = torch.tensor([[.25, .75, 0., 0.], [.5, .5, 0., 0.], [1., 0., 0., 0.]])
    run = lambda u, us, d=(0, 1, 0), off=(0, 3), probs=q: verify_ref(p, d, off, u, us, probs)
    assert run([.9, .4, 0.], [.5]) == ([0, 1, 2], [2])             # .9 * .25 < .5, .4 * .5 < .25; then p of row 2
    assert run([.9, .5, 0.], [.5]) == ([0, 3, -1], [1])            # .5 * .5 = .25: refused; r = 0, 0, 1/4, 1/4
    assert run([.9, .5, 0.], [.49]) == ([0, 2, -1], [1])
    assert run([0., 0., 0.], [0.], d=(3, 0, 0)) == ([0, -1, -1], [0])   # p = 0 is never accepted; r = 1/4, 0, 1/4
    assert run([.5, .1, 0.], [.7], probs=None) == ([2, -1, -1], [0])    # certain drafts: u < p; p without token 0
    assert run([0., 0., 0.], [.7], d=(9, 0, 0)) == ([2, -1, -1], [0])   # a draft outside the vocabulary: refused; r = 1/4, 0, 1/4
    assert run([0., 0., 0.], [.7, .7], off=(0, 0, 3)) == ([0, 1, 2], [0, 2])
    z = torch.zeros(1, 4)
    assert verify_ref(z, (0,), (0, 1), [0.], [.5], None) == ([-1], [0])
