"""A plain form of the draft verification in exact rational arithmetic (64-bit floats are exact fractions)."""
from fractions import Fraction
import math


def _clean(v):
    return Fraction(v) if math.isfinite(v) and 0 < v <= 2.0 ** 64 else Fraction(0)


def verify_ref(p, drafts, offsets, u, u_sample, q):
    """p, q: CPU tensors [R][V] (q may be None); the rest sequences.  Rows of no request hold None."""
    tokens, accepted = [None] * p.shape[0], []
    V = p.shape[1]
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if lo < 0 or hi < lo or hi > p.shape[0]:
            accepted.append(-1)
            continue
        if hi == lo:
            accepted.append(0)
            continue
        r = lo
        while r < hi - 1:
            t = int(drafts[r])
            pt = _clean(float(p[r, t])) if 0 <= t < V else 0
            qt = (_clean(float(q[r, t])) if q is not None else 1) if 0 <= t < V else 0
            if not Fraction(float(u[r])) * qt < pt:
                break
            tokens[r] = t
            r += 1
        row = [_clean(v) for v in p[r].double().tolist()]
        left = row
        if r < hi - 1:
            if q is None:
                left = [Fraction(0) if i == int(drafts[r]) else v for i, v in enumerate(row)]
            else:
                left = [max(v - _clean(w), Fraction(0)) for v, w in zip(row, q[r].double().tolist())]
            if not sum(left):
                left = row
        at, c, token = Fraction(max(0.0, float(u_sample[b]))) * sum(left), Fraction(0), -1
        for i, v in enumerate(left):
            if v > 0:
                c, token = c + v, i
                if c > at:
                    break
        tokens[r] = token
        for i in range(r + 1, hi):
            tokens[i] = -1
        accepted.append(r - lo)
    return tokens, accepted
