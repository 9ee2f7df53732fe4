"""What sample_tokens draws, in 64 bits, and the error bounds of its numbers."""
import math

import numpy as np


def sample64(x, u, T, k, p, least):
    """(token, log-probability, distribution, margin) of one row x (float64 values of its stored type): from the
    definition, sorted.  `margin`: how far the nearest decision was from its border (the nucleus' border against p, the
    draw's against u), in what the sums of weights may be off by."""
    V = len(x)
    order = np.lexsort((np.arange(V), -x))          # value descending, index ascending
    dist = np.zeros(V)
    if T == 0:
        dist[order[0]] = 1
        return int(order[0]), 0.0, dist, math.inf
    if k > 0:
        order = order[:k]
    w = np.exp((x[order] - x[order[0]]) / T)
    margin = math.inf
    keep = np.ones(len(order), bool)
    if p < 1:
        before = np.array([0.0] + [math.fsum(w[:i]) for i in range(1, len(w))]) if len(w) < 400 else \
            np.concatenate([[0.0], np.cumsum(w.astype(np.longdouble))[:-1]]).astype(float)
        target = p * math.fsum(w)
        keep &= before < target
        margin = min(margin, np.abs(before[1:] - target).min(initial=math.inf) / off(math.fsum(w), V))
    keep &= w >= least
    keep[0] = True
    kept = order[keep]
    mass = np.zeros(V)
    mass[kept] = w[keep]
    total = math.fsum(mass)
    upto = np.cumsum(mass.astype(np.longdouble)).astype(float)
    token = int(np.searchsorted(upto, u * total, side="right"))
    at = np.flatnonzero(mass)
    margin = min(margin, np.abs(upto[at] - u * total)[:-1].min(initial=math.inf) / off(total, V))
    token = min(token, int(at[-1]))
    return token, math.log(mass[token] / total), mass / total, margin


def off(mass, V):
    """What a border between sums of weights may be off by.  A weight is off by 2^-29 of itself (its table's entry 2^-31, its
    whole part 2^-30 rounded down, 2^r - 1 in fp32 2^-34), and is rounded down to units of 2^-44 of the largest; the two
    sides of a comparison together are the whole mass."""
    return 2.0 ** -29 * mass + 2.0 ** -44 * V


# The kept mass, where no border is near, may be the sum of fp32 weights 2^t, t = fma(x, c, -ref): with D = (max - x) c (in
# log2 units) a term is off by the roundings of c and t, ln 2 (2 D + 8) 2^-24, and by ex2, 2^-22; a thread's sum by ex2 once
# more, by its additions and by its rounding to whole units, 2^-22 each.  Averaged over the mass D is at most the
# distribution's entropy in bits, 19 for 2^19 entries: (ln 2 (2 * 19 + 8) + 4 * 4) 2^-24 < 2^-18 in all.
MASS = 2.0 ** -18


def logprob_bound(lp):
    """Of ln((W - w) / w + 1) in fp32: the mass W; three roundings of the quotient (2^-24 each), the logarithm's own two
    last places."""
    return MASS + 2.0 ** -22 + 2.0 ** -22 * abs(lp)


def probs_bound(p):
    """The mass; weight (2^-22, the special-function unit's) and quotient (four roundings of 2^-24); what is below the
    weights' unit."""
    return (MASS + 2.0 ** -20) * p + 2.0 ** -38
