"""Sampling in 64 bits, one row at a time: the definition in include/spec.h
(spec_sampling), written with library sorts and sums, and how near a row's
decisions are to a border.

The kernel evaluates a weight to a relative 2^-36 and rounds it to its unit,
an absolute 2^-44 at most (the largest weight is 1). A sum of up to V weights, compared
with another one, is therefore off by at most 2 * (Z * 2^-36 + V * 2^-44), Z the
whole mass: a draw is compared only where it is further from its borders than
that, `slack`. Where top-p's cut is that near to a border, the kernel may cut up
to 2 * slack of mass and one token earlier or later; the kept mass and each
partial sum then move by no more, and the draw is compared where its borders are
that much further. A row is compared where no weight is within
2^-36 min_p + 2^-44 of min_p."""
import numpy as np


def weights(l, T):
    m = l.max()
    if m == np.inf:
        return (l == np.inf).astype(np.float64)
    with np.errstate(over="ignore"):
        return np.exp((l - m) / T)


def row(l, u, T=1.0, k=0, p=1.0, q=0.0):
    """(token, probability, decided): decided is False where a border is too
    near to be held to the 64-bit answer."""
    l = np.asarray(l, np.float64)
    n = len(l)
    if np.isnan(l).any() or l.max() == -np.inf or not (0.0 <= T < np.inf):
        return -1, 0.0, True
    if T < 1e-5:
        return int(np.argmax(l)), 1.0, True
    w = weights(l, T)
    slack = 2.0 * (w.sum() * 2.0 ** -36 + n * 2.0 ** -44)
    order = np.lexsort((np.arange(n), -l))
    if 0 < k < n:
        order = order[:k]
    decided, moved = True, 0.0
    if p < 1.0:
        mass = np.concatenate([[0.0], np.cumsum(w[order])])
        target = max(p, 0.0) * mass[-1]
        if target > 0.0 and np.abs(mass - target).min() <= slack:
            at = int(np.searchsorted(mass, target - slack, "left"))
            moved = 2.0 * slack + w[order[max(0, at - 1)]]
        order = order[:max(1, int(np.searchsorted(mass[:-1], target, "left")))]
    keep = np.zeros(n, bool)
    keep[order] = True
    if q > 0.0:
        q = min(q, 1.0)
        decided &= q == 1.0 or np.abs(w - q).min() > q * 2.0 ** -36 + 2.0 ** -44
        keep &= w >= q
    at = np.flatnonzero(keep & (w > 2.0 ** -45))
    cum = np.cumsum(w[at])
    u = min(max(u, 0.0), 1.0) if u == u else 0.0
    t = u * cum[-1]
    j = min(int(np.searchsorted(cum, t, "right")), len(at) - 1)
    near = np.abs(cum[:-1] - t)
    decided &= moved <= cum[-1] * 2.0 ** -24      # (the probability follows the kept mass)
    decided &= len(near) == 0 or u == 0.0 or u == 1.0 or near.min() > slack + 2.0 * moved
    return int(at[j]), float(w[at[j]] / cum[-1]), bool(decided)


def rows(l, u, T=None, k=None, p=None, q=None):
    at = lambda v, i, off: off if v is None else float(v[i])
    out = [row(l[i], float(u[i]), at(T, i, 1.0), int(at(k, i, 0)), at(p, i, 1.0), at(q, i, 0.0))
           for i in range(len(l))]
    return np.array([o[0] for o in out]), np.array([o[1] for o in out]), np.array([o[2] for o in out])


def accept(tokens, probs, drafts):
    """The walk over sampled rows [B][k+1]: (out, n, probs)."""
    B, k1 = tokens.shape
    out, n, pr = np.full((B, k1), -1), np.zeros(B, int), np.zeros((B, k1))
    for b in range(B):
        for j in range(k1):
            if tokens[b, j] < 0:
                break
            out[b, j], pr[b, j], n[b] = tokens[b, j], probs[b, j], j + 1
            if j < k1 - 1 and drafts[b, j] != tokens[b, j]:
                break
    return out, n, pr
