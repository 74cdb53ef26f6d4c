"""spec_attention_tree's float rows on a bf16 cache as the tensor cores make them, emulated in numpy:
queries and weights in three bf16 parts, products exact, a sum of 16 products and its accumulator cut to
24 bits toward zero, blocks of 64 keys in two streams, sums taken out after 8 blocks and added up in
binary32. The arguments leave one of these out at a time, to see what a tolerance has to tell apart."""
import numpy as np
import torch

F = np.float32


def bf16(x):
    return torch.from_numpy(np.asarray(x, F)).bfloat16().float().numpy()


def parts(x, n):
    x, out = np.asarray(x, F), []
    for _ in range(n):
        p = bf16(x)
        out.append(p.astype(np.float64))
        x = (x - p).astype(F)
    return out


def product(acc, a, b):
    """acc += a b, 16 terms at a time."""
    for i in range(0, a.shape[1], 16):
        m, e = np.frexp(acc + a[:, i:i + 16] @ b[i:i + 16])
        acc = np.ldexp(np.trunc(m * 2 ** 24) / 2 ** 24, e)
    return acc


def power(m, to):
    """2^(m - to); 0 for a maximum that is not there yet."""
    return np.where(np.isinf(m), 0, np.exp2(np.where(np.isinf(m), 0, m - to).astype(np.float64))).astype(F)


def attention(q, k, v, rng, q_parts=3, p_parts=3, run=8, smallest_first=True):
    """q [rows][hd], k and v [keys][hd] (bf16 values): outputs [rows][hd]."""
    (R, hd), n = q.shape, len(k)
    scale2, Q = F(1.4426950408889634 / np.sqrt(hd)), parts(q, q_parts)
    k, v = (np.pad(x.astype(np.float64), ((0, -n % 64), (0, 0))) for x in (k, v))
    blocks = len(k) // 64
    top, total, acc = np.full(R, -np.inf, F), np.zeros(R, F), np.zeros((R, hd), F)
    m = [np.full(R, -np.inf, F), np.full(R, -np.inf, F)]
    for e0 in range(0, blocks, run):
        o, l = [np.zeros((R, hd)), np.zeros((R, hd))], [np.zeros(R, F), np.zeros(R, F)]
        for b in range(e0, min(e0 + run, blocks)):
            s, at = b & 1, slice(64 * b, 64 * b + 64)
            S = np.zeros((R, 64))
            for x in Q[::-1] if smallest_first else Q:
                S = product(S, x, k[at].T)
            S[:, max(n - 64 * b, 0):] = -np.inf
            big = (S.max(1) * scale2).astype(F)
            up = (big > m[s] + 8) | np.isinf(m[s])
            f = np.where(up, power(m[s], big), F(1))
            m[s] = np.where(up, big, m[s])
            w = np.exp2((S * scale2 - m[s][:, None]).astype(F).astype(np.float64))
            w = (w * (1 + rng.uniform(-1, 1, w.shape) * 2.0 ** -22.5)).astype(F)        # (the hardware's exponential)
            l[s] = (l[s] * f + w.astype(np.float64).sum(1)).astype(F)
            o[s] = (o[s] * f[:, None]).astype(F).astype(np.float64)
            W = parts(w, p_parts)
            for c in range(0, 64, 16):
                for x in W:
                    o[s] = product(o[s], x[:, c:c + 16], v[at][c:c + 16])
        M = np.maximum(*m)
        g = [power(x, M) for x in m]
        new = np.maximum(top, M)
        old, now = power(top, new), power(M, new)
        both = (g[0][:, None] * o[0].astype(F) + g[1][:, None] * o[1].astype(F)).astype(F)
        acc = (old[:, None] * acc + now[:, None] * both).astype(F)
        total = (old * total + now * (g[0] * l[0] + g[1] * l[1])).astype(F)
        top = new
    return acc / total[:, None]


def exact(q, k, v):
    s = q.astype(np.float64) @ k.astype(np.float64).T / np.sqrt(q.shape[1])
    p = np.exp(s - s.max(1, keepdims=True))
    return p @ v / p.sum(1, keepdims=True)


def off(got, want):
    """The error of all outputs together, relative to all outputs."""
    return np.linalg.norm(got - want) / np.linalg.norm(want)


# Limits for `off`, queries of deviation 1.5, keys and values of 1, by keys and head dim. Emulated, as built
# 4.0e-7 to 5.3e-7 at 64 keys, 1.3e-6 to 1.4e-6 and 1.4e-6 to 1.9e-6 (head dim 128) at 4200; with a part, the
# order or the runs left out 7.7e-7 and more, 2.0e-6 and 2.2e-6 and more.
LIMITS = {(64, 64): 6e-7, (64, 128): 6e-7, (4200, 64): 1.7e-6, (4200, 128): 2.1e-6}
