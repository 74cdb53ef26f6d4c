"""64-bit references of the operators for drafted trees and branching sequences
(spec_attention_tree, spec_adjust_logits, spec_pages_*, spec_rows_keep), written
from their definitions in include/spec.h with numpy, one row at a time."""
import numpy as np

PAGE = 64


def chain_up(parents, r):
    while r >= 0:
        yield r
        p = int(parents[r])
        r = p if p < r else -1


def random_parents(rng, B, R):
    return np.array([[-1] + [int(rng.integers(-1, r)) for r in range(1, R)] for _ in range(B)], np.int32)


def attention(pool, table, seq_ids, seq_len, q, nq, parents, n_rows):
    """pool [n_pages][2][nkv][64][hd] of a layer, q [B*R][nq*hd], all float64.
    Per output: (value, weighted sum of |v|, largest sum of |q k| / sqrt(hd) of its keys,
    keys); rows not in use stay NaN."""
    nkv, hd = pool.shape[2], pool.shape[4]
    B, R = len(seq_ids), len(q) // len(seq_ids)
    q = q.reshape(B, R, nq, hd)
    out = np.full(q.shape, np.nan)
    mag, big, keys = np.zeros(q.shape), np.zeros((B, R, nq)), np.zeros((B, R, nq))
    for b in range(B):
        n = int(seq_len[seq_ids[b]])
        rows = R if n_rows is None else int(n_rows[b])
        if rows == 0:
            continue
        at = np.arange(n + rows)
        page = table[seq_ids[b]][at // PAGE]
        k, v = (pool[page, i, :, at % PAGE] for i in (0, 1))        # [N][nkv][hd]
        for r in range(rows):
            up = list(chain_up(parents[b], r)) if parents is not None else list(range(r + 1))
            j = np.concatenate([np.arange(n), n + np.array(sorted(up))])
            for h in range(nq):
                kk, vv, qq = k[j, h * nkv // nq], v[j, h * nkv // nq], q[b, r, h]
                s = kk @ qq / np.sqrt(hd)
                p = np.exp(s - s.max())
                out[b, r, h] = p @ vv / p.sum()
                mag[b, r, h] = p @ np.abs(vv) / p.sum()
                big[b, r, h] = (np.abs(kk) @ np.abs(qq)).max() / np.sqrt(hd)
                keys[b, r, h] = len(j)
    shape = (B * R, nq * hd)
    each = lambda x: np.repeat(x[..., None], hd, -1).reshape(shape)
    return out.reshape(shape), mag.reshape(shape), each(big), each(keys)


def adjust(x, R, hist=None, hist_len=None, prompt_len=None, tokens=None, parents=None, rep=None, freq=None, pres=None,
           bias_tokens=None, bias_values=None, mask=None, mask_ids=None):
    """x [B*R][V] float64 -> the changed logits in 64 bits."""
    x = x.copy()
    M, V = x.shape
    B = M // R
    ok = lambda v, off, pos=False: off if v is None or not np.isfinite(v) or (pos and v <= 0) else float(v)
    for m in range(M):
        b, r, row = m // R, m % R, x[m]
        inf = row == -np.inf
        n = 0 if hist is None else hist.shape[1] if hist_len is None else min(max(int(hist_len[b]), 0), hist.shape[1])
        np_ = 0 if prompt_len is None else min(max(int(prompt_len[b]), 0), n)
        text = np.zeros(0, np.int64) if hist is None else hist[b, :n].astype(np.int64)
        path = [] if tokens is None else [tokens[b, j] for j in (
            chain_up(parents[b], r) if parents is not None else range(r + 1))]
        said = np.concatenate([text[np_:], np.array(path, np.int64)])
        rp = ok(None if rep is None else rep[b], 1.0, True)
        fr, pr = ok(None if freq is None else freq[b], 0.0), ok(None if pres is None else pres[b], 0.0)
        for t in set(int(t) for t in np.concatenate([text, said]) if 0 <= t < V):
            row[t] = row[t] / rp if row[t] > 0 else row[t] * rp
            c = int((said == t).sum())
            if c:
                row[t] = row[t] - c * fr - pr
        ban = np.zeros(V, bool)
        if bias_tokens is not None:
            last = {}
            for t, v in zip(bias_tokens[b], bias_values[b]):
                if 0 <= t < V:
                    last[int(t)] = float(v)
            for t, v in last.items():
                if v == -np.inf:
                    ban[t] = True
                elif not np.isnan(v):
                    row[t] = row[t] + v
        if mask is not None:
            i = m if mask_ids is None else int(mask_ids[m])
            if 0 <= i < len(mask):
                bits = np.unpackbits(np.ascontiguousarray(mask[i]).view(np.uint8), bitorder="little")[:V]
                ban |= bits == 0
        row[ban | inf] = -np.inf
    return x


def release(table, refs, ids, lens=None):
    for i, s in enumerate(ids):
        k = 0 if lens is None else -(-int(lens[i]) // PAGE)
        for p in table[s, k:]:
            if p >= 0:
                refs[p] -= 1
        table[s, k:] = -1


def reserve(table, refs, ids, lens):
    for s, n in zip(ids, lens):
        for k in range(-(-int(n) // PAGE)):
            if table[s, k] < 0:
                table[s, k] = np.flatnonzero(refs == 0)[0]
                refs[table[s, k]] = 1


def fork(pool, table, refs, seq_len, src, dst):
    """pool [L][n_pages][2][nkv][64][hd]; all in place."""
    release(table, refs, dst)
    for a, d in zip(src, dst):
        full, part = divmod(int(seq_len[a]), PAGE)
        table[d, :full] = table[a, :full]
        for p in table[d, :full]:
            refs[p] += 1
        if part:
            p = np.flatnonzero(refs == 0)[0]
            table[d, full] = p
            refs[p] = 1
            pool[:, p, :, :, :part] = pool[:, table[a, full], :, :, :part]
        seq_len[d] = seq_len[a]


def compact(pool, table, refs):
    """(moved, live); the rest in place."""
    live = np.flatnonzero(refs > 0)
    n = len(live)
    holes = [p for p in range(n) if refs[p] == 0]
    moved = np.full(len(refs), -1, np.int32)
    moved[live] = live
    for p in live[live >= n]:
        to = holes.pop(0)
        moved[p] = to
        pool[:, to] = pool[:, p]
        refs[to], refs[p] = refs[p], 0
    table[:] = np.where(table >= 0, moved[np.maximum(table, 0)], -1)
    return moved, n


def keep(pool, table, seq_ids, seq_len, rows, n_keep):
    for b, s in enumerate(seq_ids):
        n = int(seq_len[s])
        old = pool.copy()
        for i in range(int(n_keep[b])):
            a, d = n + int(rows[b][i]), n + i
            pool[:, table[s, d // PAGE], :, :, d % PAGE] = old[:, table[s, a // PAGE], :, :, a % PAGE]
