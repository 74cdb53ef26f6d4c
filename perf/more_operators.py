"""Cases and plain forms of the operators that serve drafted trees and sequences that branch.

`tree`    attention of the rows of drafted trees over the paged cache: row r of a sequence (its key and
          value already at position n + r, n the committed length) attends the n committed keys, its
          ancestors' and its own; scores q.k / sqrt(head_dim), softmax, sum of the values;
`adjust`  the logits of such rows made ready for sampling. Of token t with c occurrences among the
          output (the history behind the prompt, then the tokens on the row's own path): if it occurs at all,
          prompt included, x > 0 becomes x / repetition, else x * repetition; then x - c * frequency
          - (c > 0) * presence + bias; tokens that a grammar's bits (or a bias of -inf) forbid get -inf;
`fork`    a sequence continued by several slots: full pages are shared (their counts of references
          rise), the last page's rows are copied in every layer into the lowest free page; what the slots
          held before is given back first;
`compact` the pages in use moved into the lowest numbers of the pool, and the tables with them.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
PAGE = 64
INF = float("inf")


def listed():
    return [
        # the tiny fp32 model, four rows behind a short prompt: the smallest call, all latency
        dict(name="tree_1x4_tiny_f32", op="tree", B=1, R=4, nq=4, nkv=4, hd=64, lo=64, hi=64, q="f32", kv="f32",
             ragged=False, mix=1),
        # one user of an E2B-shaped model, a small tree
        dict(name="tree_1x16_e2b", op="tree", B=1, R=16, nq=12, nkv=4, hd=128, lo=2048, hi=2048, q="f32", kv="bf16",
             ragged=False, mix=2),
        # a batch of an E4B-shaped model, contexts and trees of all sizes
        dict(name="tree_8x24_e4b_ragged", op="tree", B=8, R=24, nq=20, nkv=4, hd=128, lo=1024, hi=8192, q="f32",
             kv="bf16", ragged=True, mix=3),
        # the 30B-class model at batch 8 with large trees: 384 query rows a KV head
        dict(name="tree_8x64_30b_bf16", op="tree", B=8, R=64, nq=48, nkv=8, hd=128, lo=8192, hi=8192, q="bf16",
             kv="bf16", ragged=False, mix=4),
        # one very long document
        dict(name="tree_1x7_e2b_131072", op="tree", B=1, R=7, nq=12, nkv=4, hd=128, lo=131071, hi=131071, q="bf16",
             kv="bf16", ragged=False, mix=5),
        # one row of a small vocabulary, a chat's history: all latency
        dict(name="adjust_1x1x4096", op="adjust", B=1, R=1, V=4096, ld=4096, dtype="f32", hist=300, bias=0,
             masked=False, tree=False, mix=6),
        # a verify pass of eight requests, penalties, biases, grammars on some
        dict(name="adjust_8x5x262144", op="adjust", B=8, R=5, V=262144, ld=262144, dtype="f32", hist=8192, bias=64,
             masked=True, tree=False, mix=7),
        # a plain decoding step of a full batch
        dict(name="adjust_64x1x262144", op="adjust", B=64, R=1, V=262144, ld=262144, dtype="f32", hist=2048, bias=0,
             masked=False, tree=False, mix=8),
        # trees over an odd vocabulary in padded bf16 rows
        dict(name="adjust_3x7x100003_bf16", op="adjust", B=3, R=7, V=100003, ld=100008, dtype="bf16", hist=777, bias=5,
             masked=True, tree=True, mix=9),
        # one branch of a sequence of the tiny model
        dict(name="fork_1to1_tiny", op="fork", L=2, d=256, nkv=4, hd=64, kv="f32", src=1, kids=1, lo=100, hi=100, mix=10),
        # eight samples of one prompt, 30B-class cache (48 layers)
        dict(name="fork_1to8_30b", op="fork", L=48, d=6144, nkv=8, hd=128, kv="bf16", src=1, kids=8, lo=2037, hi=2037,
             mix=11),
        # an E4B-shaped model's pool after many requests came and went
        dict(name="compact_e4b", op="compact", L=32, nkv=4, hd=128, kv="bf16", pages=160, slots=12, live=0.6, mix=12),
    ]


HEADS = [(12, 4, 128), (20, 4, 128), (48, 8, 128), (16, 8, 128), (4, 4, 64)]
CACHES = [(24, 1536, 4, 128), (32, 2560, 4, 128), (48, 6144, 8, 128), (16, 2048, 8, 128), (2, 256, 4, 64)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "adjust", "adjust", "fork", "compact"])
    mix = rng.randrange(1 << 20)
    if op == "tree":
        nq, nkv, hd = rng.choice(HEADS)
        B, R = _log(rng, 1, 16), _log(rng, 1, 64)
        # (no more keys, and no more keys times query rows, than the largest listed case; fp32 caches are for small models)
        most = min(131072, 65536 * 8 // (B * nkv), 65536 * 64 * 48 // (B * R * nq))
        kv = "f32" if hd == 64 and rng.random() < 0.6 else "bf16"
        hi = _log(rng, 1, max(2, most if kv == "bf16" else min(most, 8192)))
        ragged = rng.random() < 0.6
        return dict(op=op, B=B, R=R, nq=nq, nkv=nkv, hd=hd, lo=rng.randint(0, hi) if ragged else hi, hi=hi,
                    q="f32" if kv == "f32" else rng.choice(["f32", "bf16"]), kv=kv, ragged=ragged, mix=mix)
    if op == "adjust":
        V = _log(rng, 500, 262144)
        R = rng.choice([1, 1, 2, 4, 5, 8, 16, 33])
        return dict(op=op, B=_log(rng, 1, 64 // R if R < 64 else 1), R=R, V=V, ld=V + rng.choice([0, 0, 1, 5, 64]),
                    dtype=rng.choice(["f32", "f32", "bf16"]), hist=_log(rng, 1, 32768), bias=rng.choice([0, 0, 3, 40, 300]),
                    masked=rng.random() < 0.5, tree=rng.random() < 0.5, mix=mix)
    L, d, nkv, hd = rng.choice(CACHES)
    kv = "f32" if hd == 64 and rng.random() < 0.5 else "bf16"
    page = L * 2 * nkv * PAGE * hd * (4 if kv == "f32" else 2)
    if op == "fork":
        src, kids = rng.randint(1, 4), _log(rng, 1, 8)
        room = max(1, 600_000_000 // page - src * kids * 3 - 8)   # pages of the sources together
        hi = _log(rng, 1, max(2, min(4096, room * PAGE // src - PAGE)))
        return dict(op=op, L=L, d=d, nkv=nkv, hd=hd, kv=kv, src=src, kids=kids, lo=rng.randint(0, hi), hi=hi, mix=mix)
    return dict(op=op, L=L, nkv=nkv, hd=hd, kv=kv, pages=_log(rng, 8, max(16, min(2000, 600_000_000 // page))),
                slots=rng.randint(1, 16), live=rng.uniform(0.1, 0.95), mix=mix)


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _lens(c, n):
    r = random.Random(c["mix"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(n)]


def _rows_of(c):
    r = random.Random(c["mix"] + 1)
    return [r.randint((c["R"] + 1) // 2, c["R"]) if c["ragged"] else c["R"] for _ in range(c["B"])]


def _parents(B, R, rng, tree):
    """Parent rows of B drafted trees: row 0 the root, a node hangs on any earlier row, later ones more often."""
    return [[-1] + [r - 1 if not tree else int(r * math.sqrt(rng.random())) for r in range(1, R)] for _ in range(B)]


def _pool(c, L, pages, g):
    x = torch.empty((L, pages, 2, c["nkv"], PAGE, c["hd"]), dtype=_dt(c["kv"]), device=DEV)
    for l in range(L):
        x[l].normal_(0.0, 1.0, generator=g)
    return x


def prepare(case, seed):
    c, g, rng = case, _gen(seed), random.Random(seed)
    s = {"op": c["op"], "case": c}
    if c["op"] == "tree":
        B, R, lens, rows = c["B"], c["R"], _lens(c, c["B"]), _rows_of(c)
        need = [-(-(n + r) // PAGE) for n, r in zip(lens, rows)]
        P, total = max(need), sum(need)
        ids, table, at = list(range(total)), [], 0
        rng.shuffle(ids)
        for n in need:   # (an entry behind a sequence's last page names none)
            table.append(ids[at:at + n] + [-1] * (P - n))
            at += n
        slots = list(range(B))
        rng.shuffle(slots)
        where = sorted(range(B), key=lambda b: slots[b])
        s.update(pool=_pool(c, 1, total, g), lens=lens, rows=rows, block_table=_int([table[b] for b in where]),
                 seq_ids=_int(slots), seq_len=_int([lens[b] for b in where]), n_rows=_int(rows),
                 parents=_int(_parents(B, R, rng, True)))
        s["q"] = (torch.randn((B * R, c["nq"] * c["hd"]), generator=g, device=DEV) * 1.5).to(_dt(c["q"]))
        s["out"] = torch.zeros_like(s["q"])
        if own:
            from speculative_decoding_spec_gb300 import binding
            s["cache"] = binding.Cache(s["pool"], s["block_table"])
        return s
    if c["op"] == "adjust":
        B, R, V, H = c["B"], c["R"], c["V"], c["hist"]
        x = torch.randn((B * R, c["ld"]), generator=g, device=DEV) * 3.0
        s["logits"] = x.to(_dt(c["dtype"]))[:, :V]
        # texts repeat themselves: a few tokens often, many once
        u = torch.rand((B, H), generator=g, device=DEV)
        s["history"] = (V * u ** 3).long().clamp_max(V - 1).to(torch.int32)
        lens = [rng.randint(H // 3, H) for _ in range(B)]
        s["hist_len"], s["prompt_len"] = _int(lens), _int([int(n * rng.random()) for n in lens])
        f = lambda lo, hi: lo + (hi - lo) * torch.rand(B, generator=g, device=DEV)
        s["repetition"], s["presence"], s["frequency"] = f(1.0, 1.4), f(0.0, 1.0), f(0.0, 0.6)
        s["repetition"][1::3] = 1.0   # some requests leave a penalty out
        s["presence"][2::3] = 0.0
        s["frequency"][2::3] = 0.0
        s["tokens"] = (V * torch.rand((B, R), generator=g, device=DEV) ** 3).long().clamp_max(V - 1).to(torch.int32)
        s["parents"] = _int(_parents(B, R, rng, True)) if c["tree"] else None
        s["bias_tokens"] = s["bias_values"] = s["mask"] = s["mask_ids"] = None
        if c["bias"]:   # padded lists of distinct tokens
            n = min(c["bias"], V)
            t = torch.stack([torch.randperm(V, generator=g, device=DEV)[:n] for _ in range(B)])
            keep = torch.arange(n, device=DEV) < _int([rng.randint(0, n) for _ in range(B)])[:, None]
            s["bias_tokens"] = torch.where(keep, t, -1).to(torch.int32)
            s["bias_values"] = torch.randn((B, n), generator=g, device=DEV) * 5.0
        if c["masked"]:   # every other request under a grammar that leaves about a third of the tokens
            on = [m for m in range(B * R) if (m // R) % 2 == 0]
            words = -(-V // 32)
            s["mask"] = torch.randint(-(1 << 31), 1 << 31, (len(on), words), generator=g, device=DEV, dtype=torch.int64).to(
                torch.int32) & torch.randint(-(1 << 31), 1 << 31, (len(on), words), generator=g, device=DEV,
                                             dtype=torch.int64).to(torch.int32)
            s["mask_ids"] = _int([on.index(m) if m in on else -1 for m in range(B * R)])
        return s
    if c["op"] == "fork":
        n, kids = c["src"], c["kids"]
        lens = _lens(c, n)
        need = [-(-x // PAGE) for x in lens]
        # pages of an earlier request in the slots that are forked to (as many whatever the seed: a pool has one size)
        held = [random.Random(c["mix"] + 2 + i).randint(0, 2) for i in range(n * kids)]
        total = sum(need) + sum(held) + n * kids + 4
        P = max(max(need), 2) + 1
        ids = list(range(total))
        rng.shuffle(ids)
        slots = list(range(n * (1 + kids)))
        rng.shuffle(slots)
        src, dst = slots[:n], slots[n:]
        table, refs, seq_len = [[-1] * P for _ in slots], [0] * total, [0] * len(slots)
        for slot, k in list(zip(src, need)) + list(zip(dst, held)):
            for i in range(k):
                table[slot][i] = ids.pop()
                refs[table[slot][i]] = 1
        for slot, x in zip(src, lens):
            seq_len[slot] = x
        s.update(pool=_pool(c, c["L"], total, g), block_table=_int(table), refs=_int(refs), seq_len=_int(seq_len),
                 src=_int([src[i // kids] for i in range(n * kids)]), dst=_int(dst),
                 lens=[lens[i // kids] for i in range(n * kids)],
                 pending=torch.randint(0, 4096, (len(slots),), generator=g, device=DEV, dtype=torch.int32),
                 hid=torch.randn((len(slots), c["d"]), generator=g, device=DEV))
        if own:
            from speculative_decoding_spec_gb300 import binding
            s["cache"] = binding.Cache(s["pool"], s["block_table"], s["refs"])
        return s
    table, refs = _scattered(c, rng)
    n_live = sum(r > 0 for r in refs)
    s.update(pool=_pool(c, c["L"], c["pages"], g), block_table=_int(table), refs=_int(refs), n_live=n_live,
             n_moved=sum(r > 0 for r in refs[n_live:]))
    s["table_out"], s["refs_out"] = torch.empty_like(s["block_table"]), torch.empty_like(s["refs"])
    if own:
        from speculative_decoding_spec_gb300 import binding
        s["cache"] = binding.Cache(s["pool"], s["block_table"], s["refs"])
    return s


def _scattered(c, rng):
    """Tables of slots whose pages lie all over the pool, some of them shared by two, one page held by nobody's table."""
    n = max(2, int(c["pages"] * c["live"]))
    ids = rng.sample(range(c["pages"]), min(n, c["pages"]))
    P = -(-len(ids) // c["slots"]) + 2
    table, refs = [[-1] * P for _ in range(c["slots"])], [0] * c["pages"]
    for i, p in enumerate(ids[:-1]):
        table[i % c["slots"]][i // c["slots"]] = p
        refs[p] = 1
    refs[ids[-1]] = 1
    for b in range(1, c["slots"], 3):   # a slot that shares the first pages of the one before it
        for i in range(rng.randint(0, P)):
            old, new = table[b][i], table[b - 1][i]
            if old >= 0 and new >= 0:
                refs[old] -= 1
                refs[new] += 1
                table[b][i] = new
    return table, refs


# ---- plain forms -------------------------------------------------------------------------------

def _paths(parents):
    """[B][R][R]: whether row j is row r or an ancestor of it."""
    B, R = parents.shape
    i = torch.arange(R, device=parents.device)
    up = ((parents[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (R - 1).bit_length())):
        up = ((up @ up) > 0).float()
    return up > 0


def _plain_tree(s):
    c, pool = s["case"], s["pool"][0]
    B, R, nq, nkv, hd = c["B"], c["R"], c["nq"], c["nkv"], c["hd"]
    paths = _paths(s["parents"])
    q = s["q"].float().view(B, R, nkv, nq // nkv, hd)
    out = s["out"].view(B, R, nkv, nq // nkv, hd)
    for b in range(B):
        n, r = s["lens"][b], s["rows"][b]
        N = n + r
        pages = s["block_table"].index_select(0, s["seq_ids"][b:b + 1])[0, : -(-N // PAGE)]
        kv = pool.index_select(0, pages).float()                       # [pages][2][nkv][64][hd]
        k, v = kv.permute(1, 2, 0, 3, 4).reshape(2, nkv, -1, hd)[:, :, :N]
        x = q[b, :r].permute(1, 2, 0, 3).reshape(nkv, -1, hd)          # [nkv][group * rows][hd]
        w = (x @ k.transpose(1, 2)) / math.sqrt(hd)
        w = w.view(nkv, -1, r, N)
        w[..., n:].masked_fill_(~paths[b, :r, :r], -INF)
        w = torch.exp(w - w.amax(-1, keepdim=True))
        w = w / w.sum(-1, keepdim=True)
        y = w.view(nkv, -1, N) @ v
        out[b, :r] = y.view(nkv, -1, r, hd).permute(2, 0, 1, 3).to(out.dtype)
    return {"out": s["out"]}


def _plain_adjust(s):
    c = s["case"]
    B, R, V = c["B"], c["R"], c["V"]
    dev = s["logits"].device
    x = s["logits"].float().view(B, R, V)
    at = torch.arange(s["history"].shape[1], device=dev)
    here = at < s["hist_len"][:, None]
    output = here & (at >= s["prompt_len"][:, None])
    h = s["history"].long()
    zero = torch.zeros((B, V), dtype=torch.int32, device=dev)
    seen = zero.scatter_add(1, h, here.int())[:, None].expand(B, R, V) > 0
    count = zero.scatter_add(1, h, output.int())[:, None].repeat(1, R, 1)
    if s["parents"] is None:
        path = torch.ones((R, R), dtype=torch.int32, device=dev).tril().expand(B, R, R)
    else:
        path = _paths(s["parents"]).int()
    row = torch.arange(B * R, device=dev).view(B, R, 1) * V
    count.view(-1).scatter_add_(0, (row + s["tokens"].long()[:, None, :]).reshape(-1), path.reshape(-1))
    each = lambda t: t[:, None, None]
    seen = seen | (count > 0)
    x = torch.where(seen, torch.where(x > 0, x / each(s["repetition"]), x * each(s["repetition"])), x)
    x = x - count * each(s["frequency"]) - (count > 0) * each(s["presence"])
    if s["bias_tokens"] is not None:
        t = s["bias_tokens"].long()
        bias = torch.zeros((B, V), device=dev).scatter_add_(1, t.clamp_min(0), torch.where(t >= 0, s["bias_values"], 0.0))
        x = x + bias[:, None]
    x = x.view(B * R, V)
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        bits = bits.view(s["mask"].shape[0], -1)[:, :V] > 0
        free = (s["mask_ids"] < 0)[:, None] | bits[s["mask_ids"].clamp_min(0).long()]
        x = torch.where(free, x, -INF)
    return {"logits": x.to(s["logits"].dtype)}


def _plain_fork(s):
    pool, table, refs, src, dst = s["pool"], s["block_table"], s["refs"], s["src"].long(), s["dst"].long()
    P = table.shape[1]
    count = lambda t, by: refs.scatter_add_(0, t.clamp_min(0).long().view(-1), ((t >= 0).int() * by).view(-1))
    count(table[dst], -1)
    n = s["seq_len"][src]
    full, part = n // PAGE, n % PAGE
    free = torch.argsort((refs > 0).int(), stable=True)               # the lowest free pages first
    new = free[(torch.cumsum((part > 0).int(), 0) - 1).clamp_min(0)]
    old = table[src]
    i = torch.arange(P, device=table.device)
    mine = torch.where(i < full[:, None], old, -1)
    mine = torch.where((i == full[:, None]) & (part > 0)[:, None], new[:, None].int(), mine)
    table.index_copy_(0, dst, mine)
    count(mine, 1)
    for k, x in enumerate(s["lens"]):
        if x % PAGE:
            a = pool.index_select(1, old[k, x // PAGE: x // PAGE + 1])
            b = pool.index_select(1, new[k:k + 1])
            b[..., : x % PAGE, :] = a[..., : x % PAGE, :]
            pool.index_copy_(1, new[k:k + 1], b)
    for t in (s["seq_len"], s["pending"], s["hid"]):
        t.index_copy_(0, dst, t[src])
    return _forked(s)


def _forked(s):
    return {k: s[k] for k in ("pool", "block_table", "refs", "seq_len", "pending", "hid")}


def _plain_compact(s):
    pool, table, refs = s["pool"], s["block_table"], s["refs"]
    i = torch.arange(refs.shape[0], device=refs.device)
    live = refs > 0
    n = live.sum()
    moves, holes = live & (i >= n), ~live & (i < n)
    to = torch.argsort((~holes).int(), stable=True)                   # holes in front, ascending
    moved = torch.where(moves, to[(torch.cumsum(moves.int(), 0) - 1).clamp_min(0)], i)
    moved = torch.where(live, moved, -1).int()
    k = s["n_moved"]
    pool.index_copy_(1, to[:k], pool.index_select(1, torch.argsort((~moves).int(), stable=True)[:k]))
    s["table_out"].copy_(torch.where(table >= 0, moved[table.clamp_min(0).long()], -1))
    back = torch.argsort((~live).int(), stable=True)                  # live pages in front
    s["refs_out"].zero_().scatter_(0, moved[back[: s["n_live"]]].long(), refs[back[: s["n_live"]]])
    return {"pool": pool, "block_table": s["table_out"], "refs": s["refs_out"], "moved": moved, "n_live": n.int()}


def run(state):
    s = state
    if not own:
        return {"tree": _plain_tree, "adjust": _plain_adjust, "fork": _plain_fork, "compact": _plain_compact}[s["op"]](s)
    from speculative_decoding_spec_gb300 import binding
    if s["op"] == "tree":
        binding.spec_attention_tree(s["cache"], 0, s["seq_ids"], s["seq_len"], s["q"], s["parents"], n_rows=s["n_rows"],
                                    out=s["out"])
        return {"out": s["out"]}
    if s["op"] == "adjust":
        return {"logits": binding.spec_adjust_logits(
            s["logits"], s["case"]["R"], tokens=s["tokens"], parents=s["parents"], history=s["history"],
            hist_len=s["hist_len"], prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
            frequency=s["frequency"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], mask=s["mask"],
            mask_ids=s["mask_ids"])}
    if s["op"] == "fork":
        binding.spec_pages_fork(s["cache"], s["seq_len"], s["src"], s["dst"], pending=s["pending"], hid=s["hid"])
        return _forked(s)
    moved, n_live = binding.spec_pages_compact(s["cache"], s["table_out"], s["refs_out"])
    return {"pool": s["pool"], "block_table": s["table_out"], "refs": s["refs_out"], "moved": moved, "n_live": n_live[0]}


def work(case):
    c = case
    if c["op"] == "tree":
        es = {"f32": 4, "bf16": 2}
        lens, rows = _lens(c, c["B"]), _rows_of(c)
        # the committed keys of every row, and its own (a row's ancestors are a few more)
        pairs = sum(r * (n + 1) for n, r in zip(lens, rows)) * c["nq"]
        return {"bytes": sum(2.0 * (n + r) * c["nkv"] * c["hd"] * es[c["kv"]] + 2.0 * r * c["nq"] * c["hd"] * es[c["q"]]
                             for n, r in zip(lens, rows)) + 4.0 * c["B"] * c["R"],
                "flops": 4.0 * pairs * c["hd"]}
    if c["op"] == "adjust":
        B, R, V = c["B"], c["R"], c["V"]
        masks = (B + 1) // 2 * R * -(-V // 32) * 4.0 if c["masked"] else 0.0
        return {"bytes": 2.0 * B * R * V * (2 if c["dtype"] == "bf16" else 4) + B * (c["hist"] * 8 / 3 + 20.0) +
                masks + B * c["bias"] * 8.0 + 8.0 * B * R, "flops": 1.0 * B * R * V}
    row = 2.0 * c["L"] * c["nkv"] * c["hd"] * (4 if c["kv"] == "f32" else 2)
    if c["op"] == "fork":
        part = sum(n % PAGE for n in _lens(c, c["src"]))
        pages = sum(-(-n // PAGE) for n in _lens(c, c["src"]))
        return {"bytes": part * row * (1 + c["kids"]) + c["src"] * (1 + c["kids"]) * (c["d"] + 2) * 4.0 +
                8.0 * pages * c["kids"], "flops": 0.0}
    # (how many pages move is the pool's history: about this many)
    moves = int(c["pages"] * c["live"] * (1.0 - c["live"]))
    return {"bytes": 2.0 * PAGE * row * moves + 12.0 * c["pages"], "flops": 0.0}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _chain_up(parents, r):
    while r >= 0:
        yield r
        r = parents[r]


def _exact_tree(c, s):
    B, R, nq, nkv, hd = c["B"], c["R"], c["nq"], c["nkv"], c["hd"]
    out = torch.zeros((B, R, nq, hd), dtype=torch.float64, device=s["q"].device)
    q = s["q"].double().view(B, R, nq, hd)
    table, slots, parents = s["block_table"].tolist(), s["seq_ids"].tolist(), s["parents"].tolist()
    for b in range(B):
        n, rows = s["lens"][b], s["rows"][b]
        at = torch.arange(n + rows, device=q.device)
        page = torch.tensor(table[slots[b]], device=q.device)[at // PAGE]
        seen = torch.zeros((rows, n + rows), dtype=torch.bool, device=q.device)
        seen[:, :n] = True
        for r in range(rows):
            seen[r, [n + j for j in _chain_up(parents[b], r)]] = True
        for h in range(nkv):
            k = s["pool"][0, page, 0, h, at % PAGE].double()
            v = s["pool"][0, page, 1, h, at % PAGE].double()
            for g in range(h * nq // nkv, (h + 1) * nq // nkv):
                z = torch.einsum("rd,nd->rn", q[b, :rows, g], k) * hd ** -0.5
                out[b, :rows, g] = torch.softmax(torch.where(seen, z, -INF), -1) @ v
    return {"out": out.view(B * R, nq * hd)}


def _exact_adjust(c, s):
    B, R, V = c["B"], c["R"], c["V"]
    n = lambda k: None if s[k] is None else s[k].cpu().numpy()
    x = s["logits"].double().cpu().numpy().copy()
    hist, hl, pl, tok = n("history"), n("hist_len"), n("prompt_len"), n("tokens")
    rep, pres, freq = (n(k).astype(np.float64) for k in ("repetition", "presence", "frequency"))
    parents, mask, ids = n("parents"), n("mask"), n("mask_ids")
    for b in range(B):
        text = hist[b, : hl[b]]
        for r in range(R):
            up = list(_chain_up(parents[b], r)) if parents is not None else list(range(r + 1))
            said = np.concatenate([text[pl[b]:], tok[b, up]])
            t, k = np.unique(said, return_counts=True)
            row = x[b * R + r]
            both = np.union1d(text, said)
            row[both] = np.where(row[both] > 0, row[both] / rep[b], row[both] * rep[b])
            row[t] -= k * freq[b] + pres[b]
            if s["bias_tokens"] is not None:
                for i, v in zip(n("bias_tokens")[b], n("bias_values")[b]):
                    if i >= 0:
                        row[i] += float(v)
            if mask is not None and ids[b * R + r] >= 0:
                bits = np.unpackbits(mask[ids[b * R + r]].view(np.uint8), bitorder="little")[:V]
                row[bits == 0] = -np.inf
    return {"logits": x}


def _exact_fork(c, s):
    table, refs, seq_len = (s[k].cpu().numpy().copy() for k in ("block_table", "refs", "seq_len"))
    src, dst = s["src"].tolist(), s["dst"].tolist()
    pending, hid = s["pending"].cpu().numpy().copy(), s["hid"].double().cpu().numpy()
    for d in dst:
        for p in table[d]:
            refs[p] -= p >= 0
        table[d] = -1
    for a, d in zip(src, dst):
        full, part = divmod(int(seq_len[a]), PAGE)
        table[d, :full] = table[a, :full]
        if part:
            table[d, full] = int(np.flatnonzero(refs == 0)[0])
        for p in table[d]:
            refs[p] += p >= 0
        seq_len[d], pending[d], hid[d] = seq_len[a], pending[a], hid[a]
    return {"pool": None, "block_table": table, "refs": refs, "seq_len": seq_len, "pending": pending, "hid": hid}


def _exact_compact(c, s):
    table, refs = s["block_table"].cpu().numpy(), s["refs"].cpu().numpy()
    live = [p for p in range(len(refs)) if refs[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] == 0]
    moved, new = np.full(len(refs), -1, np.int32), np.zeros_like(refs)
    for p in live:
        moved[p] = p if p < n else holes.pop(0)
        new[moved[p]] = refs[p]
    out = np.array([[moved[p] if p >= 0 else -1 for p in row] for row in table], np.int32)
    return {"pool": None, "block_table": out, "refs": new, "moved": moved, "n_live": np.int32(n)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "adjust": _exact_adjust, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](case, s)
