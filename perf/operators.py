"""Cases and plain forms of the operators a batch of requests with settings of its own needs.

`sample`  one token per row of logits, each row with its own temperature, top-k, top-p, min-p and
          uniform number (a decoding step of B sequences, or the scored rows of a verify pass);
`accept`  the sampled accept of a speculative step: every row of [B][k+1] is sampled and a
          sequence's drafts are kept while they equal the samples;
`lora`    one shared projection plus each row's own low-rank adapter.

The definitions, in the order they are applied to a row of logits l with maximum m:
w_i = exp((l_i - m) / T); top-k keeps the first k of the order (logit descending, index ascending);
top-p keeps, of those, the tokens whose preceding mass is below p times their whole mass (always
the first); min-p keeps the tokens with w_i >= min_p; the token is the lowest index at which the
kept mass, summed in index order, exceeds u times the kept mass. T < 1e-5 takes the first token of
the order. Beside the token comes the probability it had: its weight over the kept mass. A row
without a distribution (a NaN, or nothing above -inf) gives token -1 and probability 0; +inf logits
share the whole mass equally.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
GREEDY = 1e-5


def listed():
    return [
        # one small-vocabulary row: the smallest call, all latency
        dict(name="sample_1x4096", op="sample", M=1, V=4096, ld=4096, dtype="f32", temp=0.8, top_k=0, top_p=0.0,
             min_p=0.0, spread=2.0, mixed=False, masked=False),
        # one sequence's decoding step over the full vocabulary with the usual filters
        dict(name="sample_1x262144_kp", op="sample", M=1, V=262144, ld=262144, dtype="f32", temp=0.8, top_k=50,
             top_p=0.95, min_p=0.0, spread=2.0, mixed=False, masked=False),
        # the rows of a batched verify pass, temperature only (the whole vocabulary stays)
        dict(name="sample_40x262144_t", op="sample", M=40, V=262144, ld=262144, dtype="f32", temp=1.0, top_k=0,
             top_p=0.0, min_p=0.0, spread=2.0, mixed=False, masked=False),
        # nucleus sampling of a full batch, every request with settings of its own, some greedy
        dict(name="sample_64x262144_p", op="sample", M=64, V=262144, ld=262144, dtype="f32", temp=0.9, top_k=0,
             top_p=0.9, min_p=0.0, spread=2.5, mixed=True, masked=False),
        # an odd vocabulary in padded bf16 rows, tokens banned by a grammar, k and min-p
        dict(name="sample_13x100003_bf16", op="sample", M=13, V=100003, ld=100008, dtype="bf16", temp=0.7, top_k=64,
             top_p=0.0, min_p=0.05, spread=2.0, mixed=True, masked=True),
        # a speculative step of one sequence
        dict(name="accept_b1_k3", op="accept", B=1, k=3, V=262144, ld=262144, dtype="f32", temp=0.7, top_k=40,
             top_p=0.0, min_p=0.0, spread=2.0, mixed=False, masked=False, alpha=0.8),
        # a speculative step of a batch of eight, all three filters
        dict(name="accept_b8_k4", op="accept", B=8, k=4, V=262144, ld=262144, dtype="f32", temp=0.8, top_k=200,
             top_p=0.95, min_p=0.02, spread=2.0, mixed=True, masked=False, alpha=0.8),
        # a smaller odd vocabulary in bf16
        dict(name="accept_b3_k6_odd", op="accept", B=3, k=6, V=32003, ld=32003, dtype="bf16", temp=0.9, top_k=0,
             top_p=0.9, min_p=0.0, spread=2.0, mixed=True, masked=True, alpha=0.6),
        # the QKV projection of a small decoder, four rows of one request, one adapter, fused norm
        dict(name="lora_m4_2560x1536", op="lora", N=2560, K=1536, M=4, dtype="bf16", rank=16, adapters=1, rows=4,
             none=False, gain=True),
        # gate/up of the 30B-class decoder at batch 8, five rows a request, eight adapters
        dict(name="lora_m40_49152x6144", op="lora", N=49152, K=6144, M=40, dtype="bf16", rank=16, adapters=8, rows=5,
             none=False, gain=True),
        # a 4-bit gate/up with bf16 adapters beside it, some rows without one
        dict(name="lora_m20_q4_12288x1536", op="lora", N=12288, K=1536, M=20, dtype="q4_0", rank=32, adapters=4,
             rows=5, none=True, gain=False),
        # an LM head with adapters, 40 scored rows
        dict(name="lora_m40_262144x2560", op="lora", N=262144, K=2560, M=40, dtype="bf16", rank=64, adapters=8,
             rows=5, none=True, gain=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "accept", "lora"])
    if op == "lora":
        dtype = rng.choice(["bf16", "bf16", "q4_0", "f32"])
        rows = rng.randint(1, 6)
        K = _log(rng, 8, 256) * 32
        # (32-bit weights are for small models: a few rows of a small matrix)
        N = min(_log(rng, 64, 65536), (20_000_000 if dtype == "f32" else 200_000_000) // K)
        M = rng.randint(1, 8 if dtype == "f32" else 64)
        return dict(op="lora", N=N, K=K, M=M, dtype=dtype, rank=8 * rng.randint(1, 12), adapters=_log(rng, 1, 24),
                    rows=rows, none=rng.random() < 0.4, gain=rng.random() < 0.5)
    V = _log(rng, 500, 262144)
    c = dict(op=op, V=V, ld=V + rng.choice([0, 0, 1, 5, 64]), dtype=rng.choice(["f32", "f32", "bf16"]),
             temp=rng.choice([0.5, 0.7, 0.8, 1.0, 1.3]), top_k=rng.choice([0, 0, 1, 20, 50, 500, 5000]),
             top_p=rng.choice([0.0, 0.0, 0.5, 0.8, 0.9, 0.95, 0.99]), min_p=rng.choice([0.0, 0.0, 0.02, 0.1]),
             spread=rng.uniform(1.0, 4.0), mixed=rng.random() < 0.6, masked=rng.random() < 0.3)
    if op == "sample":
        c["M"] = _log(rng, 1, 64)
    else:
        c["B"], c["k"] = _log(rng, 1, 8), rng.randint(0, 7)
        c["alpha"] = rng.uniform(0.3, 0.95)
    return c


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _logits(c, M, g):
    """Rows like a language model's: a broad body, and a few dozen tokens well above it."""
    V = c["V"]
    x = torch.randn((M, c["ld"]), generator=g, device=DEV) * c["spread"]
    at = torch.randint(0, V, (M, 48), generator=g, device=DEV)
    up = torch.empty((M, 48), device=DEV).exponential_(0.35, generator=g) + 2.5 * c["spread"]
    x.scatter_(1, at, up)
    if c["masked"]:  # banned tokens: -inf in some rows, the type's lowest value in others
        ban = torch.rand((M, c["ld"]), generator=g, device=DEV) < 0.7
        low = torch.full((M, 1), float("-inf"), device=DEV)
        low[1::2] = torch.finfo(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32).min
        x = torch.where(ban, low, x)
    x = x.to(torch.bfloat16) if c["dtype"] == "bf16" else x
    return x[:, :V]


def _settings(c, M, g):
    r = lambda: torch.rand(M, generator=g, device=DEV)
    s = {"uniform": (torch.randint(0, 1 << 23, (M,), generator=g, device=DEV).float() + 0.5) / (1 << 23),
         "temperature": c["temp"] * (0.75 + 0.5 * r()), "top_k": None, "top_p": None, "min_p": None}
    if c["top_k"]:
        s["top_k"] = (c["top_k"] * (0.5 + 0.5 * r())).ceil().to(torch.int32)
    if c["top_p"]:
        s["top_p"] = c["top_p"] - 0.1 * r()
    if c["min_p"]:
        s["min_p"] = c["min_p"] * (0.5 + r())
    if c["mixed"]:  # requests that leave a filter out, and greedy ones
        i = torch.arange(M, device=DEV)
        s["temperature"] = torch.where(i % 5 == 4, 0.0, s["temperature"])
        if c["top_k"]:
            s["top_k"] = torch.where(i % 3 == 2, 0, s["top_k"])
        if c["top_p"]:
            s["top_p"] = torch.where(i % 4 == 1, 1.0, s["top_p"])
        if c["min_p"]:
            s["min_p"] = torch.where(i % 2 == 1, 0.0, s["min_p"])
    return {k: v if v is None else v.contiguous() for k, v in s.items()}


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"op": c["op"]}
    if c["op"] == "lora":
        N, K, M, n, r = c["N"], c["K"], c["M"], c["adapters"], c["rank"]
        s["dtype"], s["scales"] = c["dtype"], None
        if c["dtype"] == "q4_0":
            s["w"] = torch.randint(0, 256, (1, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
            s["scales"] = (torch.randn((1, N, K // 32), generator=g, device=DEV) * 0.004).abs().half()
        else:
            dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
            s["w"] = torch.empty((1, N, K), dtype=dt, device=DEV).normal_(0.0, 0.02, generator=g)
        dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        s["a"] = (torch.randn((n, r, K), generator=g, device=DEV) / math.sqrt(K)).to(dt)
        s["b"] = torch.empty((n, N, r), dtype=dt, device=DEV).normal_(0.0, 0.05, generator=g)
        s["scale"] = 0.5 + torch.rand(n, generator=g, device=DEV)
        req = -(-M // c["rows"])
        ids = torch.randperm(n, generator=g, device=DEV)[torch.arange(req, device=DEV) % n]
        if c["none"]:
            ids = torch.where(torch.arange(req, device=DEV) % 4 == 3, -1, ids)
        s["ids"] = ids.repeat_interleave(c["rows"])[:M].to(torch.int32).contiguous()
        s["x"] = torch.randn((M, K), generator=g, device=DEV)
        s["gain"] = 1.0 + 0.1 * torch.randn(K, generator=g, device=DEV) if c["gain"] else None
        return s
    M = c["M"] if c["op"] == "sample" else c["B"] * (c["k"] + 1)
    s["logits"] = _logits(c, M, g)
    s["settings"] = _settings(c, M, g)
    if c["op"] == "accept":
        best = s["logits"].float().argmax(-1).view(c["B"], c["k"] + 1)[:, : c["k"]]
        other = torch.randint(0, c["V"], best.shape, generator=g, device=DEV)
        hit = torch.rand(best.shape, generator=g, device=DEV) < c["alpha"]
        s["drafts"] = torch.where(hit, best, other).to(torch.int32).contiguous()
    return s


# ---- plain forms -------------------------------------------------------------------------------

def _plain_sample(logits, uniform, temperature, top_k, top_p, min_p):
    # 64 bits for the masses: the token is decided by sums of up to V weights next to a border
    x = logits.float()
    M, V = x.shape
    idx = torch.arange(V, device=x.device)
    m = x.amax(-1, keepdim=True)
    d = torch.where(x == m, 0.0, x.double() - m.double())
    T = temperature[:, None].double()
    greedy = T < GREEDY
    first = torch.where(x == m, idx, V).amin(-1, keepdim=True)
    w = torch.where(greedy, (idx == first).double(), torch.exp(d / torch.where(greedy, 1.0, T)))
    keep = None
    if top_k is not None or top_p is not None:
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices
        ws = w.gather(-1, order)
        kept = torch.ones_like(ws, dtype=torch.bool)
        if top_k is not None:
            kept = (idx < torch.where(top_k > 0, top_k, V)[:, None])
        if top_p is not None:
            wk = torch.where(kept, ws, 0.0)
            cum = wk.cumsum(-1)
            before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], -1)
            p = top_p[:, None].double()
            kept = kept & ((before < p * cum[:, -1:]) | (p >= 1.0) | (idx == 0))
        keep = torch.zeros_like(kept).scatter_(-1, order, kept)
    if min_p is not None:
        big = w >= min_p[:, None].double()
        keep = big if keep is None else keep & big
    wk = w if keep is None else torch.where(keep, w, 0.0)
    cum = wk.cumsum(-1)
    total = cum[:, -1:]
    last = torch.where(wk > 0, idx, -1).amax(-1)
    token = torch.minimum((cum <= uniform[:, None].double() * total).sum(-1), last).clamp_min(0)
    prob = (wk.gather(-1, token[:, None]) / total)[:, 0]
    bad = torch.isnan(x).any(-1) | (m[:, 0] == float("-inf"))
    token = torch.where(bad, -1, token)
    return token.to(torch.int32), torch.where(bad, 0.0, prob).float()


def _plain_accept(logits, drafts, **settings):
    B, k = drafts.shape
    token, prob = _plain_sample(logits, **settings)
    token, prob = token.view(B, k + 1), prob.view(B, k + 1)
    live = token >= 0
    same = torch.cat([torch.ones_like(token[:, :1]), (token[:, :k] == drafts).int()], 1)
    emitted = (same.cumprod(1) * live.int().cumprod(1)).bool()
    return (torch.where(emitted, token, -1), emitted.sum(1).to(torch.int32),
            torch.where(emitted, prob, 0.0))


def _plain_weight(w, dtype, scales):
    if dtype != "q4_0":
        return w[0].float()
    N, half = w.shape[1:]
    c = w[0].view(N, half // 16, 16)
    codes = torch.cat([c & 15, c >> 4], -1).float() - 8.0
    return (codes * scales[0].float()[..., None]).view(N, 2 * half)


def _plain_lora(s, eps=1e-6):
    x, a, b = s["x"], s["a"], s["b"]
    n, r, K = a.shape
    N = b.shape[1]
    if s["gain"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * s["gain"]
    y = x @ _plain_weight(s["w"], s["dtype"], s["scales"]).t()
    mine = (s["ids"][:, None] == torch.arange(n, device=x.device)).float() * s["scale"]
    t = (x @ a.float().view(n * r, K).t()).view(-1, n, r) * mine[:, :, None]
    return y + t.view(-1, n * r) @ b.float().permute(0, 2, 1).reshape(n * r, N)


def run(state):
    s = state
    if own:
        from speculative_decoding_spec_gb300 import binding, synth
        if s["op"] == "lora":
            N, K = s["w"].shape[1], s["x"].shape[1]
            w = synth.WTensor(s["dtype"], 1, N, K, s["w"], s["scales"])
            lora = binding.Lora(s["a"], s["b"], s["scale"])
            return {"y": binding.spec_linear_lora(w, s["x"], lora, s["ids"], gain=s["gain"])}
        if s["op"] == "sample":
            token, prob = binding.spec_sample(s["logits"], **s["settings"])
            return {"token": token, "prob": prob}
        out, n, prob = binding.spec_accept_sampled(s["logits"], s["drafts"], **s["settings"])
        return {"out": out, "n": n, "prob": prob}
    if s["op"] == "lora":
        return {"y": _plain_lora(s)}
    if s["op"] == "sample":
        token, prob = _plain_sample(s["logits"], **s["settings"])
        return {"token": token, "prob": prob}
    out, n, prob = _plain_accept(s["logits"], s["drafts"], **s["settings"])
    return {"out": out, "n": n, "prob": prob}


def work(case):
    c = case
    if c["op"] == "lora":
        N, K, M, r = c["N"], c["K"], c["M"], c["rank"]
        per = {"bf16": 2.0, "f32": 4.0, "q4_0": 0.5 + 2.0 / 32}[c["dtype"]]
        req = -(-M // c["rows"])
        used = len({i % c["adapters"] for i in range(req) if not (c["none"] and i % 4 == 3)})
        ab = 4 if c["dtype"] == "f32" else 2
        on = sum(min(c["rows"], M - i * c["rows"]) for i in range(req) if not (c["none"] and i % 4 == 3))
        return {"bytes": N * K * per + used * r * (K + N) * ab + 4.0 * M * (K + N) + 4.0 * M,
                "flops": 2.0 * M * N * K + 2.0 * on * r * (K + N)}
    M = c["M"] if c["op"] == "sample" else c["B"] * (c["k"] + 1)
    # a difference, a scaling, an exponential and a sum for every logit; settings and results are a few words a row
    return {"bytes": M * c["V"] * (2 if c["dtype"] == "bf16" else 4) + 28.0 * M, "flops": 4.0 * M * c["V"]}


# ---- the definitions in 64 bits, one row at a time ---------------------------------------------

def _exact_row(l, u, T, k, p, q):
    n = len(l)
    if np.isnan(l).any() or l.max() == -np.inf:
        return -1, 0.0
    if T < GREEDY:
        return int(np.flatnonzero(l == l.max())[0]), 1.0
    if l.max() == np.inf:
        w = (l == np.inf).astype(np.float64)
    else:
        w = np.exp((l - l.max()) / T)
    keep = np.ones(n, bool)
    if (k is not None and 0 < k < n) or (p is not None and p < 1.0):
        order = np.lexsort((np.arange(n), -l))
        order = order[:k] if k is not None and k > 0 else order
        if p is not None and p < 1.0:
            mass = np.concatenate([[0.0], np.cumsum(w[order])])
            order = order[: max(1, int(np.searchsorted(mass[:-1], p * mass[-1], "left")))]
        keep[:] = False
        keep[order] = True
    if q is not None:
        keep &= w >= q
    at = np.flatnonzero(keep & (w > 0))
    cum = np.cumsum(w[at])
    j = min(int(np.searchsorted(cum, u * cum[-1], "right")), len(at) - 1)
    return int(at[j]), float(w[at[j]] / cum[-1])


def _exact_sample(logits, st):
    l = logits.float().cpu().numpy().astype(np.float64)
    v = {k: None if t is None else t.cpu().numpy().astype(np.int64 if k == "top_k" else np.float64)
         for k, t in st.items()}
    at = lambda k, i: None if v[k] is None else v[k][i]
    rows = [_exact_row(l[i], v["uniform"][i], v["temperature"][i], at("top_k", i), at("top_p", i), at("min_p", i))
            for i in range(len(l))]
    return np.array([r[0] for r in rows], np.int32), np.array([r[1] for r in rows])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        token, prob = _exact_sample(s["logits"], s["settings"])
        return {"token": token, "prob": prob}
    if case["op"] == "accept":
        B, k = s["drafts"].shape
        token, prob = _exact_sample(s["logits"], s["settings"])
        token, prob, d = token.reshape(B, k + 1), prob.reshape(B, k + 1), s["drafts"].cpu().numpy()
        out, lp, count = np.full((B, k + 1), -1, np.int32), np.zeros((B, k + 1)), np.zeros(B, np.int32)
        for b in range(B):
            for j in range(k + 1):
                if token[b, j] < 0:
                    break
                out[b, j], lp[b, j], count[b] = token[b, j], prob[b, j], j + 1
                if j < k and d[b, j] != token[b, j]:
                    break
        return {"out": out, "n": count, "prob": lp}
    x = s["x"].double()
    if s["gain"] is not None:
        x = x / torch.sqrt((x ** 2).sum(1, keepdim=True) / x.shape[1] + 1e-6) * s["gain"].double()
    y = torch.empty((case["M"], case["N"]), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 28) // case["K"])
    for n0 in range(0, case["N"], step):  # some rows of the weights at a time
        w = s["w"][0, n0:n0 + step]
        if case["dtype"] == "q4_0":
            full = torch.empty((w.shape[0], case["K"]), dtype=torch.float64, device=x.device)
            for i in range(16):
                full[:, i::32] = (w[:, i::16] % 16).double() - 8
                full[:, i + 16::32] = (w[:, i::16] // 16).double() - 8
            w = full * s["scales"][0, n0:n0 + step].double().repeat_interleave(32, 1)
        y[:, n0:n0 + step] = torch.einsum("mk,nk->mn", x, w.double())
    for i, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            t = s["a"][a].double() @ x[i]
            y[i] += float(s["scale"][a]) * (s["b"][a].double() @ t)
    return {"y": y}
