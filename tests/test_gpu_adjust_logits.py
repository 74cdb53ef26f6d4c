"""spec_adjust_logits against the 64-bit reference (tests/branch_ref.py).

Tolerance: a logit goes through at most a division or product, a count's product
with its subtraction, the presence's subtraction and the bias's addition, each
rounded once to binary32: 6 * 2^-24 of the largest magnitude on the way, and for
bf16 the result's rounding of 2^-8."""
import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding
from tests import branch_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def _case(B, R, V, dtype="f32", hist=200, bias=7, mask=True, tree=False, pad=0, seed=0):
    rng = np.random.default_rng(seed)
    cu = lambda x, t=np.int32: torch.from_numpy(np.ascontiguousarray(x, t)).cuda()
    f = np.float32
    x = (torch.randn((B * R, V + pad), generator=torch.Generator().manual_seed(seed)) * 4).to(DT[dtype])
    x[:, ::17] = -float("inf")
    x[::2, 5::23] = torch.finfo(DT[dtype]).min
    a = dict(R=R, tokens=cu((V * rng.random((B, R)) ** 2).astype(int)), parents=cu(ref.random_parents(rng, B, R)) if tree else None)
    if hist:
        h = (V * rng.random((B, hist)) ** 3).astype(int)
        h[rng.random((B, hist)) < 0.1] = -1
        h[rng.random((B, hist)) < 0.05] = V + 3
        a.update(history=cu(h), hist_len=cu(rng.integers(0, hist + 1, B)))
        a["prompt_len"] = cu((a["hist_len"].cpu().numpy() * rng.random(B)).astype(int))
    a.update(rep=cu(rng.uniform(0.7, 1.5, B), f), pres=cu(rng.uniform(-0.5, 1, B), f), freq=cu(rng.uniform(-0.2, 0.7, B), f))
    if bias:
        t = rng.integers(-1, V + 1, (B, bias))
        v = rng.normal(0, 6, (B, bias))
        v[rng.random((B, bias)) < 0.1] = -np.inf
        a.update(bias_tokens=cu(t), bias_values=cu(v, f))
    if mask:
        n = max(1, B * R // 2)
        a.update(mask=cu(rng.integers(-(1 << 31), 1 << 31, (n, (V + 31) // 32)).astype(np.int64).astype(np.int32)),
                 mask_ids=cu(rng.integers(-1, n, B * R)))
    return x.cuda()[:, :V], a


def _call(x, a, **kw):
    names = dict(rep="repetition", pres="presence", freq="frequency")
    return binding.spec_adjust_logits(x, **{names.get(k, k): v for k, v in a.items()}, **kw)


def _want(x, a):
    b = {k: _np(v) if torch.is_tensor(v) else v for k, v in a.items()}
    b["x"] = _np(x)
    if b.get("history") is not None:
        b["hist"] = b.pop("history")
    b.pop("history", None)
    return ref.adjust(b.pop("x"), b.pop("R"), **b)


def _check(x, a, got=None):
    got, want = _np(_call(x, a) if got is None else got), _want(x, a)
    big = np.abs(_np(x))
    big = np.where(np.isfinite(big), big, 0)
    for k in ("rep", "pres", "freq"):
        if a.get(k) is not None:
            v = np.abs(_np(a[k]))[:, None].repeat(a["R"], 0).reshape(-1, 1)
            n = 1 + (0 if a.get("history") is None else a["history"].shape[1]) + a["R"]
            v = np.where(np.isfinite(v), v, 0)
            big = big * np.maximum(v, np.where(v > 0, 1 / np.maximum(v, 1e-30), 1)) if k == "rep" else big + v * (n if k == "freq" else 1)
    if a.get("bias_values") is not None:
        v = np.abs(_np(a["bias_values"]))
        big = big + np.where(np.isfinite(v), v, 0).max(1).repeat(a["R"])[:, None]
    # (what rounds past the type's largest value is infinite: its lowest value, made lower by a penalty, is forbidden)
    r = torch.from_numpy(want).float().to(x.dtype).double().numpy()
    want = np.where(np.isinf(r), r, want)
    ban = want == -np.inf
    assert np.array_equal(got == -np.inf, ban)
    if x.dtype is torch.float32:
        tol = 6 * 2.0 ** -24 * big
    else:
        tol = 6 * 2.0 ** -24 * big + 2.0 ** -8 * np.abs(np.where(ban, 0, want))
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    inf = want == np.inf
    assert np.array_equal(got == np.inf, inf)
    ok = ~(ban | nan | inf)
    err = np.abs(got[ok] - want[ok])
    assert (err <= tol[ok]).all(), (err - tol[ok]).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 500, 1023, 1025, 4096, 16385, 32003, 100003])
@pytest.mark.parametrize("B,R,tree", [(1, 1, False), (3, 5, False), (2, 7, True)])
def test_matches_reference(dtype, V, B, R, tree):
    for pad in (0, 1, 6):
        x, a = _case(B, R, V, dtype, tree=tree, pad=pad, seed=V + pad)
        _check(x, a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drop", ["history", "bias", "mask", "pen", "tokens", "all"])
def test_parts_left_out(dtype, drop):
    x, a = _case(3, 4, 5003, dtype, seed=3)
    gone = dict(history=["history", "hist_len", "prompt_len"], bias=["bias_tokens", "bias_values"], mask=["mask", "mask_ids"],
                pen=["rep", "pres", "freq"], tokens=["tokens"])
    for k in sum(gone.values(), []) if drop == "all" else gone[drop]:
        a[k] = None
    _check(x, a)
    if drop == "all":
        assert torch.equal(_call(x, a), x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R,tree", [(64, True), (64, False), (200, False), (33, True)])
def test_many_rows(dtype, R, tree):
    x, a = _case(2, R, 3000, dtype, tree=tree, seed=R)
    _check(x, a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lists_and_histories(dtype):
    """Long histories of one token, empty ones, long lists with repeated entries, lengths left out."""
    x, a = _case(3, 2, 70000, dtype, hist=30000, bias=4000, seed=5)
    a["history"][0] = 17
    a["hist_len"][1] = 0
    a["bias_tokens"][2] = torch.arange(4000, dtype=torch.int32, device="cuda") % 50 * 3
    _check(x, a)
    a["hist_len"] = a["prompt_len"] = None
    _check(x, a)
    a["history"] = torch.cat([a["history"]] * 2, 1)[:, 7:20007]     # rows that start anywhere
    _check(x, a)


def test_edges_of_settings():
    x, a = _case(8, 1, 600, "f32", seed=6)
    nan, inf = float("nan"), float("inf")
    a["rep"] = torch.tensor([0.0, -1.0, nan, inf, 1.0, 1e-30, 1e30, 1.2], device="cuda")
    a["pres"] = torch.tensor([nan, inf, -inf, 0.0, 1e30, -1e30, 0.5, 0.5], device="cuda")
    a["freq"] = torch.tensor([inf, nan, 0.0, -inf, 1e30, 0.1, 0.0, 0.3], device="cuda")
    a["bias_values"][:, 3] = nan
    a["bias_values"][:, 4] = inf
    a["bias_tokens"][:, 3:5] = torch.tensor([11, 13], dtype=torch.int32, device="cuda")
    a["bias_tokens"][:, 5:] = -1
    x[:, 40] = inf
    x[:, 41] = nan
    _check(x, a)
    a["mask_ids"][:] = 0
    a["mask"][0] = 0                                      # a mask that leaves nothing
    assert (_call(x, a) == -inf).all()
    tok, prob = binding.spec_sample(_call(x, a), torch.full((8,), 0.5, device="cuda"))
    assert (tok == -1).all() and (prob == 0).all()
    a["mask"][0] = -1
    _check(x, a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,pad", [(4096, 0), (4096, 8), (5001, 0), (5001, 3), (33, 1)])
@pytest.mark.parametrize("tree", [False, True])
def test_in_place_and_given_outputs(dtype, V, pad, tree):
    x, a = _case(2, 5, V, dtype, tree=tree, pad=pad, seed=7)
    want = _call(x, a)
    full = torch.full((10, V + pad + 9), 3.0, dtype=x.dtype, device="cuda")
    for at in (0, 1, 8):
        full.fill_(3.0)
        out = full[:, at:at + V]
        assert _call(x, a, out=out) is out and torch.equal(out, want)
        assert (full[:, :at] == 3).all() and (full[:, at + V:] == 3).all()
    base = x.clone()
    got = _call(base, a, out=base)
    assert got is base and torch.equal(base, want)
    whole = torch.full((10, V + pad + 5), 2.0, dtype=x.dtype, device="cuda")
    mine = whole[:, 3:3 + V]
    mine.copy_(x)
    _call(mine, a, out=mine)
    assert torch.equal(mine, want) and (whole[:, :3] == 2).all() and (whole[:, 3 + V:] == 2).all()


def test_status_and_ids_out_of_range():
    x, a = _case(3, 4, 900, "f32", tree=True, seed=8)
    want, status = _call(x, a), torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(_call(x, a, status=status), want) and status[0] == 0
    n = a["history"].shape[1]

    def changed(key, at, bad, same):
        b = dict(a)
        b[key] = a[key].clone()
        b[key][at] = same
        want = _call(x, b)
        b[key][at] = bad
        status.zero_()
        assert torch.equal(_call(x, b, status=status), want) and status[0] == 2
        assert torch.equal(_call(x, b), want)

    for bad, same in ((-1, 0), (-(1 << 31), 0), (n + 1, n), ((1 << 31) - 1, n)):
        changed("hist_len", 1, bad, same)
    for bad in (3, 2, -2, 1 << 30):
        changed("parents", (1, 2), bad, -1)
    for bad in (-2, a["mask"].shape[0], 1 << 30):
        changed("mask_ids", 5, bad, -1)


def test_graph_streams_and_two_at_once():
    x, a = _case(8, 5, 100003, "f32", seed=9)
    y, b = _case(2, 9, 32003, "bf16", tree=True, seed=10)
    wx, wy = _call(x, a), _call(y, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(_call(x, a, stream=s1), _call(y, b, stream=s2)) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, wx) and torch.equal(q, wy) for p, q in got)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _call(x, a, out=out)
    a["hist_len"] //= 2
    a["prompt_len"] //= 2
    want = _call(x, dict(a))
    g.replay()          # (the captured call reads the tensors it was given)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not torch.equal(want, wx)


def test_then_sampled():
    """Greedy rows of the changed logits are the reference's largest allowed logits."""
    x, a = _case(4, 3, 50021, "f32", seed=11)
    y = _call(x, a)
    u = torch.full((12,), 0.5, device="cuda")
    tok, _ = binding.spec_sample(y, u, temperature=torch.zeros(12, device="cuda"))
    w = _want(x, a)
    for m, t in enumerate(tok.tolist()):
        assert w[m, t] >= w[m].max() - 1e-5 and np.isfinite(w[m, t])


def test_refusals():
    x, a = _case(3, 4, 900, "f32", seed=12)
    run = lambda logits=x, **k: _call(logits, {**a, **k})
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    bad = [
        lambda: run(x.half()), lambda: run(x.cpu()), lambda: run(x[0]), lambda: run(x[:0]), lambda: run(x.t().contiguous().t()),
        lambda: run(x[:11]), lambda: run(R=0), lambda: run(tokens=i32(3, 3)), lambda: run(tokens=a["tokens"].long()),
        lambda: run(parents=i32(12).cpu()), lambda: run(history=a["history"].long()), lambda: run(history=a["history"][:2]),
        lambda: run(history=i32(200, 3).t()), lambda: run(hist_len=i32(2)), lambda: run(prompt_len=i32(3).float()),
        lambda: run(rep=a["rep"].double()), lambda: run(pres=a["pres"][:2]), lambda: run(freq=a["freq"].cpu()),
        lambda: run(bias_tokens=None), lambda: run(bias_values=None), lambda: run(bias_values=a["bias_values"][:, :3]),
        lambda: run(bias_tokens=i32(2, 2), bias_values=i32(2, 2).float()), lambda: run(mask=a["mask"][:, :5]),
        lambda: run(mask=a["mask"].long()), lambda: run(mask_ids=None), lambda: run(mask_ids=i32(5)),
        lambda: run(mask=a["mask"][:1].expand(3, -1)),
        lambda: run(history=i32(3, 1 << 19)), lambda: run(bias_tokens=i32(3, 4096), bias_values=i32(3, 4096).float()),
        lambda: _call(x, a, out=x[:5]), lambda: _call(x, a, out=torch.empty_like(x, dtype=torch.bfloat16)),
        lambda: _call(x, a, out=torch.empty((900, 12), device="cuda").t()), lambda: _call(x, a, status=i32(2)),
        lambda: _call(x, a, out=x[:1].expand(12, -1)),
        lambda: binding.spec_adjust_logits(torch.zeros((65, 40), device="cuda"), 65, tokens=i32(1, 65), parents=i32(1, 65)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(binding.SpecError):
            f()
            pytest.fail("call %d was not refused" % i)
    _check(x, a)


# Calls of a megabyte and more, whose tokens are counted in hash tables beside the copy.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,pad", [(300032, 0), (300007, 1), (300007, 2)])
@pytest.mark.parametrize("mask", [False, True])
def test_large_in_place_and_given_outputs(dtype, V, pad, mask):
    x, a = _case(2, 3, V, dtype, tree=True, pad=pad, seed=13, mask=mask, hist=3000, bias=50)
    want = _call(x, a)
    _check(x, a, want)
    full = torch.full((6, V + pad + 9), 3.0, dtype=x.dtype, device="cuda")
    for at in (0, 1, 8):
        full.fill_(3.0)
        assert torch.equal(_call(x, a, out=full[:, at:at + V]), want)
        assert (full[:, :at] == 3).all() and (full[:, at + V:] == 3).all()
    for at in (0, 3):
        full.fill_(2.0)
        mine = full[:, at:at + V]
        mine.copy_(x)
        _call(mine, a, out=mine)
        assert torch.equal(mine, want) and (full[:, :at] == 2).all() and (full[:, at + V:] == 2).all()


@pytest.mark.parametrize("R,tree", [(64, True), (64, False), (65, False)])
def test_large_with_many_rows(R, tree):
    x, a = _case(1, R, 20011, "f32", tree=tree, seed=14, hist=400)
    a["tokens"][0, 1::2] = a["tokens"][0, 0]              # the same token on many paths
    a["history"][0, :200] = a["tokens"][0, 0]
    _check(x, a)


@pytest.mark.parametrize("hist", [1, 12000, 12288, 12300])
def test_large_with_as_many_tokens_as_a_table_holds(hist):
    V = 262144
    x, a = _case(2, 2, V, "f32", seed=15, hist=hist, bias=0, mask=False)
    a["history"] = (torch.arange(2 * hist, device="cuda", dtype=torch.int32) * 21 % V).view(2, hist)   # all different
    a["hist_len"] = a["prompt_len"] = None
    _check(x, a)
    a["history"].zero_()                                  # all the same
    _check(x, a)
    nan, inf = float("nan"), float("inf")
    a["rep"][0], a["pres"][0], a["freq"][0] = 1.0, 0.0, nan   # a sequence that leaves all out, beside one that does not
    x[:, 7] = inf
    x[:, 0] = nan
    a["bias_tokens"] = torch.tensor([[5, 7, 5, -1], [0, V, 9, 9]], dtype=torch.int32, device="cuda")
    a["bias_values"] = torch.tensor([[1.0, -inf, nan, 2.0], [3.0, 1.0, -inf, 2.0]], device="cuda")
    _check(x, a)


@pytest.mark.parametrize("V", [600, 300007])
def test_forbidden_stays_forbidden_with_infinite_rewards(V):
    """Two occurrences at a frequency of -3e38 sum to an infinite reward."""
    x, a = _case(2, 1, V, "f32", hist=0, bias=0, mask=False, seed=12)
    x[:, 5:9] = -float("inf")
    a["history"] = torch.tensor([[5, 5, 6, 7], [8, 8, 8, 5]], dtype=torch.int32, device="cuda")
    a["hist_len"] = a["prompt_len"] = None
    a["freq"] = torch.full((2,), -3e38, device="cuda")
    a["tokens"] = torch.tensor([[7], [20]], dtype=torch.int32, device="cuda")
    got = _call(x, a)
    assert (got[:, 5:9] == -float("inf")).all() and not torch.isnan(got).any()


@pytest.mark.parametrize("V", [40, 4096, 5001, 300032, 300011])
@pytest.mark.parametrize("pen", [False, True])
def test_in_place_leaves_what_stays(V, pen):
    """In place, a logit that stays as it is keeps its bits beside forbidden ones: a NaN's (a rewrite gives the type's own NaN)."""
    x, a = _case(2, 2, V, "bf16", hist=20 if pen else 0, bias=0, seed=V, mask=True)
    a["mask_ids"] = torch.tensor([0, 1, 0, 1], dtype=torch.int32, device="cuda")
    if not pen:
        a["rep"] = a["pres"] = a["freq"] = a["tokens"] = None
    full = torch.zeros((4, (V + 7) // 8 * 8 + 8), dtype=torch.bfloat16, device="cuda")    # (rows on 16-byte boundaries, and 6 bytes behind them)
    for at in (0, 3):
        mine = full[:, at:at + V]
        bits = mine.view(torch.int16)
        g = torch.Generator(device="cuda").manual_seed(V)
        bits.copy_(torch.randint(0x7f81, 0x7fff, (4, V), generator=g, device="cuda", dtype=torch.int16))
        was = bits.clone()
        _call(mine, a, out=mine)
        words = a["mask"][a["mask_ids"].long()]
        t = torch.arange(V, device="cuda")
        banned = ((words[:, t // 32] >> (t % 32).int()) & 1) == 0
        said = torch.zeros((4, V + 4), dtype=torch.bool, device="cuda")
        if pen:
            rows = torch.arange(4, device="cuda")[:, None]
            said[rows, a["history"].repeat_interleave(2, 0).long()] = True      # (padding: -1 and V + 3 are columns behind)
            said[rows, a["tokens"].repeat_interleave(2, 0).long()] = True
        said = said[:, :V]
        assert (mine[banned] == -float("inf")).all()
        stays = ~banned & ~said
        assert torch.equal(bits[stays], was[stays])


@pytest.mark.parametrize("V", [600, 300007])
def test_status_of_what_does_not_count(V):
    """A length, prompt or parent that no penalty uses is not recorded, in small calls and in large ones."""
    x, a = _case(3, 4, V, "f32", tree=True, seed=8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    off = dict(a, rep=None, pres=None, freq=None)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for key, bad in (("hist_len", i32(-1, 1 << 30, 0)), ("prompt_len", i32(-7, 0, 1 << 30)),
                     ("parents", torch.full_like(a["parents"], 99))):
        b = dict(off, **{key: bad})
        assert torch.equal(_call(x, b, status=status), _call(x, off)) and status[0] == 0, key
        ones, zeros = torch.ones(3, device="cuda"), torch.zeros(3, device="cuda")
        b.update(rep=ones, pres=zeros, freq=zeros)            # settings that change nothing
        assert torch.equal(_call(x, b, status=status), _call(x, off)) and status[0] == 0, key
        b["rep"] = torch.tensor([1.0, 1.0, 1.25], device="cuda")
        _call(x, b, status=status)                            # the last sequence's count (a prompt longer than no history too)
        assert status[0] == 2, key
        status.zero_()
    b = dict(off, rep=torch.tensor([1.0, 1.0, 1.25], device="cuda"), hist_len=i32(-1, 1 << 30, int(a["hist_len"][2])))
    assert int(a["prompt_len"][2]) > 0
    _call(x, b, status=status)                                # the others' do not
    assert status[0] == 0
    b = dict(a, tokens=None, parents=torch.full_like(a["parents"], 99))
    assert torch.equal(_call(x, b, status=status), _call(x, dict(b, parents=None))) and status[0] == 0
