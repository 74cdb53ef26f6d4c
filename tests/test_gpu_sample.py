"""GPU parity of spec_sample, spec_accept_sampled and spec_verify_sampled with
the 64-bit reference (tests/sampling_ref.py): tokens are equal wherever the
reference's decisions are not on a border, probabilities to 2^-21 relative (a
weight to 2^-24, the kept mass rounded to binary32 and one division: under four
roundings of 2^-24, and the mass's own 2^-36 and V * 2^-44)."""
import dataclasses

import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding, configs, synth
from tests import sampling_ref as ref

pytestmark = pytest.mark.gpu
PTOL = 2.0 ** -21


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _check(x, got, u, T=None, k=None, p=None, q=None, most_undecided=0.02):
    tok, prob = (t.cpu().numpy() for t in got)
    n = lambda t: None if t is None else t.cpu().numpy()
    rt, rp, decided = ref.rows(x.float().cpu().numpy(), n(u), n(T), n(k), n(p), n(q))
    assert decided.mean() >= 1 - most_undecided or (~decided).sum() <= 1
    assert np.array_equal(tok[decided], rt[decided]), (tok, rt, decided)
    assert np.all(np.abs(prob - rp)[decided] <= PTOL * rp[decided]), (prob, rp)


SETTINGS = {
    "plain": {},
    "temp": dict(T=0.7),
    "k": dict(T=0.9, k=7),
    "k_large": dict(T=1.2, k=900),
    "p": dict(T=0.8, p=0.9),
    "p_small": dict(T=1.5, p=0.05),
    "q": dict(T=1.0, q=0.05),
    "kpq": dict(T=0.8, k=50, p=0.95, q=0.01),
    "p_all": dict(T=1.0, p=0.9999),
    "cold": dict(T=0.01, p=0.5),
    "hot": dict(T=40.0, k=1000, p=0.7),
}


def _vec(v, M, dtype=torch.float32):
    return None if v is None else torch.full((M,), v, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 5, 33, 1000, 4099, 32003, 100003, 262144])
@pytest.mark.parametrize("name", list(SETTINGS))
def test_sample_matches_reference(dtype, V, name):
    c = SETTINGS[name]
    M = 6 if V > 50000 else 11
    g = _gen(V + len(name))
    x = (torch.randn((M, V), generator=g, device="cuda") * 2.5).to(dtype)
    u = torch.rand(M, generator=g, device="cuda")
    T, k, p, q = _vec(c.get("T"), M), _vec(c.get("k"), M, torch.int32), _vec(c.get("p"), M), _vec(c.get("q"), M)
    _check(x, binding.spec_sample(x, u, T, k, p, q), u, T, k, p, q)


# Top-p's cut found in a few bins: nuclei from a token to most of the row, values so
# coarse that thousands of tokens share one, and min-p's end around top-p's.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2500, 32003, 262144])
@pytest.mark.parametrize("kind", ["smooth", "coarse", "halves", "equal", "masked", "inf", "huge"])
def test_nuclei(dtype, V, kind):
    M = 12
    g = _gen(V + len(kind))
    x = torch.randn((M, V), generator=g, device="cuda") * 2.5
    if kind == "coarse":
        x = (x * 2).round() / 2
    elif kind == "halves":
        x = (x > 0).float() * 1.5
    elif kind == "equal":
        x.fill_(3.25)
    elif kind == "masked":
        x[torch.rand((M, V), generator=g, device="cuda") < 0.97] = -float("inf")
        x[:, V // 2] = 1.0
    elif kind == "inf":
        x[torch.rand((M, V), generator=g, device="cuda") < 0.3] = float("inf")
        x[:, V // 2] = float("inf")
    elif kind == "huge":
        x = x * 1e37
    x = x.to(dtype)
    u = torch.rand(M, generator=g, device="cuda")
    T = torch.linspace(0.4, 3.0, M, device="cuda")
    if kind == "huge":
        T = T * 1e37
    p = torch.tensor([0.9, 0.5, 0.05, 0.99, 0.9999, 0.7, 0.2, 0.95, 0.999, 0.31, 0.83, 0.61], device="cuda")
    _check(x, binding.spec_sample(x, u, T, None, p), u, T, None, p, most_undecided=0.1)
    q = torch.tensor([0.5, 0.3, 0.9, 1e-4, 1e-9, 0.1, 0.03, 0.01, 0.003, 0.6, 0.2, 0.05], device="cuda")
    _check(x, binding.spec_sample(x, u, T, None, p, q), u, T, None, p, q, most_undecided=0.1)
    k = torch.randint(1, V, (M,), generator=g, device="cuda").int()
    _check(x, binding.spec_sample(x, u, T, k, p, q), u, T, k, p, q, most_undecided=0.1)
    _check(x, binding.spec_sample(x, u, T, k, p), u, T, k, p, most_undecided=0.1)
    _check(x, binding.spec_sample(x, u, T, k), u, T, k, most_undecided=0.1)


# min-p's end moved across the bins in which top-p's cut lies
def test_min_p_around_the_nucleus():
    V, M = 100003, 96
    g = _gen(5)
    x = (torch.randn((1, V), generator=g, device="cuda") * 2.5).expand(M, V)
    u = torch.rand(M, generator=g, device="cuda")
    T, p = _vec(1.0, M), _vec(0.8, M)
    w = torch.sort(torch.exp((x[0] - x[0].max()).double()), descending=True).values
    at = w[int((torch.cumsum(w, 0) < 0.8 * w.sum()).sum())].item()   # the weight of the last token of the nucleus
    q = (at * torch.exp(torch.linspace(-0.08, 0.08, M, dtype=torch.float64))).float().cuda()
    x = x.contiguous()
    _check(x, binding.spec_sample(x, u, T, None, p, q), u, T, None, p, q)


# top_p a rounding away from where a token enters the nucleus: nearer than the plain
# float sums that decide most narrow nuclei can tell.
@pytest.mark.parametrize("V", [4099, 262144])
def test_top_p_beside_a_border(V):
    M = 96
    g = _gen(V)
    x = (torch.randn((1, V), generator=g, device="cuda") * 9).repeat(M, 1)
    u = torch.rand(M, generator=g, device="cuda")
    w = torch.sort(torch.exp((x[0].double() - x[0].max().double())), descending=True).values
    at = (torch.cumsum(w, 0) / w.sum())[1:33].repeat_interleave(3).float()
    p = torch.nextafter(at, torch.tensor([0.0, 2.0, 1.0], device="cuda").repeat(32))
    p[2::3] = at[2::3] * (1 - 2.0 ** -19)
    _check(x, binding.spec_sample(x, u, None, None, p), u, None, None, p, most_undecided=0.1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,ld,off", [(1000, 1003, 0), (4097, 4097, 1), (32003, 32010, 3), (50001, 50001, 7)])
def test_strided_and_unaligned_rows(dtype, V, ld, off):
    M = 5
    g = _gen(ld)
    buf = (torch.randn(off + M * ld, generator=g, device="cuda") * 3).to(dtype)
    x = buf[off:off + M * ld].view(M, ld)[:, :V]
    u = torch.rand(M, generator=g, device="cuda")
    T, k, p = _vec(0.8, M), _vec(100, M, torch.int32), _vec(0.9, M)
    _check(x, binding.spec_sample(x, u, T, k, p), u, T, k, p)
    _check(x, binding.spec_sample(x, u, T), u, T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,ld,off", [(64, 32773, 32773, 0), (22, 100003, 100010, 3), (9, 262144, 262144, 0),
                                         (5, 500000, 500003, 1), (40, 57344, 57344, 0)])
def test_large_calls(dtype, M, V, ld, off):
    """Calls that read their rows in chunks first: every row with settings of its
    own (plain, filtered, greedy), with masks and without."""
    g = _gen(M + V)
    buf = (torch.randn(off + M * ld, generator=g, device="cuda") * 2.5).to(dtype)
    x = buf[off:off + M * ld].view(M, ld)[:, :V]
    x[:, torch.randint(0, V, (40,), generator=g, device="cuda")] += 9.0
    x[1, torch.rand(V, generator=g, device="cuda") < 0.9] = -float("inf")
    x[3, ::2] = torch.finfo(dtype).min
    x[4, :V - 1] = -float("inf")
    u = torch.rand(M, generator=g, device="cuda")
    i = torch.arange(M, device="cuda")
    T = torch.where(i % 7 == 6, 0.0, 0.5 + 0.1 * (i % 9)).contiguous()
    k = torch.where(i % 4 == 1, 30 + i, torch.where(i % 4 == 3, 3000, 0)).to(torch.int32)
    p = torch.where(i % 3 == 0, 1.0, 0.7 + 0.29 * (i % 5) / 4).contiguous()
    q = torch.where(i % 5 == 2, 0.02, 0.0).contiguous()
    assert binding.lib().spec_sample_workspace_bytes(M, V) > 0
    _check(x, binding.spec_sample(x, u, T, k, p, q), u, T, k, p, q)
    _check(x, binding.spec_sample(x, u, T), u, T)
    _check(x, binding.spec_sample(x, u, T, None, p), u, T, None, p)
    x[0, V // 2] = float("nan")
    x[2, [5, V - 1]] = float("inf")
    x[3] = -float("inf")
    tok, prob = binding.spec_sample(x, u)
    assert tok[0] == -1 and prob[0] == 0 and tok[2] == (5 if u[2] < 0.5 else V - 1) and prob[2] == 0.5 and tok[3] == -1


def test_settings_differ_by_row():
    M, V = 64, 5003
    g = _gen(3)
    x = torch.randn((M, V), generator=g, device="cuda") * 3
    u = torch.rand(M, generator=g, device="cuda")
    T = torch.rand(M, generator=g, device="cuda") * 2
    T[::5] = 0.0
    k = torch.randint(-3, 300, (M,), generator=g, device="cuda", dtype=torch.int32)
    p = torch.rand(M, generator=g, device="cuda") * 1.2
    q = torch.rand(M, generator=g, device="cuda") * 0.4 - 0.1
    _check(x, binding.spec_sample(x, u, T, k, p, q), u, T, k, p, q)


@pytest.mark.parametrize("V", [3, 700, 40000])
def test_ties_go_to_the_lowest_index(V):
    """Rows of one value, and of a few values: the cuts fall inside ties."""
    M = 12
    g = _gen(V)
    x = torch.randint(0, 3, (M, V), generator=g, device="cuda").float()
    x[:3] = 1.25
    x[3] = -0.0
    x[3, ::2] = 0.0
    u = (torch.arange(M, device="cuda") + 0.37) / M
    for k, p in ((2, 2.0), (V // 2 + 1, 2.0), (0, 0.3141), (0, 0.777), (V // 3 + 1, 0.5123)):
        kk, pp = _vec(k, M, torch.int32), _vec(p, M)
        _check(x, binding.spec_sample(x, u, None, kk, pp), u, None, kk, pp, most_undecided=0.5)
    assert binding.spec_sample(x, u, _vec(0.0, M))[0].tolist() == x.cpu().numpy().argmax(1).tolist()


def test_masks_infinities_and_nan():
    V = 3001
    inf, low = float("inf"), torch.finfo(torch.float32).min
    g = _gen(1)
    x = torch.randn((12, V), generator=g, device="cuda")
    x[0] = -inf                                    # nothing left
    x[1] = -inf
    x[1, 1234] = -50.0                             # one token left
    x[2, 17] = float("nan")
    x[3] = low                                     # every token at the type's lowest value: equal mass
    x[4] = low
    x[4, 2999] = 3.0
    x[5, 100::700] = inf                           # equal mass among the infinities
    x[6, torch.rand(V, generator=g, device="cuda") < 0.99] = -inf
    x[7] = -inf
    x[7, :2] = low
    x[8, 5] = -float("nan")
    x[9] = torch.finfo(torch.float32).max          # the largest finite value, and the lowest beside it
    x[9, ::2] = low
    u = torch.rand(12, generator=g, device="cuda")
    for T, k, p, q in ((1.0, 0, 2.0, 0.0), (0.7, 5, 0.9, 0.0), (1.0, 2000, 2.0, 0.3), (2.0, 0, 0.5, 1.5), (0.0, 3, 0.5, 0.5)):
        s = (_vec(T, 12), _vec(k, 12, torch.int32), _vec(p, 12), _vec(q, 12))
        got = binding.spec_sample(x, u, *s)
        _check(x, got, u, *s, most_undecided=0.5)
        assert got[0][0] == -1 and got[1][0] == 0 and got[0][2] == -1 and got[0][8] == -1
        assert got[0][1] == 1234 and got[1][1] == 1 and got[0][4] == 2999


def test_settings_out_of_range():
    nan, inf = float("nan"), float("inf")
    x = torch.randn((8, 100), generator=_gen(2), device="cuda")
    T = torch.tensor([-1.0, nan, inf, 1.0, 1.0, 1.0, 1.0, 1e-6], device="cuda")
    u = torch.tensor([0.5, 0.5, 0.5, -1.0, nan, 1.0, 7.0, 0.9], device="cuda")
    p = torch.tensor([0.5, 0.5, 0.5, nan, -1.0, 2.0, 0.5, 0.5], device="cuda")
    tok, prob = binding.spec_sample(x, u, T, None, p)
    assert tok[:3].tolist() == [-1, -1, -1] and prob[:3].tolist() == [0, 0, 0]
    assert tok[3] == 0                             # u below 0: the first token
    best = x.argmax(1)
    assert tok[4] == best[4] and prob[4] == 1      # p below 0: the most likely token
    assert tok[5] == 99                            # u >= 1: the last token kept
    assert tok[7] == best[7] and prob[7] == 1      # a temperature below 1e-5 is greedy
    _check(x[6:7], (tok[6:7], prob[6:7]), torch.tensor([1.0]), T[6:7], None, p[6:7])


@pytest.mark.parametrize("V", [100, 262144])
def test_min_p_out_of_range_is_off(V):
    x = torch.randn((4, V), generator=_gen(3), device="cuda") * 2.5
    q = torch.tensor([float("nan"), -0.5, 0.0, -float("inf")], device="cuda")
    u = torch.rand(4, generator=_gen(4), device="cuda")
    plain, got = binding.spec_sample(x, u), binding.spec_sample(x, u, None, None, None, q)
    _check(x, got, u)
    assert torch.equal(plain[0], got[0])
    one = binding.spec_sample(x, u, None, None, None, torch.full((4,), 7.0, device="cuda"))
    assert torch.equal(one[0].long(), x.argmax(1)) and one[1].tolist() == [1.0] * 4   # at most 1



def test_a_row_depends_on_nothing_else():
    """Bit-identical tokens and probabilities alone, in a batch, at another
    alignment, and from run to run."""
    M, V = 33, 40001
    g = _gen(9)
    x = torch.randn((M, V), generator=g, device="cuda") * 2
    u = torch.rand(M, generator=g, device="cuda")
    T, k, p, q = _vec(0.9, M), _vec(3000, M, torch.int32), _vec(0.93, M), _vec(0.001, M)
    tok, prob = binding.spec_sample(x, u, T, k, p, q)
    again = binding.spec_sample(x, u, T, k, p, q)
    assert torch.equal(tok, again[0]) and torch.equal(prob, again[1])
    for i in (0, 7, 32):
        one = binding.spec_sample(x[i:i + 1].clone(), u[i:i + 1], T[:1], k[:1], p[:1], q[:1])
        assert one[0][0] == tok[i] and one[1][0] == prob[i]


def test_frequencies():
    """Inverse CDF over equal steps of u: each token's share is within one step
    of its probability."""
    n, V = 4096, 50
    x = (torch.randn(V, generator=_gen(5), device="cuda") * 1.5).expand(n, V)
    u = (torch.arange(n, device="cuda").float() + 0.5) / n
    tok, _ = binding.spec_sample(x.contiguous(), u, _vec(0.8, n))
    share = torch.bincount(tok.long(), minlength=V).double() / n
    want = torch.softmax(x[0].double() / np.float32(0.8), 0)
    assert (share - want).abs().max() <= 1.0 / n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,k,V", [(1, 0, 100), (1, 3, 262144), (3, 6, 32003), (8, 4, 4096), (300, 1, 64)])
def test_accept_matches_reference(dtype, B, k, V):
    M = B * (k + 1)
    g = _gen(B * 100 + k)
    x = (torch.randn((M, V), generator=g, device="cuda") * 4).to(dtype)
    u = torch.rand(M, generator=g, device="cuda")
    T, p = _vec(0.5, M), _vec(0.9, M)
    best = x.float().argmax(1).view(B, k + 1)[:, :k]
    d = torch.where(torch.rand((B, k), generator=g, device="cuda") < 0.8, best, best * 0 + V // 2).int().contiguous()
    out, ne, pr = (t.cpu().numpy() for t in binding.spec_accept_sampled(x, d, u, T, None, p))
    n = lambda t: t.cpu().numpy()
    rt, rp, dec = ref.rows(x.float().cpu().numpy(), n(u), n(T), None, n(p), None)
    ro, rn, rpr = ref.accept(rt.reshape(B, -1), rp.reshape(B, -1), n(d))
    ok = dec.reshape(B, -1).all(1)
    assert ok.mean() > 0.9
    assert np.array_equal(out[ok], ro[ok]) and np.array_equal(ne[ok], rn[ok])
    assert np.all(np.abs(pr - rpr)[ok] <= PTOL * rpr[ok])


def test_accept_ends_before_a_row_without_a_distribution():
    V = 500
    x = torch.randn((8, V), generator=_gen(4), device="cuda")
    x[1] = float("nan")            # sequence 0, row 1
    x[4] = -float("inf")           # sequence 1, row 0
    T = _vec(0.0, 8)
    d = x.nan_to_num(-1e9).argmax(1).view(2, 4)[:, :3].int().contiguous()
    out, ne, pr = binding.spec_accept_sampled(x, d, _vec(0.5, 8), T)
    assert ne.tolist() == [1, 0] and out[0].tolist() == [int(d[0, 0]), -1, -1, -1] and out[1].tolist() == [-1] * 4
    assert pr[0].tolist() == [1, 0, 0, 0] and pr[1].tolist() == [0] * 4


def test_other_stream_and_captured_graph():
    M, V = 9, 20000
    g = _gen(6)
    x = torch.randn((M, V), generator=g, device="cuda") * 2
    u = torch.rand(M, generator=g, device="cuda")
    T, p = _vec(0.8, M), _vec(0.9, M)
    want = binding.spec_sample(x, u, T, None, p)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = binding.spec_sample(x, u, T, None, p, stream=st)
    st.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    graph = torch.cuda.CUDAGraph()
    d = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    with torch.cuda.graph(graph):
        t1 = binding.spec_sample(x, u, T, None, p)
        t2 = binding.spec_accept_sampled(x, d, u, T, None, p)
    for seed in (1, 2):
        x.copy_(torch.randn((M, V), generator=_gen(seed), device="cuda") * 2)
        graph.replay()
        torch.cuda.synchronize()
        now = binding.spec_sample(x, u, T, None, p)
        assert torch.equal(now[0], t1[0]) and torch.equal(now[1], t1[1])
        assert all(torch.equal(a, b) for a, b in zip(t2, binding.spec_accept_sampled(x, d, u, T, None, p)))


def test_two_calls_at_once():
    """Calls on two streams, large enough to overlap, leave what each leaves alone."""
    g = _gen(11)
    x = [torch.randn((24, 100003), generator=g, device="cuda") * 2.5 for _ in range(2)]
    u = [torch.rand(24, generator=g, device="cuda") for _ in range(2)]
    p = _vec(0.9, 24)
    for top_p in (None, p):
        alone = [binding.spec_sample(x[i], u[i], None, None, top_p) for i in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = [[binding.spec_sample(x[i], u[i], None, None, top_p, stream=streams[i]) for i in range(2)]
               for _ in range(8)]
        torch.cuda.synchronize()
        for both in got:
            for i in range(2):
                assert torch.equal(both[i][0], alone[i][0]) and torch.equal(both[i][1], alone[i][1])


def test_refusals():
    x, u = torch.zeros((2, 8), device="cuda"), torch.zeros(2, device="cuda")
    bad = [
        lambda: binding.spec_sample(x.double(), u),
        lambda: binding.spec_sample(x, u.double()),
        lambda: binding.spec_sample(x, u[:1]),
        lambda: binding.spec_sample(x, u.cpu()),
        lambda: binding.spec_sample(x, None),
        lambda: binding.spec_sample(x.t(), torch.zeros(8, device="cuda")),
        lambda: binding.spec_sample(x, u, top_k=u),
        lambda: binding.spec_sample(x[:0], u[:0]),
        lambda: binding.spec_sample(x[0].expand(2, 8), u),
        lambda: binding.spec_accept_sampled(x, torch.zeros((1, 2), dtype=torch.int32, device="cuda"), u),
        lambda: binding.spec_accept_sampled(x, torch.zeros((1, 1), dtype=torch.int64, device="cuda"), u),
    ]
    for f in bad:
        with pytest.raises(binding.SpecError):
            f()


# ---- the sampled verify of a context ----------------------------------------------------------

W = configs.WORKLOADS["tiny_f32_b1_k3"]


def _engine(dt, B):
    tshape = W.target if dt == configs.F32 else dataclasses.replace(W.target, wdtype=dt, kvdtype=configs.BF16)
    dshape = W.drafter if dt == configs.F32 else dataclasses.replace(W.drafter, wdtype=dt)
    tw = synth.make_target(tshape, device="cuda")
    dw = synth.make_drafter(dshape, device="cuda")
    eng = binding.Engine(tw, dw, n_slots=B, B_max=B, rows_max=64, max_ctx=512, shuffle_pages=True)
    ids = eng.seq_ids(list(range(B)))
    prompt = synth.make_tokens(40 * B, tshape.V).view(B, 40).cuda()
    eng.spec_prefill(ids, eng._in("prompt", prompt))
    eng.sync()
    return eng, ids, tshape


@pytest.mark.parametrize("dt", [configs.F32, configs.BF16])
@pytest.mark.parametrize("B,k", [(1, 0), (1, 3), (3, 4)])
def test_verify_sampled(dt, B, k):
    """The pass emits what spec_accept_sampled gives for the pass's own logits,
    commits that many rows, and decoding goes on from there: a second pass from
    the new state agrees with plain sampled decoding of the same state."""
    eng, ids, t = _engine(dt, B)
    M = B * (k + 1)
    g = _gen(k)
    u = torch.rand(M, generator=g, device="cuda")
    T, p = _vec(0.2, M), _vec(0.95, M)
    drafts = eng.spec_draft(ids, B, k) if k else torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    # the first draft is the likeliest token, so that some drafts are accepted
    logits = torch.empty((M, t.V), device="cuda")
    saved = [x.clone() for x in (eng.seq_len, eng.pending, eng.hid, eng.stats)]
    if k:
        eng.spec_verify_sampled(ids, drafts, u, _vec(0.0, M), None, None, None, logits)
        eng.sync()
        for dst, src in zip((eng.seq_len, eng.pending, eng.hid, eng.stats), saved):
            dst.copy_(src)
        drafts = drafts.clone()
        drafts[:, 0] = logits.view(B, k + 1, -1)[:, 0].argmax(-1)
    out, ne, pr = (x.clone() for x in eng.spec_verify_sampled(ids, drafts, u, T, None, p, None, logits))
    eng.sync()
    want = binding.spec_accept_sampled(logits, drafts.contiguous(), u, T, None, p)
    assert torch.equal(out, want[0]) and torch.equal(ne, want[1]) and torch.equal(pr, want[2])
    assert torch.equal(eng.seq_len, saved[0] + ne)
    last = out.gather(1, (ne - 1).long()[:, None])[:, 0]
    assert torch.equal(eng.pending, last)
    st = eng.spec_stats(0)
    assert st.passes == 1 and st.drafted == k and st.accepted == int(ne[0]) - 1 and st.emitted == int(ne[0])
    # greedy settings reproduce spec_verify from the same state
    state = [x.clone() for x in (eng.seq_len, eng.pending, eng.hid, eng.stats)]
    o1, n1 = (x.clone() for x in eng.spec_verify(ids, drafts))
    eng.sync()
    end = [x.clone() for x in (eng.seq_len, eng.pending, eng.hid)]
    for dst, src in zip((eng.seq_len, eng.pending, eng.hid, eng.stats), state):
        dst.copy_(src)
    o2, n2, _ = eng.spec_verify_sampled(ids, drafts, u, _vec(0.0, M))
    eng.sync()
    assert torch.equal(o1, o2) and torch.equal(n1, n2)
    for a, b in zip(end, (eng.seq_len, eng.pending, eng.hid)):
        assert torch.equal(a, b)
    eng.close()


def test_speculative_sampling_equals_plain_sampling():
    """With one number per position, speculating emits the tokens that sampling
    one token a pass emits."""
    n, k = 12, 3
    u = torch.rand(64, generator=_gen(11), device="cuda")
    eng, ids, t = _engine(configs.F32, 1)
    plain = []
    for i in range(n):
        out, ne, _ = eng.spec_verify_sampled(ids, torch.zeros((1, 0), dtype=torch.int32, device="cuda"), u[i:i + 1],
                                             _vec(0.3, 1), None, _vec(0.9, 1))
        plain.append(int(out[0, 0]))
    eng.sync()
    eng.close()
    eng, ids, t = _engine(configs.F32, 1)
    got, accepted = [], 0
    while len(got) < n:
        at = len(got)
        right = [plain[min(at + j, n - 1)] for j in range(k)]
        right[2] = (right[2] + (at % 2)) % t.V       # sometimes a wrong draft
        d = torch.tensor([right], dtype=torch.int32, device="cuda")
        out, ne, _ = eng.spec_verify_sampled(ids, d, u[at:at + k + 1], _vec(0.3, k + 1), None, _vec(0.9, k + 1))
        got += out[0, :int(ne[0])].tolist()
        accepted += int(ne[0]) - 1
    eng.sync()
    eng.close()
    assert got[:n] == plain and accepted >= 4


def test_verify_sampled_commits_nothing_without_a_distribution():
    eng, ids, t = _engine(configs.F32, 2)
    saved = [x.clone() for x in (eng.seq_len, eng.pending, eng.hid, eng.stats)]
    d = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    T = torch.tensor([1.0, 1.0, -1.0, 1.0], device="cuda")   # sequence 1, row 0
    eng.spec_verify_sampled(ids, d, torch.full((4,), 0.5, device="cuda"), T)
    with pytest.raises(binding.SpecError) as e:
        eng.sync()
    assert e.value.code == binding.SPEC_EINVAL
    for a, b in zip(saved, (eng.seq_len, eng.pending, eng.hid, eng.stats)):
        assert torch.equal(a, b)
    out, ne, _ = eng.spec_verify_sampled(ids, d, torch.full((4,), 0.5, device="cuda"), torch.ones(4, device="cuda"))
    eng.sync()
    assert torch.equal(eng.seq_len, saved[0] + ne)
    eng.close()
