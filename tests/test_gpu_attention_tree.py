"""spec_attention_tree against the 64-bit reference (tests/branch_ref.py).

Tolerances, per output o = sum p v / sum p with A = sum p |v| / sum p and S the
largest sum |q k| / sqrt(hd) of the row:
 - a score is off by at most (hd + 8) 2^-23 S (hd products and sums, of which a
   tensor core may cut instead of round, and the scaling), its exponential by 2^-21
   more (the hardware's exponential and its argument's rounding up to scores of 16);
   that moves a weight, and twice that an output, relative to A;
 - sums over n keys: n 2^-23 A;
 - float rows on a bf16 cache: probabilities to 2^-16 (two bf16 planes): 2 * 2^-16 A;
 - bf16 rows: probabilities rounded to bf16 (2^-8) in both sums, 2 * 2^-8 A, and
   the result's rounding 2^-8 |o|."""
import ctypes as C

import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding
from tests import branch_ref as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, nq, nkv, hd, lens, R, q="f32", kv="bf16", rows=None, parents="tree", layers=2, seed=0, spare=3,
                 scale=1.5, garbage=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        B = len(lens)
        self.B, self.R, self.nq, self.hd = B, R, nq, hd
        rows = [R] * B if rows is None else rows
        need = [-(-(n + r) // 64) for n, r in zip(lens, rows)]
        P, pages = max(max(need), 1) + 1, sum(need) + spare
        pool = torch.randn((layers, pages, 2, nkv, 64, hd), generator=g, device="cuda").to(DT[kv])
        ids = rng.permutation(pages)
        slots = rng.permutation(B + 1)[:B]          # a slot that no sequence of the call has
        table, at = np.full((B + 1, P), -1, np.int32), 0
        for b, n in enumerate(need):
            table[slots[b], :n] = ids[at:at + n]
            at += n
        if garbage:                                  # what lies behind a sequence's last key, and pages of nobody
            for b in range(B):
                n = lens[b] + rows[b]
                if n % 64:
                    pool[:, int(table[slots[b], n // 64]), :, :, n % 64:] = float("nan")
            pool[:, torch.from_numpy(ids[at:].copy()).cuda()] = float("inf")
        seq_len = np.zeros(B + 1, np.int32)
        seq_len[slots] = lens
        self.parents = None if parents is None else ref.random_parents(rng, B, R) if parents == "tree" else np.array(parents, np.int32)
        self.rows = np.array(rows, np.int32)
        cu = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
        self.pool, self.table, self.seq_ids, self.seq_len = pool, cu(table), cu(slots), cu(seq_len)
        self.q = (torch.randn((B * R, nq * hd), generator=g, device="cuda") * scale).to(DT[q])
        self.cache = binding.Cache(pool, self.table)
        self.layer = layers - 1
        self.alive = []

    def call(self, **kw):
        par = None if self.parents is None else torch.from_numpy(self.parents).cuda()
        kw.setdefault("n_rows", torch.from_numpy(self.rows).cuda())
        self.alive.append((par, kw["n_rows"]))     # (a call on another stream may still read them)
        return binding.spec_attention_tree(self.cache, self.layer, self.seq_ids, self.seq_len, self.q, par, **kw)

    def want(self):
        return ref.attention(_np(self.pool[self.layer]), self.table.cpu().numpy(), self.seq_ids.cpu().numpy(),
                             self.seq_len.cpu().numpy(), _np(self.q), self.nq, self.parents, self.rows)

    def tol(self, o, A, S, n):
        t = A * (2 * ((self.hd + 8) * 2.0 ** -23 * S + 2.0 ** -21) + (n + 16) * 2.0 ** -23)
        if self.q.dtype is torch.bfloat16:
            return t + A * 2 * 2.0 ** -8 + 2.0 ** -8 * np.abs(o)
        return t + (A * 2 * 2.0 ** -16 if self.pool.dtype is torch.bfloat16 else 0)

    def check(self, out=None):
        out = self.call(sync=True) if out is None else out
        o, A, S, n = self.want()
        got, used = _np(out), ~np.isnan(o)
        assert np.isfinite(got[used]).all()
        err, tol = np.abs(got - o)[used], self.tol(o, A, S, n)[used]
        assert (err <= tol).all(), "worst %.3g of its tolerance" % (err / tol).max()
        return out


KINDS = [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")]
HEADS = [(12, 4, 128), (20, 4, 128), (48, 8, 128), (4, 4, 64), (16, 8, 128)]


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n,R", [(0, 1), (1, 1), (62, 1), (63, 1), (64, 1), (0, 2), (60, 5), (63, 2), (127, 7), (128, 16), (500, 33), (1000, 64)])
def test_one_sequence(q, kv, heads, n, R):
    Case(*heads, [n], R, q, kv, seed=n + R).check()


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("heads", [(6, 2, 96), (5, 1, 40), (3, 3, 8), (8, 1, 256), (32, 4, 64), (71, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("n,R", [(3, 1), (130, 9), (300, 40)])
def test_other_heads(q, kv, heads, n, R):
    Case(*heads, [n], R, q, kv, seed=n).check()


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("heads", [(12, 4, 128), (48, 8, 128), (4, 4, 64)])
@pytest.mark.parametrize("R,rows", [(24, [24, 1, 0, 13, 7, 24]), (64, [64, 22, 43, 1, 0, 64]), (3, [3, 3, 1, 2, 0, 3])])
def test_ragged_batch(q, kv, heads, R, rows):
    c = Case(*heads, [0, 700, 65, 1283, 64, 40], R, q, kv, rows=rows, seed=R)
    out = torch.full_like(c.q, 7.0)
    assert c.call(out=out, sync=True) is out
    c.check(out)
    free = torch.from_numpy(np.arange(R)[None] >= c.rows[:, None]).reshape(-1).cuda()
    assert (out[free] == 7.0).all()                         # rows that are not in use stay as they are
    made = c.call()
    assert (made[free] == 0).all() and torch.equal(made[~free], out[~free])


@pytest.mark.parametrize("q,kv", KINDS[:3])
def test_long_context_and_many_sequences(q, kv):
    hd = 128 if kv == "bf16" else 64
    Case(4, 2, hd, [20000], 5, q, kv, layers=1, seed=1).check()
    Case(4, 2, hd, [(i * 37) % 211 for i in range(70)], 3, q, kv, layers=1, seed=2).check()


@pytest.mark.parametrize("q,kv", KINDS)
def test_chain_and_star(q, kv):
    heads = (12, 4, 128)
    chain = Case(*heads, [333, 64], 9, q, kv, parents=None)
    star = [[-1] + [0] * 8] * 2
    forest = [[-1] * 9, [-1, -1, 0, 1, 1, 2, -1, 6, 7]]
    a = chain.check()
    chain.parents = np.array([[r - 1 for r in range(9)]] * 2, np.int32)
    assert torch.equal(a, chain.call())
    Case(*heads, [333, 64], 9, q, kv, parents=star).check()
    Case(*heads, [333, 64], 9, q, kv, parents=forest).check()


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("n", [0, 100, 127])
def test_values_of_unseen_rows_do_not_count(q, kv, n):
    """Infinities and NaN in a row's key and value reach only the rows that see it."""
    c = Case(12, 4, 128, [n], 6, q, kv, parents=[[-1, 0, 0, 1, 2, 0]])
    want = c.check()
    for plane in (0, 1):
        for bad in (float("inf"), float("-inf"), float("nan")):
            pool = c.pool.clone()
            at = n + 2
            pool[:, int(c.table[int(c.seq_ids[0]), at // 64]), plane, :, at % 64, 3::5] = bad
            c.cache = binding.Cache(pool, c.table)
            got = c.call(sync=True)
            clean = [0, 1, 3, 5]
            assert torch.isfinite(got[clean]).all()
            o, A, S, k = c.want()
            assert (np.abs(_np(got) - o)[clean] <= c.tol(o, A, S, k)[clean]).all()
            touched = got[[2, 4]].view(2, 12, 128)
            if plane == 0:
                assert torch.isnan(touched).any(-1).all() or bad == float("-inf") or bad == float("inf")
            else:
                assert not torch.isfinite(touched[..., 3::5]).any()
                assert torch.isfinite(touched[..., 0::5]).all()


@pytest.mark.parametrize("q,kv", KINDS)
def test_strided_rows(q, kv):
    c = Case(12, 4, 128, [77, 300], 5, q, kv)
    want = c.call()
    wide = torch.full((10, 12 * 128 + 24), float("nan"), dtype=c.q.dtype, device="cuda")
    wide[:, 8:8 + 12 * 128] = c.q
    c.q = wide[:, 8:8 + 12 * 128]
    out = torch.full((10, 12 * 128 + 40), 3.0, dtype=c.q.dtype, device="cuda")
    got = c.call(out=out[:, 16:16 + 12 * 128])
    assert torch.equal(got, want) and (out[:, :16] == 3).all() and (out[:, 16 + 12 * 128:] == 3).all()


@pytest.mark.parametrize("q,kv", KINDS)
def test_large_scores(q, kv):
    """Peaked rows: one key takes nearly all of the weight, and the maximum moves often."""
    c = Case(12, 4, 128, [900], 8, q, kv, scale=12.0)
    c.check()
    c = Case(4, 4, 64, [900], 8, q, kv, scale=0.0)          # all scores equal
    c.check()


@pytest.mark.parametrize("q,kv", KINDS)
def test_recorded_errors(q, kv):
    c = Case(12, 4, 128, [100, 200, 300], 4, q, kv)
    want = c.check()
    mark = lambda: torch.full_like(want, 5.0)
    rows = torch.from_numpy(c.rows).cuda()

    def run(out, **kw):
        ws = torch.full((1 << 26,), 0xAB, dtype=torch.uint8, device="cuda")
        c.call(out=out, workspace=ws, **kw)
        return int(ws[:4].view(torch.int32))

    out = mark()
    assert run(out) == 0 and torch.equal(out, want)
    for bad in (-1, 5, 1 << 30, -(1 << 31)):               # a row count: that sequence stays as it was
        r = rows.clone()
        r[1] = bad
        out = mark()
        assert run(out, n_rows=r) == 2
        assert (out[4:8] == 5).all() and torch.equal(out[:4], want[:4]) and torch.equal(out[8:], want[8:])
    keep = c.seq_ids
    for bad in (-1, 4, 1 << 30):
        c.seq_ids = keep.clone()
        c.seq_ids[2] = bad
        out = mark()
        assert run(out) == 2 and (out[8:] == 5).all() and torch.equal(out[:8], want[:8])
    c.seq_ids = keep
    lens = c.seq_len
    for bad in (-1, c.cache.max_pages * 64 - 3, (1 << 31) - 1):
        c.seq_len = lens.clone()
        c.seq_len[int(keep[0])] = bad
        out = mark()
        assert run(out) == 2 and (out[:4] == 5).all() and torch.equal(out[4:], want[4:])
    c.seq_len = lens
    for bad in (4, 3, -2, 1 << 30):                         # a parent that is no earlier row counts as none
        c.parents[1, 3] = -1
        fixed = c.call()
        c.parents[1, 3] = bad
        out = mark()
        assert run(out) == 2 and torch.equal(out, fixed)
    c.parents[1, 3] = -1
    fixed = c.call()
    table = c.table.clone()
    for bad in (-1, c.cache.n_pages, 1 << 30):
        c.table.copy_(table)
        c.table[int(keep[1]), 1] = bad
        out = mark()
        assert run(out) == 2 and torch.equal(out[:4], fixed[:4]) and torch.equal(out[8:], fixed[8:])
        with pytest.raises(binding.SpecError) as e:
            c.call(sync=True)
        assert e.value.code == binding.SPEC_ECAPACITY


@pytest.mark.parametrize("q,kv", KINDS)
def test_graph_streams_and_two_at_once(q, kv):
    c = Case(48, 8, 128, [700, 90, 1500], 12, q, kv)
    d = Case(48, 8, 128, [10, 4000], 5, q, kv, seed=9)
    a, b = c.call(), d.call()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(c.call(stream=s1), d.call(stream=s2)) for _ in range(4)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, a) and torch.equal(y, b)
    rows, par = torch.from_numpy(c.rows).cuda(), torch.from_numpy(c.parents).cuda()
    out = torch.zeros_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.spec_attention_tree(c.cache, c.layer, c.seq_ids, c.seq_len, c.q, par, n_rows=rows, out=out)
    for shift in (0, 1, 64):                                # other lengths on replay
        c.seq_len -= shift
        want = c.call()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes (and elements), pages from its end."""
    nkv, hd = 8, 128
    page = 2 * nkv * 64 * hd
    n = (1 << 32) // page + 9
    pool = torch.empty((1, n, 2, nkv, 64, hd), dtype=torch.bfloat16, device="cuda")
    c = Case(16, nkv, hd, [150, 100], 6, "bf16", "bf16", layers=1, garbage=False)
    k = c.pool.shape[1]
    pool[:, n - k:] = c.pool
    table = torch.where(c.table >= 0, c.table + (n - k), -1).to(torch.int32)
    want = c.check()
    c.cache = binding.Cache(pool, table)
    assert torch.equal(c.call(sync=True), want)


def test_refusals():
    c = Case(12, 4, 128, [100, 200], 4)
    run = binding.spec_attention_tree
    a = (c.cache, 0, c.seq_ids, c.seq_len)
    bad = [
        lambda: run(*a, c.q.half()), lambda: run(*a, c.q.cpu()), lambda: run(*a, c.q[:7]), lambda: run(*a, c.q[:, :-128]),
        lambda: run(*a, c.q.t().contiguous().t()), lambda: run(*a, c.q[:0]), lambda: run(c.cache, 2, *a[2:], c.q),
        lambda: run(c.cache, -1, *a[2:], c.q), lambda: run(*a, c.q, torch.zeros((2, 3), dtype=torch.int32, device="cuda")),
        lambda: run(*a, c.q, torch.zeros((2, 4), device="cuda")), lambda: run(*a, c.q, n_rows=c.seq_len),
        lambda: run(*a, c.q, out=torch.empty_like(c.q, dtype=torch.bfloat16)), lambda: run(*a, c.q, out=c.q[:4]),
        lambda: run(c.cache, 0, c.seq_ids.long(), c.seq_len, c.q), lambda: run(c.cache, 0, c.seq_ids, c.seq_len[:2], c.q),
        lambda: run(*a, torch.zeros((8, 12 * 128 + 4), device="cuda")[:, 2:-2]),
        lambda: run(*a, torch.zeros((8, 12 * 128 + 4), device="cuda")[:, :-4]),
        lambda: run(*a, c.q, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        lambda: run(*a, torch.zeros((130, 12 * 128), device="cuda")),
        lambda: binding.Cache(c.pool[0], c.table), lambda: binding.Cache(c.pool.half(), c.table),
        lambda: binding.Cache(c.pool, c.table.long()), lambda: binding.Cache(c.pool, c.table.cpu()),
        lambda: binding.Cache(c.pool[:, :, :, ::2], c.table), lambda: binding.Cache(c.pool, c.table, c.seq_len),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(binding.SpecError):
            f()
            pytest.fail("call %d was not refused" % i)
    c.check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("grow", [0.0, 3.0])
def test_float_rows_over_many_blocks(hd, grow):
    """Sums of float rows leave the tensor cores every 8 blocks of 64 keys, whatever the length: a run cuts at most
    3 * 8 * 64 / 16 = 96 times (2^-23 each), and runs, pieces, streams and weights take some 100 more additions.
    Scores that grow along the sequence raise the maximum in every run."""
    c = Case(4, 2, hd, [130001], 3, "f32", "bf16", layers=1, seed=hd)
    slot, n = int(c.seq_ids[0]), -(-130004 // 64)
    pages = c.table[slot, :n].long()
    c.pool[0, pages, 0] *= (1 + grow * torch.arange(n, device="cuda") / n).to(torch.bfloat16)[:, None, None, None]
    out = c.call(sync=True)
    o, A, S, _ = c.want()
    tol = A * (2 * ((hd + 8) * 2.0 ** -23 * S + 2.0 ** -21) + (96 + 100) * 2.0 ** -23)
    err = np.abs(_np(out) - o)
    assert (err <= tol).all(), (err / tol).max()
    c.pool[0, pages[-1], 1, :, 130001 % 64 + 1] = float("inf")     # the second row's values: seen by it and its children
    out = c.call(sync=True)
    assert torch.isinf(out[1]).all() and torch.isfinite(out[0]).all()


@pytest.mark.parametrize("q,kv", KINDS)
def test_a_slot_named_twice(q, kv):
    """Two trees over one slot's cache, as many rows each: the calls only read it."""
    c = Case(12, 4, 128, [333], 9, q, kv, seed=21)
    ids = c.seq_ids.repeat(2)
    par = torch.from_numpy(np.concatenate([c.parents, np.arange(-1, 8, dtype=np.int32)[None]])).cuda()
    out = binding.spec_attention_tree(c.cache, c.layer, ids, c.seq_len, c.q.repeat(2, 1), par, sync=True)
    c.check(out[:9])
    c.parents = par[1:].cpu().numpy()
    c.check(out[9:])


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("back", [0, 3, 200, 251])
def test_lengths_next_to_the_32nd_bit(q, kv, back):
    """A table wide enough for 2^31 positions: a length whose last blocks pass 2^31 - 256 is out of range, and the
    sequence beside it is as it is in a table of its own width."""
    R, nq, hd = 4, 2, 64
    c = Case(nq, 1, hd, [100], R, q, kv, layers=1, seed=back)
    wide = torch.full((2, (1 << 25) + 4), -1, dtype=torch.int32, device="cuda")
    wide[0, :c.table.shape[1]] = c.table[c.seq_ids[0]]
    wide[1] = 0
    lens = torch.tensor([100, (1 << 31) - 1 - back], dtype=torch.int64).to(torch.int32).cuda()
    cache, ids = binding.Cache(c.pool, wide), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    par = torch.from_numpy(np.concatenate([c.parents, c.parents])).cuda()
    out = torch.full((2 * R, nq * hd), 5.0, dtype=c.q.dtype, device="cuda")
    with pytest.raises(binding.SpecError) as e:
        binding.spec_attention_tree(cache, 0, ids, lens, c.q.repeat(2, 1), par, out=out, sync=True)
    assert e.value.code == binding.SPEC_ECAPACITY and (out[:R] == 5).all()
    c.check(out[R:])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("seed", range(3))
def test_error_of_float_rows(hd, seed):
    """All 24 bits of float rows and their weights, over one block of keys and over runs of many (160 sequences of one
    slot, so that a CTA has some 70 blocks to itself): the limits are what a part, the order or the runs would cost."""
    from tests import float_rows_ref as fr
    c = Case(8, 2, hd, [60], 4, "f32", "bf16", layers=1, seed=seed)
    assert fr.off(_np(c.call(sync=True)), c.want()[0]) <= fr.LIMITS[64, hd]
    c = Case(4, 1, hd, [4199], 1, "f32", "bf16", layers=1, seed=seed)
    q = torch.randn((160, 4 * hd), generator=torch.Generator(device="cuda").manual_seed(seed + 1000), device="cuda") * 1.5
    out = binding.spec_attention_tree(c.cache, 0, c.seq_ids.repeat(160), c.seq_len, q, sync=True)
    pages = c.table[int(c.seq_ids[0]), : -(-4200 // 64)].long()
    k, v = (_np(c.pool[0, pages, i, 0]).reshape(-1, hd)[:4200] for i in (0, 1))
    assert fr.off(_np(out).reshape(-1, hd), fr.exact(_np(q).reshape(-1, hd), k, v)) <= fr.LIMITS[4200, hd]


@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("lens,R", [([100, 30], 5), ([60], 1), ([700, 1500, 40], 24)])
def test_a_wait_that_runs_out(q, lens, R):
    """Every CTA waits for weights that are never handed over: the call gives up after about a second, records the
    timeout (in tables without cuts and with them) and returns, and the next call in the same workspace is right."""
    c = Case(20, 4, 128, lens, R, q, "bf16")
    ws = torch.full((1 << 26,), 0xAB, dtype=torch.uint8, device="cuda")
    wait = binding.lib().spec_test_attention_tree_wait
    wait.argtypes, wait.restype = [C.c_int32], None
    want = c.call(workspace=ws, sync=True)
    for _ in range(2):
        wait(1)
        try:
            with pytest.raises(binding.SpecError) as e:
                c.call(workspace=ws, sync=True)
        finally:
            wait(0)
        assert e.value.code == binding.SPEC_ETIMEOUT and int(ws[:4].view(torch.int32)) == 4
        assert torch.equal(c.call(workspace=ws, sync=True), want)
