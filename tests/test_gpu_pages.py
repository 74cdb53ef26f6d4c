"""Pages of the cache (spec_pages_*, spec_rows_keep) against the reference
(tests/branch_ref.py): tables, counts, lengths and the bytes of the pool are equal."""
import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding
from tests import branch_ref as ref

pytestmark = pytest.mark.gpu


def cu(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


class State:
    """A pool and its tables on the GPU, and the reference's beside them."""

    def __init__(self, slots, pages, P, L=2, nkv=2, hd=64, dtype=torch.bfloat16, d=24, seed=0):
        self.rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = torch.randn((L, pages, 2, nkv, 64, hd), generator=g, device="cuda").to(dtype)
        self.np_pool = self.pool.float().cpu().numpy()
        self.table, self.refs = np.full((slots, P), -1, np.int32), np.zeros(pages, np.int32)
        self.seq_len, self.pending = np.zeros(slots, np.int32), self.rng.integers(0, 100, slots).astype(np.int32)
        self.hid = self.rng.standard_normal((slots, d)).astype(np.float32)
        self.g = dict(table=cu(self.table), refs=cu(self.refs), seq_len=cu(self.seq_len), pending=cu(self.pending),
                      hid=torch.from_numpy(self.hid.copy()).cuda())
        self.cache = binding.Cache(self.pool, self.g["table"], self.g["refs"])

    def fill(self, slots, lens):
        """Lengths, and pages for them."""
        ref.reserve(self.table, self.refs, slots, lens)
        binding.spec_pages_reserve(self.cache, cu(slots), cu(lens), sync=True)
        self.seq_len[slots] = lens
        self.g["seq_len"].copy_(cu(self.seq_len))

    def fork(self, src, dst, **kw):
        binding.spec_pages_fork(self.cache, self.g["seq_len"], cu(src), cu(dst), pending=self.g["pending"],
                                hid=self.g["hid"], **kw)

    def ref_fork(self, src, dst):
        ref.fork(self.np_pool, self.table, self.refs, self.seq_len, src, dst)
        for a, d in zip(src, dst):
            self.pending[d], self.hid[d] = self.pending[a], self.hid[a]

    def same(self):
        for k in ("table", "refs", "seq_len", "pending", "hid"):
            assert np.array_equal(self.g[k].cpu().numpy(), getattr(self, k)), k
        assert np.array_equal(self.pool.float().cpu().numpy(), self.np_pool)
        assert (self.refs >= 0).all()
        count = np.bincount(self.table[self.table >= 0], minlength=len(self.refs))
        assert np.array_equal(count, self.refs)


SHAPES = [dict(), dict(dtype=torch.float32, hd=8, nkv=1), dict(hd=128, nkv=4, L=3), dict(hd=40, nkv=3), dict(L=1, nkv=1, hd=256)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(4))
def test_a_life_of_requests(shape, seed):
    """Slots filled, forked, cut, released and compacted at random, all compared after every call."""
    s = State(9, 70, 12, seed=seed, **shape)
    for step in range(14):
        kind = s.rng.integers(0, 5) if step > 1 else 0
        slots = s.rng.permutation(9)[: s.rng.integers(1, 4)]
        if kind == 0:
            lens = np.array([max(int(s.seq_len[x]), int(s.rng.integers(0, 400))) for x in slots])
            s.fill(slots, lens)
        elif kind == 1:
            src = s.rng.permutation(9)
            dst, src = src[:3], s.rng.choice(src[3:], 3)
            s.ref_fork(src, dst)
            s.fork(src, dst, sync=True)
        elif kind == 2:
            lens = np.array([int(s.rng.integers(0, s.seq_len[x] + 1)) for x in slots])
            ref.release(s.table, s.refs, slots, lens)
            binding.spec_pages_release(s.cache, cu(slots), cu(lens), sync=True)
            s.seq_len[slots] = lens
            s.g["seq_len"].copy_(cu(s.seq_len))
        elif kind == 3:
            ref.release(s.table, s.refs, slots)
            binding.spec_pages_release(s.cache, cu(slots), sync=True)
            s.seq_len[slots] = 0
            s.g["seq_len"].copy_(cu(s.seq_len))
        else:
            was = s.refs.copy()
            moved, n = ref.compact(s.np_pool, s.table, s.refs)
            got, live = binding.spec_pages_compact(s.cache)
            assert np.array_equal(got.cpu().numpy(), moved) and int(live) == n == (was > 0).sum()
        s.same()


@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 640, 767, 768])
@pytest.mark.parametrize("kids", [1, 7])
def test_fork_lengths(n, kids):
    s = State(9, 60, 12, seed=n)
    s.fill([3], [n])
    dst = [x for x in range(9) if x != 3][:kids]
    for _ in range(2):                       # the second time the slots give back what the first one gave them
        s.ref_fork([3] * kids, dst)
        s.fork([3] * kids, dst, sync=True)
        s.same()
    with pytest.raises(binding.SpecError):
        s.fork([], [])


def test_fork_without_state():
    s = State(4, 30, 8)
    s.fill([0], [100])
    pending, hid = s.g["pending"].clone(), s.g["hid"].clone()
    binding.spec_pages_fork(s.cache, s.g["seq_len"], cu([0]), cu([2]), sync=True)
    ref.fork(s.np_pool, s.table, s.refs, s.seq_len, [0], [2])
    s.same()
    assert torch.equal(s.g["pending"], pending) and torch.equal(s.g["hid"], hid)


def test_large_pools():
    """More pages than one round of the planning CTA takes, live ones at either end, many slots."""
    for live_end in (0, 1, 2):
        s = State(1024, 9001, 9, L=1, nkv=1, hd=8, d=8, seed=live_end)
        slots = s.rng.permutation(1024)
        lens = s.rng.integers(0, 9 * 64 + 1, 1024)
        s.fill(slots, lens)
        drop = slots[: 600] if live_end == 0 else slots[400:] if live_end == 1 else s.rng.permutation(1024)[:700]
        ref.release(s.table, s.refs, drop)
        binding.spec_pages_release(s.cache, cu(drop), sync=True)
        s.same()
        moved, n = ref.compact(s.np_pool, s.table, s.refs)
        got, live = binding.spec_pages_compact(s.cache)
        assert np.array_equal(got.cpu().numpy(), moved) and int(live) == n
        s.same()
        left = np.setdiff1d(np.arange(1024), drop)
        src = s.rng.choice(left, len(drop))
        s.seq_len[drop] = 0
        s.g["seq_len"].copy_(cu(s.seq_len))
        s.ref_fork(src, drop)
        s.fork(src, drop, sync=True)
        s.same()


def test_compact_into_other_tables():
    s = State(4, 40, 10)
    s.fill([0, 1, 2], [300, 200, 500])
    binding.spec_pages_release(s.cache, cu([0]), sync=True)
    ref.release(s.table, s.refs, [0])
    table, refs = s.g["table"].clone(), s.g["refs"].clone()
    t2, r2 = torch.full_like(table, 77), torch.full_like(refs, 77)
    pool = s.pool.clone()
    moved, n = binding.spec_pages_compact(s.cache, t2, r2)
    assert torch.equal(s.g["table"], table) and torch.equal(s.g["refs"], refs)
    want, k = ref.compact(s.np_pool, s.table, s.refs)
    assert np.array_equal(moved.cpu().numpy(), want) and int(n) == k
    assert np.array_equal(t2.cpu().numpy(), s.table) and np.array_equal(r2.cpu().numpy(), s.refs)
    for i in range(k):                       # what is in use reads the same under its new number
        a = int(np.flatnonzero(want == i)[0])
        assert torch.equal(s.pool[:, i], pool[:, a])
    # a page that no table names but the caller counts moves too
    refs[39] = 1
    moved, n = binding.spec_pages_compact(binding.Cache(s.pool, table, refs), t2, r2)
    assert int(n) == k + 1 and 0 <= int(moved[39]) <= k


def _unchanged(s, call, code=binding.SPEC_ECAPACITY):
    before = {k: v.clone() for k, v in s.g.items()}
    pool = s.pool.clone()
    with pytest.raises(binding.SpecError) as e:
        call()
    assert e.value.code == code
    for k, v in before.items():
        assert torch.equal(s.g[k], v), k
    assert torch.equal(s.pool, pool)
    s.same()


def test_calls_that_change_nothing():
    s = State(6, 12, 8)
    s.fill([0, 1], [300, 130])              # 5 + 3 pages, 4 are free
    B = binding
    for ids in ([2, 2], [-1, 2], [6, 2], [1 << 30, 0]):
        _unchanged(s, lambda: B.spec_pages_reserve(s.cache, cu(ids), cu([64, 64]), sync=True))
        _unchanged(s, lambda: B.spec_pages_release(s.cache, cu(ids), sync=True))
        _unchanged(s, lambda: s.fork([0, 0], ids, sync=True))
    for lens in ([64, -1], [64, 8 * 64 + 1], [64, (1 << 31) - 1], [200, 65]):   # (the last: 4 + 2 pages)
        _unchanged(s, lambda: B.spec_pages_reserve(s.cache, cu([2, 3]), cu(lens), sync=True))
    _unchanged(s, lambda: B.spec_pages_release(s.cache, cu([0, 1]), cu([64, -5]), sync=True))
    _unchanged(s, lambda: s.fork([0, 2], [2, 3], sync=True))                     # a source that is forked to
    _unchanged(s, lambda: s.fork([0], [0], sync=True))
    for src in (-1, 6, 1 << 30):
        _unchanged(s, lambda: s.fork([0, src], [2, 3], sync=True))
    for n in (-1, 8 * 64 + 1, 321):                                              # (321: a page more than the source has)
        s.seq_len[0] = n
        s.g["seq_len"].copy_(cu(s.seq_len))
        _unchanged(s, lambda: s.fork([0], [2], sync=True))
    s.seq_len[0] = 300
    s.g["seq_len"].copy_(cu(s.seq_len))
    s.fill([5], [190])                                                           # one page is free
    _unchanged(s, lambda: s.fork([0, 0], [2, 3], sync=True))
    s.ref_fork([0, 1], [5, 2])                                                   # (slot 5 gives three back first)
    s.fork([0, 1], [5, 2], sync=True)
    s.same()
    good = int(s.g["table"][0, 1])
    for bad in (12, 1 << 30):
        s.g["table"][0, 1] = bad
        s.table[0, 1] = bad
        for call in (lambda: B.spec_pages_release(s.cache, cu([0]), sync=True), lambda: s.fork([0], [3], sync=True)):
            with pytest.raises(binding.SpecError):
                call()
        assert np.array_equal(s.g["table"].cpu().numpy(), s.table) and np.array_equal(s.g["refs"].cpu().numpy(), s.refs)
    s.g["table"][0, 1] = good


@pytest.mark.parametrize("shape", SHAPES)
def test_rows_keep(shape):
    s = State(5, 40, 8, seed=3, **shape)
    for step in range(4):
        lens = s.rng.integers(0, 300, 5)
        s.fill(np.arange(5), lens + 64)
        s.seq_len[:] = lens
        s.g["seq_len"].copy_(cu(s.seq_len))
        n = [1, 7, 40, 64][step]
        slots = s.rng.permutation(5)[:3]
        rows = np.sort(np.array([s.rng.permutation(64)[:n] for _ in range(3)]), 1)
        k = s.rng.integers(0, n + 1, 3)
        k[0] = n
        ref.keep(s.np_pool, s.table, slots, s.seq_len, rows, k)
        binding.spec_rows_keep(s.cache, cu(slots), s.g["seq_len"], cu(rows), cu(k), sync=True)
        s.same()


def test_rows_keep_records():
    s = State(3, 20, 4)
    s.fill([0, 1, 2], [100, 120, 10])
    lens = s.g["seq_len"]
    ok = [[1, 3, 5], [0, 2, 7], [0, 1, 30]]

    def run(ids, rows, k, moved):
        for b in moved:
            ref.keep(s.np_pool, s.table, [ids[b]], s.seq_len, [rows[b]], [k[b]])
        with pytest.raises(binding.SpecError) as e:
            binding.spec_rows_keep(s.cache, cu(ids), lens, cu(rows), cu(k), sync=True)
        assert e.value.code == binding.SPEC_ECAPACITY
        s.same()

    run([0, 1, 3], ok, [3, 3, 3], [0, 1])
    run([0, -1, 2], ok, [3, 3, 3], [0, 2])
    run([0, 1, 2], [[3, 1, 5], [0, 2, 7], [0, 1, 30]], [3, 3, 3], [1, 2])
    run([0, 1, 2], [[1, 1, 5], [0, 2, 7], [0, 1, 30]], [3, 3, 3], [1, 2])
    run([0, 1, 2], [[1, 3, 5], [-1, 2, 7], [0, 1, 30]], [3, 3, 3], [0, 2])
    run([0, 1, 2], [[1, 3, 60], [0, 2, 7], [0, 1, 30]], [3, 3, 3], [1, 2])       # past the slot's pages
    run([0, 1, 2], ok, [3, 4, -1], [0])
    run([0, 1, 1], ok, [3, 3, 3], [0])


def test_captured_and_replayed():
    s = State(9, 60, 12, seed=4)
    s.fill([0, 1], [200, 333])
    src, dst, all_ = cu([0, 1, 1]), cu([4, 5, 6]), cu([4, 5, 6])
    more = cu([300, 400, 500])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.spec_pages_fork(s.cache, s.g["seq_len"], src, dst, pending=s.g["pending"], hid=s.g["hid"])
        binding.spec_pages_reserve(s.cache, all_, more)
        binding.spec_pages_release(s.cache, all_, s.g["seq_len"][4:7])
    for _ in range(3):
        s.ref_fork([0, 1, 1], [4, 5, 6])
        ref.reserve(s.table, s.refs, [4, 5, 6], [300, 400, 500])
        ref.release(s.table, s.refs, [4, 5, 6], s.seq_len[4:7])
        g.replay()
        torch.cuda.synchronize()
        s.same()


def test_refusals():
    s = State(4, 20, 6)
    s.fill([0], [100])
    B, c, n = binding, s.cache, s.g["seq_len"]
    bare = B.Cache(s.pool, s.g["table"])
    i = cu([1])
    bad = [
        lambda: B.spec_pages_reserve(bare, i, cu([64])), lambda: B.spec_pages_release(bare, i),
        lambda: B.spec_pages_fork(bare, n, cu([0]), i), lambda: B.spec_pages_compact(bare),
        lambda: B.spec_pages_reserve(c, i.long(), cu([64])), lambda: B.spec_pages_reserve(c, i, cu([64, 64])),
        lambda: B.spec_pages_reserve(c, i, cu([64]).cpu()), lambda: B.spec_pages_reserve(c, cu([]), cu([])),
        lambda: B.spec_pages_reserve(c, cu(range(1025)), cu(range(1025))),
        lambda: B.spec_pages_fork(c, n, cu([0, 0]), i), lambda: B.spec_pages_fork(c, n[:2], cu([0]), i),
        lambda: B.spec_pages_fork(c, n, cu([0]), i, pending=n.float()), lambda: B.spec_pages_fork(c, n, cu([0]), i, hid=s.g["hid"][:2]),
        lambda: B.spec_pages_fork(c, n, cu([0]), i, hid=s.g["hid"][:, :9]),
        lambda: B.spec_pages_compact(c, s.g["table"][:2]), lambda: B.spec_pages_compact(c, None, s.g["refs"][:3]),
        lambda: B.spec_pages_release(c, i, workspace=torch.empty(100, dtype=torch.uint8, device="cuda")),
        lambda: B.spec_rows_keep(c, i, n, cu([1]), i), lambda: B.spec_rows_keep(c, i, n, cu([[1]]).long(), i),
        lambda: B.spec_rows_keep(c, i, n, cu(np.zeros((1, 65))), i), lambda: B.spec_rows_keep(c, i, n, cu([[1]]), cu([1, 1])),
    ]
    odd = torch.zeros((1, 20, 2, 1, 64, 4), dtype=torch.bfloat16, device="cuda")     # rows of 8 bytes
    co = B.Cache(odd, s.g["table"], s.g["refs"])
    bad += [lambda: B.spec_pages_fork(co, n, cu([0]), i), lambda: B.spec_pages_compact(co),
            lambda: B.spec_rows_keep(co, i, n, cu([[1]]), i)]
    for k, f in enumerate(bad):
        with pytest.raises(binding.SpecError):
            f()
            pytest.fail("call %d was not refused" % k)
    s.same()


@pytest.mark.parametrize("bad", [12, 1 << 30])
def test_reserve_follows_no_entry_out_of_range(bad):
    s = State(6, 12, 70)
    s.fill([0, 1], [300, 130])
    good = int(s.table[0, 1])
    s.g["table"][0, 1] = s.table[0, 1] = bad
    with pytest.raises(binding.SpecError):
        binding.spec_pages_reserve(s.cache, cu([2, 0]), cu([64, 400]), sync=True)
    assert np.array_equal(s.g["table"].cpu().numpy(), s.table) and np.array_equal(s.g["refs"].cpu().numpy(), s.refs)
    s.g["table"][0, 1] = s.table[0, 1] = good
    s.g["table"][0, 40] = s.table[0, 40] = bad              # (behind the row's end: nothing follows it)
    s.fill([2, 0], [64, 310])
    s.g["table"][0, 40] = s.table[0, 40] = -1
    s.same()


@pytest.mark.parametrize("lens", [(100, 70), (70, 100), (100, 100), (65, 127), (127, 65)])
@pytest.mark.parametrize("shape", SHAPES[:3])
def test_fork_of_slots_cut_back_into_one_page(shape, lens):
    """Slots that share a last page and hold different numbers of its rows, forked in one call: each child
    gets its own source's rows."""
    s = State(9, 60, 6, seed=sum(lens), **shape)
    s.fill([0], [128])
    s.ref_fork([0], [1])
    s.fork([0], [1], sync=True)
    s.seq_len[[0, 1]] = lens
    s.g["seq_len"].copy_(cu(s.seq_len))
    binding.spec_pages_release(s.cache, cu([0, 1]), cu(lens), sync=True)
    s.same()                                                  # (both still name the page)
    for src, dst in (([0, 1], [2, 3]), ([1, 0], [2, 3]), ([0, 0, 1, 1, 0, 1], [2, 3, 4, 5, 6, 7])):
        s.ref_fork(src, dst)
        s.fork(src, dst, sync=True)
        s.same()


@pytest.mark.parametrize("slots,width", [(1024, (1 << 21) + 64), (513, 1 << 22)])
def test_reserve_of_more_pages_than_32_bits_count(slots, width):
    """1024 slots that want some 2^21 pages each (2^31 together), and 513 that want 2^22: refused, and nothing is written."""
    pool = torch.zeros((1, 9, 2, 1, 64, 8), dtype=torch.bfloat16, device="cuda")
    table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(9, dtype=torch.int32, device="cuda")
    table[3, 0], refs[4] = 4, 1
    cache = binding.Cache(pool, table, refs)
    ids = torch.arange(slots, dtype=torch.int32, device="cuda")
    with pytest.raises(binding.SpecError) as e:
        binding.spec_pages_reserve(cache, ids, torch.full_like(ids, width * 64 - 1), sync=True)
    assert e.value.code == binding.SPEC_ECAPACITY
    assert refs.tolist() == [0, 0, 0, 0, 1, 0, 0, 0, 0] and int(table[3, 0]) == 4 and int(table.amax(1).sum()) == 4 - (slots - 1)
    binding.spec_pages_reserve(cache, ids[:4], torch.full_like(ids[:4], 65), sync=True)
    assert table[:5, :3].tolist() == [[0, 1, -1], [2, 3, -1], [5, 6, -1], [4, 7, -1], [-1, -1, -1]]
    assert refs.tolist() == [1] * 8 + [0]


@pytest.mark.parametrize("back", [0, 3, 64, 200])
def test_rows_keep_next_to_the_32nd_bit(back):
    """Rows whose positions pass 2^31 - 256, in a table wide enough for them, are out of range; the sequence beside them moves."""
    pool = torch.randn((2, 7, 2, 1, 64, 8), device="cuda")
    table = torch.full((2, (1 << 25) + 4), -1, dtype=torch.int32, device="cuda")
    table[0, :3] = cu([2, 5, 1])
    table[1, -16:] = 3
    lens = np.array([100, (1 << 31) - 1 - back])
    rows, want, was = [[1, 3, 30], [1, 9, 63]], pool.cpu().numpy(), table[:, -16:].clone()
    ref.keep(want, table[:, :3].cpu().numpy(), [0], lens, [rows[0]], [3])
    with pytest.raises(binding.SpecError) as e:
        binding.spec_rows_keep(binding.Cache(pool, table), cu([1, 0]), cu(lens), cu(rows[::-1]), cu([3, 3]), sync=True)
    assert e.value.code == binding.SPEC_ECAPACITY
    assert np.array_equal(pool.cpu().numpy(), want) and torch.equal(table[:, -16:], was)
