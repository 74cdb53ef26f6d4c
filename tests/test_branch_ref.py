"""Pins of tests/branch_ref.py, the reference of the operators for drafted trees and
branching sequences (CPU)."""
import numpy as np
import pytest

from tests import branch_ref as ref


def _pool(rng, pages, nkv=2, hd=4):
    return rng.standard_normal((pages, 2, nkv, 64, hd))


def test_attention_of_one_key_is_its_value():
    rng = np.random.default_rng(1)
    pool, q = _pool(rng, 2), rng.standard_normal((1, 8))
    o, mag, _, n = ref.attention(pool, np.array([[1, -1]]), [0], [0], q, 2, None, None)
    assert np.allclose(o, pool[1, 1, :, 0].reshape(1, 8)) and np.allclose(mag, np.abs(o)) and (n == 1).all()


def test_attention_with_zero_queries_is_the_mean_over_the_path():
    rng = np.random.default_rng(2)
    pool = _pool(rng, 3)
    table = np.array([[2, 0, 1]])
    parents = np.array([[-1, 0, 0, 2]], np.int32)
    o = ref.attention(pool, table, [0], [63], np.zeros((4, 8)), 2, parents, np.array([4]))[0].reshape(4, 2, 4)
    keys = np.concatenate([pool[p, 1] for p in table[0]], 1)
    for r, up in enumerate([[0], [0, 1], [0, 2], [0, 2, 3]]):
        j = list(range(63)) + [63 + u for u in up]
        assert np.allclose(o[r], keys[:, j].mean(1))


def test_attention_matches_a_library_softmax():
    from scipy.special import softmax
    rng = np.random.default_rng(3)
    pool, q = _pool(rng, 2), rng.standard_normal((3, 16))
    o = ref.attention(pool, np.array([[0, 1]]), [0], [70], q, 4, None, None)[0].reshape(3, 4, 4)
    k, v = (np.concatenate([pool[0, i], pool[1, i]], 1) for i in (0, 1))
    for r in range(3):
        for h in range(4):
            s = k[h // 2, : 71 + r] @ q.reshape(3, 4, 4)[r, h] / 2.0
            assert np.allclose(o[r, h], softmax(s) @ v[h // 2, : 71 + r])


def test_adjust_by_hand():
    x = np.array([[1.0, -2.0, 3.0, 0.5, -np.inf, 4.0], [1.0, -2.0, 3.0, 0.5, 9.0, 4.0]])
    one = np.array([1.0], np.float32)
    y = ref.adjust(x, 2, hist=np.array([[0, 1, 2, 2, -1, 7]]), hist_len=[6], prompt_len=[2], tokens=np.array([[3, 2]]),
                   rep=one * 2, freq=one * 0.25, pres=one * 0.5, bias_tokens=np.array([[5, 5, 4]]),
                   bias_values=np.array([[9.0, 1.0, 2.0]]), mask=np.array([[0b111110], [0b111111]], np.int32),
                   mask_ids=[1, 0])
    # 0, 1: prompt only; 2: twice in the output (three times in the second row); 3: once, fed
    assert np.allclose(y[0, [0, 1, 2, 3, 5]], [0.5, -4.0, 1.5 - 0.5 - 0.5, 0.25 - 0.25 - 0.5, 5.0]) and y[0, 4] == -np.inf
    assert y[1, 0] == -np.inf and np.allclose(y[1, [2, 4]], [1.5 - 0.75 - 0.5, 11.0])


def test_chain_is_the_tree_of_a_chain():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((5, 40))
    a = dict(hist=rng.integers(0, 40, (1, 9)), tokens=rng.integers(0, 40, (1, 5)), rep=[1.3], freq=[0.2], pres=[0.1])
    assert np.array_equal(ref.adjust(x, 5, **a), ref.adjust(x, 5, parents=np.array([[-1, 0, 1, 2, 3]]), **a))


@pytest.mark.parametrize("n", [0, 1, 64, 100])
def test_fork_then_release_leaves_the_source(n):
    rng = np.random.default_rng(5)
    pool = rng.standard_normal((1, 8, 2, 1, 64, 2))
    table, refs, lens = np.full((3, 4), -1, np.int32), np.zeros(8, np.int32), np.array([n, 0, 0])
    ref.reserve(table, refs, [0], [n])
    was = table.copy(), refs.copy(), pool.copy()
    ref.fork(pool, table, refs, lens, [0, 0], [1, 2])
    full = n // 64
    assert (table[1, :full] == table[0, :full]).all() and lens.tolist() == [n] * 3
    assert refs.sum() == 3 * -(-n // 64)
    if n % 64:
        assert len({table[i, full] for i in range(3)}) == 3
        assert (pool[:, table[2, full], ..., : n % 64, :] == pool[:, table[0, full], ..., : n % 64, :]).all()
    ref.release(table, refs, [1, 2])
    assert np.array_equal(table, was[0]) and np.array_equal(refs, was[1])


def test_compact_keeps_what_every_slot_reads():
    rng = np.random.default_rng(6)
    pool = rng.standard_normal((2, 20, 2, 1, 64, 2))
    table, refs = np.full((4, 6), -1, np.int32), np.zeros(20, np.int32)
    ref.reserve(table, refs, [0, 1, 2, 3], [300, 200, 100, 350])
    ref.release(table, refs, [1])
    read = [[pool[:, p].copy() for p in table[s] if p >= 0] for s in range(4)]
    moved, n = ref.compact(pool, table, refs)
    assert (refs[:n] > 0).all() and (refs[n:] == 0).all() and (moved >= 0).sum() == n
    for s in range(4):
        for a, p in zip(read[s], table[s][table[s] >= 0]):
            assert np.array_equal(a, pool[:, p])


def test_keep_moves_rows_together():
    rng = np.random.default_rng(7)
    pool = rng.standard_normal((1, 2, 2, 1, 64, 2))
    table = np.array([[1, 0]])
    was = np.concatenate([pool[0, p].copy() for p in table[0]], 2)
    ref.keep(pool, table, [0], [60], [[1, 4, 9]], [3])
    now = np.concatenate([pool[0, p] for p in table[0]], 2)
    assert np.array_equal(now[:, :, 60:63], was[:, :, [61, 64, 69]])
    assert np.array_equal(now[:, :, :60], was[:, :, :60]) and np.array_equal(now[:, :, 63:], was[:, :, 63:])
