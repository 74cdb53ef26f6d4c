"""Calls of the operators for drafted trees and branching sequences that are refused
on the host, before anything is launched (no GPU needed)."""
import ctypes as C

import pytest

from speculative_decoding_spec_gb300 import binding, configs

P = 1 << 20        # an address that no refused call reads
EINVAL, EUNSUPPORTED, ECAPACITY = binding.SPEC_EINVAL, binding.SPEC_EUNSUPPORTED, binding.SPEC_ECAPACITY


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_spec_gb300 import build
    build.build()
    return binding.lib()


def _kv(**kw):
    v = dict(pool=P, n_pages=9, page_size=64, block_table=P, max_pages_per_seq=4, n_slots=3)
    v.update(kw)
    return binding.spec_kv_desc(*(v[k] for k in ("pool", "n_pages", "page_size", "block_table", "max_pages_per_seq", "n_slots")))


def _md(**kw):
    m = binding.model_desc(configs.E2B)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


def test_attention_tree(lib):
    def call(m=None, kv=None, **kw):
        a = dict(layer=0, B=2, seq_ids=P, seq_len=P, R=4, nq=12, parents=P, rows=P, dt=1, q=P, ldq=1536, out=2 * P, ldo=1536,
                 ws=P, n=1 << 40)
        a.update(kw)
        return lib.spec_attention_tree(C.byref(m or _md()), C.byref(kv or _kv()), *a.values(), None)
    for kw in (dict(layer=-1), dict(layer=24), dict(B=0), dict(B=-3), dict(seq_ids=None), dict(seq_len=None), dict(R=0), dict(nq=0),
               dict(nq=13), dict(dt=2), dict(dt=-1), dict(q=None), dict(out=None), dict(ws=None), dict(q=P + 8), dict(out=P + 4),
               dict(ws=P + 8), dict(ldq=1535), dict(ldq=1540), dict(ldo=1528), dict(ldo=1537), dict(m=_md(head_dim=0)),
               dict(m=_md(n_kv_heads=5)), dict(kv=_kv(pool=None)), dict(kv=_kv(page_size=32)), dict(kv=_kv(block_table=None)),
               dict(kv=_kv(n_pages=0)), dict(kv=_kv(max_pages_per_seq=0)), dict(kv=_kv(n_slots=0)), dict(kv=_kv(pool=P + 8))):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(B=1025), dict(R=65), dict(m=_md(head_dim=100), ldq=2000, ldo=2000)):
        assert call(**kw) == EUNSUPPORTED, kw
    n = lib.spec_attention_tree_workspace_bytes(C.byref(_md()), 2, 4, 12, 4)
    assert n > 0 and call(n=n - 1) == ECAPACITY
    for bad in ((0, 4, 12, 4), (2, 0, 12, 4), (2, 65, 12, 4), (1025, 4, 12, 4), (2, 4, 13, 4), (2, 4, 12, 0)):
        assert lib.spec_attention_tree_workspace_bytes(C.byref(_md()), *bad) == 0


def test_rows_keep(lib):
    def call(m=None, kv=None, **kw):
        a = dict(B=2, seq_ids=P, seq_len=P, n=4, rows=P, keep=P, ws=P, size=256)
        a.update(kw)
        return lib.spec_rows_keep(C.byref(m or _md()), C.byref(kv or _kv()), *a.values(), None)
    for kw in (dict(B=0), dict(seq_ids=None), dict(seq_len=None), dict(n=0), dict(rows=None), dict(keep=None), dict(ws=None),
               dict(kv=_kv(n_slots=0)), dict(m=_md(n_layers=0))):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(B=1025), dict(n=65), dict(m=_md(head_dim=4)), dict(kv=_kv(pool=P + 8))):
        assert call(**kw) == EUNSUPPORTED, kw
    assert call(size=255) == ECAPACITY


def test_pages(lib):
    size = lib.spec_pages_workspace_bytes(9, 2)
    assert size > 0
    for bad in ((0, 1), (9, 0), (9, 1025), ((1 << 20) + 1, 1)):
        assert lib.spec_pages_workspace_bytes(*bad) == 0
    for f in (lib.spec_pages_reserve, lib.spec_pages_release):
        def call(kv=None, **kw):
            a = dict(refs=P, n=2, ids=P, lens=P, ws=P, size=size)
            a.update(kw)
            return f(C.byref(kv or _kv()), *a.values(), None)
        for kw in (dict(refs=None), dict(n=0), dict(n=-1), dict(ids=None), dict(ws=None), dict(ws=P + 4), dict(kv=_kv(block_table=None)),
                   dict(kv=_kv(n_pages=0)), dict(kv=_kv(n_slots=0)), dict(kv=_kv(max_pages_per_seq=0))):
            assert call(**kw) == EINVAL, kw
        assert call(n=1025) == EUNSUPPORTED and call(kv=_kv(n_pages=(1 << 20) + 1)) == EUNSUPPORTED
        assert call(size=size - 1) == ECAPACITY
    assert lib.spec_pages_reserve(C.byref(_kv()), P, 2, P, None, P, size, None) == EINVAL

    def fork(m=None, kv=None, **kw):
        a = dict(refs=P, state=C.byref(binding.spec_state(P, P, P, None)), n=2, src=P, dst=P, ws=P, size=size)
        a.update(kw)
        return lib.spec_pages_fork(C.byref(m or _md()), C.byref(kv or _kv()), *a.values(), None)
    for kw in (dict(refs=None), dict(state=None), dict(state=C.byref(binding.spec_state(None, P, P, None))), dict(n=0), dict(src=None),
               dict(dst=None), dict(ws=None), dict(kv=_kv(pool=None)), dict(m=_md(n_kv_heads=0))):
        assert fork(**kw) == EINVAL, kw
    assert fork(n=1025) == EUNSUPPORTED and fork(m=_md(head_dim=4)) == EUNSUPPORTED and fork(size=64) == ECAPACITY

    def compact(m=None, kv=None, **kw):
        a = dict(refs=P, table=P, refs_out=P, moved=P, live=P, ws=P, size=size)
        a.update(kw)
        return lib.spec_pages_compact(C.byref(m or _md()), C.byref(kv or _kv()), *a.values(), None)
    for k in ("refs", "table", "refs_out", "moved", "live", "ws"):
        assert compact(**{k: None}) == EINVAL, k
    assert compact(m=_md(head_dim=4)) == EUNSUPPORTED and compact(size=8) == ECAPACITY


def test_adjust_logits(lib):
    def call(s=None, **kw):
        v = dict(history=P, ld_history=50, n_history=50, bias_tokens=P, bias_values=P, n_bias=3, mask=P, ld_mask=32, n_masks=8,
                 mask_ids=P, parents=P)
        v.update(s or {})
        a = dict(dt=0, logits=P, ld=1000, B=2, R=4, V=1000, s=C.byref(binding.spec_adjust(**v)), out=2 * P, ldo=1000)
        a.update(kw)
        return lib.spec_adjust_logits(*a.values(), None)
    for kw in (dict(dt=2), dict(dt=-1), dict(logits=None), dict(ld=999), dict(B=0), dict(R=0), dict(V=0), dict(out=None),
               dict(ldo=999), dict(out=P, ldo=1001), dict(logits=P + 2), dict(out=2 * P + 1, dt=1)):
        assert call(**kw) == EINVAL, kw
    assert lib.spec_adjust_logits(0, P, 1000, 2, 4, 1000, None, P, 1000, None) == EINVAL
    for s in (dict(n_history=-1), dict(n_bias=-1), dict(ld_history=49), dict(bias_tokens=None), dict(bias_values=None),
              dict(n_masks=0), dict(ld_mask=31), dict(mask_ids=None, n_masks=7)):
        assert call(s) == EINVAL, s
    assert call(dict(mask=None), V=(1 << 19) + 1, ld=1 << 20, ldo=1 << 20) == EUNSUPPORTED
    assert call(R=65) == EUNSUPPORTED and call(dict(parents=None), R=1025) == EUNSUPPORTED and call(B=65536) == EUNSUPPORTED
    assert call(dict(n_bias=4096)) == EUNSUPPORTED
    assert call(dict(n_history=1 << 19, ld_history=1 << 19)) == EUNSUPPORTED


def test_attention_tree_in_place_and_wide_heads(lib):
    """One tensor for queries and results; more query rows on a KV head than a row's number has bits for."""
    def call(q, out, nq, R):
        return lib.spec_attention_tree(C.byref(_md()), C.byref(_kv()), 0, 1, P, P, R, nq, P, P, 1, q, nq * 128, out, nq * 128, P,
                                       1 << 40, None)
    assert call(P, P, 12, 4) == EINVAL
    for R, G in ((64, 1025), (1, (1 << 16) + 1), (33, 2000)):
        assert call(P, 2 * P, 4 * G, R) == EUNSUPPORTED, (R, G)
        assert lib.spec_attention_tree_workspace_bytes(C.byref(_md()), 1, R, 4 * G, 4) == 0
    for R, G in ((64, 1024), (1, 1 << 16)):
        assert lib.spec_attention_tree_workspace_bytes(C.byref(_md()), 1, R, 4 * G, 4) > 0


def test_rows_keep_workspace_alignment(lib):
    for ws in (P + 1, P + 2, P + 4, P + 8):
        assert lib.spec_rows_keep(C.byref(_md()), C.byref(_kv()), 2, P, P, 4, P, P, ws, 256, None) == EINVAL


def test_stream_of_another_gpu(lib):
    """A call whose stream is not on its tensors' GPU is refused, not sent to a stream of that GPU."""
    import types
    import torch
    cache = types.SimpleNamespace(dev=0)
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    logits = types.SimpleNamespace(get_device=lambda: 0)
    B = binding
    for call in (lambda: B.spec_attention_tree(cache, 0, None, None, None, stream=other),
                 lambda: B.spec_rows_keep(cache, None, None, None, None, stream=other),
                 lambda: B.spec_pages_reserve(cache, None, None, stream=other),
                 lambda: B.spec_pages_release(cache, None, stream=other),
                 lambda: B.spec_pages_fork(cache, None, None, None, stream=other),
                 lambda: B.spec_pages_compact(cache, stream=other),
                 lambda: B.spec_adjust_logits(logits, stream=other)):
        with pytest.raises(B.SpecError) as e:
            call()
        assert e.value.code == EINVAL and "another GPU" in str(e.value)
