"""The operators for drafted trees and branching sequences as they are used together:
slots of an engine that take pages from a pool, fork, go on differently and give
their pages back; a pass's logits adjusted and sampled; a tree attended in the
engine's cache and its accepted rows kept."""
import dataclasses
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding, configs, synth
from tests import branch_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
W = configs.WORKLOADS["tiny_f32_b1_k3"]


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _shape(kind):
    return W.target if kind == "f32" else dataclasses.replace(W.target, wdtype=configs.BF16, kvdtype=configs.BF16)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_forked_slots_go_on_alone(kind):
    """A prompt prefilled once and forked gives every branch the tokens that an engine
    of its own gives it, whatever the other branches do, before and after compaction."""
    t = _shape(kind)
    tw = synth.make_target(t, device="cuda")
    eng = binding.Engine(tw, None, n_slots=4, B_max=1, rows_max=160, max_ctx=256, n_pages=11)
    prompt = synth.make_tokens(130, t.V).view(1, -1).cuda()
    one = [_int([s]) for s in range(4)]
    eng.spec_pages_reserve(one[2], _int([131]))
    eng.spec_prefill(one[2], prompt)
    eng.sync()
    eng.spec_pages_fork(_int([2, 2]), _int([0, 3]))
    firsts = {0: 11, 2: None, 3: 77}                  # the branches' next tokens (None: the target's own)
    alone = {}
    for s, tok in firsts.items():
        other = binding.Engine(tw, None, n_slots=1, B_max=1, rows_max=160, max_ctx=256)
        other.spec_prefill(_int([0]), prompt)
        other.sync()
        if tok is not None:
            other.pending[0] = tok
            eng.pending[s] = tok
        alone[s] = other
    got, want = {s: [] for s in firsts}, {s: [] for s in firsts}
    for step in range(70):                            # (past the second page's end)
        for s in firsts:
            eng.spec_pages_reserve(one[s], eng.seq_len[s:s + 1] + 1)
            got[s].append(int(eng.spec_decode(one[s], 1)[0]))
            want[s].append(int(alone[s].spec_decode(_int([0]), 1)[0]))
        eng.sync()
        if step == 20:                                # a branch ends, its pages are used again
            eng.spec_pages_release(one[3])
            del firsts[3]
            moved, live = eng.spec_pages_compact()
            assert int(live) == int((eng.page_refs > 0).sum())
            assert (eng.page_refs[: int(live)] > 0).all() and (eng.page_refs[int(live):] == 0).all()
    assert got == want
    shared = eng.block_table[0][:2].tolist()
    assert shared == eng.block_table[2][:2].tolist() and int(eng.block_table[0][2]) != int(eng.block_table[2][2])
    assert eng.page_refs[shared].tolist() == [2, 2]
    eng.spec_pages_release(_int([0, 2]))
    assert (eng.page_refs == 0).all() and (eng.block_table == -1).all()
    for e in [eng, *alone.values()]:
        e.close()


def test_a_pass_without_pages_is_refused_on_the_gpu():
    t = _shape("f32")
    eng = binding.Engine(synth.make_target(t, device="cuda"), None, n_slots=2, B_max=1, rows_max=64, max_ctx=128, n_pages=3)
    ids = _int([0])
    eng.spec_pages_reserve(ids, _int([64]))
    eng.spec_prefill(ids, synth.make_tokens(64, t.V).view(1, -1).cuda())
    eng.sync()
    eng.spec_decode(ids, 1)
    with pytest.raises(binding.SpecError) as e:       # position 64 has no page yet
        eng.sync()
    assert e.value.code == binding.SPEC_ECAPACITY and int(eng.seq_len[0]) == 64
    eng.spec_pages_reserve(ids, _int([65]))
    eng.spec_decode(ids, 1)
    eng.sync()
    assert int(eng.seq_len[0]) == 65
    with pytest.raises(binding.SpecError):
        eng.spec_pages_reserve(_int([1]), _int([128]))
    eng.close()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_tree_rows_in_the_engines_cache(kind):
    """A chain through spec_attention_tree is spec_attention's; a tree's accepted rows,
    kept, read as the chain of them alone."""
    t = _shape(kind)
    eng = binding.Engine(synth.make_target(t, device="cuda"), None, n_slots=2, B_max=2, rows_max=16, max_ctx=256)
    g = torch.Generator(device="cuda").manual_seed(1)
    eng.pool.normal_(generator=g)
    lens, R = [100, 63], 6
    eng.seq_len.copy_(_int(lens))
    ids = _int([1, 0])
    q = torch.randn((2 * R, t.nq * t.hd), generator=g, device="cuda")
    a = binding.spec_attention(t, eng.pool, eng.block_table, 1, ids, eng.seq_len, R, t.nq, 1, q)
    b = binding.spec_attention_tree(eng.cache, 1, ids, eng.seq_len, q, sync=True)
    assert float((a - b).abs().max()) <= 1e-4 * float(a.abs().max())
    parents = _int([[-1, 0, 0, 1, 2, 4], [-1, 0, 1, 1, 3, 3]])
    tree = binding.spec_attention_tree(eng.cache, 1, ids, eng.seq_len, q, parents, sync=True).view(2, R, -1)
    path, keep = _int([[0, 2, 4, 5], [0, 1, 3, 0]]), _int([4, 3])
    binding.spec_rows_keep(eng.cache, ids, eng.seq_len, path, keep, sync=True)
    rows = torch.stack([q.view(2, R, -1)[i, path[i].long()] for i in range(2)]).view(8, -1)
    chain = binding.spec_attention_tree(eng.cache, 1, ids, eng.seq_len, rows, n_rows=keep, sync=True).view(2, 4, -1)
    for i in range(2):
        for j in range(int(keep[i])):
            x, y = tree[i, int(path[i, j])], chain[i, j]
            assert float((x - y).abs().max()) <= 1e-4 * float(x.abs().max())
    eng.close()


def test_adjusted_and_sampled_pass():
    """A verify pass's logits, adjusted for its rows and accepted by sampling: the greedy
    rows take the reference's largest changed logits."""
    t = _shape("f32")
    eng = binding.Engine(synth.make_target(t, device="cuda"), None, n_slots=2, B_max=2, rows_max=64, max_ctx=256)
    prompt = synth.make_tokens(120, t.V).view(2, 60)
    ids, k = eng.seq_ids([0, 1]), 3
    eng.spec_prefill(ids, prompt.cuda())
    eng.sync()
    fed = torch.cat([eng.pending[:2, None].cpu(), synth.make_tokens(6, t.V, seed=9).view(2, 3)], 1).to(torch.int32)
    logits = torch.empty((8, t.V), device="cuda")
    eng.spec_verify(ids, fed[:, 1:].contiguous().cuda(), logits)
    eng.sync()
    f = lambda *v: torch.tensor(v, device="cuda")
    got = binding.spec_adjust_logits(logits, k + 1, tokens=fed.cuda(), history=prompt.cuda(), repetition=f(1.3, 1.0),
                                     presence=f(0.5, 2.0), frequency=f(0.1, 0.0))
    want = ref.adjust(logits.double().cpu().numpy(), k + 1, prompt.numpy(), None, None, fed.numpy(), None,
                      np.float32([1.3, 1.0]), np.float32([0.1, 0.0]), np.float32([0.5, 2.0]))
    assert np.abs(got.double().cpu().numpy() - want).max() <= 6 * 2.0 ** -24 * (np.abs(want).max() + 10)
    drafts = fed[:, 1:].contiguous()
    best = want.argmax(1).reshape(2, k + 1)
    drafts[0, 0] = best[0, 0]
    out, n, _ = binding.spec_accept_sampled(got, drafts.cuda(), torch.full((8,), 0.5, device="cuda"),
                                            temperature=torch.zeros(8, device="cuda"))
    for b in range(2):
        e = [int(best[b, 0])]
        for j in range(k):
            if int(drafts[b, j]) != best[b, j]:
                break
            e.append(int(best[b, j + 1]))
        assert out[b, : len(e)].tolist() == e and int(n[b]) == len(e)
    eng.close()


FIRST = """
import torch
from speculative_decoding_spec_gb300 import binding
g = torch.Generator(device="cuda").manual_seed(1)
i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
pool = torch.randn((2, 9, 2, 2, 64, 128), generator=g, device="cuda").bfloat16()
table = i([3, 1, -1], [0, 5, 7])
refs = torch.bincount(table[table >= 0].long(), minlength=9).int()
cache = binding.Cache(pool, table, refs)
lens = i(100, 140)
q = torch.randn((8, 6 * 128), generator=g, device="cuda")
x = torch.randn((8, 300001), generator=g, device="cuda")
f = torch.full((2,), 1.25, device="cuda")
outs = [torch.zeros_like(q), torch.zeros_like(q, dtype=torch.bfloat16), torch.zeros_like(x[:, :4000]), torch.zeros_like(x)]
h = torch.randint(0, 4000, (2, 50), generator=g, device="cuda").int()
def tree32(): binding.spec_attention_tree(cache, 1, i_01, lens, q, out=outs[0]); return outs[0]
def tree16(): binding.spec_attention_tree(cache, 1, i_01, lens, qb, out=outs[1]); return outs[1]
def small(): binding.spec_adjust_logits(x[:, :4000], 4, tokens=tok, history=h, repetition=f, out=outs[2]); return outs[2]
def large(): binding.spec_adjust_logits(x, 4, tokens=tok, history=h, repetition=f, out=outs[3]); return outs[3]
i_01, tok, qb = i(1, 0), h[:, :4].contiguous(), q.bfloat16()
def compact():
    t2, r2 = torch.empty_like(table), torch.empty_like(refs)
    binding.spec_pages_compact(cache, t2, r2)
    return t2
call = dict(tree32=tree32, tree16=tree16, small=small, large=large, compact=compact)[%r]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
got = got.clone()
assert torch.equal(got, call()) and got.any()
print("same")
"""


@pytest.mark.parametrize("call", ["tree32", "tree16", "small", "large", "compact"])
def test_first_call_is_captured(call):
    r = subprocess.run([sys.executable, "-c", FIRST % call], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_engine_buffers_of_ids():
    """Engine.seq_ids has one buffer for lists of one length: a fork of one tensor onto itself is named as such."""
    t = _shape("f32")
    eng = binding.Engine(synth.make_target(t, device="cuda"), None, n_slots=3, B_max=1, rows_max=4, max_ctx=128, n_pages=6)
    eng.spec_pages_reserve(eng.seq_ids([0]), _int([100]))
    eng.seq_len[0] = 100
    with pytest.raises(binding.SpecError) as e:
        eng.spec_pages_fork(eng.seq_ids([0]), eng.seq_ids([1]))
    assert e.value.code == binding.SPEC_EINVAL and "one tensor" in str(e.value)
    eng.spec_pages_fork(eng.seq_ids([0]), _int([1]))
    assert eng.seq_len.tolist() == [100, 100, 0] and int(eng.block_table[0, 0]) == int(eng.block_table[1, 0])
    eng.close()


def test_prefilled_contents_need_pages():
    """Contents for a slot of a pooled engine that has no pages for them are refused: no other slot's page is written."""
    t = _shape("f32")
    eng = binding.Engine(synth.make_target(t, device="cuda"), None, n_slots=2, B_max=1, rows_max=4, max_ctx=192, n_pages=4)
    kv = synth.make_prefilled_kv(t, 100, device="cuda")
    eng.pool.fill_(7.0)
    for pages in (0, 64):
        if pages:
            eng.spec_pages_reserve(_int([1]), _int([pages]))
        with pytest.raises(binding.SpecError) as e:
            eng.load_prefilled(1, kv)
        assert e.value.code == binding.SPEC_ECAPACITY and (eng.pool == 7.0).all() and int(eng.seq_len[1]) == 0
    eng.spec_pages_reserve(_int([1]), _int([100]))
    eng.load_prefilled(1, kv)
    assert int(eng.seq_len[1]) == 100 and torch.equal(eng.pool[:, 0], kv[:, :, :, :64].to(eng.pool.dtype))
    assert (eng.pool[:, 2:] == 7.0).all()
    eng.close()
