"""The first token of a sampled request. spec_prefill leaves the target's greedy choice
pending; a caller that samples feeds all prompt tokens but the last, writes that one
into pending and samples the row behind it with spec_verify_sampled, k = 0."""
import dataclasses

import pytest
import torch

from speculative_decoding_spec_gb300 import binding, configs, synth

pytestmark = pytest.mark.gpu
W = configs.WORKLOADS["tiny_f32_b1_k3"]


def _engine(dt, B):
    tshape = W.target if dt == configs.F32 else dataclasses.replace(W.target, wdtype=dt, kvdtype=configs.BF16)
    dshape = W.drafter if dt == configs.F32 else dataclasses.replace(W.drafter, wdtype=dt)
    eng = binding.Engine(synth.make_target(tshape, device="cuda"), synth.make_drafter(dshape, device="cuda"), n_slots=B,
                         B_max=B, rows_max=64, max_ctx=512, shuffle_pages=True)
    return eng, eng.seq_ids(list(range(B))), tshape


@pytest.mark.parametrize("dt", [configs.F32, configs.BF16])
@pytest.mark.parametrize("B,R", [(1, 40), (3, 17), (2, 1)])
def test_first_token_sampled(dt, B, R):
    g = torch.Generator(device="cuda").manual_seed(R)
    none = torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    u = torch.rand(B, generator=g, device="cuda")
    T = torch.full((B,), 0.7, device="cuda")
    # the greedy start, for the state to compare with
    eng, ids, t = _engine(dt, B)
    prompt = synth.make_tokens(R * B, t.V).view(B, R).cuda().to(torch.int32).contiguous()
    eng.spec_prefill(ids, eng._in("prompt", prompt))
    eng.sync()
    greedy, length = eng.pending.clone(), eng.seq_len.clone()
    eng.close()
    for temp in (torch.zeros(B, device="cuda"), T):
        eng, ids, t = _engine(dt, B)
        if R > 1:
            eng.spec_prefill(ids, eng._in("prompt", prompt[:, :-1].contiguous()))
        eng.pending.copy_(prompt[:, -1])
        logits = torch.empty((B, t.V), device="cuda")
        out, n, prob = (x.clone() for x in eng.spec_verify_sampled(ids, none, u, temp, logits=logits))
        eng.sync()
        want = binding.spec_sample(logits, u, temp)
        assert torch.equal(out[:, 0], want[0]) and torch.equal(prob[:, 0], want[1]) and (n == 1).all()
        assert torch.equal(eng.seq_len, length) and torch.equal(eng.pending, out[:, 0])
        if not temp.any():
            assert torch.equal(out[:, 0], greedy)
        # drafting goes on from there
        d = eng.spec_draft(ids, B, 2)
        _, n, _ = eng.spec_verify_sampled(ids, d, torch.rand(3 * B, generator=g, device="cuda"), T.repeat_interleave(3))
        eng.sync()
        assert (n >= 1).all() and torch.equal(eng.seq_len, length + n)
        eng.close()
