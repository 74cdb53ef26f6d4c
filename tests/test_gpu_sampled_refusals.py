"""Calls that spec_verify_sampled of an engine refuses before anything is launched:
their tensors would be read or written out of range, or as another type."""
import pytest
import torch

from speculative_decoding_spec_gb300 import binding, configs, synth

pytestmark = pytest.mark.gpu


def test_verify_sampled_refuses():
    W = configs.WORKLOADS["tiny_f32_b1_k3"]
    eng = binding.Engine(synth.make_target(W.target, device="cuda"), None, n_slots=2, B_max=2, rows_max=8, max_ctx=128)
    ids, V = eng.seq_ids([0, 1]), W.target.V
    d = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    u = torch.full((4,), 0.5, device="cuda")
    state = [t.clone() for t in (eng.seq_len, eng.pending, eng.hid)]
    run = eng.spec_verify_sampled
    bad = [
        lambda: run(ids, d.long(), u),
        lambda: run(ids, d.cpu(), u),
        lambda: run(ids, d[0], u),
        lambda: run(ids, torch.zeros((1, 2), dtype=torch.int32, device="cuda").t().expand(2, 2).t(), u),
        lambda: run(ids[:1], d, u),
        lambda: run(ids.long(), d, u),
        lambda: run(ids, d, u[:3]),
        lambda: run(ids, d, None),
        lambda: run(ids, d, u, torch.ones(2, device="cuda")),
        lambda: run(ids, d, u, logits=torch.empty((3, V), device="cuda")),
        lambda: run(ids, d, u, logits=torch.empty((4, V), dtype=torch.bfloat16, device="cuda")),
        lambda: run(ids, d, u, logits=torch.empty((V, 4), device="cuda").t()),
    ]
    for f in bad:
        with pytest.raises(binding.SpecError):
            f()
    eng.sync()
    for a, b in zip(state, (eng.seq_len, eng.pending, eng.hid)):
        assert torch.equal(a, b)
    logits = torch.empty((2, 2, V), device="cuda")
    out, n, prob = run(ids, d, u.view(2, 2), logits=logits)     # (flat or [B][k+1])
    eng.sync()
    want = binding.spec_accept_sampled(logits.view(4, V), d, u)
    assert torch.equal(out, want[0]) and torch.equal(n, want[1]) and torch.equal(prob, want[2])
    eng.close()
