"""What a spec_linear_lora call records of its own errors, on both of its routes (bf16
weights and adapters in one stream; shrink, projection and expand for the other
types, in either order), and that it leaves its result to nothing a workspace held."""
import pytest
import torch

from speculative_decoding_spec_gb300 import binding, configs, synth

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _adapters(g, n, r, N, K, dtype):
    a = (torch.randn((n, r, K), generator=g, device="cuda") / K ** 0.5).to(dtype)
    b = (torch.randn((n, N, r), generator=g, device="cuda") * 0.1).to(dtype)
    return binding.Lora(a, b)


KINDS = [(configs.BF16, torch.bfloat16), (configs.Q4_0, torch.bfloat16), (configs.F32, torch.float32),
         (configs.BF16, torch.float32)]


@pytest.mark.parametrize("dtype,adt", KINDS)
@pytest.mark.parametrize("N", [640, 641, 642])
@pytest.mark.parametrize("M", [6, 12, 40])
def test_ids_out_of_range_and_a_dirty_workspace(dtype, adt, N, M):
    g = _gen(N + M)
    K, r = 256, 16
    w = synth.make_matrix(g, dtype, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, 3, r, N, K, adt)
    x = torch.randn((M, K), generator=g, device="cuda")
    odd = [0, 1, 3, -2, 2, 1 << 30, -1, -(1 << 31), 2147483647]
    ids = torch.tensor([odd[i % len(odd)] for i in range(M)], dtype=torch.int32, device="cuda")
    fixed = torch.where((ids < 0) | (ids >= 3), -1, ids).to(torch.int32)
    want = binding.spec_linear_lora(w, x, lora, fixed, sync=True)
    size = binding.lib().spec_linear_lora_workspace_bytes(N, K, M, r)
    ws = torch.full((size + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    word = ws[:4].view(torch.int32)
    for _ in range(2):                       # the second call on what the first one left
        y = binding.spec_linear_lora(w, x, lora, ids, workspace=ws[:size])
        assert word[0] == 2 and torch.equal(y, want)
    assert torch.equal(binding.spec_linear_lora(w, x, lora, fixed, workspace=ws[:size]), want) and word[0] == 0
    assert (ws[size:] == 0xAB).all()
    with pytest.raises(binding.SpecError) as e:
        binding.spec_linear_lora(w, x, lora, ids, sync=True)
    assert e.value.code == binding.SPEC_ECAPACITY
    with pytest.raises(binding.SpecError):
        binding.spec_linear_lora(w, x, lora, ids, stream=torch.cuda.Stream(), sync=True)


def test_one_workspace_for_both_routes():
    """Calls of the two routes one after the other, each on what the other left."""
    g = _gen(5)
    N, K, M, r = 768, 512, 12, 16
    size = binding.lib().spec_linear_lora_workspace_bytes(N, K, M, r)
    ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")
    x = torch.randn((M, K), generator=g, device="cuda")
    ids = (torch.arange(M, device="cuda") % 4 - 1).to(torch.int32)
    calls = []
    for dtype, adt in KINDS:
        w = synth.make_matrix(g, dtype, 1, N, K, 0.02, "cuda")
        lora = _adapters(g, 3, r, N, K, adt)
        calls.append((w, lora, binding.spec_linear_lora(w, x, lora, ids, sync=True)))
    for _ in range(3):
        for w, lora, want in calls + calls[::-1]:
            assert torch.equal(binding.spec_linear_lora(w, x, lora, ids, workspace=ws), want)
