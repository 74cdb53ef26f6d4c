"""GPU parity of spec_linear_lora with a 64-bit reference. The whole output is
held to the projection tests' kernel-level bound (1e-4 of a row's largest value:
the activations enter the tensor cores as two 16-bit planes). With W = 0 the
adapters' part stands alone and is held to the bound of its binary32 sums: a sum
of n products is off by at most n * 2^-24 of the sum of their magnitudes, here
K + rank products and a few scalings."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_spec_gb300 import binding, configs, synth
from tests import sampling_ref as ref
from tests.parity import assert_rows_close

pytestmark = pytest.mark.gpu
KTOL = 1e-4


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _adapters(g, n, r, N, K, dtype, scale=True):
    a = (torch.randn((n, r, K), generator=g, device="cuda") / K ** 0.5).to(dtype)
    b = (torch.randn((n, N, r), generator=g, device="cuda") * 0.1).to(dtype)
    return binding.Lora(a, b, torch.rand(n, generator=g, device="cuda") + 0.5 if scale else None)


def _delta(x, lora, ids, gain, eps=1e-6):
    """The adapters' part and the sum of magnitudes behind it, in 64 bits."""
    xd = x.double()
    if gain is not None:
        xd = xd / torch.sqrt((xd ** 2).mean(1, keepdim=True) + eps) * gain.double()
    y = torch.zeros((x.shape[0], lora.N), dtype=torch.float64, device="cuda")
    mag = y.clone()
    for m, i in enumerate(ids.tolist()):
        if 0 <= i < lora.n:
            s = float(lora.scale[i]) if lora.scale is not None else 1.0
            A, B = lora.a[i].double(), lora.b[i].double()
            y[m] = s * (B @ (A @ xd[m]))
            mag[m] = s * (B.abs() @ (A.abs() @ xd[m].abs()))
    return y.cpu().numpy(), mag.cpu().numpy()


def _base(w, x, gain):
    xd = x.double().cpu().numpy()
    if gain is not None:
        xd = np.stack([oracle.rmsnorm(r, gain.cpu().numpy(), 1e-6) for r in xd])
    return oracle.linear(w, xd)


@pytest.mark.parametrize("dtype,adt", [(configs.BF16, torch.bfloat16), (configs.Q4_0, torch.bfloat16),
                                       (configs.F32, torch.float32), (configs.BF16, torch.float32)])
@pytest.mark.parametrize("M", [1, 3, 8, 9, 40, 64])
@pytest.mark.parametrize("N,K,r,norm", [(300, 256, 16, True), (1001, 512, 8, False), (97, 1536, 64, True),
                                        (2048, 256, 128, False), (3, 128, 24, True), (224, 288, 72, True),
                                           (515, 1000, 16, False)])
def test_lora_matches_reference(dtype, adt, M, N, K, r, norm):
    if dtype == configs.Q4_0 and K % 32:
        pytest.skip("Q4_0 rows are whole blocks")
    g = _gen(N + K + M)
    w = synth.make_matrix(g, dtype, 1, N, K, 0.02, "cuda")
    n = 5
    lora = _adapters(g, n, r, N, K, adt)
    ids = torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((M, K), generator=g, device="cuda") * 2
    gain = torch.rand(K, generator=g, device="cuda") + 0.5 if norm else None
    y = binding.spec_linear_lora(w, x, lora, ids, gain=gain)
    want = _base(w, x, gain) + _delta(x, lora, ids, gain)[0]
    assert_rows_close(y.cpu().numpy(), want, KTOL, "lora")


@pytest.mark.parametrize("adt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,r,norm", [(1, 512, 1536, 16, True), (5, 514, 6144, 64, False), (40, 2560, 512, 128, True),
                                          (64, 130, 24576, 32, False), (33, 4099, 1536, 8, True)])
def test_adapter_part_alone(adt, M, N, K, r, norm):
    g = _gen(M + N)
    w = synth.WTensor(configs.BF16, 1, N, K, torch.zeros((1, N, K), dtype=torch.bfloat16, device="cuda"))
    lora = _adapters(g, 7, r, N, K, adt)
    ids = torch.randint(-1, 7, (M,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((M, K), generator=g, device="cuda")
    gain = torch.rand(K, generator=g, device="cuda") + 0.5 if norm else None
    y = binding.spec_linear_lora(w, x, lora, ids, gain=gain).double().cpu().numpy()
    want, mag = _delta(x, lora, ids, gain)
    assert np.all(np.abs(y - want) <= (K + r + 8) * 2.0 ** -24 * mag)
    # (and far inside it, as errors of alternating sign are)
    assert np.linalg.norm(y - want) <= 1e-6 * np.linalg.norm(want) + 1e-30


@pytest.mark.parametrize("dtype", [configs.BF16, configs.Q4_0, configs.F32])
@pytest.mark.parametrize("N,M", [(1024, 8), (1024, 40), (1023, 5), (80001, 12)])
def test_rows_without_an_adapter(dtype, N, M):
    """Bit for bit those of a call without adapters, whatever the other rows
    bring; unused adapters are not read into any row."""
    g = _gen(2)
    w = synth.make_matrix(g, dtype, 1, N, 512, 0.02, "cuda")
    lora = _adapters(g, 4, 16, N, 512, torch.bfloat16)
    lora.a[2] = float("nan")
    lora.b[2] = float("inf")
    x = torch.randn((M, 512), generator=g, device="cuda")
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    none = binding.spec_linear_lora(w, x, lora, ids)
    assert_rows_close(none.cpu().numpy(), _base(w, x, None), KTOL, "no adapters")
    ids[::3] = 1
    ids[1::3] = 3
    y = binding.spec_linear_lora(w, x, lora, ids)
    assert torch.equal(y[ids < 0], none[ids < 0]) and torch.isfinite(y).all()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 1536), (12, 2560, 6144), (40, 3000, 2560), (64, 130, 24576),
                                   (3, 26001, 2048), (37, 8201, 6144), (64, 7000, 6144), (46, 2000, 608)])
def test_bf16_is_a_binary32_projection(M, N, K):
    """bf16 weights and adapters: activations in three 16-bit planes (2^-25), exact
    products, binary32 sums. A sum of n products of random sign is off by about
    sqrt(n) * 2^-24 of a product's size times the number of roundings of a partial
    sum, relative to a result of sqrt(n) such products: well below 2^-20."""
    g = _gen(N)
    w = synth.make_matrix(g, configs.BF16, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, 5, 16, N, K, torch.bfloat16)
    ids = torch.randint(-1, 5, (M,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((M, K), generator=g, device="cuda")
    want = torch.as_tensor(_delta(x, lora, ids, None)[0], device="cuda") + x.double() @ w.data[0].double().t()
    y = binding.spec_linear_lora(w, x, lora, ids).double()
    assert (y - want).norm() <= 2.0 ** -20 * want.norm()


def test_a_row_depends_on_its_adapter_only():
    g = _gen(3)
    N, K = 768, 1536
    w = synth.make_matrix(g, configs.BF16, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, 9, 32, N, K, torch.bfloat16)
    x = torch.randn((8, K), generator=g, device="cuda")
    ids = torch.tensor([3, 3, 0, 8, -1, 5, 3, 0], dtype=torch.int32, device="cuda")
    full = binding.spec_linear_lora(w, x, lora, ids)
    again = binding.spec_linear_lora(w, x, lora, ids)
    assert torch.equal(full, again)
    perm = torch.tensor([6, 2, 0, 7, 1, 3, 5, 4], device="cuda")
    assert torch.equal(binding.spec_linear_lora(w, x[perm].contiguous(), lora, ids[perm].contiguous()), full[perm])
    for m in (0, 4, 7):
        assert torch.equal(binding.spec_linear_lora(w, x[m:m + 1], lora, ids[m:m + 1])[0], full[m])


def test_ids_out_of_range_and_a_dirty_workspace():
    g = _gen(4)
    N, K, M = 640, 256, 12
    w = synth.make_matrix(g, configs.BF16, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, 3, 8, N, K, torch.bfloat16, scale=False)
    x = torch.randn((M, K), generator=g, device="cuda")
    ids = torch.tensor([0, 1, 2, 3, -2, 1 << 30, -1, 0, 1, 2, 0, -(1 << 31)], dtype=torch.int32, device="cuda")
    ws = torch.full((binding.lib().spec_linear_lora_workspace_bytes(N, K, M, 8),), 0xAB, dtype=torch.uint8, device="cuda")
    y = binding.spec_linear_lora(w, x, lora, ids, workspace=ws)
    assert ws[:4].view(torch.int32)[0] == 2
    bad = (ids < 0) | (ids >= 3)
    fixed = torch.where(bad, -1, ids).to(torch.int32)
    assert torch.equal(y, binding.spec_linear_lora(w, x, lora, fixed, workspace=ws))
    assert ws[:4].view(torch.int32)[0] == 0
    want = _base(w, x, None) + _delta(x, lora, fixed, None)[0]
    assert_rows_close(y.cpu().numpy(), want, KTOL, "lora")


def test_infinities_stay_in_their_rows():
    g = _gen(5)
    w = synth.make_matrix(g, configs.BF16, 1, 256, 256, 0.02, "cuda")
    lora = _adapters(g, 2, 8, 256, 256, torch.bfloat16)
    x = torch.randn((4, 256), generator=g, device="cuda")
    ids = torch.tensor([0, 1, -1, 0], dtype=torch.int32, device="cuda")
    y = binding.spec_linear_lora(w, x, lora, ids)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    z = binding.spec_linear_lora(w, x, lora, ids)
    assert torch.equal(z[0], y[0]) and torch.equal(z[3], y[3]) and torch.isnan(z[1]).all()


# An adapter with infinities and NaN is its own rows' trouble.
@pytest.mark.parametrize("dtype,adt", [(configs.BF16, torch.bfloat16), (configs.Q4_0, torch.bfloat16),
                                       (configs.BF16, torch.float32)])
@pytest.mark.parametrize("M,N,K,r", [(7, 300, 256, 16), (40, 1001, 1536, 72), (20, 130, 24576, 8)])
def test_a_broken_adapter_stays_in_its_rows(dtype, adt, M, N, K, r):
    g = _gen(N)
    w = synth.make_matrix(g, dtype, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, 3, r, N, K, adt)
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % 4 - 1
    x = torch.randn((M, K), generator=g, device="cuda")
    want = _base(w, x, None) + _delta(x, lora, ids, None)[0]
    lora.b[1, ::2, 0] = float("nan")
    lora.b[1, 1::3, r - 1] = float("inf")
    lora.a[2, r // 2, K // 2] = float("-inf")
    y = binding.spec_linear_lora(w, x, lora, ids).cpu().numpy()
    rows = (ids.cpu().numpy() < 1)
    assert_rows_close(y[rows], want[rows], KTOL, "rows of sound adapters")
    one = y[ids.cpu().numpy() == 1]
    assert np.isnan(one[:, ::2]).all() and np.isfinite(np.delete(one, np.r_[0:N:2, 1:N:3], 1)).all()
    assert not np.isfinite(y[ids.cpu().numpy() == 2]).any()


def test_other_stream_captured_graph_and_layers():
    g = _gen(6)
    N, K, M = 1536, 512, 20
    w = synth.make_matrix(g, configs.BF16, 3, N, K, 0.02, "cuda")
    lora = _adapters(g, 4, 16, N, K, torch.bfloat16)
    x = torch.randn((M, K), generator=g, device="cuda")
    ids = torch.randint(-1, 4, (M,), generator=g, device="cuda", dtype=torch.int32)
    want = [binding.spec_linear_lora(w, x, lora, ids, layer=l) for l in range(3)]
    assert not torch.equal(want[0], want[2])
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [binding.spec_linear_lora(w, x, lora, ids, layer=l, stream=st[l % 2]) for l in (0, 1, 2, 0)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[l]) for a, l in zip(got, (0, 1, 2, 0)))
    graphs = []
    for l in (1, 2):                      # two graphs: each has scratch of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = binding.spec_linear_lora(w, x, lora, ids, layer=l)
        graphs.append((graph, out, l))
    for seed in (1, 2):
        x.copy_(torch.randn((M, K), generator=_gen(seed), device="cuda"))
        ids.copy_(torch.randint(-1, 4, (M,), generator=_gen(seed), device="cuda", dtype=torch.int32))
        torch.cuda.synchronize()
        for (graph, _, _), s in zip(graphs, st):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, l in graphs:
            assert torch.equal(out, binding.spec_linear_lora(w, x, lora, ids, layer=l))


@pytest.mark.parametrize("dtype", [configs.BF16, configs.Q4_0])
def test_two_calls_at_once(dtype):
    g = _gen(12)
    N, K, M = 5000, 2048, 24
    w = synth.make_matrix(g, dtype, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, 4, 16, N, K, torch.bfloat16)
    x = [torch.randn((M, K), generator=g, device="cuda") for _ in range(2)]
    ids = [torch.randint(-1, 4, (M,), generator=g, device="cuda", dtype=torch.int32) for _ in range(2)]
    alone = [binding.spec_linear_lora(w, x[i], lora, ids[i]) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[binding.spec_linear_lora(w, x[i], lora, ids[i], stream=streams[i]) for i in range(2)] for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(both[i], alone[i]) for both in got for i in range(2))


def test_refusals():
    g = _gen(7)
    w = synth.make_matrix(g, configs.BF16, 1, 64, 64, 0.02, "cuda")
    lora = _adapters(g, 2, 8, 64, 64, torch.bfloat16)
    x = torch.zeros((4, 64), device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    run = binding.spec_linear_lora
    bad = [
        lambda: run(w, x.half(), lora, ids),
        lambda: run(w, x[:, :32].contiguous(), lora, ids),
        lambda: run(w, x.expand(4, 64).t(), lora, ids),
        lambda: run(w, x.cpu(), lora, ids),
        lambda: run(w, x, lora, ids.long()),
        lambda: run(w, x, lora, ids[:3]),
        lambda: run(w, x, lora, ids, gain=torch.ones(32, device="cuda")),
        lambda: run(w, x, lora, ids, y=torch.zeros((4, 32), device="cuda")),
        lambda: run(w, x, lora, ids, layer=1),
        lambda: run(w, torch.zeros((65, 64), device="cuda"), lora, torch.zeros(65, dtype=torch.int32, device="cuda")),
        lambda: run(w, x, lora, ids, workspace=torch.zeros(512, dtype=torch.uint8, device="cuda")),
        lambda: run(w, x, _adapters(g, 2, 8, 32, 64, torch.bfloat16), ids),
        lambda: run(w, x, _adapters(g, 2, 12, 64, 64, torch.bfloat16), ids),
        lambda: run(w, x, _adapters(g, 2, 136, 64, 64, torch.bfloat16), ids),
        lambda: binding.Lora(lora.a, lora.b.float()),
        lambda: binding.Lora(lora.a[:1], lora.b),
        lambda: binding.Lora(lora.a, lora.b, torch.ones(3, device="cuda")),
    ]
    for f in bad:
        with pytest.raises(binding.SpecError):
            f()


@pytest.mark.parametrize("B,k,V", [(1, 3, 4096), (4, 2, 5003)])
def test_adapters_logits_samples_and_accept_together(B, k, V):
    """A verify step of requests with settings of their own: hidden rows -> LM
    head with each request's adapter -> each request's sampling -> accept. The
    logits are held to the projection's bound, the tokens to the 64-bit
    reference on those logits."""
    M, K, g = B * (k + 1), 512, _gen(V)
    w = synth.make_matrix(g, configs.BF16, 1, V, K, 0.1, "cuda")
    lora = _adapters(g, 3, 16, V, K, torch.bfloat16)
    ids = (torch.arange(B, device="cuda") % 4 - 1).repeat_interleave(k + 1).to(torch.int32)
    h = torch.randn((M, K), generator=g, device="cuda")
    gain = torch.rand(K, generator=g, device="cuda") + 0.5
    T = (0.3 + 0.2 * torch.arange(B, device="cuda")).repeat_interleave(k + 1).contiguous()
    tk = (20 + 5 * torch.arange(B, device="cuda")).repeat_interleave(k + 1).to(torch.int32)
    p = torch.full((M,), 0.95, device="cuda")
    u = torch.rand(M, generator=g, device="cuda")
    logits = binding.spec_linear_lora(w, h, lora, ids, gain=gain)
    token, _ = binding.spec_sample(logits, u, T, tk, p)
    drafts = token.view(B, k + 1)[:, :k].clone()
    drafts[0, k - 1] += 1
    out, ne, pr = binding.spec_accept_sampled(logits, drafts.contiguous(), u, T, tk, p)
    assert_rows_close(logits.cpu().numpy(), _base(w, h, gain) + _delta(h, lora, ids, gain)[0], KTOL, "logits")
    n = lambda t: t.cpu().numpy()
    rt, rp, dec = ref.rows(n(logits), n(u), n(T), n(tk), n(p))
    assert dec.all() and np.array_equal(rt, n(token))
    ro, rn, rpr = ref.accept(rt.reshape(B, -1), rp.reshape(B, -1), n(drafts))
    assert np.array_equal(n(out), ro) and np.array_equal(n(ne), rn) and n(ne)[0] == k and (n(ne)[1:] == k + 1).all()
    assert np.all(np.abs(n(pr) - rpr) <= 2.0 ** -21 * rpr)
