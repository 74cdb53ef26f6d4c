"""Infinities and NaN among the weights, the adapters and the activations of
spec_linear_lora: a row's result follows from its own x, W and its own adapter
alone, bit for bit, and is infinite or NaN where a binary32 projection's is."""
import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding, configs, synth

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _adapters(g, n, r, N, K, dtype=torch.bfloat16):
    a = (torch.randn((n, r, K), generator=g, device="cuda") / K ** 0.5).to(dtype)
    b = (torch.randn((n, N, r), generator=g, device="cuda") * 0.1).to(dtype)
    return binding.Lora(a, b, torch.rand(n, generator=g, device="cuda") + 0.5)


def _break(lora, i, how):
    N, r, K = lora.N, lora.rank, lora.K
    if how == "b nan":
        lora.b[i] = NAN
    elif how == "b inf":
        lora.b[i, ::3, r - 1] = INF
        lora.b[i, 1::5, 0] = -INF
    elif how == "a nan":
        lora.a[i, r // 2, K // 3] = NAN
    else:
        lora.a[i] = INF
        lora.b[i, ::2] = INF
    return lora


# (tiles of one and of two MMAs, split and whole; adapters of one chunk and of two;
# one adapter for several rows and one a row)
SHAPES = [(7, 300, 256, 16, 3), (40, 1001, 1536, 72, 5), (20, 130, 24576, 8, 3), (64, 2560, 512, 128, 64),
          (33, 700, 2560, 64, 33), (40, 20011, 2048, 16, 40), (64, 20011, 2048, 24, 9)]


@pytest.mark.parametrize("dtype,adt", [(configs.BF16, torch.bfloat16), (configs.Q4_0, torch.bfloat16),
                                       (configs.BF16, torch.float32), (configs.F32, torch.float32)])
@pytest.mark.parametrize("M,N,K,r,n", SHAPES)
def test_another_rows_adapter_changes_nothing(dtype, adt, M, N, K, r, n):
    """The rows of sound adapters and those without one, bit for bit: beside a sound
    adapter, beside the same one broken, and beside none."""
    if adt == torch.float32 and N * K > 20_000_000:
        pytest.skip("as the smaller ones")
    g = _gen(M + N)
    w = synth.make_matrix(g, dtype, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, n, r, N, K, adt)
    ids = (torch.arange(M, device="cuda") * n // M).to(torch.int32)
    ids[M - 1] = -1
    x = torch.randn((M, K), generator=g, device="cuda")
    want = binding.spec_linear_lora(w, x, lora, ids)
    assert torch.isfinite(want).all()
    bad = n // 2
    other = ids != bad
    assert other.any() and not other.all()
    gone = torch.where(other, ids, -1).to(torch.int32)
    assert torch.equal(binding.spec_linear_lora(w, x, lora, gone)[other], want[other])
    for how in ("b nan", "b inf", "a nan", "all inf"):
        a, b = lora.a.clone(), lora.b.clone()
        y = binding.spec_linear_lora(w, x, _break(binding.Lora(a, b, lora.scale), bad, how), ids)
        assert torch.equal(y[other], want[other]), how
        own = y[~other]
        assert not torch.isfinite(own).all(), how
        if how in ("b nan", "a nan"):
            assert torch.isnan(own).all(), how


def _same_kind(y, want):
    """Infinite and NaN where the 64-bit result is."""
    y, want = y.double().cpu(), want.cpu()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y == INF, want == INF) and torch.equal(y == -INF, want == -INF)
    fine = torch.isfinite(want)
    assert (y[fine] - want[fine]).abs().max() <= 2.0 ** -18 * want[fine].abs().max()


def _exact(w, x, lora, ids):
    # (one product at a time, in float64: library sums of infinities are left out of it)
    W, xd = w.data[0].double(), x.double()
    y = torch.stack([(W * xd[m]).sum(1) for m in range(x.shape[0])])
    for m, i in enumerate(ids.tolist()):
        if i >= 0:
            t = (lora.a[i].double() * xd[m]).sum(1)
            y[m] += float(lora.scale[i]) * (lora.b[i].double() * t).sum(1)
    return y


@pytest.mark.parametrize("M,N,K,r", [(5, 300, 256, 16), (40, 700, 1536, 72), (9, 20011, 2048, 8)])
@pytest.mark.parametrize("where", ["x", "w", "b", "a"])
def test_infinite_and_nan_where_a_projection_is(where, M, N, K, r):
    g = _gen(N + M)
    w = synth.make_matrix(g, configs.BF16, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, 3, r, N, K)
    ids = (torch.arange(M, device="cuda") % 4 - 1).to(torch.int32)
    x = torch.randn((M, K), generator=g, device="cuda")
    if where == "x":
        x[0, 3] = INF
        x[1, K - 1] = -INF
        x[2, 5], x[2, K // 2] = INF, -INF
        x[3, 7] = NAN
    elif where == "w":
        w.data[0, 1, 2] = INF
        w.data[0, N - 1, K - 1] = -INF
        w.data[0, N // 2, 9] = NAN
        w.data[0, 7, ::64] = INF
        x[1, 0::64] = x[1, 0::64].abs()     # one sign: infinite; elsewhere infinities of both signs
    elif where == "b":
        lora.b[1, 0, 0] = INF
        lora.b[2, N - 1, r - 1] = -INF
        lora.b[2, 5, 1] = NAN
    else:
        lora.a[1, 0, 0] = INF
    _same_kind(binding.spec_linear_lora(w, x, lora, ids), _exact(w, x, lora, ids))


def test_activations_beyond_the_16_bit_range():
    """Finite activations that round to an infinity in 16 bits."""
    N, K, M = 260, 128, 4
    g = _gen(1)
    w = synth.make_matrix(g, configs.BF16, 1, N, K, 0.02, "cuda")
    lora = _adapters(g, 2, 8, N, K)
    lora.a.zero_()
    x = torch.randn((M, K), generator=g, device="cuda")
    x[0, 5] = torch.finfo(torch.float32).max
    x[1, 6] = -3.4e38
    ids = torch.tensor([0, -1, 1, -1], dtype=torch.int32, device="cuda")
    y = binding.spec_linear_lora(w, x, lora, ids).double()
    want = x.double() @ w.data[0].double().t()
    assert torch.isfinite(y).all()
    assert ((y - want).norm(dim=1) <= 2.0 ** -20 * want.norm(dim=1)).all()
