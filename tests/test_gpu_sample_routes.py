"""A row without filters is sampled by one of two routes: in a large call its chunks
of 4096 tokens are spread over the GPU, in a small one, or where the call gives
filters that leave the row as it is, a cluster of CTAs takes the row. Both give the
same token and the same probability, bit for bit: what a row emits depends neither
on the rows beside it nor on where it lies in memory."""
import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding

pytestmark = pytest.mark.gpu
LAST = 1.0 - 2.0 ** -24   # the largest number below 1


def _rows(V, M, dtype, seed):
    """A broad body, a few likely tokens, and tokens far below them: from 2^-40 to
    2^-60 of the largest weight, in a last chunk of their own, spread over the row,
    and as its last token alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, V), generator=g, device="cuda") * 2.5
    x[:, ::997] += 6.0
    i = torch.arange(M, device="cuda")
    top = x.amax(1, keepdim=True)
    x = torch.where((i % 4 == 1)[:, None] & (torch.arange(V, device="cuda") >= (V - 1) // 4096 * 4096)[None], top - 35.0, x)
    x = torch.where((i % 4 == 2)[:, None] & (torch.rand((M, V), generator=g, device="cuda") < 0.9), top - 30.0, x)
    x[i % 4 == 3, V - 1] = (top - 30.8)[i % 4 == 3, 0]
    u = torch.rand(M, generator=g, device="cuda")
    u[1::8], u[2::8], u[3::8] = 1.0, LAST, LAST
    u[5::8], u[6::8], u[7::8], u[4::8] = LAST, 1.0, 1.0, 0.0
    T = torch.where(i % 3 == 0, 1.0, 0.6 + 0.01 * i).contiguous()
    return x.to(dtype), u, T


def _same(a, b, what):
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), (what, a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [8192, 8193, 32003, 40001, 100003, 262144])
def test_a_row_without_filters_depends_on_nothing_else(dtype, V):
    M = 33
    x, u, T = _rows(V, M, dtype, V)
    assert binding.lib().spec_sample_workspace_bytes(M, V) > 0            # in chunks
    got = binding.spec_sample(x, u, T)
    _same(binding.spec_sample(x, u, T), got, "again")
    # filters that are given and leave every row as it is
    f = lambda v, t=torch.float32: torch.full((M,), v, dtype=t, device="cuda")
    _same(binding.spec_sample(x, u, T, None, None, f(0.0)), got, "min_p 0")
    _same(binding.spec_sample(x, u, T, f(0, torch.int32), f(1.0)), got, "top_k 0, top_p 1")
    _same(binding.spec_sample(x, u, T, f(V, torch.int32), f(float("nan")), f(-1.0)), got, "top_k V")
    # a row alone, and behind rows that have filters
    for i in (0, 1, 2, 3, 7, 32):
        one = binding.spec_sample(x[i:i + 1].clone(), u[i:i + 1].clone(), T[i:i + 1].clone())
        _same(one, (got[0][i:i + 1], got[1][i:i + 1]), "row %d alone" % i)
    p = torch.where(torch.arange(M, device="cuda") % 2 == 0, 0.9, 1.0).contiguous()
    some = binding.spec_sample(x, u, T, None, p)
    _same((some[0][1::2], some[1][1::2]), (got[0][1::2], got[1][1::2]), "beside filtered rows")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [9000, 32003, 131071])
@pytest.mark.parametrize("M", [3, 21])
def test_a_row_without_filters_at_every_alignment(dtype, V, M):
    x, u, T = _rows(V, M, dtype, V + M)
    want = binding.spec_sample(x, u, T)
    zero = torch.zeros(M, device="cuda")
    for off in range(8):
        ld = V + (-V) % 8 + (off % 3) * 8 + off      # rows of one call at different places too
        buf = torch.full((off + M * ld,), float("nan"), dtype=dtype, device="cuda")
        y = buf[off:off + M * ld].view(M, ld)[:, :V]
        y.copy_(x)
        _same(binding.spec_sample(y, u, T), want, off)
        _same(binding.spec_sample(y, u, T, None, None, zero), want, (off, "min_p 0"))
        greedy = binding.spec_sample(y, u, zero)
        assert greedy[0].tolist() == x.float().cpu().numpy().argmax(1).tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [32003, 100003])
def test_tokens_of_little_mass(dtype, V):
    """The token is the 64-bit one up to the mass by which sums may be off: a weight to
    2^-36 of itself and 2^-44 of the largest, both twice (the draw's border and the
    kept mass follow the same sums)."""
    M = 32
    x, u, T = _rows(V, M, dtype, 5)
    tok, prob = (t.cpu().numpy() for t in binding.spec_sample(x, u, T))
    l, us, ts = x.float().cpu().numpy().astype(np.float64), u.cpu().numpy().astype(np.float64), T.cpu().numpy().astype(np.float64)
    for i in range(M):
        w = np.exp((l[i] - l[i].max()) / ts[i])
        cum = np.cumsum(w)
        slack = 2.0 * (cum[-1] * 2.0 ** -36 + V * 2.0 ** -44)
        t = min(us[i], 1.0) * cum[-1]
        assert cum[tok[i]] > t - slack and (tok[i] == 0 or cum[tok[i] - 1] <= t + slack)
        assert abs(prob[i] - w[tok[i]] / cum[-1]) <= 2.0 ** -21 * w[tok[i]] / cum[-1]


@pytest.mark.parametrize("V", [32003, 50001])
def test_drafts_beside_a_token_alone(V):
    """Four rows of a sequence's step, and the same rows as steps without drafts."""
    k = 3
    x, u, T = _rows(V, k + 1, torch.float32, 3)
    d = torch.zeros((1, k), dtype=torch.int32, device="cuda")
    alone = [binding.spec_accept_sampled(x[j:j + 1].clone(), d[:, :0].contiguous(), u[j:j + 1].clone(), T[j:j + 1].clone())
             for j in range(k + 1)]
    for j in range(k):
        d[0, j] = alone[j][0][0, 0]
    out, n, prob = binding.spec_accept_sampled(x, d, u, T)
    assert n.item() == k + 1
    assert torch.equal(out[0], torch.cat([a[0][0] for a in alone]))
    assert torch.equal(prob[0], torch.cat([a[2][0] for a in alone]))
