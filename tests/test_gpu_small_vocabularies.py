"""Sampling and the sampled accept on small vocabularies, where a few dozen likely
tokens are a good part of the row: every row with settings of its own (filters left
out by some, greedy rows), against the 64-bit reference on one and the same tensor.
Probabilities to 2^-21 relative, as in the tests of the larger ones: a weight to
2^-24, the kept mass rounded to binary32 and one division are under four roundings
of 2^-24. The likely tokens lie at distinct places: a scatter to repeated places
leaves open which value lands, and with it what the right token is."""
import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding
from tests import sampling_ref as ref

pytestmark = pytest.mark.gpu
PTOL = 2.0 ** -21


def _rows(V, ld, M, dtype, spread, masked, g):
    x = torch.randn((M, ld), generator=g, device="cuda") * spread
    at = torch.rand((M, V), generator=g, device="cuda").argsort(1)[:, :48]
    up = torch.empty((M, 48), device="cuda").exponential_(0.35, generator=g) + 2.5 * spread
    x.scatter_(1, at, up)
    if masked:
        low = torch.full((M, 1), float("-inf"), device="cuda")
        low[1::2] = torch.finfo(dtype).min
        x = torch.where(torch.rand((M, ld), generator=g, device="cuda") < 0.7, low, x)
    return x.to(dtype)[:, :V]


def _settings(M, g, k, p, q):
    i = torch.arange(M, device="cuda")
    r = lambda: torch.rand(M, generator=g, device="cuda")
    T = torch.where(i % 5 == 4, 0.0, 0.6 + 0.6 * r()).contiguous()
    kk = torch.where(i % 3 == 2, 0, (k * (0.5 + 0.5 * r())).ceil().int()).to(torch.int32).contiguous() if k else None
    pp = torch.where(i % 4 == 1, 1.0, p - 0.1 * r()).contiguous() if p else None
    qq = torch.where(i % 2 == 1, 0.0, q * (0.5 + r())).contiguous() if q else None
    u = (torch.randint(0, 1 << 23, (M,), generator=g, device="cuda").float() + 0.5) / (1 << 23)
    return u, T, kk, pp, qq


def _np(*ts):
    return [None if t is None else t.cpu().numpy() for t in ts]


FILTERS = [(0, 0, 0), (20, 0, 0), (500, 0.95, 0), (0, 0.9, 0), (0, 0.5, 0.1), (5000, 0.8, 0.02), (1, 0, 0), (0, 0, 0.02)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,ld", [(500, 500), (504, 505), (730, 735), (1028, 1092), (1616, 1616), (3564, 3565)])
@pytest.mark.parametrize("masked", [False, True])
def test_small_rows_with_settings_of_their_own(dtype, V, ld, masked):
    g = torch.Generator(device="cuda").manual_seed(V)
    M = 60
    for n, (k, p, q) in enumerate(FILTERS):
        x = _rows(V, ld, M, dtype, 1.0 + 0.4 * n, masked, g)
        s = _settings(M, g, k, p, q)
        tok, prob = _np(*binding.spec_sample(x, s[0], *s[1:]))
        rt, rp, decided = ref.rows(x.float().cpu().numpy(), *_np(*s))
        assert decided.sum() >= M - 2
        assert np.array_equal(tok[decided], rt[decided]), (k, p, q)
        assert np.all(np.abs(prob - rp)[decided] <= PTOL * rp[decided]), (k, p, q)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,k,V,ld", [(1, 7, 573, 573), (8, 3, 517, 522), (5, 0, 1289, 1289), (3, 6, 2003, 2004)])
def test_small_accepts_with_settings_of_their_own(dtype, B, k, V, ld):
    g = torch.Generator(device="cuda").manual_seed(V)
    M = B * (k + 1)
    for n, (tk, p, q) in enumerate(FILTERS):
        x = _rows(V, ld, M, dtype, 1.0 + 0.4 * n, n % 2 == 1, g)
        s = _settings(M, g, tk, p, q)
        best = x.float().argmax(-1).view(B, k + 1)[:, :k]
        hit = torch.rand((B, k), generator=g, device="cuda") < 0.8
        d = torch.where(hit, best, torch.randint(0, V, (B, k), generator=g, device="cuda")).int().contiguous()
        out, ne, pr = _np(*binding.spec_accept_sampled(x, d, s[0], *s[1:]))
        rt, rp, decided = ref.rows(x.float().cpu().numpy(), *_np(*s))
        ro, rn, rpr = ref.accept(rt.reshape(B, -1), rp.reshape(B, -1), d.cpu().numpy())
        ok = decided.reshape(B, -1).all(1)
        assert (~ok).sum() <= 1
        assert np.array_equal(out[ok], ro[ok]) and np.array_equal(ne[ok], rn[ok])
        assert np.all(np.abs(pr - rpr)[ok] <= PTOL * rpr[ok])
