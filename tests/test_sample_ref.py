"""The 64-bit sampling reference against closed forms, and the host-side
refusals of the per-request entry points (no GPU)."""
import ctypes as C

import numpy as np
import pytest
import torch

from speculative_decoding_spec_gb300 import binding
from tests import sampling_ref as ref


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_spec_gb300 import build
    build.build()
    return binding.lib()


def test_frequencies_are_the_softmax():
    l = np.array([0.0, 1.0, -2.0, 1.0, 3.0])
    n = 20000
    got = np.bincount([ref.row(l, (i + 0.5) / n, 0.7)[0] for i in range(n)], minlength=5) / n
    w = np.exp(l / 0.7)
    # an inverse CDF on n equal steps is within one step of each probability
    assert np.abs(got - w / w.sum()).max() <= 1.0 / n


def test_filters_by_hand():
    l = np.log([0.1, 0.4, 0.2, 0.2, 0.1])
    assert [ref.row(l, u, k=2)[0] for u in (0.0, 0.6, 0.7, 0.99)] == [1, 1, 2, 2]      # the tie at 0.2: lower index
    assert {ref.row(l, u, p=0.5)[0] for u in np.linspace(0, 0.999, 50)} == {1, 2}      # 0.4 < 0.5, 0.6 reaches it
    assert {ref.row(l, u, p=0.0)[0] for u in np.linspace(0, 0.999, 50)} == {1}
    assert {ref.row(l, u, q=0.49)[0] for u in np.linspace(0, 0.999, 50)} == {1, 2, 3}  # at least 0.49 * 0.4
    assert ref.row(l, 0.3, T=0.0)[:2] == (1, 1.0)
    assert abs(ref.row(l, 0.3, k=2)[1] - 0.4 / 0.6) < 1e-12


def test_rows_without_a_distribution():
    inf = np.inf
    assert ref.row(np.array([-inf, -inf]), 0.5)[0] == -1
    assert ref.row(np.array([0.0, np.nan]), 0.5)[0] == -1
    assert ref.row(np.array([0.0, 1.0]), 0.5, T=-1.0)[0] == -1
    assert ref.row(np.array([0.0, inf, 3.0, inf]), 0.6)[0] == 3


def test_accept_walk():
    t = np.array([[5, 6, 7], [5, 6, 7], [-1, 6, 7], [5, -1, 7]])
    d = np.array([[5, 6], [5, 9], [1, 2], [5, 6]])
    out, n, _ = ref.accept(t, np.ones((4, 3)), d)
    assert n.tolist() == [3, 2, 0, 1]
    assert out.tolist() == [[5, 6, 7], [5, 6, -1], [-1, -1, -1], [5, -1, -1]]


def test_host_refusals(lib):
    E, U, CAP = binding.SPEC_EINVAL, binding.SPEC_EUNSUPPORTED, binding.SPEC_ECAPACITY
    s = binding.spec_sampling(uniform=256)       # never read: every call below is refused on the host
    none = binding.spec_sampling()
    p = 256
    sample = lambda dt=0, lg=p, ld=8, M=1, V=8, st=s, tok=p, ws=None, nws=0: lib.spec_sample(dt, lg, ld, M, V, C.byref(st), tok, p, ws, nws, None)
    assert sample(dt=2) == E and sample(lg=None) == E and sample(ld=7) == E and sample(M=0) == E
    assert sample(V=0) == E and sample(st=none) == E and sample(tok=None) == E
    assert lib.spec_sample(0, p, 8, 1, 8, None, p, p, None, 0, None) == E
    big = dict(M=64, V=1 << 18, ld=1 << 18)      # needs a workspace
    need = lib.spec_sample_workspace_bytes(64, 1 << 18)
    assert need > 0 and sample(**big) == CAP and sample(ws=p, nws=need - 1, **big) == CAP
    assert sample(ws=p + 8, nws=need, **big) == E
    assert lib.spec_sample_workspace_bytes(1, 4096) == 0 and lib.spec_sample_workspace_bytes(0, 8) == 0
    assert sample(V=(1 << 19) + 1, ld=1 << 22) == U and sample(M=(1 << 20) + 1) == U
    acc = lambda B=1, k=2, d=p, st=s, out=p, ne=p: lib.spec_accept_sampled(0, p, 8, B, k, 8, d, C.byref(st), out, ne,
                                                                           None, None, 0, None)
    assert acc(B=0) == E and acc(k=-1) == E and acc(d=None) == E and acc(st=none) == E
    assert acc(out=None) == E and acc(ne=None) == E and acc(k=1024) == U and acc(B=1 << 20) == U
    assert lib.spec_verify_sampled(None, 1, None, 0, None, C.byref(s), None, None, None, None, None) == E


def test_binding_refusals(lib):
    x, u = torch.zeros(2, 8), torch.zeros(2)
    with pytest.raises(binding.SpecError):
        binding.spec_sample(x, u)                # not on a GPU
    with pytest.raises(binding.SpecError):
        binding.spec_accept_sampled(x, torch.zeros(1, 1, dtype=torch.int64), u)


def test_lora_host_refusals(lib):
    E, U, CAP = binding.SPEC_EINVAL, binding.SPEC_EUNSUPPORTED, binding.SPEC_ECAPACITY
    p = 256                                       # never read: every call below is refused on the host
    w = binding.spec_matrix(1, p, None)

    def call(w=w, N=64, K=64, x=p, M=4, gain=None, dt=1, n=2, r=8, a=p, b=p, ids=p, y=p, ws=p, nws=0):
        lo = binding.spec_lora(dt, n, r, a, b, None)
        return lib.spec_linear_lora(C.byref(w), N, K, x, M, gain, 1e-6, C.byref(lo), ids, y, ws, nws, None)
    assert call() == CAP and call(ws=None) == CAP  # a workspace too small, or none
    for kw in (dict(N=0), dict(K=0), dict(K=12), dict(x=None), dict(M=0), dict(M=65), dict(dt=2), dict(n=0), dict(r=0),
               dict(a=None), dict(b=None), dict(ids=None), dict(y=None), dict(x=260), dict(a=264), dict(b=258),
               dict(y=252), dict(gain=4), dict(ws=8)):
        assert call(**kw) == E, kw
    assert call(r=12) == U and call(r=136) == U
    assert lib.spec_linear_lora(C.byref(w), 64, 64, p, 4, None, 1e-6, None, p, p, p, 1 << 30, None) == E
    assert lib.spec_linear_lora_workspace_bytes(0, 64, 4, 8) == 0
    assert lib.spec_linear_lora_workspace_bytes(64, 64, 4, 0) == 0
