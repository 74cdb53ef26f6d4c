"""The limits that float rows of spec_attention_tree are held to on the GPU tell the kernel's sums from
cheaper ones: without a third part of the queries or of the weights, with the largest parts first, or with
one long sum in the tensor cores."""
import numpy as np
import pytest

from tests import float_rows_ref as fr


@pytest.mark.parametrize("keys,hd", sorted(fr.LIMITS))
@pytest.mark.parametrize("seed", [0, 1])
def test_limits(keys, hd, seed):
    rng = np.random.default_rng(100 * seed + hd)
    q = (rng.standard_normal((24, hd)) * 1.5).astype(np.float32)
    k, v = fr.bf16(rng.standard_normal((keys, hd))), fr.bf16(rng.standard_normal((keys, hd)))
    want = fr.exact(q, k, v)
    assert fr.off(fr.attention(q, k, v, rng), want) <= fr.LIMITS[keys, hd]
    for less in (dict(q_parts=2), dict(p_parts=2), dict(smallest_first=False)) + ((dict(run=1 << 30),) if keys > 64 else ()):
        assert fr.off(fr.attention(q, k, v, rng, **less), want) > fr.LIMITS[keys, hd], less
