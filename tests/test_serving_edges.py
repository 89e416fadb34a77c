"""Calls of the serving operators that their documentation allows and that ordinary use seldom makes: odd strides, shared and
overlapping tensors, infinities, numbers that do not fit."""
import math

import pytest
import torch

from tests import serving_reference as ref
from tests.test_serving import BF16, F32, ints, normal, rope_bound


@pytest.fixture(scope="module")
def s2():
    from longlora_shifted_sparse_b200 import build
    build.build()
    from longlora_shifted_sparse_b200 import s2attn
    return s2attn


# --------------------------------------------------------------------------------- rope

@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("row", [65, 66, 68, 72])
def test_rope_rows_of_any_stride(s2, row, dtype, layout):
    """Rows [..., :64] of an aligned tensor, that lie an odd number of elements apart (or 2, 4, 8 more than a dense one's): no wider
    access than the rows' own alignment allows, in place or not, whichever of q and k has such rows."""
    T, Hq, Hkv, d = 41, 3, 2, 64
    pos = torch.arange(5, 5 + T, device="cuda")
    f, theta = s2.rope_freqs(d, pi_scale=2.0), ref.freqs(d, pi_scale=2.0)
    wide_q, wide_k = normal(1, 2, T, Hq, row, dtype=dtype), normal(2, 2, T, Hkv, row, dtype=dtype)
    q, k = wide_q[..., :d], wide_k[..., :d]
    assert q.data_ptr() % 16 == 0 and k.data_ptr() % 16 == 0 and q.stride() == (T * Hq * row, Hq * row, row, 1)
    for a, b in ((q, k), (q, k.contiguous()), (q.contiguous(), k), (q, None)):
        a2, b2 = s2.rope(a, b, pos, f, layout=layout, mscale=1.5)
        for x, got in ((a, a2), (b, b2)):
            if x is None:
                assert got is None
                continue
            want = ref.rope(x, pos.expand(2, T), theta, layout, 1.5)
            assert ((got.double() - want).abs() <= rope_bound(x, want, d, layout, 1.5)).all()
    rest = wide_q[..., d:].clone(), wide_k[..., d:].clone()
    q2, k2 = s2.rope(q, k, pos, f, layout=layout, mscale=1.5)
    s2.rope(q, k, pos, f, layout=layout, mscale=1.5, in_place=True)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    assert torch.equal(wide_q[..., d:], rest[0]) and torch.equal(wide_k[..., d:], rest[1])
    # a token of one head a row, and rows of which a part is turned
    y = normal(3, T, 1, row, dtype=dtype)[..., :d]
    part, theta = s2.rope_freqs(18), ref.freqs(18)
    want = ref.rope(y.unsqueeze(0), pos.view(1, T), theta, layout)[0]
    assert ((s2.rope(y, None, pos, part, layout=layout)[0].double() - want).abs() <= rope_bound(y, want, 18, layout, 1.0)).all()
