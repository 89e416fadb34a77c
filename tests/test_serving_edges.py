"""Calls of the serving operators that their documentation allows and that ordinary use seldom makes: odd strides, shared and
overlapping tensors, infinities, numbers that do not fit."""
import math
import os
import re

import pytest
import torch

from tests import serving_reference as ref
from tests.test_serving import BF16, F32, filled, ints, normal, rope_bound
from tests.test_serving_many import wide


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


# --------------------------------------------------------------------------------- block tables

def overlapping(table, R, step):
    """R rows of the table's width, each `step` elements behind the last, in the memory of one."""
    return table.as_strided((R, table.shape[1] - (R - 1) * step), (step, 1))


def test_plans_refuse_tables_whose_rows_overlap(s2):
    i, table = torch.zeros(4, dtype=torch.int32), torch.zeros(1, 9, dtype=torch.int32)
    for bad in (table.expand(4, 9), overlapping(table, 4, 1), table[:, :1].expand(4, 1)):
        with pytest.raises(ValueError, match="overlap"):
            s2.page_plan(i, i, i, i[:1], bad, 16, 4)


def test_one_row_of_pages_for_all_requests_is_accepted(s2):
    # (the page size is refused last of the shape's checks)
    from tests.test_serving_abi import attn
    assert attn(s2, ts=0, p=20) == s2.S2_ERR_ARG and attn(s2, ts=2, p=20) == s2.S2_ERR_SHAPE and attn(s2, ts=-4, p=20) == s2.S2_ERR_SHAPE


@pytest.mark.gpu
def test_plans_refuse_tables_whose_rows_overlap_on_the_gpu(s2):
    n, free, table = ints([20] * 4), ints(list(range(50))), torch.full((1, 9), 77, dtype=torch.int32, device="cuda")
    for bad in (table.expand(4, 9), overlapping(table, 4, 1), table[:, :1].expand(4, 1)):
        with pytest.raises(ValueError, match="overlap"):
            s2.page_plan(ints([0] * 4), n, free, ints([50]), bad, 16, 80)
    assert (table == 77).all()
    alone = table.expand(3, 9)[1:2]                  # one row: its stride of 0 says nothing
    s2.page_plan(ints([0]), ints([20]), free, ints([50]), alone, 16, 20)
    assert table[0, :3].tolist() == [49, 48, 77]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,new", [(BF16, 128, 1), (BF16, 64, 70), (F32, 96, 2), (BF16, 256, 5)])
@pytest.mark.parametrize("R", [3, 40])
def test_requests_that_share_pages(s2, R, dtype, d, new):
    """One row of pages expanded over requests, and rows that overlap, give what a table with a row for each gives; on both paths of
    the call, over every kernel. The memory behind the row is no table: page numbers there would give NaN."""
    L, H, P = 300, 2, 16
    cache, one, _ = filled(s2, [L], P, H, d, 4)
    room = torch.full((8, one.shape[1]), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    room[0] = one[0]
    g = torch.Generator().manual_seed(R)
    lens = ints(torch.randint(new, L + 1, (R,), generator=g).tolist())
    q, cu = normal(3, R * new, 4, d, dtype=dtype), ints([r * new for r in range(R + 1)])
    for columns in (one.shape[1], 1 << 14):
        row = wide(room[:1], columns) if columns > one.shape[1] else room[:1]
        want = s2.cache4_attention(q, cache, row.repeat(R, 1), lens, cu, new, return_lse=True)
        assert want[0].isfinite().all()
        for q2 in (q, torch.cat((q, q), -1)[..., 4:4 + d].copy_(q)):   # the second: rows off 16 bytes, for the Python path
            got = s2.cache4_attention(q2, cache, row.expand(R, -1), lens, cu, new, return_lse=True)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if R == 3:   # each request's pages begin one page behind the last one's
        windows = overlapping(one, 3, 1)
        seen = lens.clamp(max=windows.shape[1] * P)
        args = (seen, cu, new)
        assert torch.equal(s2.cache4_attention(q, cache, windows, *args), s2.cache4_attention(q, cache, windows.clone().contiguous(), *args))


# --------------------------------------------------------------------------------- kernels' sources

def test_waits_for_own_copies_are_followed_by_a_barrier():
    """A thread's wait for its asynchronous copies says nothing of other threads' copies, nor does a vote: a barrier of the warp or
    block stands between the wait and whatever the kernel does next with shared memory (or the function ends)."""
    root = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "longlora_shifted_sparse_b200", "csrc")
    waits = 0
    for name in ("cache4_attn.cu", "cache4_tc.cu", "cache4_simt.cu"):
        with open(os.path.join(root, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"(cp_async_wait_all\(\);|cp_async_wait<[^>]*>\(\);|\"cp\.async\.wait_all;\")", text):
            waits += 1
            rest = text[m.end():]
            barrier = re.search(r"__syncwarp\(\)|__syncthreads\(\)|\n}", rest)
            between = rest[:barrier.start()]
            # sums over lanes into places of their own (the few-row kernel's maxima and sums) read nothing that was copied
            assert not re.search(r"ld_shared|load_words|__all_sync|__any_sync|copy\(|issue\(", between), (name, between)
    assert waits == 5
