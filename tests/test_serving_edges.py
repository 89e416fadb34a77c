"""Calls of the serving operators that their documentation allows and that ordinary use seldom makes: odd strides, shared and
overlapping tensors, infinities, numbers that do not fit."""
import ctypes
import importlib.util
import math
import os
import re
import shutil

import pytest
import torch

from tests import serving_reference as ref
from tests.test_serving import BF16, F32, HALF, filled, ints, normal, rope_bound
from tests.test_serving_many import launches, wide


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


# --------------------------------------------------------------------------------- attention

@pytest.mark.gpu
@pytest.mark.parametrize("below", [26.3, 31.0])
@pytest.mark.parametrize("dtype,d,new,kernel", [(BF16, 64, 1, "cache4_attn"), (BF16, 128, 3, "cache4_attn"), (BF16, 256, 1, "cache4_attn"),
                                                (BF16, 64, 80, "cache4_tc"), (BF16, 128, 70, "cache4_tc"), (F32, 96, 1, "cache4_attn_simt")])
def test_a_tail_of_small_weights_counts(s2, dtype, d, new, kernel, below):
    """Every 32nd key is far above the others and has v = 0, so that the output is all made of weights 2^-below of the largest.
    A weight may be off by half a step of fp16 (2^-11 of it) and, subnormal, by 2^-40 of the largest with few rows, 2^-33 with many."""
    L, H, P, Hq = 4000, 1, 64, 2
    a = math.sqrt(below * math.log(2) / (d * d ** -0.5))
    k, v = torch.full((L, H, d), 0.4 / below * a, device="cuda"), 1 + 0.1 * normal(1, L, H, d)   # (0.4: no whole power of two)
    k[::32], v[::32] = (1 + 0.4 / below) * a, 0.0
    k, v = k.to(dtype), v.to(dtype)
    q = torch.full((new, Hq, d), a, device="cuda").to(dtype)
    cache = s2.cache4(L // P + 1, P, H, d)
    s2.cache4_append(k, v, cache, torch.arange(L, dtype=torch.int32, device="cuda"))
    table = torch.arange(L // P + 1, device="cuda", dtype=torch.int32).view(1, -1)
    (o, lse), n = launches(s2, kernel, lambda: s2.cache4_attention(q, cache, wide(table), ints([L]), ints([0, new]), new, return_lse=True))
    assert n == 1
    kd, vd = ref.quantised(k)[0], ref.quantised(v)[0]
    want, wl, pv = ref.attention(q, kd, vd, [L - (new - 1 - i) for i in range(new)], d ** -0.5)
    score = (q.double().abs().sum(-1) * kd.abs().amax() * d ** -0.5).amax()
    # scores: k in fp16 with many rows (half a step 2^-11), fp32 sums
    err = score * (2.0 ** -11 if kernel == "cache4_tc" else 2.0 ** -20)
    most = math.exp(score - wl.min())                       # the largest weight
    floor = {"cache4_attn": 2.0 ** -40, "cache4_tc": 2.0 ** -33, "cache4_attn_simt": 0.0}[kernel]
    bound = HALF[dtype] * want.abs() * 1.01 + (3 * 2.0 ** -11 + 2 * err) * pv + floor * most * vd.abs().sum(0).amax()
    assert (want >= 2.0 ** -30).all() and ((o.double() - want).abs() <= bound).all()
    assert ((lse.T.double() - wl).abs() <= err + 2.0 ** -20 * (4 + wl.abs())).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,new,kernel", [(BF16, 64, 1, "cache4_attn"), (BF16, 128, 3, "cache4_attn"), (BF16, 64, 70, "cache4_tc"),
                                                (BF16, 128, 64, "cache4_tc"), (F32, 96, 2, "cache4_attn_simt"), (BF16, 32, 2, "cache4_attn_simt")])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("inf", [math.inf, -math.inf])
def test_an_infinite_query_spoils_its_row(s2, inf, sign, dtype, d, new, kernel):
    """Every score of such a row is infinite, here of one sign: the softmax of the row is NaN where it sees a key, whichever kernel
    runs, and 0 where it sees none; other rows are as they were."""
    L, H, P, Hq = 66, 1, 16, 2
    k, v = sign * (1 + 0.1 * normal(1, L, H, d).abs()).to(dtype), normal(2, L, H, d).to(dtype)
    q = normal(3, new, Hq, d).to(dtype)
    cache = s2.cache4(L // P + 1, P, H, d)
    s2.cache4_append(k, v, cache, torch.arange(L, dtype=torch.int32, device="cuda"))
    table = wide(torch.arange(L // P + 1, device="cuda", dtype=torch.int32).view(1, -1))
    for held in (L, new, 1, 0):
        args = (cache, table, ints([held]), ints([0, new]), new)
        good, good_l = s2.cache4_attention(q, *args, return_lse=True)
        bad, row = q.clone(), new - 1
        bad[row, 1, 7] = inf
        if new > 1:
            bad[0, 0] = inf                     # sees held - (new - 1) keys: none, one or more
        (o, lse), n = launches(s2, kernel, lambda: s2.cache4_attention(bad, *args, return_lse=True))
        assert n == 1
        spoilt = {(row, 1): held} | ({(0, 0): max(0, held - (new - 1))} if new > 1 else {})
        for (i, h), keys in spoilt.items():
            if keys:
                assert o[i, h].isnan().all() and lse[h, i].isnan()
            else:
                assert (o[i, h] == 0).all() and lse[h, i] == -math.inf
            o[i, h], lse[h, i] = good[i, h], good_l[h, i]
        assert torch.equal(o, good) and torch.equal(lse, good_l)


# --------------------------------------------------------------------------------- rope and autograd

def tangents(s2, q, k, t, u, pos, f):
    """rope's forward-mode derivatives: of q and k together, of q alone, without k, and of the backward pass."""
    from torch.autograd import forward_ad as fw
    with fw.dual_level():
        out = [fw.unpack_dual(x).tangent for x in s2.rope(fw.make_dual(q, t), fw.make_dual(k, u), pos, f, layout="half", mscale=1.5)]
        out += [fw.unpack_dual(x).tangent for x in s2.rope(fw.make_dual(q, t), k, pos, f, layout="half", mscale=1.5)]
        out.append(fw.unpack_dual(s2.rope(fw.make_dual(q, t), None, pos, f, layout="half", mscale=1.5)[0]).tangent)
        x = fw.make_dual(q.clone().requires_grad_(), t)
        (g,) = torch.autograd.grad(s2.rope(x, None, pos, f, layout="half", mscale=1.5)[0].square().sum() / 2, x)
        out.append(fw.unpack_dual(g).tangent)        # R^T R t
        with pytest.raises(ValueError, match="no gradient"):
            s2.rope(fw.make_dual(q, t), None, pos, f, in_place=True)
        assert all(fw.unpack_dual(x).tangent is None for x in s2.rope(q.detach(), k.detach(), pos, f))
    return out


def check_tangents(s2, q, k, t, u, pos, f, theta):
    out = tangents(s2, q, k, t, u, pos, f)
    turn = lambda x: ref.rope(x, pos.view(1, -1), theta, "half", 1.5)  # noqa: E731
    assert not out[3].any()
    twice = t.double().clone()
    twice[..., :2 * theta.numel()] *= 1.5 ** 2
    for got, want in ((out[0], turn(t)), (out[1], turn(u)), (out[2], turn(t)), (out[4], turn(t)), (out[5], twice)):
        assert (got.double() - want).abs().max() <= 2.0 ** -20 * want.abs().max()      # a few roundings of fp32


def test_rope_carries_tangents(s2, monkeypatch):
    """Forward-mode derivatives are not lost on the way to the launch (a plain form stands in for it here)."""
    def plain(q, k, pos, f, layout, mscale, inverse, in_place):
        return tuple(None if x is None else ref.rope(x, pos.view(1, -1), 2 * math.pi * f, layout, mscale, inverse).to(x.dtype) for x in (q, k))

    monkeypatch.setattr(s2, "_rope_launch", plain)
    q, k, t, u = (torch.randn(1, 5, 2, 16, generator=torch.Generator().manual_seed(s)) for s in range(4))
    check_tangents(s2, q, k, t, u, torch.arange(5), s2.rope_freqs(12, device="cpu"), ref.freqs(12))


@pytest.mark.gpu
def test_rope_carries_tangents_on_the_gpu(s2):
    q, k, t, u = (normal(s, 1, 5, 2, 16) for s in range(4))
    check_tangents(s2, q, k, t, u, torch.arange(5, device="cuda"), s2.rope_freqs(12), ref.freqs(12))


def test_what_is_overwritten_says_so(s2, monkeypatch):
    """The version counters that autograd checks saved tensors by move with every call that writes a caller's tensor (the launch
    itself is left out here)."""
    monkeypatch.setattr(s2, "_call", lambda *a: None)
    x = torch.zeros(2, 4, 64)
    i, cache, ws = torch.zeros(2, dtype=torch.int32), s2.cache4(2, 16, 4, 64, device="cpu"), torch.zeros(8, dtype=torch.uint8)
    table, cu = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q, k, out = x.clone(), x.clone(), x.clone()
    f = s2.rope_freqs(64, device="cpu")
    s2.rope(q, k, i, f, in_place=True)
    assert (q._version, k._version) == (1, 1)
    s2.rope(q, None, i, f, in_place=True)
    s2.rope(q, k, i, f)
    assert (q._version, k._version) == (2, 1)
    s2.cache4_append(q, k, cache, i)
    s2.page_plan(i, i, i, i[:1], table, 16, 4)
    s2.cache4_attention(x, cache, table, i, cu, 1, ws=ws, out=out)
    s2.cache4_attention(x, cache, table, i, cu, 1, ws=ws)
    assert (cache._version, table._version, out._version) == (1, 1, 1)
    assert (x._version, i._version, q._version, k._version) == (0, 0, 2, 1)
    with torch.inference_mode():
        y = torch.zeros(2, 4, 64)
        s2.rope(y, None, i, f, in_place=True)
    s2.rope(y, None, i, f, in_place=True)               # (tensors of inference mode have no counter)


@pytest.mark.gpu
def test_a_backward_over_what_was_overwritten_says_so(s2):
    f, pos = s2.rope_freqs(64), ints([0, 1])
    cache, table, _ = filled(s2, [40], 16, 2, 64, 1)
    args = (cache, table, ints([40]), ints([0, 2]), 2)
    w = torch.ones(2, 4, 64, device="cuda", requires_grad=True)

    def over(write):
        x = normal(1, 2, 4, 64)
        y = (x * w).sum()                                # saves x
        write(x)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()

    over(lambda x: s2.rope(x, None, pos, f, in_place=True))
    over(lambda x: s2.cache4_attention(normal(2, 2, 4, 64), *args, out=x))
    over(lambda x: s2.cache4_attention(normal(2, 2, 4, 128)[..., 1:65], *args, out=x))    # rows off 16 bytes: the Python path
    was = cache._version, table._version
    s2.cache4_append(normal(3, 1, 2, 64), normal(4, 1, 2, 64), cache, ints([5]))
    s2.page_plan(ints([0]), ints([1]), ints([0]), ints([1]), table, 16, 1)
    assert (cache._version, table._version) == (was[0] + 1, was[1] + 1)
    with torch.inference_mode():
        x = normal(1, 2, 4, 64)
    s2.rope(x, None, pos, f, in_place=True)
    s2.cache4_attention(normal(2, 2, 4, 64), *args, out=x)


def addresses(t):
    at = torch.full(t.shape, t.data_ptr() // t.element_size())
    for i, (n, s) in enumerate(zip(t.shape, t.stride())):
        at += (s * torch.arange(n)).view([-1 if i == j else 1 for j in range(t.dim())])
    return set(at.flatten().tolist())


def test_rope_in_place_refuses_what_would_turn_twice(s2, monkeypatch):
    """q and k that share an element would both write it. Rows that only interleave, as those of one projection do, are taken."""
    monkeypatch.setattr(s2, "_call", lambda *a: None)
    f, pos, buf = s2.rope_freqs(4, device="cpu"), torch.arange(64), torch.zeros(4000)
    g = torch.Generator().manual_seed(0)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    met = 0
    for _ in range(600):
        B, T, d, heads = pick(1, 3), pick(1, 5), 4 * pick(1, 2), (pick(1, 4), pick(1, 4))
        hs = d + 4 * pick(0, 3)
        ts = 4 * hs + 4 * pick(0, 20)
        bs = T * ts + 4 * pick(0, 9)
        if pick(0, 3) == 0:                                # head-major
            hs, ts = T * hs, hs
            bs = max(bs, 4 * hs)
        q, k = (buf.as_strided((B, T, h, d), (bs, ts, hs, 1), 4 * pick(0, 80)) for h in heads)
        if addresses(q) & addresses(k):
            met += 1
            with pytest.raises(ValueError, match="overlap"):
                s2.rope(q, k, pos[:T], f, in_place=True)
        else:
            s2.rope(q, k, pos[:T], f, in_place=True)
    assert 100 < met < 500
    x = torch.zeros(2, 3, 2, 8)
    for q, k in ((x, x), (x, x[:, :, :1]), (x[:, :, :2], x.view(2, 3, 2, 8)[:, :, 1:])):
        with pytest.raises(ValueError, match="overlap"):
            s2.rope(q, k, pos[:3], f, in_place=True)
    s2.rope(x[:, :, :1], x[:, :, 1:], pos[:3], f, in_place=True)
    s2.rope(x, x, pos[:3], f)                              # (outputs of their own)


# --------------------------------------------------------------------------------- what is built

def test_training_calls_do_without_the_compiled_serving_calls(s2, tmp_path):
    package = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "longlora_shifted_sparse_b200")
    for name in ("s2attn.py", "libs2attn.so"):
        shutil.copy(os.path.join(package, name), tmp_path / name)
    spec = importlib.util.spec_from_file_location("s2attn_alone", tmp_path / "s2attn.py")
    alone = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(alone)
    x, alone._stream_ptr = torch.zeros(1, 3, 2, 64), lambda device: 0
    with pytest.raises(alone.S2Error, match="invalid shape"):      # the library's own refusal of the group size
        alone.forward(x, x, x, 2, 1.0)
    with pytest.raises(ImportError, match="not built"):
        alone.cache4_append(x[0], x[0], x, x)


def test_the_library_is_built_without_torch(s2, monkeypatch):
    from longlora_shifted_sparse_b200 import build
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == build.LIB
    assert build.build_calls(force=True) is None       # and makes no attempt


def test_a_workspace_is_dense_bytes(s2, monkeypatch):
    """Its number of elements is taken for its size: a tensor that repeats its elements would be shorter than it says."""
    launched = []
    monkeypatch.setattr(s2, "_call", lambda *a: launched.append(a))
    i, cache, x = torch.zeros(1, dtype=torch.int32), s2.cache4(2, 16, 4, 64, device="cpu"), torch.zeros(1, 4, 64)
    size = s2.s2attn_cache4_workspace_bytes()
    attend = lambda ws: s2.cache4_attention(x, cache, i.view(1, 1), i, torch.zeros(2, dtype=torch.int32), 1, ws=ws)  # noqa: E731
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(size), torch.zeros(16, 2, dtype=torch.uint8)[:, 0], torch.zeros(size // 4, dtype=torch.int32)):
        with pytest.raises(ValueError, match="workspace"):
            attend(bad)
    assert not launched
    attend(s2.cache4_workspace("cpu"))
    assert len(launched) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("columns", [1, (2 ** 31 - 256) // 256])
def test_the_hint_may_be_anything(s2, columns):
    """The largest hint and the widest table together (their product with the requests and heads is beyond 64 bits)."""
    R, H, P, d = 4096, 32, 256, 256
    cache, one, _ = filled(s2, [40], P, H, d, 1)
    table = (one if columns == 1 else wide(one, columns)).expand(R, -1)
    q = normal(2, 5, H, d, dtype=BF16)
    cu = torch.full((R + 1,), 5, dtype=torch.int32, device="cuda")       # requests 0 and 7 have rows, the others none
    cu[0], cu[1:8] = 0, 2
    lens = torch.full((R,), 40, dtype=torch.int32, device="cuda")
    few = s2.cache4_attention(q, cache, one.expand(2, -1), ints([40, 40]), ints([0, 2, 5]), 3)
    assert few.isfinite().all()
    for said in (2 ** 31 - 1, 3):
        got = s2.cache4_attention(q, cache, table, lens, cu, said)
        # tiles of 8 or 16 rows: other orders of the same sums
        assert (got.float() - few.float()).abs().max() <= 2.0 ** -7 * few.float().abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,columns", [(BF16, 64, 0), (BF16, 256, 0), (BF16, 128, 1 << 15), (F32, 64, 0), (F32, 96, 1 << 15), (BF16, 32, 0)])
def test_a_request_whose_rows_leave_the_buffer(s2, dtype, d, columns):
    """page_plan leaves a request out whose tokens do not fit the step and still counts its rows: the attention writes none of them."""
    cache, table, _ = filled(s2, [90, 120, 40], 16, 2, d, 3)
    if columns:
        table = wide(table, columns)
    q, out = normal(1, 70, 4, d, dtype=dtype), torch.full((70, 4, d), 7.0, dtype=dtype, device="cuda")
    lens, cu = ints([90, 120, 40]), [0, 66, 66 + 40, 66 + 41]
    o = s2.cache4_attention(q, cache, table, lens, ints(cu), 66, out=out)
    want = s2.cache4_attention(q[:66], cache, table[:1], lens[:1], ints([0, 66]), 66)
    assert o.data_ptr() == out.data_ptr() and (o[66:] == 7.0).all()
    assert (o[:66].float() - want.float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()     # (other cuts of the same sums)


# --------------------------------------------------------------------------------- plans

@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [80, 148 * 256 + 1])
@pytest.mark.parametrize("page", [-1, -2 ** 27, -2 ** 28, 2 ** 27, 2 ** 28 + 3, 2 ** 31 - 1, -2 ** 31, 2 ** 27 - 1])
def test_plans_with_pages_that_are_none(s2, page, tokens):
    """A page number that no slot can have gives slots of -1, and not those of another page by its low bits: 2^28 pages of 16 tokens
    are 2^32 slots. The last page whose slots have numbers is taken."""
    P, n = 16, tokens // 2
    table = torch.zeros(2, -(-n // P) + 1, dtype=torch.int32, device="cuda")
    free = torch.arange(5, 5 + 2 * table.shape[1], dtype=torch.int32, device="cuda")
    free[-2] = page                                   # the first request's second page
    table[1, 0] = page                                # the second request's first, held already
    p = s2.page_plan(ints([0, 10]), ints([n, n - 10]), free, ints([free.numel()]), table, P, 2 * n)
    count = free.numel()
    slots = p.slots.tolist()
    last = page == 2 ** 27 - 1
    want = [(-1 if page_no == page and not last else page_no * P + i % P)
            for i in range(n) for page_no in [free[count - 1 - i // P].item()]] if n < 1000 else None
    assert slots[16:32] == ([page * P + i for i in range(16)] if last else [-1] * 16)
    assert slots[n:n + 6] == ([page * P + i for i in range(10, 16)] if last else [-1] * 6)
    if want:
        assert slots[:n] == want
    rest = p.slots[32:n].tolist() + p.slots[n + 6:2 * n - 10].tolist()
    assert all(5 * P <= x < (5 + count) * P for x in rest + slots[:16]) and len(set(rest)) == len(rest)
    assert p.left_out.tolist() == [0]


LARGE_SCORES = [(BF16, 64, 1, "cache4_attn"), (BF16, 128, 3, "cache4_attn"), (BF16, 256, 2, "cache4_attn"), (F32, 96, 2, "cache4_attn_simt"),
                (BF16, 64, 70, "cache4_tc"), (BF16, 128, 64, "cache4_tc")]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,new,kernel", LARGE_SCORES)
@pytest.mark.parametrize("power", [16, 20, 22, 23, 24, 25, 26, 27, 30, 60])
def test_large_scores(s2, power, dtype, d, new, kernel):
    """Scores of 2^power and some times it, where fp32 rounds to whole numbers and more: the softmax is the value of the largest."""
    L, H, P, Hq = 200, 1, 16, 2
    k, v = normal(power, L, H, d).to(dtype), normal(2, L, H, d).to(dtype)
    k[::2] = 0.0                                            # scores that are exactly 0
    cache = s2.cache4(L // P + 1, P, H, d)
    s2.cache4_append(k, v, cache, torch.arange(L, dtype=torch.int32, device="cuda"))
    table = wide(torch.arange(L // P + 1, device="cuda", dtype=torch.int32).view(1, -1))
    q = (normal(3, new, Hq, d) * 2.0 ** power).to(dtype)
    kd, vd = ref.quantised(k)[0], ref.quantised(v)[0]
    hidden = torch.arange(L, device="cuda") >= torch.tensor([L - (new - 1 - i) for i in range(new)], device="cuda").view(-1, 1, 1)
    for sign in (1, -1):
        sc = sign * d ** -0.5
        (o, lse), n = launches(s2, kernel, lambda: s2.cache4_attention(q, cache, table, ints([L]), ints([0, new]), new, scale=sc, return_lse=True))
        assert n == 1 and o.isfinite().all()
        score = sc * torch.einsum("nhd,ld->nhl", q.double(), kd[:, 0])
        top, at = score.masked_fill(hidden, -math.inf).topk(2, -1)
        # k in fp16 with many rows (half a step 2^-11 of each product), fp32 sums otherwise
        off = abs(sc) * torch.einsum("nhd,ld->nhl", q.double().abs(), kd[:, 0].abs()).amax(-1) * (2.0 ** -11 if kernel == "cache4_tc" else 2.0 ** -20)
        clear = top[..., 0] - top[..., 1] > 2 * off + 40   # the others' weights are below 2^-50 together
        assert clear.double().mean() > 0.5
        want = vd[at[..., 0], 0]
        assert ((o.double() - want).abs() <= (HALF[dtype] + 2.0 ** -10) * want.abs())[clear].all()       # v in fp16, and the output
        assert ((lse.T.double() - top[..., 0]).abs() <= off + 2.0 ** -20 * top[..., 0].abs() + 0.7).all()   # (two equal ones: log 2)


@pytest.mark.gpu
@pytest.mark.parametrize("first,then", [(0.0, 2.0 ** 24), (2.0 ** 24, 0.0), (2.0 ** 21, 2.0 ** 23), (-2.0 ** 25, 3.0), (2.0 ** 30, -2.0 ** 30)])
def test_many_rows_whose_scores_change_their_size(s2, first, then):
    """Scores of one size over the first tiles of keys, of another over the rest: a row's maximum passes from ordinary to large or stays
    large. The larger ones' value is the result."""
    L, H, P, d, new = 900, 1, 64, 64, 64
    k = torch.empty(L, H, d, device="cuda")
    k[:400], k[400:] = first / 2 ** 20, then / 2 ** 20
    v = torch.empty(L, H, d, device="cuda")
    v[:400], v[400:] = 1.0, -2.0
    cache = s2.cache4(L // P + 1, P, H, d)
    s2.cache4_append(k, v, cache, torch.arange(L, dtype=torch.int32, device="cuda"))
    table = wide(torch.arange(L // P + 1, device="cuda", dtype=torch.int32).view(1, -1))
    q = torch.full((new, 1, d), 2.0 ** 20, device="cuda", dtype=BF16)       # scores: 64 times first, or then
    o, lse = s2.cache4_attention(q, cache, table, ints([L]), ints([0, new]), new, scale=1.0, return_lse=True)
    assert (o == (1.0 if first > then else -2.0)).all()
    count = torch.arange(L - new + 1, L + 1, device="cuda").double() - 400 if then > first else torch.full((new,), 400.0, device="cuda")
    want = 64 * max(first, then) + count.log()
    assert ((lse[0].double() - want).abs() <= 2.0 ** -20 * (4 + want.abs())).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,new,kernel", LARGE_SCORES)
@pytest.mark.parametrize("qscale,scale", [(2.0 ** 117, None), (2.0 ** 105, 2.0 ** 11), (2.0 ** 112, -2.0), (2.0 ** -100, 2.0 ** 115), (2.0 ** -120, 2.0 ** 118)])
def test_scores_near_the_end_of_fp32(s2, qscale, scale, dtype, d, new, kernel):
    """Queries and scales of any size whose product with the keys is finite: no NaN, also for the scores that are 0 and where the
    scales alone, taken out of a row, would be infinite or 0."""
    L, H, P, Hq = 200, 1, 16, 2
    k, v = normal(1, L, H, d).to(dtype), normal(2, L, H, d).to(dtype)
    k[::2] = 0.0
    cache = s2.cache4(L // P + 1, P, H, d)
    s2.cache4_append(k, v, cache, torch.arange(L, dtype=torch.int32, device="cuda"))
    table = wide(torch.arange(L // P + 1, device="cuda", dtype=torch.int32).view(1, -1))
    q = (normal(3, new, Hq, d) * qscale).to(dtype)
    (o, lse), n = launches(s2, kernel, lambda: s2.cache4_attention(q, cache, table, ints([L]), ints([0, new]), new, scale=scale, return_lse=True))
    assert n == 1 and o.isfinite().all() and lse.isfinite().all()
    sc = d ** -0.5 if scale is None else scale
    kd, vd = ref.quantised(k)[0], ref.quantised(v)[0]
    keys = [L - (new - 1 - i) for i in range(new)]
    want, _, pv = ref.attention(q, kd, vd, keys, sc)
    score = sc * torch.einsum("nhd,ld->nhl", q.double(), kd[:, 0])
    hidden = torch.arange(L, device="cuda") >= torch.tensor(keys, device="cuda").view(-1, 1, 1)
    top = score.masked_fill(hidden, -math.inf).topk(2, -1).values
    off = abs(sc) * torch.einsum("nhd,ld->nhl", q.double().abs(), kd[:, 0].abs()).amax(-1) * (2.0 ** -11 if kernel == "cache4_tc" else 2.0 ** -20)
    # as in the tests above: one weight is 1, or all scores are known to their rounding
    clear = (top[..., 0] - top[..., 1] > 2 * off + 40) | (off < 0.1)
    assert clear.double().mean() > 0.5
    small = torch.where(off < 0.1, off, torch.zeros_like(off)).unsqueeze(-1)
    assert ((o.double() - want).abs() <= HALF[dtype] * 1.01 * want.abs() + (3 * 2.0 ** -11 + 4 * small) * pv)[clear].all()


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,Hq,H,d,P", [([1, 16, 100, 257], [1, 1, 1, 1], 4, 2, 64, 32), ([700, 33], [3, 1], 8, 2, 128, 16),
                                               ([5000], [1], 2, 2, 128, 64), ([900, 40], [2, 5], 4, 1, 256, 16)])
@pytest.mark.parametrize("shift", [0.0, 6.0])
def test_scores_and_small_weights_tightly(s2, lens, new, Hq, H, d, P, shift):
    """The few-row kernel's scores to fp32: products with the codes (0..15) are exact and so are those with the minima's two parts, so
    that a sum of them is off by 2^-22 of the sum of their sizes; keys far from zero make the minima's part the larger one. Weights
    are off by half a step of fp16, or by 2^-40 of the largest."""
    cache, table, kv = filled(s2, lens, P, H, d, 17)
    if shift:
        kv = []
        for r, n in enumerate(lens):
            k, v = normal(7 * r, n, H, d, dtype=BF16) + shift, normal(7 * r + 1, n, H, d, dtype=BF16)
            s2.cache4_append(k, v, cache, (table[r].repeat_interleave(P)[:n] * P + torch.arange(n, device="cuda") % P).int())
            kv.append((ref.quantised(k), ref.quantised(v)))
    cu = [sum(new[:r]) for r in range(len(new) + 1)]
    q = normal(3, cu[-1], Hq, d, dtype=BF16)
    (o, lse), n = launches(s2, "cache4_attn", lambda: s2.cache4_attention(q, cache, table, ints(lens), ints(cu), max(new), return_lse=True))
    assert n == 1
    sc = d ** -0.5
    for r, m in enumerate(new):
        rows = slice(cu[r], cu[r + 1])
        (k, ks), (v, _) = kv[r]
        keys = [max(0, lens[r] - (m - 1 - i)) for i in range(m)]
        want, wl, pv = ref.attention(q[rows], k, v, keys, sc)
        g = q[rows].double().abs().view(m, H, Hq // H, d // 32, 32).sum(-1)                # |q| over a group
        sizes = 15 * ks.double().amax(0) + k.unflatten(-1, (-1, 32)).abs().amax(-1).amax(0)  # codes' part, and the minima's
        err = sc * 2.0 ** -22 * (g * sizes.view(1, H, 1, -1)).sum(-1).reshape(m, Hq) + 2.0 ** -22 * wl.abs()
        live = torch.tensor([x > 0 for x in keys], device="cuda")
        assert ((lse[:, rows].T.double() - wl).abs() <= err + 2.0 ** -21)[live].all()
        bound = HALF[BF16] * 1.01 * want.abs() + (2 * 2.0 ** -11 + 2 * err.unsqueeze(-1) + 2.0 ** -18) * pv + 2.0 ** -40 * max(keys) * v.abs().max()
        assert ((o[rows].double() - want).abs() <= bound)[live].all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_at_every_scale(s2, dtype):
    """Values on, just below and just above the borders of any two codes, for every mantissa that a scale may have: the code is that of
    the exact division (the nearest, ties to even)."""
    S = 1024
    scale = (1024 + torch.arange(S, device="cuda")).double() * 2.0 ** -12          # fp16 numbers from 1/4 to 1/2
    border = (torch.arange(15, device="cuda").double() + 0.5).view(1, 15) * scale.view(S, 1)
    step = lambda x, way: torch.nextafter(x.float(), torch.full_like(x, way, dtype=F32)).double()  # noqa: E731
    if dtype is F32:
        sets = [border.float().double(), step(border, math.inf), step(border, 0.0), step(step(border, math.inf), math.inf)]
    else:
        sets = [border.to(BF16).double()]
    H = 2
    for x in sets:
        # a group: 0, fifteen scales (its maximum), and the fifteen values, twice; its minimum is 0, so that x - minimum is x
        top = (15 * scale).to(dtype).double().view(S, 1)
        rows = torch.cat((torch.zeros(S, 1, device="cuda"), top, x, x), -1).to(dtype).view(S, 1, 32).repeat(1, H, 1)
        cache, slots = s2.cache4(S // 16, 16, H, 32), torch.arange(S, dtype=torch.int32, device="cuda")
        s2.cache4_append(rows, rows, cache, slots)
        g = rows.float()
        held = ((g.amax(-1, keepdim=True) - 0) * (1 / 15)).half().double()
        if dtype is F32:
            assert torch.equal(held[:, 0, 0], scale)
        quotient = g.double() / held                       # 24 bits by 11: a border is hit exactly or missed by more than fp64 rounds
        want = quotient.round().clamp(0, 15) * held
        for got in s2.cache4_read(cache, slots, F32):
            assert torch.equal(got.double(), want)


# --------------------------------------------------------------------------------- rows that are copied first

def odd_rows():
    """[T, H, d] tensors that are dense, or all but, and yet not what the kernels read: an address off 16 bytes, and strides that are
    odd where there is one token, or one head."""
    flat = torch.arange(2 * 4 * 64 + 9, dtype=F32)
    yield flat[1:513].view(2, 4, 64)
    yield flat[:256].view(1, 4, 64).as_strided((1, 4, 64), (257, 64, 1))
    yield flat.as_strided((1, 1, 64), (65, 65, 1))


def test_dense_rows_off_their_alignment_are_copied(s2, monkeypatch):
    calls = []

    def launch(device, fn, *args):
        tensors, strides = args[:2], [list(a) for a in args if isinstance(a, ctypes.Array)]
        calls.append((fn, [p for p in tensors if p], strides))

    monkeypatch.setattr(s2, "_call", launch)
    ws = s2.cache4_workspace("cpu")
    for x in odd_rows():
        T, H, d = x.shape
        assert x.data_ptr() % 16 or x.stride(0) % 4 or x.stride(1) % 4
        i, cache = torch.zeros(T, dtype=torch.int32), s2.cache4(2, 16, H, d, device="cpu")
        s2.cache4_append(x, x, cache, i)
        s2.cache4_attention(x, cache, i[:1].view(1, 1), i[:1], i.new_zeros(2), 1, ws=ws)
        for fn, pointers, strides in calls:
            assert all(p % 16 == 0 for p in pointers) and all(s % 4 == 0 for row in strides for s in row)
        calls.clear()
        s2.rope(x, None, i, s2.rope_freqs(d, device="cpu"))
        assert all(p % 16 == 0 for p in calls[0][1])
        calls.clear()


@pytest.mark.gpu
def test_dense_rows_off_their_alignment(s2):
    f = s2.rope_freqs(64)
    for x in odd_rows():
        x = torch.arange(1024, dtype=F32, device="cuda").as_strided(x.shape, x.stride(), x.storage_offset())
        T, H, d = x.shape
        y, slots = x.clone(memory_format=torch.contiguous_format), torch.arange(T, dtype=torch.int32, device="cuda")
        one, two = s2.cache4(1, 16, H, d), s2.cache4(1, 16, H, d)
        s2.cache4_append(x, x, one, slots)
        s2.cache4_append(y, y, two, slots)
        assert torch.equal(one, two) and one.any()
        args = (one, ints([[0]]), ints([T]), ints([0, T]), T)
        for dtype in (F32, BF16):
            assert torch.equal(s2.cache4_attention(x.to(dtype) if dtype is BF16 else x, *args), s2.cache4_attention(y.to(dtype), *args))
        assert torch.equal(s2.rope(x, None, slots, f)[0], s2.rope(y, None, slots, f)[0])
