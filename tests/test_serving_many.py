"""The serving operators where their other kernels take over: many query rows of a kv head over the 4-bit cache (tiles of 256
rows), large page plans, caches beyond 4 GB, the limits of the cache's numbers, captured calls and expired waits."""
import math

import pytest
import torch

from tests import serving_reference as ref
from tests.test_serving import BF16, F32, HALF, check_attention, filled, ints, normal, plan_both, rope_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def s2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from longlora_shifted_sparse_b200 import s2attn
    return s2attn


def launches(s2, name, call):
    """What call() returns, and how often it launched the kernel `name`."""
    s2.check(s2.s2attn_profile_enable(1))
    out = call()
    n = {k: v[0] for k, v in ((s2.s2attn_profile_query(i)[0], s2.s2attn_profile_query(i)[1:])
                              for i in range(s2.s2attn_profile_num_kernels()))}
    s2.check(s2.s2attn_profile_enable(0))
    return out, n[name]


def wide(table, columns=1 << 14):
    """The same table with room for many more pages, as a server keeps it: a call may then be a large one."""
    t = torch.full((table.shape[0], columns), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    t[:, :table.shape[1]] = table
    return t


def check_rows(o, lse, q, k, v, keys, sc):
    """One request's rows against the 64-bit form. k and v are held in fp16 (half a step 2^-11 of the value), and so is P, whose
    sum is at least 2^3 (subnormal ones are off by 2^-25); sums and maxima are fp32."""
    want, wl, pv = ref.attention(q, k, v, keys, sc)
    n, Hq, d = q.shape
    H = k.shape[1]
    big = torch.einsum("nhgd,lhd->nhgl", q.double().abs().view(n, H, Hq // H, d), k.abs()).amax(-1).reshape(n, Hq) if k.shape[0] else 0.0
    err = abs(sc) * big * (2.0 ** -11 + 2.0 ** -18)
    dead = torch.tensor([x == 0 for x in keys], device="cuda")
    got = lse.T.double()
    assert (got[dead] == -math.inf).all() and (o[dead] == 0).all()
    live = ~dead
    if not live.any():
        return
    assert ((got - wl).abs()[live] <= (err + 2.0 ** -20 * (4 + wl.abs()))[live]).all()
    vmax = float(v.abs().max())
    bound = HALF[BF16] * want.abs() * 1.01 + (4 * 2.0 ** -11 + 2 * err.unsqueeze(-1)) * pv + max(keys) * 2.0 ** -28 * vmax
    assert ((o.double() - want).abs() <= bound)[live].all()


def check_many(s2, lens, new, Hq, H, d, P, seed=0, scale=None, qscale=1.0):
    cache, table, kv = filled(s2, lens, P, H, d, seed)
    cu = [sum(new[:r]) for r in range(len(new) + 1)]
    q = normal(seed + 99, cu[-1] + 3, Hq, d, dtype=BF16) * qscale
    out = torch.full_like(q, 7.0)
    ws = s2.cache4_workspace()
    args = (q, cache, wide(table), ints(lens), ints(cu), max(new))
    (o, lse), n = launches(s2, "cache4_tc", lambda: s2.cache4_attention(*args, scale=scale, ws=ws, out=out, return_lse=True))
    assert n == 1 and s2.device_status(ws) == s2.S2_OK
    again = s2.cache4_attention(*args, scale=scale, ws=ws)
    assert (o[cu[-1]:] == 7.0).all()
    for r, n in enumerate(new):
        if n:
            rows = slice(cu[r], cu[r + 1])
            check_rows(o[rows], lse[:, rows], q[rows], kv[r][0][0], kv[r][1][0], [max(0, lens[r] - (n - 1 - i)) for i in range(n)],
                       d ** -0.5 if scale is None else scale)
            assert torch.equal(again[rows], o[rows])                    # the same bits each time


@pytest.mark.parametrize("lens,new", [
    ([64], [64]), ([100, 700, 3000], [64, 128, 129]), ([5, 0, 1], [70, 1, 300]), ([127, 128, 129, 257], [127, 128, 2, 257]),
    ([1, 1, 1], [1, 64, 1]), ([40, 9000], [0, 65])])
@pytest.mark.parametrize("Hq,H,d", [(1, 1, 128), (2, 2, 64), (6, 2, 128), (16, 1, 64), (8, 4, 128)])
def test_many_rows(s2, lens, new, Hq, H, d):
    check_many(s2, lens, new, Hq, H, d, 32, seed=len(lens) + Hq)


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_many_rows_pages(s2, P):
    check_many(s2, [333, P, P + 1, 1500], [100, P, 77, 65], 4, 2, 128, P, seed=P)


def test_many_rows_many_requests(s2):
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 400, (120,), generator=g).tolist()
    new = [min(n, x) for n, x in zip(lens, torch.randint(0, 90, (120,), generator=g).tolist())]
    new[7] = lens[7] = 200
    check_many(s2, lens, new, 4, 2, 64, 16, seed=31)


def test_many_rows_of_a_wide_group(s2):
    check_many(s2, [50, 300], [3, 2], 300, 1, 64, 16, seed=4)           # more heads than a tile has rows


@pytest.mark.parametrize("d,dtype", [(96, F32), (128, F32), (256, F32), (160, BF16), (32, BF16)])
def test_long_rows_of_the_other_types(s2, d, dtype):
    """Head dims and types that take no tensor instructions, split over their keys; no key at all among them."""
    check_attention(s2, [5000, 0, 127, 129], [1, 0, 2, 1], 4, 2, d, 64, dtype, seed=d)
    check_attention(s2, [20000], [1], 1, 1, d, 16, dtype, seed=d + 1)


@pytest.mark.parametrize("scale,qscale", [(-0.1, 1.0), (0.0, 1.0), (1e-5, 3e4), (1e19, 1e-20), (0.2, 3.0)])
def test_many_rows_scales(s2, scale, qscale):
    check_many(s2, [300, 1000], [80, 64], 4, 2, 128, 64, seed=9, scale=scale, qscale=qscale)


@pytest.mark.parametrize("slope", [0.02, 0.3, 3.0, -3.0])
@pytest.mark.parametrize("n", [1, 64])
def test_scores_that_rise_and_fall(s2, slope, n):
    """The maximum moves again and again (or never): with one token, and with many."""
    L, H, d, P = 1200, 1, 128, 64
    cache = s2.cache4(L // P + 1, P, H, d)
    k = (torch.arange(L, device="cuda", dtype=F32).view(L, 1, 1) * slope / 10).expand(L, H, d) / 12 + 0.1 * normal(1, L, H, d)
    k, v = k.to(BF16), normal(2, L, H, d, dtype=BF16)
    s2.cache4_append(k, v, cache, torch.arange(L, dtype=torch.int32, device="cuda"))
    table = wide(torch.arange(L // P + 1, device="cuda", dtype=torch.int32).view(1, -1))
    q = (torch.ones(n, 1, d, device="cuda") + 0.1 * normal(3, n, 1, d)).to(BF16)
    o, lse = s2.cache4_attention(q, cache, table, ints([L]), ints([0, n]), n, return_lse=True)
    check_rows(o, lse, q, ref.quantised(k)[0], ref.quantised(v)[0], [L - (n - 1 - i) for i in range(n)], d ** -0.5)


def test_many_rows_poison_and_bad_pages(s2):
    H, P, L, n, d = 2, 16, 400, 70, 64
    cache, table, _ = filled(s2, [L, 90], P, H, d, 1)
    q = normal(5, 2 * n, 4, d, dtype=BF16)
    lens, cu = ints([L, 90]), ints([0, n, 2 * n])

    def attend(t):
        return s2.cache4_attention(q, cache, wide(t), lens, cu, n)

    good = attend(table)
    assert good.isfinite().all()
    k, v = normal(6, 1, H, d, dtype=BF16), normal(7, 1, H, d, dtype=BF16)
    place = L - n + 30                                       # seen by rows 30.. of the first request
    was = cache.clone()
    for bad, x in ((math.nan, k), (math.inf, v)):
        y = x.clone()
        y[0, 1, 5] = bad
        s2.cache4_append(y if x is k else k, y if x is v else v, cache, table[0, place // P].view(1) * P + place % P)
        o = attend(table)
        assert o[30:n, 2:].isnan().all() and o[30:n, :2].isfinite().all()
        assert torch.equal(o[:30], good[:30]) and torch.equal(o[n:], good[n:])
    cache.copy_(was)
    for page in (-1, cache.shape[0]):
        t = table.clone()
        t[1, 2] = page                                       # keys 32.. of 90: rows that see key 32 or more
        o = attend(t)
        first = 32 - (90 - n)
        assert o[n + first:].isnan().all() and torch.equal(o[:n + first], good[:n + first])
    q[3, 1, 0] = math.nan                                    # a query spoils its own row alone
    o = attend(table)
    assert o[3, 1].isnan().all()
    o[3, 1] = good[3, 1]
    assert torch.equal(o, good)


@pytest.mark.parametrize("new", [1, 64])
def test_beyond_four_gigabytes(s2, new):
    H, P, d, L = 2, 64, 128, 150
    pages = (5 << 30) // (P // 16 * H * 20 * d)
    cache = s2.cache4(pages, P, H, d)
    assert cache.numel() > 1 << 32
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    k, v = normal(1, L, H, d, dtype=BF16), normal(2, L, H, d, dtype=BF16)
    slots = (table[0].long().repeat_interleave(P) * P + torch.arange(P, device="cuda").repeat(3))[:L].int()
    s2.cache4_append(k, v, cache, slots)
    kq, vq = ref.quantised(k)[0], ref.quantised(v)[0]
    for x, y in zip((kq, vq), s2.cache4_read(cache, slots, F32)):
        assert (x - y.double()).abs().max() <= 2.0 ** -21
    q = normal(3, new, 4, d, dtype=BF16)
    o, lse = s2.cache4_attention(q, cache, wide(table), ints([L]), ints([0, new]), new, return_lse=True)
    check_rows(o, lse, q, kq, vq, [L - (new - 1 - i) for i in range(new)], d ** -0.5)


@pytest.mark.parametrize("new", [1, 64])
def test_the_largest_values_stay_finite(s2, new):
    """A group whose values span fp16: its top is held within what fp16 can round, so that readers need no wider numbers."""
    H, P, d, L = 1, 16, 64, 20
    cache = s2.cache4(2, P, H, d)
    v = normal(1, L, H, d)
    v[3, 0, 1], v[3, 0, 2], v[9, 0, 40] = 1e6, -1e6, 65504.0
    slots = torch.arange(L, dtype=torch.int32, device="cuda")
    s2.cache4_append(normal(2, L, H, d), v, cache, slots)
    held = s2.cache4_read(cache, slots, F32)[1]
    assert held.abs().max() < 65520 and held[3, 0, 1] >= 65000 and held[3, 0, 2] == -65504
    o = s2.cache4_attention(normal(3, new, 1, d, dtype=BF16), cache, wide(ints([[0, 1]])), ints([L]), ints([0, new]), new)
    assert o.isfinite().all()


def test_codes_at_borders(s2):
    """Values that lie on the borders of two codes, groups far from zero, narrow groups: the codes of the exact division."""
    H, d, P = 4, 64, 16
    g = torch.Generator().manual_seed(0)
    x = torch.randint(0, 31, (64, H, d), generator=g).float() * 0.5        # quotients at halves where the scale is 1
    x[..., 0], x[..., 1], x[..., 32], x[..., 33] = 0.0, 15.0, 0.0, 15.0
    x[16:32] = x[16:32] * 2.0 ** -9 + 3.0                                    # the minimum rounds, for the group's width
    x[32:48] = x[32:48] * 2.0 ** -20 + 1000.25                               # narrower than fp16's step there
    x[48:] = normal(1, 16, H, d).cpu() * torch.logspace(-7, 6, 16).view(16, 1, 1)
    for dtype in (F32, BF16):
        y = x.cuda().to(dtype)
        cache = s2.cache4(4, P, H, d)
        slots = torch.arange(64, dtype=torch.int32, device="cuda")
        s2.cache4_append(y, y, cache, slots)
        want = ref.quantised(y)[0]
        for got in s2.cache4_read(cache, slots, F32):
            assert ((got.double() - want).abs() <= 2.0 ** -23 * want.abs() + 1e-30).all()


@pytest.mark.parametrize("d,dtype", [(128, F32), (96, F32), (128, BF16)])
def test_codes_of_many_groups(s2, d, dtype):
    """Every scale, minimum and code of many groups: the values held are the format's, to the rounding of one product and sum."""
    T, H, P = 5000, 2, 64
    k, v = normal(1, T, H, d, dtype=dtype), normal(2, T, H, d, dtype=dtype) * torch.logspace(-3, 3, T, device="cuda").view(T, 1, 1).to(dtype)
    cache = s2.cache4(T // P + 1, P, H, d)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    s2.cache4_append(k, v, cache, slots)
    for x, got in zip((k, v), s2.cache4_read(cache, slots, F32)):
        want = ref.quantised(x)[0]
        assert ((got.double() - want).abs() <= 2.0 ** -23 * want.abs() + 1e-30).all()


@pytest.mark.parametrize("T_extra", [0, 1, 2, 3])
def test_large_plans(s2, T_extra):
    g = torch.Generator().manual_seed(3)
    R, P = 200, 32
    cached = torch.randint(0, 200, (R,), generator=g).tolist()
    new = torch.randint(0, 500, (R,), generator=g).tolist()
    new[5:9] = [0, 0, 1, 0]
    free = torch.randperm(6000, generator=g).tolist()
    table = torch.randint(0, 9000, (R, 23), generator=g).tolist()
    plan_both(s2, cached, new, free, len(free), table, P, sum(new) + T_extra)


def test_large_plan_with_unaligned_outputs(s2):
    R, P, n = 50, 16, 1000
    cached, new, free = ints([3] * R), ints([n] * R), torch.randperm(R * 70, device="cuda").int()
    count, table = ints([R * 70]), torch.zeros(R, 64, dtype=torch.int32, device="cuda")
    want = s2.page_plan(cached, new, free, count, table.clone(), P, R * n)
    T = R * n
    pos, slots, rest = (torch.full((T + 4,), 99, dtype=torch.int32, device="cuda") for _ in range(3))
    code = s2.s2attn_page_plan(cached.data_ptr(), new.data_ptr(), free.data_ptr(), count.data_ptr(), table.data_ptr(), rest.data_ptr(),
                               rest.data_ptr() + 400, pos.data_ptr() + 4, slots.data_ptr() + 8, rest.data_ptr() + 800, R, T, free.numel(),
                               64, 64, P, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    assert torch.equal(pos[1:T + 1], want.positions) and torch.equal(slots[2:T + 2], want.slots)
    assert pos[0] == 99 and (pos[T + 1:] == 99).all() and (slots[:2] == 99).all() and (slots[T + 2:] == 99).all()


def test_captured_chunks_and_two_streams(s2):
    """A chunk captured once and replayed over a longer context; two chunks at once, a workspace each."""
    lens, n, d, P = [900, 2000], 64, 64, 32
    cache, table, kv = filled(s2, lens, P, 2, d, 3)
    table, cu = wide(table), ints([0, n, 2 * n])
    q, at, ws = normal(1, 2 * n, 4, d, dtype=BF16), ints([500, 700]), s2.cache4_workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s2.cache4_attention(q, cache, table, at, cu, n, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = s2.cache4_attention(q, cache, table, at, cu, n, ws=ws)
    for seen in ([500, 700], [900, 2000], [64, 65]):
        at.copy_(ints(seen))
        graph.replay()
        assert torch.equal(o, s2.cache4_attention(q, cache, table, at, cu, n))
    want = [s2.cache4_attention(q * (i + 1), cache, table, ints(lens), cu, n) for i in range(3)]
    x, full = [q * (i + 1) for i in range(3)], ints(lens)
    torch.cuda.synchronize()
    streams, spaces = [torch.cuda.Stream() for _ in x], [s2.cache4_workspace() for _ in x]
    torch.cuda.synchronize()
    got = []
    for y, st, w in zip(x, streams, spaces):
        with torch.cuda.stream(st):
            for _ in range(5):
                z = s2.cache4_attention(y, cache, table, full, cu, n, ws=w)
            got.append(z)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_wait_that_gave_up_is_reported(s2):
    """A status word that is set makes every wait of the call give up at its next look: the call ends, the status is read and
    cleared, and the next call is whole."""
    cache, table, _ = filled(s2, [6000], 64, 2, 128, 1)
    q, table = normal(2, 256, 16, 128, dtype=BF16), wide(table)
    args = (q, cache, table, ints([6000]), ints([0, 256]), 256)
    want = s2.cache4_attention(*args)
    ws = s2.cache4_workspace()
    ws[:4] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8, device="cuda")
    s2.cache4_attention(*args, ws=ws)
    assert s2.device_status(ws) == s2.S2_ERR_DEVICE_TIMEOUT
    assert torch.equal(s2.cache4_attention(*args, ws=ws), want)
    assert s2.device_status(ws) == s2.S2_OK


@pytest.mark.parametrize("Hq,H", [(6, 2), (8, 2), (10, 5), (3, 1)])
@pytest.mark.parametrize("d", [32, 64, 192])
def test_shared_heads_of_the_other_types(s2, Hq, H, d):
    """Groups of one to four heads a block, one or many splits, requests without tokens between."""
    check_attention(s2, [700, 3, 40, 2000, 129], [40, 0, 5, 60, 2], Hq, H, d, 16, F32, seed=Hq + d)
    check_attention(s2, [12000, 900], [1, 1], Hq, H, d, 128, F32, seed=Hq * d)


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_pages_outside_the_cache_of_the_other_types(s2, bad):
    """A page that is none makes its request's rows NaN and no other's; one that lies behind every seen key is not read."""
    lens, new, Hq, H, d, P = [3000, 500, 2000], [1, 1, 1], 4, 1, 96, 64
    cache, table, _ = filled(s2, lens, P, H, d, 5)
    q = normal(6, 3, Hq, d, dtype=F32)
    args = (ints(lens), ints([0, 1, 2, 3]), 1)
    ws = s2.cache4_workspace()
    o = s2.cache4_attention(q, cache, table, *args, ws=ws)
    wrong = table.clone()
    wrong[0, 20] = bad
    wrong[1, 8:] = bad
    got = s2.cache4_attention(q, cache, wrong, *args, ws=ws)
    assert got[0].isnan().all() and torch.equal(got[1:], o[1:])
    assert torch.equal(s2.cache4_attention(q, cache, table, *args, ws=ws), o)      # nothing of it stays in the workspace


def test_captured_calls_of_the_other_types(s2):
    """Replays follow the lengths on the GPU, also to none, and share a workspace with calls between."""
    lens, P, Hq, H, d = [6000, 2500], 64, 8, 2, 64
    cache, table, _ = filled(s2, lens, P, H, d, 8)
    q = normal(9, 2, Hq, d, dtype=F32)
    n, cu, ws = ints(lens), ints([0, 1, 2]), s2.cache4_workspace()
    out = torch.empty_like(q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        s2.cache4_attention(q, cache, table, n, cu, 1, ws=ws, out=out)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            s2.cache4_attention(q, cache, table, n, cu, 1, ws=ws, out=out)
        for now in ([6000, 2500], [1, 0], [129, 2400], [5999, 128]):
            n.copy_(ints(now))
            graph.replay()
            want = s2.cache4_attention(q, cache, table, n, cu, 1, ws=ws)
            assert torch.equal(out, want)
            if 0 in now:
                assert (out[now.index(0)] == 0).all()
    torch.cuda.current_stream().wait_stream(stream)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", [(5, 1001, 2, 2, 128, 128), (900, 3, 1, 1, 64, 64), (3, 2000, 3, 1, 80, 80),
                                              (2, 3001, 5, 2, 256, 256), (4, 700, 3, 2, 44, 24), (1, 9001, 1, 1, 8, 8)])
def test_rope_few_heads(s2, layout, dtype, B, N, Hq, Hkv, d, rot):
    """Threads share out tokens as well as heads, over the ends of a batch's rows; rows that start on 8 bytes only."""
    q, k = normal(1, B, N, Hq, d, dtype=dtype), normal(2, B, N, Hkv, d, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (B, N), generator=torch.Generator().manual_seed(5)).cuda()
    theta, table = ref.freqs(rot, 10000.0, 8.0, 4096), s2.rope_freqs(rot, 10000.0, 8.0, 4096)
    q2, k2 = s2.rope(q, k, pos, table, layout=layout, mscale=1.25)
    for got, x in ((q2, q), (k2, k)):
        want = ref.rope(x, pos, theta, layout, 1.25, False)
        assert ((got.double() - want).abs() <= rope_bound(x, want, rot, layout, 1.25)).all()
    alone = s2.rope(k, None, pos, table, layout=layout, mscale=1.25)[0]
    assert torch.equal(alone, k2)
    q3, k3 = s2.rope(q, k, pos, table, layout=layout, mscale=1.25, in_place=True)
    assert torch.equal(q3, q2) and torch.equal(k3, k2) and q3.data_ptr() == q.data_ptr()
