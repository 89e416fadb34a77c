"""The serving operators on the GPU against their 64-bit forms: rotary positions and their gradient, page plans, the
4-bit cache, attention over it, and a whole step of them."""
import math

import pytest
import torch

from tests import serving_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}   # half a step of a value's rounding


@pytest.fixture(scope="module")
def s2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from longlora_shifted_sparse_b200 import s2attn
    return s2attn


def normal(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------------------- rope

def rope_bound(x, want, rot, layout, mscale):
    """sin and cos: 2 ulp, the angle's rounding to fp32 (pi 2^-24) and the product with mscale: below 7 * 2^-24; two products and
    a sum: 1.5 * 2^-24 of |a| + |b|; then the output's rounding (which is exact where the channels pass through)."""
    y = x.double().abs().clone()
    even, odd = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    both = y[..., even] + y[..., odd]
    y[..., even], y[..., odd] = both, both
    y[..., rot:] = 0
    return 9 * 2.0 ** -24 * abs(mscale) * y + HALF[x.dtype] * want.abs() * 1.001 + 1e-38


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", [(1, 1, 1, 1, 64, 64), (2, 7, 3, 1, 80, 40), (1, 33, 8, 2, 128, 128), (3, 5, 2, 2, 256, 32),
                                              (1, 2500, 4, 4, 96, 64), (1, 3, 2, 1, 6, 2), (2, 9, 2, 2, 128, 18)])
def test_rope_and_gradient(s2, layout, dtype, B, N, Hq, Hkv, d, rot):
    q, k = normal(1, B, N, Hq, d, dtype=dtype), normal(2, B, N, Hkv, d, dtype=dtype)
    dq, dk = normal(3, B, N, Hq, d, dtype=dtype), normal(4, B, N, Hkv, d, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (B, N), generator=torch.Generator().manual_seed(5)).cuda()
    theta = ref.freqs(rot, 10000.0, 8.0, 4096)
    table = s2.rope_freqs(rot, 10000.0, 8.0, 4096)
    assert torch.allclose(table.cpu() * 2 * math.pi, theta, rtol=1e-14, atol=0)
    q.requires_grad_()
    k.requires_grad_()
    q2, k2 = s2.rope(q, k, pos, table, layout=layout, mscale=1.25)
    g = torch.autograd.grad((q2, k2), (q, k), (dq, dk))
    for got, x, inv in ((q2, q, False), (k2, k, False), (g[0], dq, True), (g[1], dk, True)):
        want = ref.rope(x.detach(), pos, theta, layout, 1.25, inv)
        assert ((got.double() - want).abs() <= rope_bound(x.detach(), want, rot, layout, 1.25)).all()


def test_rope_gradient_against_differences(s2):
    # the map is linear: <dq, (rope(x + h) - rope(x - h)) / 2> is <rope^T dq, h>, up to the fp32 roundings of 64 terms
    x, h, dy = (normal(s, 1, 2, 2, 16) for s in (1, 2, 3))
    pos, f = ints([3, 70001]), s2.rope_freqs(12)
    x.requires_grad_()
    y, none = s2.rope(x, None, pos, f, layout="half", mscale=0.5)
    assert none is None
    (dx,) = torch.autograd.grad(y, x, dy)
    with torch.no_grad():
        diff = (s2.rope(x + h, None, pos, f, "half", 0.5)[0].double() - s2.rope(x - h, None, pos, f, "half", 0.5)[0].double()) / 2
    a, b = (diff * dy.double()).sum(), (dx.double() * h.double()).sum()
    assert abs(a - b) <= 64 * 16 * 16 * 2.0 ** -24


def test_rope_strides_positions_in_place(s2):
    T, Hq, Hkv, d = 37, 4, 2, 64
    f = s2.rope_freqs(64, pi_scale=2.0)
    theta = ref.freqs(64, pi_scale=2.0)
    fused = normal(7, T, (Hq + 2 * Hkv) * d, dtype=BF16)     # q, k, v of one projection
    q = fused[:, :Hq * d].unflatten(1, (Hq, d))
    k = fused[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    before = fused.clone()
    pos = torch.arange(100, 100 + T, device="cuda")
    q2, k2 = s2.rope(q, k, pos.int(), f)
    assert torch.equal(fused, before)
    want = ref.rope(q.unsqueeze(0), pos.view(1, -1), theta, "interleaved")[0]
    assert ((q2.double() - want).abs() <= rope_bound(q, want, 64, "interleaved", 1.0)).all()
    q3, k3 = s2.rope(q, k, pos, f, in_place=True)             # int64 positions, the same numbers
    assert q3.data_ptr() == q.data_ptr() and torch.equal(q, q2) and torch.equal(k, k2)
    assert torch.equal(fused[:, (Hq + Hkv) * d:], before[:, (Hq + Hkv) * d:])
    # one row of positions for a batch; a transposed (head-major) input; a slice that is not 16-byte aligned
    x = normal(8, 2, 3, T, 65, dtype=F32)
    y = s2.rope(x.transpose(1, 2)[..., 1:], None, pos, f)[0]
    want = ref.rope(x.transpose(1, 2)[..., 1:], pos.expand(2, T), theta, "interleaved")
    assert ((y.double() - want).abs() <= rope_bound(x.transpose(1, 2)[..., 1:], want, 64, "interleaved", 1.0)).all()
    assert s2.rope(x[:0].transpose(1, 2), None, pos, f)[0].shape == (0, T, 3, 65)


def test_rope_agrees_with_the_attention_calls(s2):
    # dense attention of plain inputs with the call's own rotation, and of rotated ones with none to speak of (far interpolation)
    q, k, v = (normal(s, 1, 64, 2, 64) for s in (1, 2, 3))
    o, _ = s2.forward(q, k, v, 64, 4.0, shift="none")
    q2, k2 = s2.rope(q, k, torch.arange(64, device="cuda"), s2.rope_freqs(64, pi_scale=4.0))
    o2, _ = s2.forward(q2, k2, v, 64, 1e30, shift="none")
    assert (o - o2).abs().max() <= 1e-5 * o.abs().max()


# --------------------------------------------------------------------------------- plans

def plan_both(s2, cached, new, free, count, table, P, T):
    t = ints(table)
    got = s2.page_plan(ints(cached), ints(new), ints(free), ints([count]), t, P, T)
    cu, lens, pos, slots, left, out, tab = ref.plan(cached, new, free, count, table, P, T)
    assert got.cu_new.tolist() == cu and got.lens.tolist() == lens
    assert got.slots.tolist() == slots
    assert got.positions.tolist() == pos
    assert got.free_count.tolist() == [left] and got.left_out.tolist() == [out]
    assert t.tolist() == tab
    return got


@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("R", [1, 2, 31, 300, 1025])
def test_plan(s2, R, P):
    g = torch.Generator().manual_seed(R + P)
    cached = torch.randint(0, 5 * P, (R,), generator=g).tolist()
    new = [0 if x < 2 else 1 if x < 8 else 3 * P + x for x in torch.randint(0, 12, (R,), generator=g).tolist()]
    cached[0] = 0
    free = torch.randperm(R * 10, generator=g).tolist()
    table = torch.randint(0, 1000, (R, 10), generator=g).tolist()
    plan_both(s2, cached, new, free, len(free), table, P, sum(new) + 5)


@pytest.mark.parametrize("cached,new,count,width,T", [
    ([16, 0, 3], [16, 20, 1], 2, 4, 64),          # the pages run out at the second; the third needs none
    ([16, 0, 0], [16, 20, 1], 2, 4, 64),          # ... or needs one
    ([16, 60, 3], [1, 10, 20], 9, 4, 64),         # the table is too narrow for the second
    ([0, 5, 7, 9], [30, 30, 30, 0], 50, 4, 64),   # the token buffer ends inside the third
    ([-1, 5, 7], [3, -2, 4], 50, 4, 8),           # lengths below zero
    ([0, 5], [2 ** 31 - 1, 2 ** 31 - 1], 50, 4, 8),   # sums beyond 32 bits
    ([4, 4], [4, 4], 0, 4, 8),                    # no page needed, none there
    ([4, 4], [14, 14], 99, 4, 40),                # a count beyond the list
    ([4], [0], 3, 1, 0),                          # nothing to do
])
def test_plan_left_out(s2, cached, new, count, width, T):
    if max(new) > 1 << 20:   # the loops of the plain form would not end: both are left out, nothing is taken
        t = ints([[7] * width] * 2)
        got = s2.page_plan(ints(cached), ints(new), ints(list(range(50))), ints([count]), t, 16, T)
        assert got.left_out.tolist() == [2] and got.free_count.tolist() == [count] and got.lens.tolist() == cached
        assert set(got.slots.tolist()) == {-1} and t.tolist() == [[7] * width] * 2
        return
    plan_both(s2, cached, new, list(range(100, 150)), count, [[10 * r + c for c in range(width)] for r in range(len(cached))], 16, T)


# --------------------------------------------------------------------------------- the cache

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 192, 224, 256])
def test_append_and_read(s2, d, dtype):
    T, H, P, pages = 53, 3, 32, 4
    k, v = normal(1, T, H, d, dtype=dtype), normal(2, T, H, d, dtype=dtype) * 100
    k[5] = 0.25                     # a group with no range
    v[6, 0, :32] = 1e-30            # below fp16
    k[7, 1, 3] = 1e30               # beyond fp16: limited
    cache = s2.cache4(pages, P, H, d)
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(3))[:T].int().cuda()
    slots[9], slots[10], slots[11] = -1, pages * P, 2 ** 31 - 1     # skipped
    s2.cache4_append(k, v, cache, slots)
    got = s2.cache4_read(cache, slots, dtype)
    kept = torch.ones(T, dtype=torch.bool)
    kept[9:12] = False
    for x, y in ((k, got[0]), (v, got[1])):
        want, _ = ref.quantised(x)
        # one product and sum, rounded to the output's type
        assert ((y.double() - want).abs()[kept] <= (HALF[dtype] * want.abs() * 1.001 + 1e-38)[kept]).all()
        assert (y[9:12] == 0).all()
    others = torch.ones(pages * P, dtype=torch.bool, device="cuda")
    others[slots[kept.cuda()].long()] = False
    rest = torch.arange(pages * P, device="cuda", dtype=torch.int32)[others]
    assert all((x == 0).all() for x in s2.cache4_read(cache, rest, F32))     # no other slot was touched


def test_append_strides_and_sizes(s2):
    d, H, P = 64, 2, 16
    fused = normal(4, 21, 4, 3 * H, d, dtype=BF16)
    k, v = fused[:, 1, :H], fused[:, 2, H:2 * H]
    cache = s2.cache4(2, P, H, d)
    slots = torch.arange(21, device="cuda", dtype=torch.int32)
    s2.cache4_append(k, v, cache, slots)
    for x, y in zip((k, v), s2.cache4_read(cache, slots, F32)):
        assert torch.equal(y.double(), ref.quantised(x)[0])        # 5 bits times 11 bits plus 11: exact here
    odd = normal(5, 3, H, d + 1)[..., 1:]                          # rows off 16 bytes: copied first
    s2.cache4_append(odd, odd, cache, slots[:3])
    assert (s2.cache4_read(cache, slots[:3], F32)[0].double() - ref.quantised(odd)[0]).abs().max() <= 2.0 ** -22
    s2.cache4_append(k[:0], v[:0], cache, slots[:0])
    assert s2.cache4_read(cache, slots[:0])[0].shape == (0, H, d)


# --------------------------------------------------------------------------------- attention

def filled(s2, lens, P, H, d, seed, spare=1, dtype=BF16):
    """A cache with random pages of each request's k, v; everything else in it is NaN."""
    pages = [-(-n // P) for n in lens]
    total = sum(pages) + spare
    cache = s2.cache4(total, P, H, d)
    cache.fill_(255)
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(1, max(pages))
    table, kv = [], []
    for r, n in enumerate(lens):
        mine = [order.pop() for _ in range(pages[r])]
        table.append(mine + [2 ** 31 - 1] * (width - len(mine)))   # never to be read
        k, v = normal(seed + 7 * r, n, H, d, dtype=dtype), normal(seed + 7 * r + 1, n, H, d, dtype=dtype)
        slots = ints([mine[i // P] * P + i % P for i in range(n)])
        s2.cache4_append(k, v, cache, slots)
        kv.append((ref.quantised(k), ref.quantised(v)))
    return cache, ints(table), kv


def check_attention(s2, lens, new, Hq, H, d, P, dtype, seed=0, scale=None, qscale=1.0, order=None):
    cache, table, kv = filled(s2, lens, P, H, d, seed)
    cu = [sum(new[:r]) for r in range(len(new) + 1)]
    behind = 3
    q = normal(seed + 99, cu[-1] + behind, Hq, d, dtype=dtype) * qscale
    out = torch.full_like(q, 7.0)
    ws = s2.cache4_workspace()
    args = (q, cache, table, ints(lens), ints(cu), max(1, max(new)))
    o, lse = s2.cache4_attention(*args, scale=scale, ws=ws, out=out, return_lse=True)
    assert o.data_ptr() == out.data_ptr()
    again = s2.cache4_attention(*args, scale=scale, ws=ws)
    assert (o[cu[-1]:] == 7.0).all()
    sc = d ** -0.5 if scale is None else scale
    for r, n in enumerate(new):
        rows = slice(cu[r], cu[r + 1])
        if n == 0:
            continue
        (k, ks), (v, _) = kv[r]
        keys = [max(0, lens[r] - (n - 1 - i)) for i in range(n)]
        want, wl, pv = ref.attention(q[rows], k, v, keys, sc)
        qa = q[rows].double().abs()
        # scores: fp32 sums. On the tensor cores a group's products are formed with codes offset by up to 1024 before the
        # offset is taken off again, so that their error is 2^-22 of 1100 sum |q|, times the group's scale
        biggest = (ks.amax(0).double() if ks.shape[0] else torch.zeros(H, d // 32, device="cuda", dtype=torch.float64)).repeat_interleave(Hq // H, 0)
        span = 1100 if dtype is BF16 else 16
        err = sc * 2.0 ** -22 * (span * (qa.unflatten(-1, (-1, 32)).sum(-1) * biggest).sum(-1)
                                 + 16 * qa.sum(-1) * (k.abs().amax() if k.numel() else 0))
        dead = torch.tensor([x == 0 for x in keys], device="cuda")
        got_l = lse[:, rows].T.double()
        assert (got_l[dead] == -math.inf).all() and (o[rows][dead] == 0).all()
        live = ~dead
        assert ((got_l - wl).abs()[live] <= (err + 2.0 ** -21 * (4 + wl.abs()))[live]).all()
        # probabilities and values in fp16 (half a step 2^-11 each, 2^-25 where they are subnormal), sums of `keys` terms in fp32
        half = 3 * 2.0 ** -11 if dtype is BF16 else 2.0 ** -21
        vmax = float(v.abs().max()) if v.numel() else 0.0
        tail = (max(keys) * 2.0 ** -25 * vmax if dtype is BF16 else 0.0) + 1e-30
        bound = HALF[dtype] * want.abs() * 1.01 + (half + 2 * err.unsqueeze(-1) + math.sqrt(max(keys) + 1) * 2.0 ** -22) * pv + tail
        assert ((o[rows].double() - want).abs() <= bound)[live].all()
        assert torch.equal(again[rows], o[rows])                    # the same bits each time
    return o


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 192, 224, 256])
def test_attention_head_dims(s2, d, dtype):
    check_attention(s2, [1, 16, 100, 257], [1, 1, 1, 1], 4, 2, d, 32, dtype)


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(1, 1), (6, 2), (8, 1), (32, 2), (3, 3)])
def test_attention_pages_and_heads(s2, P, Hq, H):
    check_attention(s2, [31, 1, 0, 500, 64, 65], [1, 1, 1, 1, 0, 1], Hq, H, 64, P, BF16, seed=P)


@pytest.mark.parametrize("new", [[2, 5, 8], [16, 1, 0], [40, 33, 100], [3, 300, 7]])
@pytest.mark.parametrize("Hq,H,d", [(2, 2, 128), (8, 1, 64), (12, 4, 128), (4, 2, 256)])
def test_attention_many_tokens(s2, new, Hq, H, d):
    # lengths at and below the number of the step's own tokens among them: the first rows then see no key
    check_attention(s2, [1700, max(0, new[1] - 2), new[2]], new, Hq, H, d, 32, BF16, seed=11)


@pytest.mark.parametrize("new", [[3, 1], [20, 2]])
def test_attention_many_tokens_f32(s2, new):
    check_attention(s2, [333, 1], new, 6, 2, 96, 16, F32, seed=5)


def test_attention_long(s2):
    check_attention(s2, [20011, 3], [1, 1], 4, 2, 128, 64, BF16, seed=3)
    check_attention(s2, [9000], [2], 8, 1, 128, 16, BF16, seed=4, scale=0.3, qscale=3.0)


def test_attention_batch_of_many(s2):
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 300, (200,), generator=g).tolist()
    check_attention(s2, lens, [1 if n else 0 for n in lens], 4, 2, 64, 16, BF16, seed=21)


def test_attention_large_and_small_queries(s2):
    check_attention(s2, [77, 130], [1, 2], 8, 2, 128, 32, BF16, seed=8, qscale=3e4, scale=1e-5)
    check_attention(s2, [77, 130], [1, 2], 8, 2, 128, 32, BF16, seed=8, qscale=1e-20, scale=1e19)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 96)])
def test_attention_poison_stays_where_it_is(s2, dtype, d):
    """A NaN or infinity in a token reaches the rows that see it, in its kv head, and no other."""
    H, P, L, n = 2, 16, 70, 6
    cache, table, _ = filled(s2, [L, 40], P, H, d, 1)
    q = normal(5, n + 1, 4, d, dtype=dtype)
    args = (ints([L, 40]), ints([0, n, n + 1]), n)
    good = s2.cache4_attention(q, cache, table, *args)
    assert good.isfinite().all()
    k, v = normal(6, 1, H, d, dtype=dtype), normal(7, 1, H, d, dtype=dtype)
    place = L - n + 3                                        # seen by rows 3, 4, 5 of the first request
    slot = table[0, place // P].item() * P + place % P
    for bad in (math.nan, math.inf, -math.inf):
        for x in (k, v):
            was, x[0, 1, 5] = x[0, 1, 5].item(), bad         # kv head 1: query heads 2, 3
            s2.cache4_append(k, v, cache, ints([slot]))
            o = s2.cache4_attention(q, cache, table, *args)
            assert o[3:n, 2:].isnan().all()
            assert torch.equal(o[:3], good[:3]) and torch.equal(o[n:], good[n:]) and o[3:n, :2].isfinite().all()
            assert s2.cache4_read(cache, ints([slot]))[0][0, 1].isnan().all()
            x[0, 1, 5] = was
    # a query that holds one spoils its own row alone
    s2.cache4_append(k, v, cache, ints([slot]))
    clean = s2.cache4_attention(q, cache, table, *args)
    q[1, 0, 3] = math.inf
    o = s2.cache4_attention(q, cache, table, *args)
    assert o[1, 0].isnan().all()
    o[1, 0], clean[1, 0] = 0, 0
    assert torch.equal(o, clean)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 32)])
def test_attention_bad_numbers_on_the_device(s2, dtype, d):
    H, P = 1, 16
    cache, table, _ = filled(s2, [40, 40, 40], P, H, d, 1)
    q = normal(5, 4, 2, d, dtype=dtype)
    good = s2.cache4_attention(q, cache, table, ints([40, 40, 40]), ints([0, 1, 2, 3]), 1)
    for page in (-1, -2 ** 31, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 1] = page
        o = s2.cache4_attention(q, cache, t, ints([40, 40, 40]), ints([0, 1, 2, 3]), 1)
        assert o[1].isnan().all() and torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
    # lengths beyond the table, and below zero
    o = s2.cache4_attention(q, cache, table, ints([48, 2 ** 31 - 1, -5]), ints([0, 0, 1, 2]), 1)
    full = s2.cache4_attention(q, cache, table, ints([48, 48, 0]), ints([0, 0, 1, 2]), 1)
    assert torch.equal(o[1], full[1]) and (o[1] == 0).all()
    # row numbers that fall, or lie beyond q
    s2.cache4_attention(q, cache, table, ints([40, 40, 40]), ints([3, 1, -7, 2 ** 31 - 1]), 1)
    torch.cuda.synchronize()


def test_attention_strided_query_and_table(s2):
    H, P, d, Hq = 2, 32, 128, 4
    cache, table, _ = filled(s2, [90, 200], P, H, d, 2)
    wide = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    fused = normal(9, 2, 3 * Hq, d, dtype=BF16)
    q = fused[:, Hq:2 * Hq]
    a = s2.cache4_attention(q, cache, table, ints([90, 200]), ints([0, 1, 2]), 1)
    b = s2.cache4_attention(q.contiguous(), cache, wide[:, :table.shape[1]], ints([90, 200]), ints([0, 1, 2]), 1)
    assert torch.equal(a, b)


# --------------------------------------------------------------------------------- together

def serving_model(s2, lens, steps, page, Hq, H, d, captured):
    """`steps` decode steps of requests with `lens` cached tokens; returns the outputs, and all that they attend to."""
    R, width = len(lens), -(-(max(lens) + steps) // page)
    total = R * width
    cache = s2.cache4(total, page, H, d)
    f = s2.rope_freqs(d, pi_scale=8.0)
    table = torch.zeros(R, width, dtype=torch.int32, device="cuda")
    free = torch.randperm(total, generator=torch.Generator().manual_seed(1)).int().cuda()
    count, cached, ws = ints([total]), ints([0] * R), s2.cache4_workspace()
    kept = [([], []) for _ in lens]

    def step(q, k, v, new, tokens, most):
        p = s2.page_plan(cached, new, free, count, table, page, tokens)
        q2, k2 = s2.rope(q, k, p.positions, f)
        s2.cache4_append(k2, v, cache, p.slots)
        o = s2.cache4_attention(q2, cache, table, p.lens, p.cu_new, most, ws=ws)
        cached.copy_(p.lens)
        count.copy_(p.free_count)
        return q2, k2, o

    def keep(new, k2, v):
        at = 0
        for r, n in enumerate(new):
            kept[r][0].append(k2[at:at + n].clone())
            kept[r][1].append(v[at:at + n].clone())
            at += n

    T = sum(lens)
    q, k, v = (normal(s, T, h, d, dtype=BF16) for s, h in ((1, Hq), (2, H), (3, H)))
    q2, k2, o = step(q, k, v, ints(lens), T, max(lens))
    keep(lens, k2, v)
    outs = [(lens, q2.clone(), o.clone())]
    one = ints([1] * R)
    q, k, v = (torch.empty(R, h, d, dtype=BF16, device="cuda") for h in (Hq, H, H))
    graph = None
    for i in range(steps):
        for x, s in ((q, 10), (k, 20), (v, 30)):
            x.copy_(normal(100 * i + s, *x.shape, dtype=BF16))
        if captured and graph is None:
            was = cached.clone(), count.clone(), table.clone(), cache.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step(q, k, v, one, R, 1)
            torch.cuda.current_stream().wait_stream(side)
            for x, y in zip((cached, count, table, cache), was):
                x.copy_(y)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                q2, k2, o = step(q, k, v, one, R, 1)
        if captured:
            graph.replay()
        else:
            q2, k2, o = step(q, k, v, one, R, 1)
        keep([1] * R, k2, v)
        outs.append(([1] * R, q2.clone(), o.clone()))
    return outs, kept, cached, count, total


@pytest.mark.parametrize("captured", [False, True])
def test_a_prompt_and_decode_steps(s2, captured):
    lens, steps, page, Hq, H, d = [5, 63, 200], 20, 16, 8, 2, 128
    outs, kept, cached, count, total = serving_model(s2, lens, steps, page, Hq, H, d, captured)
    assert cached.tolist() == [n + steps for n in lens]
    assert count.item() == total - sum(-(-(n + steps) // page) for n in lens)
    done = [0] * len(lens)
    for new, q2, o in outs:
        at = 0
        for r, n in enumerate(new):
            done[r] += n
            k, v = (ref.quantised(torch.cat(x))[0][:done[r]] for x in kept[r])
            keys = [done[r] - (n - 1 - i) for i in range(n)]
            want, _, pv = ref.attention(q2[at:at + n], k, v, keys, d ** -0.5)
            # as in check_attention, with |q|, |k| of unit normals: the scores' error stays below 2^-10
            assert ((o[at:at + n].double() - want).abs() <= HALF[BF16] * 1.01 * want.abs() + (3 * 2.0 ** -11 + 2.0 ** -9) * pv + 2e-5).all()
            at += n


def test_two_streams_with_a_workspace_each(s2):
    cache, table, _ = filled(s2, [3000], 64, 2, 128, 1)
    q = [normal(s, 1, 8, 128, dtype=BF16) for s in range(4)]
    args = (cache, table, ints([3000]), ints([0, 1]), 1)
    want = [s2.cache4_attention(x, *args) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    spaces = [s2.cache4_workspace() for _ in q]
    torch.cuda.synchronize()
    got = []
    for x, st, ws in zip(q, streams, spaces):
        with torch.cuda.stream(st):
            for _ in range(10):
                o = s2.cache4_attention(x, *args, ws=ws)
            got.append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
