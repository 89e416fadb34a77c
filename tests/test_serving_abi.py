"""The serving calls' refusals, on the CPU: bad arguments are answered with the documented codes before any GPU call."""
import ctypes
import math

import pytest
import torch

from tests import serving_reference as ref

P = 1 << 20   # an aligned address that nothing reads: the calls below fail before any launch


@pytest.fixture(scope="module")
def s2():
    from longlora_shifted_sparse_b200 import build
    build.build()
    from longlora_shifted_sparse_b200 import s2attn
    return s2attn


def strides(*x):
    return (ctypes.c_longlong * len(x))(*x)


def test_freqs(s2):
    for kw in (dict(), dict(pi_scale=8.0), dict(rope_base=80000.0), dict(pi_scale=25.0, original_len=4096),
               dict(pi_scale=25.0, original_len=4096, slow_turns=0.0, fast_turns=1.0)):
        got = s2.rope_freqs(64, device="cpu", **kw)
        want = ref.freqs(64, kw.get("rope_base", 10000.0), kw.get("pi_scale", 1.0), kw.get("original_len", 0),
                         kw.get("slow_turns", 1.0), kw.get("fast_turns", 32.0))
        assert got.dtype == torch.float64 and torch.allclose(got * 2 * math.pi, want, rtol=1e-14, atol=0)
    for kw in (dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=258), dict(rotary_dim=64, pi_scale=0.0),
               dict(rotary_dim=64, rope_base=-1.0), dict(rotary_dim=64, pi_scale=math.nan), dict(rotary_dim=64, original_len=-1),
               dict(rotary_dim=64, original_len=9, slow_turns=2.0, fast_turns=2.0)):
        with pytest.raises(s2.S2Error):
            s2.rope_freqs(device="cpu", **kw)


def rope(s2, **kw):
    a = dict(q=P, qo=P, k=P, ko=P, pos=P, p64=0, f=P, B=1, N=4, Hq=4, Hkv=2, d=64, rot=64, qs=strides(1024, 256, 64),
             ks=strides(512, 128, 64), ps=strides(0, 1), layout=0, inv=0, m=1.0, dt=0, st=None)
    a.update(kw)
    return s2.s2attn_rope(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(f=None), 1),
    (dict(qs=None), 1), (dict(ks=None), 1), (dict(ps=None), 1), (dict(dt=2), 3), (dict(B=0), 2), (dict(N=0), 2), (dict(Hq=0), 2),
    (dict(Hkv=0), 2), (dict(B=1 << 16, N=1 << 16), 2), (dict(Hq=1 << 16), 2), (dict(d=0), 4), (dict(d=65), 4), (dict(d=258), 4),
    (dict(rot=0), 4), (dict(rot=66), 4), (dict(rot=7), 4), (dict(layout=2), 9), (dict(m=math.inf), 9), (dict(q=P + 8), 5),
    (dict(ko=P + 2), 5), (dict(f=P + 4), 5), (dict(pos=P + 4, p64=1), 5), (dict(pos=P + 2), 5)])
def test_rope_refuses(s2, kw, code):
    assert rope(s2, **kw) == code


def plan(s2, **kw):
    a = dict(c=P, n=P, f=P, fc=P, t=P, cu=P, le=P, pos=P, sl=P, co=P, R=4, T=8, nf=9, mp=4, ts=4, ps=16, st=None)
    a.update(kw)
    return s2.s2attn_page_plan(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(c=None), 1), (dict(n=None), 1), (dict(f=None), 1), (dict(fc=None), 1), (dict(t=None), 1), (dict(cu=None), 1),
    (dict(le=None), 1), (dict(pos=None), 1), (dict(sl=None), 1), (dict(co=None), 1), (dict(R=0), 2), (dict(R=4097), 2),
    (dict(T=-1), 2), (dict(nf=-1), 2), (dict(mp=0), 2), (dict(ts=3), 2), (dict(ps=8), 9), (dict(ps=48), 9), (dict(ps=512), 9),
    (dict(mp=1 << 27, ts=1 << 27), 2)])
def test_plan_refuses(s2, kw, code):
    assert plan(s2, **kw) == code


def test_cache_bytes(s2):
    # 5 bits a value, k and v
    assert s2.s2attn_cache4_bytes(7, 64, 8, 128) == 7 * 64 * 8 * 128 * 2 * 5 // 8
    assert s2.s2attn_cache4_bytes(1 << 20, 64, 32, 128) == (1 << 26) * 32 * 160
    for bad in ((0, 64, 8, 128), (7, 24, 8, 128), (7, 512, 8, 128), (7, 64, 0, 128), (7, 64, 8, 48), (7, 64, 8, 288), (1 << 27, 16, 1, 32)):
        assert s2.s2attn_cache4_bytes(*bad) == 0
    with pytest.raises(s2.S2Error):
        s2.cache4(7, 24, 8, 128, device="cpu")


def append(s2, **kw):
    a = dict(k=P, v=P, c=P, s=P, T=4, H=2, d=64, n=4, p=16, ks=strides(128, 64), vs=strides(128, 64), dt=0, st=None)
    a.update(kw)
    return s2.s2attn_cache4_append(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(c=None), 1), (dict(s=None), 1), (dict(ks=None), 1), (dict(vs=None), 1),
    (dict(dt=3), 3), (dict(T=0), 2), (dict(H=0), 2), (dict(n=0), 2), (dict(n=1 << 27), 2), (dict(d=48), 4), (dict(d=512), 4),
    (dict(p=15), 9), (dict(k=P + 4), 5), (dict(c=P + 8), 5), (dict(ks=strides(130, 64)), 5), (dict(vs=strides(128, 66)), 5)])
def test_append_refuses(s2, kw, code):
    assert append(s2, **kw) == code


def read(s2, **kw):
    a = dict(c=P, s=P, k=P, v=P, T=4, H=2, d=64, n=4, p=16, dt=0, st=None)
    a.update(kw)
    return s2.s2attn_cache4_read(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(c=None), 1), (dict(s=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(dt=-1), 3), (dict(T=0), 2), (dict(H=-2), 2),
    (dict(n=0), 2), (dict(d=40), 4), (dict(p=0), 9), (dict(v=P + 4), 5)])
def test_read_refuses(s2, kw, code):
    assert read(s2, **kw) == code


def attn(s2, **kw):
    a = dict(q=P, c=P, t=P, l=P, cu=P, o=P, lse=None, R=2, T=4, Hq=4, H=2, d=64, n=4, p=16, mp=4, ts=4, qs=strides(256, 64), mn=1,
             sc=0.1, dt=0, ws=P, wsb=1 << 40, st=None)
    a.update(kw)
    return s2.s2attn_cache4_attn(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(c=None), 1), (dict(t=None), 1), (dict(l=None), 1), (dict(cu=None), 1), (dict(o=None), 1),
    (dict(qs=None), 1), (dict(dt=9), 3), (dict(R=0), 2), (dict(T=0), 2), (dict(Hq=3), 2), (dict(H=0), 2), (dict(mp=0), 2),
    (dict(ts=3), 2), (dict(mn=0), 2), (dict(n=1 << 27), 2), (dict(mp=1 << 27, ts=1 << 27), 2), (dict(d=80), 4), (dict(p=20), 9),
    (dict(sc=math.nan), 9), (dict(q=P + 8), 5), (dict(o=P + 8), 5), (dict(qs=strides(256, 68)), 5), (dict(ws=None), 6),
    (dict(wsb=8), 6), (dict(ws=P + 4), 5)])
def test_attention_refuses(s2, kw, code):
    assert attn(s2, **kw) == code


def test_torch_layer_refuses(s2):
    """Checks of the torch layer that come before any CUDA call."""
    x = torch.zeros(2, 3, 4, 64)
    f, pos = s2.rope_freqs(64, device="cpu"), torch.arange(3)
    for bad in (lambda: s2.rope(x, None, pos, f, layout="pairs"), lambda: s2.rope(x, None, torch.arange(4), f),
                lambda: s2.rope(x, x[:1], pos, f), lambda: s2.rope(x[0, 0], None, pos, f),
                lambda: s2.rope(x.clone().requires_grad_(), None, pos, f, in_place=True),
                lambda: s2.rope(x, None, pos, f.view(2, -1))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: s2.rope(x.half(), None, pos, f), lambda: s2.rope(x, None, pos.float(), f), lambda: s2.rope(x, None, pos, f.float())):
        with pytest.raises(TypeError):
            bad()
    i = torch.zeros(2, dtype=torch.int32)
    one = torch.ones(1, dtype=torch.int32)
    table = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        s2.page_plan(i.long(), i, one, one, table, 16, 4)
    for bad in (lambda: s2.page_plan(i, one, one, one, table, 16, 4), lambda: s2.page_plan(i, i, one, one, table.T, 16, 4)):
        with pytest.raises(ValueError):
            bad()
    cache = s2.cache4(2, 16, 4, 64, device="cpu")
    k = torch.zeros(2, 4, 64)
    for bad in (lambda: s2.cache4_append(k[:, :2], k[:, :2], cache, i), lambda: s2.cache4_append(k, k.bfloat16(), cache, i),
                lambda: s2.cache4_append(k, k, cache, one), lambda: s2.cache4_append(k, k, cache.view(2, 4, -1), i),
                lambda: s2.cache4_attention(k[..., :32], cache, table, i, torch.zeros(3, dtype=torch.int32), 1),
                lambda: s2.cache4_attention(k, cache, table[:1], i, torch.zeros(3, dtype=torch.int32), 1),
                lambda: s2.cache4_attention(k, cache, table, i, i, 1)):
        with pytest.raises(ValueError):
            bad()
