"""The compiled serving calls and the Python layer behind them: both give the same, and a missing build is named."""
import importlib.util
import os
import shutil

import pytest
import torch

from tests.test_serving import BF16, F32, filled, ints, normal

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "longlora_shifted_sparse_b200")


@pytest.fixture(scope="module")
def s2():
    from longlora_shifted_sparse_b200 import build
    build.build()
    from longlora_shifted_sparse_b200 import s2attn
    return s2attn


def test_a_missing_build_is_named(s2, tmp_path):
    shutil.copy(os.path.join(PKG, "s2attn.py"), tmp_path / "s2attn.py")
    shutil.copy(os.path.join(PKG, "libs2attn.so"), tmp_path / "libs2attn.so")     # and no _serve_calls.so
    spec = importlib.util.spec_from_file_location("s2attn_without_calls", tmp_path / "s2attn.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    with pytest.raises(ImportError, match="not built"):
        mod.rope(torch.zeros(1, 2, 64), None, torch.zeros(1), None)


def test_cpu_tensors_are_refused(s2):
    x, pos = torch.zeros(2, 4, 64), torch.arange(2, dtype=torch.int32)
    i, cache = torch.zeros(2, dtype=torch.int32), s2.cache4(2, 16, 4, 64, device="cpu")
    for call in (lambda: s2.rope(x, None, pos, s2.rope_freqs(64, device="cpu")), lambda: s2.cache4_append(x, x, cache, i),
                 lambda: s2.cache4_read(cache, i), lambda: s2.page_plan(i, i, i, i[:1], i.view(2, 1), 16, 4),
                 lambda: s2.cache4_attention(x, cache, i.view(2, 1), i, torch.zeros(3, dtype=torch.int32), 1, ws=torch.zeros(8, dtype=torch.uint8))):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()


@pytest.fixture
def both(s2, monkeypatch):
    """A call made through the compiled path, then through the Python one; the outputs of both."""
    def run(call):
        first = call()
        monkeypatch.setattr(s2, "_plain", lambda *a: None)
        second = call()
        monkeypatch.undo()
        return first, second
    return run


def same(a, b):
    if isinstance(a, torch.Tensor):
        assert a.shape == b.shape and a.dtype == b.dtype and a.stride() == b.stride() and torch.equal(a, b)
    elif a is None:
        assert b is None
    else:
        assert len(a) == len(b) and type(a) is type(b)
        for x, y in zip(a, b):
            same(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_both_paths_give_the_same(s2, both, dtype):
    q, k = normal(1, 3, 5, 4, 64, dtype=dtype), normal(2, 3, 5, 2, 64, dtype=dtype)
    f, pos = s2.rope_freqs(64, pi_scale=4.0), torch.arange(5, device="cuda")
    same(*both(lambda: s2.rope(q, k, pos, f, layout="half", mscale=1.5)))
    same(*both(lambda: s2.rope(q, None, pos.int().expand(3, 5), f)))
    same(*both(lambda: s2.rope(q[0], k[0], pos.view(1, 5), f)))
    same(*both(lambda: s2.rope(q.transpose(0, 1)[:, :2], k.transpose(0, 1)[:, :2], pos[:2], f)))
    g = torch.Generator().manual_seed(0)
    new = torch.randint(0, 40, (9,), generator=g).int().cuda()
    plan = [ints([3 * r for r in range(9)]), new, torch.randperm(99, generator=g).int().cuda(), ints([90]), None, 16, int(new.sum()) + 1]

    def planned():
        plan[4] = torch.zeros(9, 12, dtype=torch.int32, device="cuda")[:, :10]
        return s2.page_plan(*plan), plan[4].clone()

    same(*both(planned))
    cache, table, _ = filled(s2, [40, 90], 16, 2, 64, 1)
    rows, slots = normal(3, 6, 2, 64, dtype=dtype), ints([5, 1, 17, 33, -1, 40])

    def stored():
        c = cache.clone()
        s2.cache4_append(rows, 2 * rows, c, slots)
        return c, s2.cache4_read(c, slots, dtype), s2.cache4_read(c, slots)

    same(*both(stored))
    x, out = normal(4, 5, 6, 64, dtype=dtype), torch.zeros(5, 6, 64, dtype=dtype, device="cuda")
    args = (x, cache, table, ints([40, 90]), ints([0, 2, 5]), 3)
    same(*both(lambda: s2.cache4_attention(*args, return_lse=True)))
    same(*both(lambda: s2.cache4_attention(*args, scale=0.25, ws=s2.cache4_workspace(), out=out).clone()))
    same(*both(lambda: s2.cache4_attention(torch.nn.Parameter(x), *args[1:], scale=1)))
    same(*both(lambda: s2.cache4_attention(normal(6, 5, 6, 128, dtype=dtype)[..., 64:], *args[1:])))


@pytest.mark.gpu
def test_refusals_of_the_library_reach_the_caller(s2):
    cache, table, _ = filled(s2, [40], 16, 2, 64, 1)
    q, f = normal(1, 1, 4, 64, dtype=BF16), s2.rope_freqs(64)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(s2.S2Error, match="workspace"):
        s2.cache4_attention(q, cache, table, ints([40]), ints([0, 1]), 1, ws=small)
    with pytest.raises(s2.S2Error):
        s2.cache4_attention(q, cache, table, ints([40]), ints([0, 1]), 0)
    with pytest.raises(s2.S2Error):
        s2.cache4_attention(normal(1, 1, 3, 64, dtype=BF16), cache, table, ints([40]), ints([0, 1]), 1)
    with pytest.raises(s2.S2Error):
        s2.rope(normal(1, 1, 2, 32), None, ints([0]), f)               # more rotated channels than there are
    with pytest.raises(s2.S2Error):
        s2.rope(normal(1, 1, 2, 64), None, ints([0]), f, mscale=float("inf"))
    with pytest.raises(s2.S2Error):
        s2.page_plan(ints([0]), ints([1]), ints([0]), ints([1]), ints([[0]]), 17, 1)
    with pytest.raises(TypeError):
        s2.cache4_append(q[:, :2].half(), q[:, :2].half(), cache, ints([0]))
    with pytest.raises(ValueError):
        s2.rope(normal(1, 1, 2, 64).expand(3, 2, 64), None, ints([0, 1, 2]), f, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("said", [1, 7, 5000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_max_new_is_only_a_hint(s2, said, dtype):
    cache, table, _ = filled(s2, [300, 70], 16, 2, 64, 1, dtype=BF16)
    q = normal(1, 110, 4, 64, dtype=dtype)
    args = (q, cache, table, ints([300, 70]), ints([0, 100, 110]))
    a, b = s2.cache4_attention(*args, said), s2.cache4_attention(*args, 100)
    # other tiles, other orders of the same sums: P and v in fp16 for bf16, all fp32 otherwise
    assert (a.float() - b.float()).abs().max() <= (2.0 ** -7 if dtype is BF16 else 2.0 ** -20) * b.abs().max()


@pytest.mark.gpu
def test_on_a_stream_of_its_own(s2):
    """Work goes to the current stream: a call on a side stream waits for what that stream waits for."""
    cache, table, _ = filled(s2, [500], 16, 2, 64, 1)
    args = (cache, table, ints([500]), ints([0, 1]), 1)
    ws, side = s2.cache4_workspace(), torch.cuda.Stream()
    q = normal(1, 1, 4, 64, dtype=BF16)
    want = s2.cache4_attention(q, *args)
    x, late = torch.zeros_like(q), torch.empty(1 << 26, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            late.normal_()
        x.copy_(q)
        o = s2.cache4_attention(x, *args, ws=ws)
    side.synchronize()
    assert torch.equal(o, want)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_gradients_of_parts(s2, both, layout):
    """Gradients where only one output is used, through sums, for q alone, and of the gradient itself."""
    f, pos = s2.rope_freqs(32, pi_scale=2.0), torch.arange(7, 12, device="cuda")
    q, k, w = (normal(s, 2, 5, 3, 48).requires_grad_() for s in (1, 2, 3))
    turn = lambda x, **kw: s2.rope(x, None, pos, f, layout, 1.5, **kw)[0]  # noqa: E731

    def parts():
        y, z = s2.rope(q, k, pos, f, layout, 1.5)
        gq, gk = torch.autograd.grad((y * w).sum() + z.sum(), (q, k), create_graph=True)
        only_k = torch.autograd.grad(s2.rope(q, k, pos, f, layout, 1.5)[1].square().sum(), (q, k), allow_unused=True)
        (second,) = torch.autograd.grad((gq * gq.detach()).sum(), w)
        return gq.detach(), gk, only_k[1], second, only_k[0] is None or not only_k[0].any()

    for gq, gk, only_k, second, unused in both(parts):
        assert unused
        # the map is linear, R^T R = 1.5^2 on the rotated channels and 1 beyond: each gradient by the map itself
        with torch.no_grad():
            probe = normal(9, 2, 5, 3, 48)
            assert abs((turn(probe) * w).sum() - (probe * gq).sum()) <= 1e-3
            assert abs(turn(probe).sum() - (probe * gk).sum()) <= 1e-3
            scale = torch.ones(48, device="cuda")
            scale[:32] = 1.5 ** 2
            assert torch.allclose(only_k, 2 * k * scale, rtol=1e-5, atol=1e-5)
            assert torch.allclose(second, w * scale, rtol=1e-5, atol=1e-5)


@pytest.mark.gpu
def test_captured_rope_step(s2):
    q, f, pos = normal(1, 2, 9, 4, 64, dtype=BF16).requires_grad_(), s2.rope_freqs(64), torch.arange(9, device="cuda")
    dy = normal(2, 2, 9, 4, 64, dtype=BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(s2.rope(q, None, pos, f)[0], q, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = s2.rope(q, None, pos, f)[0]
        (dq,) = torch.autograd.grad(y, q, dy)
    for s in (3, 4):
        with torch.no_grad():
            q.copy_(normal(s, 2, 9, 4, 64, dtype=BF16))
            dy.copy_(normal(s + 5, 2, 9, 4, 64, dtype=BF16))
        graph.replay()
        z = s2.rope(q, None, pos, f)[0]
        assert torch.equal(y, z) and torch.equal(dq, torch.autograd.grad(z, q, dy)[0])
