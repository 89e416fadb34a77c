"""Thin ctypes binding of libs2attn.so (argument marshalling only; every step runs in the
library's CUDA kernels).

Two layers:
* the C ABI under its own names (``s2attn_fwd``, ``s2attn_bwd``, ...), taking raw device
  pointers and sizes exactly like ``include/s2attn.h``;
* torch conveniences (``forward``, ``backward``, ``S2AttnFunction``) that allocate outputs
  and the workspace with torch and pass their pointers and the current CUDA stream; and the
  serving step (``page_plan``, ``rope``, ``cache4_append``, ``cache4_attention``).

Importing this module raises ImportError when the library has not been built: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libs2attn.so")

S2_OK, S2_ERR_NULL, S2_ERR_SHAPE, S2_ERR_DTYPE, S2_ERR_HEADDIM, S2_ERR_ALIGN, \
    S2_ERR_WORKSPACE, S2_ERR_CUDA, S2_ERR_DEVICE_TIMEOUT, S2_ERR_ARG, \
    S2_ERR_STALE_WORKSPACE = range(11)
S2_BF16, S2_FP32 = 0, 1
S2_CAUSAL, S2_SHIFT_HALF, S2_SHIFT_ALTERNATE, S2_SHIFT_NONE = 0x01, 0x00, 0x10, 0x20
S2_INJECT_FWD, S2_INJECT_DKDV = 1, 2
S2_ROPE_INTERLEAVED, S2_ROPE_HALF = 0, 1
ROPE_LAYOUTS = {"interleaved": S2_ROPE_INTERLEAVED, "half": S2_ROPE_HALF}
SHIFT_PATTERNS = {"half": S2_SHIFT_HALF, "alternate": S2_SHIFT_ALTERNATE, "none": S2_SHIFT_NONE}
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # S2ATTN_NOALLOC_SCRATCH_BYTES

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libs2attn.so is not built (expected at %s); build it with "
        "`python -m longlora_shifted_sparse_b200.build`" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_SHAPE = [_i] * 7 + [_f, _f, _i]

_lib.s2attn_workspace_bytes.argtypes = [_i] * 6
_lib.s2attn_workspace_bytes.restype = _sz
_lib.s2attn_fwd.argtypes = [_vp] * 5 + _SHAPE + [_vp, _sz, _vp]
_lib.s2attn_fwd.restype = _i
_lib.s2attn_bwd.argtypes = [_vp] * 9 + _SHAPE + [_vp, _sz, _vp]
_lib.s2attn_bwd.restype = _i
_lib.s2attn_bwd_after_fwd.argtypes = [_vp] * 9 + _SHAPE + [_vp, _sz, _vp]
_lib.s2attn_bwd_after_fwd.restype = _i
_lib.s2attn_fwd_noalloc.argtypes = [_vp] * 5 + _SHAPE + [_vp]
_lib.s2attn_fwd_noalloc.restype = _i
_lib.s2attn_noalloc_device_status.argtypes = [_vp]
_lib.s2attn_noalloc_device_status.restype = _i
_lib.s2attn_kernel_path.argtypes = [_i] * 8
_lib.s2attn_kernel_path.restype = _i
_lib.s2attn_selftest_wait_timeout.argtypes = [_vp, _sz, _vp]
_lib.s2attn_selftest_wait_timeout.restype = _i
_lib.s2attn_selftest_inject.argtypes = [_i] + [_vp] * 9 + _SHAPE + [_vp, _sz, _vp]
_lib.s2attn_selftest_inject.restype = _i
_lib.s2attn_selftest_exp2.argtypes = [_vp, _vp, _i, _vp]
_lib.s2attn_selftest_exp2.restype = _i
_lib.s2attn_device_status.argtypes = [_vp, _sz, _vp]
_lib.s2attn_device_status.restype = _i
_ll, _dbl = ctypes.c_longlong, ctypes.c_double
_lib.s2attn_rope_freqs.argtypes = [ctypes.POINTER(_dbl), _i, _dbl, _dbl, _i, _dbl, _dbl]
_lib.s2attn_rope_freqs.restype = _i
_lib.s2attn_rope.argtypes = [_vp] * 5 + [_i, _vp] + [_i] * 6 + [_vp] * 3 + [_i, _i, _f, _i, _vp]
_lib.s2attn_rope.restype = _i
_lib.s2attn_page_plan.argtypes = [_vp] * 10 + [_i] * 4 + [_ll, _i, _vp]
_lib.s2attn_page_plan.restype = _i
_lib.s2attn_cache4_bytes.argtypes = [_i] * 4
_lib.s2attn_cache4_bytes.restype = _sz
_lib.s2attn_cache4_append.argtypes = [_vp] * 4 + [_i] * 5 + [_vp, _vp, _i, _vp]
_lib.s2attn_cache4_append.restype = _i
_lib.s2attn_cache4_read.argtypes = [_vp] * 4 + [_i] * 6 + [_vp]
_lib.s2attn_cache4_read.restype = _i
_lib.s2attn_cache4_workspace_bytes.argtypes = []
_lib.s2attn_cache4_workspace_bytes.restype = _sz
_lib.s2attn_cache4_attn.argtypes = [_vp] * 7 + [_i] * 8 + [_ll, _vp, _i, _f, _i, _vp, _sz, _vp]
_lib.s2attn_cache4_attn.restype = _i
_lib.s2attn_status_string.argtypes = [_i]
_lib.s2attn_status_string.restype = ctypes.c_char_p
_lib.s2attn_profile_enable.argtypes = [_i]
_lib.s2attn_profile_enable.restype = _i
_lib.s2attn_profile_num_kernels.argtypes = []
_lib.s2attn_profile_num_kernels.restype = _i
_lib.s2attn_profile_query.argtypes = [_i, ctypes.POINTER(ctypes.c_char_p),
                                      ctypes.POINTER(_i), ctypes.POINTER(ctypes.c_double)]
_lib.s2attn_profile_query.restype = _i
_lib.s2attn_profile_dropped.argtypes = []
_lib.s2attn_profile_dropped.restype = _i

# C ABI, same names and argument order as include/s2attn.h
s2attn_workspace_bytes = _lib.s2attn_workspace_bytes
s2attn_fwd = _lib.s2attn_fwd
s2attn_bwd = _lib.s2attn_bwd
s2attn_bwd_after_fwd = _lib.s2attn_bwd_after_fwd
s2attn_fwd_noalloc = _lib.s2attn_fwd_noalloc
s2attn_noalloc_device_status = _lib.s2attn_noalloc_device_status
s2attn_kernel_path = _lib.s2attn_kernel_path
s2attn_device_status = _lib.s2attn_device_status
s2attn_selftest_wait_timeout = _lib.s2attn_selftest_wait_timeout
s2attn_selftest_inject = _lib.s2attn_selftest_inject
s2attn_selftest_exp2 = _lib.s2attn_selftest_exp2
s2attn_rope_freqs = _lib.s2attn_rope_freqs
s2attn_rope = _lib.s2attn_rope
s2attn_page_plan = _lib.s2attn_page_plan
s2attn_cache4_bytes = _lib.s2attn_cache4_bytes
s2attn_cache4_append = _lib.s2attn_cache4_append
s2attn_cache4_read = _lib.s2attn_cache4_read
s2attn_cache4_workspace_bytes = _lib.s2attn_cache4_workspace_bytes
s2attn_cache4_attn = _lib.s2attn_cache4_attn
s2attn_profile_enable = _lib.s2attn_profile_enable
s2attn_profile_num_kernels = _lib.s2attn_profile_num_kernels
s2attn_profile_dropped = _lib.s2attn_profile_dropped


def s2attn_status_string(status: int) -> str:
    return _lib.s2attn_status_string(int(status)).decode()


def s2attn_profile_query(kernel_id: int):
    """(name, launches, total_ms) of one kernel id."""
    name = ctypes.c_char_p()
    n = _i()
    ms = ctypes.c_double()
    rc = _lib.s2attn_profile_query(kernel_id, ctypes.byref(name), ctypes.byref(n),
                                   ctypes.byref(ms))
    check(rc)
    return name.value.decode(), n.value, ms.value


def profile_summary():
    """{kernel name: (launches, total_ms)} for every kernel that launched."""
    out = {}
    for i in range(s2attn_profile_num_kernels()):
        name, n, ms = s2attn_profile_query(i)
        if n:
            out[name] = (n, ms)
    return out


class S2Error(RuntimeError):
    def __init__(self, status: int):
        super().__init__("s2attn: %s (status %d)" % (s2attn_status_string(status), status))
        self.status = status


def check(status: int) -> None:
    if status != S2_OK:
        raise S2Error(status)


# ----------------------------------------------------------------------------- torch layer

def _dtype_code(t) -> int:
    _torch or _lazy()
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("s2attn supports bfloat16 and float32 tensors, got %s" % t.dtype)
    return code


def _stream_ptr(device) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def mode(causal: bool = True, shift: str = "half") -> int:
    """The ABI's mode argument: the causal flag ORed with a shifted-head pattern."""
    if shift not in SHIFT_PATTERNS:
        raise ValueError("shift must be one of %s, got %r" % (sorted(SHIFT_PATTERNS), shift))
    return (S2_CAUSAL if causal else 0) | SHIFT_PATTERNS[shift]


def workspace(B, N, Hq, Hkv, d, dtype_code, device):
    import torch
    nbytes = s2attn_workspace_bytes(B, N, Hq, Hkv, d, dtype_code)
    if nbytes == 0:
        raise S2Error(S2_ERR_SHAPE)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def forward(q, k, v, G: int, pi_scale: float, rope_base: float = 10000.0, causal: bool = True,
            ws=None, out=None, lse=None, shift: str = "half", check_status: bool = False):
    """q [B,N,Hq,d], k/v [B,N,Hkv,d] CUDA tensors -> (o, lse). shift picks the shifted
    heads: "half" (the method), "alternate" (odd kv heads) or "none".

    check_status=True waits for the stream after the launch and raises S2Error if a bounded
    wait in a kernel expired (the outputs are then undefined)."""
    import torch
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    dt = _dtype_code(q)
    if ws is None:
        ws = workspace(B, N, Hq, Hkv, d, dt, q.device)
    o = out if out is not None else torch.empty_like(q)
    lse = lse if lse is not None else torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    check(s2attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                     B, N, Hq, Hkv, d, G, mode(causal, shift), pi_scale, rope_base, dt,
                     ws.data_ptr(), ws.numel(), _stream_ptr(q.device)))
    if check_status:
        check(device_status(ws))
    return o, lse


def backward(q, k, v, o, lse, dout, G: int, pi_scale: float, rope_base: float = 10000.0,
             causal: bool = True, ws=None, grads=None, after_forward: bool = False,
             shift: str = "half", check_status: bool = False):
    """Returns (dq, dk, dv) for the forward that produced (o, lse).

    after_forward=True calls s2attn_bwd_after_fwd: `ws` must then be the workspace the
    forward of these q, k used, unchanged since (it holds their rotation).
    check_status=True waits for the stream after the launch and raises S2Error if a bounded
    wait in a kernel expired (the gradients are then undefined)."""
    import torch
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    dt = _dtype_code(q)
    if ws is None:
        if after_forward:
            raise ValueError("after_forward=True needs the forward's workspace")
        ws = workspace(B, N, Hq, Hkv, d, dt, q.device)
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dv = grads
    fn = s2attn_bwd_after_fwd if after_forward else s2attn_bwd
    check(fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                     dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                     B, N, Hq, Hkv, d, G, mode(causal, shift), pi_scale, rope_base, dt,
                     ws.data_ptr(), ws.numel(), _stream_ptr(q.device)))
    if check_status:
        check(device_status(ws))
    return dq, dk, dv


def device_status(ws) -> int:
    """Waits for the current stream, then reads and clears the status word of `ws`."""
    return s2attn_device_status(ws.data_ptr(), ws.numel(), _stream_ptr(ws.device))


def noalloc_device_status(device=None) -> int:
    """Status of the last s2attn_fwd_noalloc on `device` (waits for its current stream)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        return s2attn_noalloc_device_status(_stream_ptr(dev))


def _make_function():
    import torch

    class S2AttnFunction(torch.autograd.Function):
        """Autograd wrapper: o = S2Attn(q, k, v); backward through the library's kernels."""

        @staticmethod
        def forward(ctx, q, k, v, G, pi_scale, rope_base=10000.0, causal=True, shift="half"):
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
            B, N, Hq, d = q.shape
            ws = workspace(B, N, Hq, k.shape[2], d, _dtype_code(q), q.device)
            o, lse = forward(q, k, v, G, pi_scale, rope_base, causal, ws=ws, shift=shift)
            # the workspace keeps the rotated q, k for the backward (q, k are saved too, so
            # autograd's version check catches an in-place change in between)
            ctx.save_for_backward(q, k, v, o, lse, ws)
            ctx.args = (G, pi_scale, rope_base, causal, shift)
            return o

        @staticmethod
        def backward(ctx, do):
            q, k, v, o, lse, ws = ctx.saved_tensors
            G, pi_scale, rope_base, causal, shift = ctx.args
            # The backward's first kernel resets the workspace's status word, so a bounded
            # wait that expired in the forward is read here, before it would be lost, and the
            # backward's own status right after it (the workspace is dropped afterwards):
            # two stream synchronisations per backward.
            check(device_status(ws))
            dq, dk, dv = backward(q, k, v, o, lse, do.contiguous(), G, pi_scale, rope_base, causal,
                                  ws=ws, after_forward=True, shift=shift, check_status=True)
            return dq, dk, dv, None, None, None, None, None

    return S2AttnFunction


_fn = None


def s2_attention(q, k, v, G: int, pi_scale: float, rope_base: float = 10000.0,
                 causal: bool = True, shift: str = "half"):
    """Differentiable S2-Attn on CUDA tensors."""
    global _fn
    if _fn is None:
        _fn = _make_function()
    return _fn.apply(q, k, v, G, pi_scale, rope_base, causal, shift)


# ----------------------------------------------------------------------------- serving
#
# Calls on tensors of another device than the current one make that device current for the
# launch; work goes to that device's current stream. These calls run once per layer and token, so
# their host time counts: the plain case (tensors of the current device, in the layouts that the
# library takes) goes from tensors to the C ABI in one compiled call (csrc/serve_calls.cpp), which
# leaves every other case, and what to say about it, to the code here.

CALLS_PATH = os.path.join(_HERE, "_serve_calls.so")
_torch = _calls = None


def _lazy():
    """torch, imported on the first call, with the names that every call needs."""
    global _torch, _device_now, _raw_stream, _i32, _DTYPES, _forward_ad
    import torch
    _device_now, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _i32, _DTYPES = torch.int32, {torch.bfloat16: S2_BF16, torch.float32: S2_FP32}
    _forward_ad = torch.autograd.forward_ad
    _torch = torch
    return torch


def _load_calls():
    """The compiled serving calls, loaded on the first of them (the training calls do without)."""
    global _calls
    _torch or _lazy()
    if not os.path.exists(CALLS_PATH):
        raise ImportError("_serve_calls.so is not built (expected at %s); build it with "
                          "`python -m longlora_shifted_sparse_b200.build`" % CALLS_PATH)
    from importlib import machinery, util
    spec = util.spec_from_file_location("_serve_calls", CALLS_PATH,
                                        loader=machinery.ExtensionFileLoader("_serve_calls", CALLS_PATH))
    calls = util.module_from_spec(spec)
    spec.loader.exec_module(calls)
    _calls = calls


def _plain(call, *args):
    """What a compiled call returns: outputs, or None where the case is not the plain one."""
    if _calls is None:
        _load_calls()
    if not args[0].is_cuda:   # (before any CUDA call: there may be no device)
        return None
    out = getattr(_calls, call)(*args)
    if type(out) is int and out:
        raise S2Error(out)
    return out


def _call(device, fn, *args) -> None:
    index = device.index
    if index is not None and index == _device_now():
        status = fn(*args, _raw_stream(index))
    else:
        with _torch.cuda.device(device):
            status = fn(*args, _stream_ptr(device))
    if status:
        raise S2Error(status)


def _written(*tensors) -> None:
    """Tells autograd that the library wrote these tensors: a backward pass that saved one before then says so."""
    _torch.autograd.graph.increment_version([t for t in tensors if t is not None and not t.is_inference()])


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _ints(t, name, device, shape=None):
    """Address of a dense int32 CUDA tensor of this device (and shape)."""
    if t.dtype is _i32 and t.device == device and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    if t.dtype is not _i32:
        raise TypeError("%s must be int32, got %s" % (name, t.dtype))
    _need(t.device == device, "%s is on %s, not on %s" % (name, t.device, device))
    raise ValueError("%s must be dense%s" % (name, "" if shape is None else " with shape %s" % (shape,)))


def _table(t, device, R):
    """Columns and row stride of a block table of R requests. Rows may all be one (stride 0), as in a
    table that is expanded over requests which share their pages; a caller that writes refuses that."""
    if t.dtype is not _i32:
        raise TypeError("block_table must be int32, got %s" % t.dtype)
    shape = t.shape
    if len(shape) != 2 or shape[0] != R or t.device != device or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("block_table must be [R, max_pages] on %s with dense rows" % device)
    return shape[1], shape[1] if R == 1 else t.stride(0)


def _dense_like(x):
    """An uninitialised dense tensor of x's shape (empty_like is the quicker call, but keeps strides)."""
    return _torch.empty_like(x) if x.is_contiguous() else _torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _copied(x):
    """A dense copy of x, on 16 bytes (contiguous() returns x itself where only its address or a stride that
    nothing steps along is odd)."""
    return x.clone(memory_format=_torch.contiguous_format)


@functools.lru_cache(maxsize=512)
def _strides(*s):
    return (_ll * len(s))(*s)


def rope_freqs(rotary_dim: int, rope_base: float = 10000.0, pi_scale: float = 1.0,
               original_len: int = 0, slow_turns: float = 1.0, fast_turns: float = 32.0,
               device="cuda"):
    """Frequencies of the channel pairs in turns per token: float64 [rotary_dim / 2] on `device`,
    made once and kept for ``rope``. pi_scale: linear position interpolation; base scaling is a
    larger rope_base; original_len > 0 interpolates by parts (a pair that makes fast_turns or
    more over original_len tokens is kept, slow_turns or fewer interpolated, blended between)."""
    import torch
    host = (_dbl * max(1, int(rotary_dim) // 2))()
    check(s2attn_rope_freqs(host, rotary_dim, rope_base, pi_scale, original_len, slow_turns,
                            fast_turns))
    return torch.tensor(list(host), dtype=torch.float64).to(device)


def _rope_rows(x, name):
    """x with dense, 16-byte aligned channels, and its strides of batch, token and head (a [T, H, d]
    tensor is one batch entry)."""
    st = x.stride()
    if st[-1] != 1 or x.data_ptr() % 16:
        x = _copied(x)
        st = x.stride()
    return x, _strides(st[0], st[1], st[2]) if len(st) == 4 else _strides(0, st[0], st[1])


def _rope_launch(q, k, positions, freqs, layout, mscale, inverse, in_place):
    if not in_place:
        out = _plain("rope", q, k, positions, freqs, layout == "half", mscale, inverse)
        if out is not None:
            return out
    torch = _torch or _lazy()
    dt, dev, shape = _DTYPES.get(q.dtype), q.device, q.shape
    if dt is None:
        _dtype_code(q)
    nd = len(shape)
    if nd == 4:
        B, N, Hq, d = shape
    else:
        _need(nd == 3, "q must be [T, H, d] or [B, N, H, d], got %s" % (tuple(shape),))
        (N, Hq, d), B = shape, 1
    wide = positions.dtype is torch.int64
    if not wide and positions.dtype is not _i32:
        raise TypeError("positions must be int32 or int64, got %s" % positions.dtype)
    if freqs.dtype is not torch.float64:
        raise TypeError("freqs must be float64 (see rope_freqs), got %s" % freqs.dtype)
    pshape, pst = positions.shape, positions.stride()
    if len(pshape) == 1 and pshape[0] == N:
        pst = _strides(0, pst[0])
    else:
        _need(len(pshape) == 2 and pshape[1] == N and pshape[0] in (1, B),
              "positions must be [N] or [B, N], got %s" % (tuple(pshape),))
        pst = _strides(0 if pshape[0] == 1 else pst[0], pst[1])
    _need(freqs.dim() == 1 and freqs.is_contiguous(), "freqs must be one dense row")
    _need(dev == positions.device == freqs.device, "q, positions and freqs must share a device")
    q4, qst = _rope_rows(q, "q")
    out = q if in_place else _dense_like(q)
    kp = kop = kst = kout = None
    Hkv = 0
    same = q4 is q
    if k is not None:
        kshape = k.shape
        _need(k.dtype is q.dtype and k.device == dev, "q and k must share dtype and device")
        _need(len(kshape) == nd and kshape[-1] == d and kshape[:-2] == shape[:-2],
              "q %s and k %s must share all but heads" % (tuple(shape), tuple(kshape)))
        k4, kst = _rope_rows(k, "k")
        same = same and k4 is k
        kout = k if in_place else _dense_like(k)
        Hkv, kp, kop = kshape[-2], k4.data_ptr(), kout.data_ptr()
    if in_place:
        _need(same, "in place needs dense, 16-byte aligned channels")
        _need(all(not _overlaps(x) for x in (q, k) if x is not None), "in place needs rows that do not overlap")
        _need(k is None or not _meet(q, k), "in place needs q and k that do not overlap")
    if B * N * (Hq + Hkv):
        _call(dev, s2attn_rope, q4.data_ptr(), out.data_ptr(), kp, kop, positions.data_ptr(), wide,
              freqs.data_ptr(), B, N, Hq, Hkv, d, 2 * freqs.shape[0], qst, kst, pst,
              ROPE_LAYOUTS[layout], inverse, mscale, dt)
        if in_place:
            _written(q, k)
    return out, kout


def _overlaps(x) -> bool:
    """True where two elements of x may share an address."""
    reach = 0
    for stride, size in sorted(zip(x.stride(), x.shape)):
        if size > 1:
            if stride <= reach:
                return True
            reach += (size - 1) * stride
    return False


def _meet(x, y) -> bool:
    """True where an element of x and one of y (of one type, neither overlapping itself) may share an address."""
    size, apart = x.element_size(), y.data_ptr() - x.data_ptr()
    if x.is_contiguous() and y.is_contiguous():
        return -size * y.numel() < apart < size * x.numel() and x.numel() > 0 < y.numel()
    if x.numel() == 0 or y.numel() == 0:
        return False
    return apart % size != 0 or _meet_at(x.shape, x.stride(), y.shape, y.stride(), apart // size)


@functools.lru_cache(maxsize=4096)
def _meet_at(x_shape, x_strides, y_shape, y_strides, apart) -> bool:
    """The same by shapes and strides, y beginning `apart` elements behind x."""
    # Some sum of a_s * s over the strides s has to be `apart`: a_s runs from minus y's places along s to x's.
    reach = {}
    for shape, steps, way, end in ((x_shape, x_strides, 1, 1), (y_shape, y_strides, -1, 0)):
        for n, s in zip(shape, steps):
            if n > 1:
                reach.setdefault(s, [0, 0])[end] += way * (n - 1)
    strides = sorted(reach, reverse=True)
    tries = 0

    def found(i, left):
        nonlocal tries
        tries += 1
        if tries > 10000:   # (strides of no order: taken to overlap)
            return True
        if i == len(strides):
            return left == 0
        s, (low, high) = strides[i], reach[strides[i]]
        down = sum(reach[r][0] * r for r in strides[i + 1:])
        up = sum(reach[r][1] * r for r in strides[i + 1:])
        return any(found(i + 1, left - a * s) for a in range(max(low, -((up - left) // s)), min(high, (left - down) // s) + 1))

    return found(0, apart)


_rope_fn = None


def _dual() -> bool:
    """True inside a level of forward-mode differentiation: a tensor may carry a tangent that requires_grad does not show."""
    return _forward_ad._current_level >= 0


def _make_rope_function():
    import torch

    class RopeFunction(torch.autograd.Function):
        """Autograd wrapper: the gradient is the same rotation the other way round, a tangent turns as its value."""

        @staticmethod
        def forward(ctx, q, k, positions, freqs, layout, mscale, inverse):
            ctx.save_for_backward(positions, freqs)
            ctx.save_for_forward(positions, freqs)
            ctx.args = (layout, mscale, not inverse)
            return _rope_launch(q, k, positions, freqs, layout, mscale, inverse, False)

        @staticmethod
        def backward(ctx, dq, dk):
            call = (dq, dk, *ctx.saved_tensors, *ctx.args)
            # (the launch itself unless a gradient or tangent of the gradient may be asked for)
            dq, dk = RopeFunction.apply(*call) if torch.is_grad_enabled() or _dual() else _rope_launch(*call, False)
            return dq, dk, None, None, None, None, None

        @staticmethod
        def jvp(ctx, tq, tk, *_):
            layout, mscale, other_way = ctx.args
            return RopeFunction.apply(tq, tk, *ctx.saved_tensors, layout, mscale, not other_way)

    return RopeFunction


def rope(q, k, positions, freqs, layout: str = "interleaved", mscale: float = 1.0,
         in_place: bool = False):
    """Rotary positions of q [B,N,Hq,d] and k [B,N,Hkv,d] (or [T,H,d]; k may be None) -> (q', k').

    positions: int32 or int64, [N] (or [T]) or [B, N]; freqs: ``rope_freqs``, whose length gives
    the rotated channels, the first 2 * len(freqs); the rest pass through. layout: pair i is
    channels (2i, 2i+1) ("interleaved", as in the attention calls) or (i, i + half)
    ("half"). mscale multiplies the rotated channels. Differentiable in q and k (both
    modes); in_place=True overwrites them (they must not overlap) instead and has no gradient. (To
    capture a training step into a graph, drop eager graphs of the same leaves first: torch's accumulation nodes keep the stream
    that they were made on.)"""
    if layout not in ROPE_LAYOUTS:
        raise ValueError("layout must be one of %s, got %r" % (sorted(ROPE_LAYOUTS), layout))
    _torch or _lazy()
    grad = (q.requires_grad or (k is not None and k.requires_grad)) and _torch.is_grad_enabled()
    if not grad and _forward_ad._current_level < 0:   # (_dual(), for a call a token)
        return _rope_launch(q, k, positions, freqs, layout, mscale, False, in_place)
    _need(not in_place, "in_place=True has no gradient")
    global _rope_fn
    if _rope_fn is None:
        _rope_fn = _make_rope_function()
    return _rope_fn.apply(q, k, positions, freqs, layout, mscale, False)


class PagePlan(NamedTuple):
    """What ``page_plan`` gives: see there."""
    cu_new: "torch.Tensor"
    lens: "torch.Tensor"
    positions: "torch.Tensor"
    slots: "torch.Tensor"
    free_count: "torch.Tensor"
    left_out: "torch.Tensor"


def page_plan(cached_lens, new_lens, free_pages, free_count, block_table, page_size: int,
              max_tokens: int) -> PagePlan:
    """Pages, positions and slots of one step's new tokens, from the requests' lengths.

    cached_lens, new_lens [R], free_pages [F], free_count [1], block_table [R, max_pages]: int32
    CUDA tensors. The pages that the new tokens need are taken from the end of
    free_pages[:free_count] and written into block_table (in place, behind each request's own).
    Returns cu_new [R+1], lens [R] (cached + new), positions and slots [max_tokens] (slots -1
    in rows that no request owns), free_count [1] (what is left) and left_out [1]: the number
    of requests that did not fit (too long for the table or for max_tokens, or no pages left),
    whose slots are -1 and whose lengths stay. The rows of block_table must not overlap."""
    out = _plain("page_plan", cached_lens, new_lens, free_pages, free_count, block_table, page_size, max_tokens)
    if out is not None:
        return tuple.__new__(PagePlan, out)
    torch = _torch
    dev, R = cached_lens.device, cached_lens.numel()
    c, n = _ints(cached_lens, "cached_lens", dev, (R,)), _ints(new_lens, "new_lens", dev, (R,))
    f, fc = _ints(free_pages, "free_pages", dev), _ints(free_count, "free_count", dev, (1,))
    cols, stride = _table(block_table, dev, R)
    _need(stride >= cols, "block_table is written: its rows must not overlap")
    rows = (max_tokens + 3) & ~3   # positions and slots on 16 bytes
    out = torch.empty(2 * rows + 2 * R + 3, dtype=_i32, device=dev)
    p = out.data_ptr()
    cu = p + 8 * rows
    _call(dev, s2attn_page_plan, c, n, f, fc, block_table.data_ptr(), cu, cu + 4 * (R + 1), p, p + 4 * rows,
          cu + 4 * (2 * R + 1), R, max_tokens, free_pages.numel(), cols, stride, page_size)
    _written(block_table)
    pos, slots, cu, lens, left, out_of = out.split_with_sizes((rows, rows, R + 1, R, 1, 1))
    if rows != max_tokens:
        pos, slots = pos[:max_tokens], slots[:max_tokens]
    return PagePlan(cu, lens, pos, slots, left, out_of)


def cache4(n_pages: int, page_size: int, Hkv: int, d: int, device="cuda"):
    """An empty 4-bit cache: uint8 [n_pages, Hkv, page_size / 16, 20 d]."""
    import torch
    if s2attn_cache4_bytes(n_pages, page_size, Hkv, d) == 0:
        raise S2Error(S2_ERR_SHAPE)
    return torch.zeros(n_pages, Hkv, page_size // 16, 20 * d, dtype=torch.uint8, device=device)


def _cache4_shape(cache):
    """(n_pages, page_size, Hkv, d) of a cache tensor."""
    torch = _torch or _lazy()
    shape = cache.shape
    if cache.dtype is not torch.uint8 or len(shape) != 4 or shape[3] % 20 or not cache.is_contiguous():
        raise ValueError("cache must be a tensor that cache4() made")
    return shape[0], 16 * shape[2], shape[1], shape[3] // 20


def _cache4_rows(x):
    """x [T, H, d] with rows of 16-byte pieces, and its strides of token and head."""
    s0, s1, s2 = x.stride()
    if s2 != 1 or (x.data_ptr() | (s0 | s1) * x.element_size()) % 16:
        x = _copied(x)
        s0, s1, s2 = x.stride()
    return x, _strides(s0, s1)


def cache4_append(k, v, cache, slots) -> None:
    """Stores k, v [T, Hkv, d] in the cache's slots (int32 [T]; rows with a negative slot, or one
    beyond the cache, are skipped; the others must differ)."""
    if _plain("append", k, v, cache, slots) is not None:
        return
    n_pages, P, Hkv, d = _cache4_shape(cache)
    dev, shape = cache.device, k.shape
    _need(len(shape) == 3 and shape == v.shape and shape[1] == Hkv and shape[2] == d,
          "k %s and v %s must be [T, %d, %d]" % (tuple(shape), tuple(v.shape), Hkv, d))
    _need(k.dtype is v.dtype and k.device == dev and v.device == dev,
          "k, v must share a dtype, and their device with the cache")
    T, dt = shape[0], _dtype_code(k)
    at = _ints(slots, "slots", dev, (T,))
    if T:
        k, ks = _cache4_rows(k)
        v, vs = _cache4_rows(v)
        _call(dev, s2attn_cache4_append, k.data_ptr(), v.data_ptr(), cache.data_ptr(), at, T, Hkv, d,
              n_pages, P, ks, vs, dt)
        _written(cache)


def cache4_read(cache, slots, dtype=None):
    """(k, v) [T, Hkv, d] that the slots (int32 [T]) hold, in bfloat16 or float32; slots outside
    the cache give zeros."""
    out = _plain("read", cache, slots, S2_BF16 if dtype is None else _DTYPES.get(dtype, -1)) if _torch or _lazy() else None
    if out is not None:
        return out
    n_pages, P, Hkv, d = _cache4_shape(cache)
    dev, T = cache.device, slots.numel()
    at = _ints(slots, "slots", dev, (T,))
    k = _torch.empty((T, Hkv, d), dtype=dtype or _torch.bfloat16, device=dev)
    v = _torch.empty_like(k)
    dt = _dtype_code(k)
    if T:
        _call(dev, s2attn_cache4_read, cache.data_ptr(), at, k.data_ptr(), v.data_ptr(), T, Hkv, d,
              n_pages, P, dt)
    return k, v


def cache4_workspace(device="cuda"):
    """The workspace of ``cache4_attention``: one for each stream that runs it, kept between calls."""
    import torch
    return torch.zeros(s2attn_cache4_workspace_bytes(), dtype=torch.uint8, device=device)


def cache4_attention(q, cache, block_table, lens, cu_new, max_new: int, scale=None, ws=None,
                     out=None, return_lse: bool = False):
    """Attention of a step's tokens over all that the cache holds of their requests.

    q [T, Hq, d]; request r has its rows cu_new[r] .. cu_new[r+1]-1 (int32 [R+1]), the pages
    block_table[r] (int32 [R, max_pages]; an expanded row serves requests that share all pages) and
    lens[r] stored tokens, those of this step included (int32 [R]); a row sees its own place and all before. max_new: the largest number
    of rows of a request (known to the caller; it picks the kernel's tile). scale: 1 / sqrt(d)
    by default. ws: ``cache4_workspace``, made anew where it is None. Returns o [T, Hq, d] (out, if
    given, which must not overlap q), or (o, lse) with lse [Hq, T]; rows that no request owns, or one
    whose rows do not all lie within q, are not written. There is no gradient. A row that sees no key
    gets 0 and -inf. ``device_status(ws)`` reads whether a wait inside the call expired."""
    if ws is None:
        ws = cache4_workspace(q.device)
    plain = _plain("attention", q, cache, block_table, lens, cu_new, max_new, scale, ws, out, return_lse)
    if plain is not None:
        return plain
    n_pages, P, Hkv, d = _cache4_shape(cache)
    dev, shape = cache.device, q.shape
    _need(len(shape) == 3 and shape[2] == d and q.device == dev,
          "q must be [T, Hq, %d] on %s, got %s on %s" % (d, dev, tuple(shape), q.device))
    T, Hq, _ = shape
    dt, R = _dtype_code(q), lens.numel()
    ln, cu = _ints(lens, "lens", dev, (R,)), _ints(cu_new, "cu_new", dev, (R + 1,))
    cols, stride = _table(block_table, dev, R)
    if 0 < stride < cols:   # rows that overlap
        block_table, stride = block_table.contiguous(), cols
    q, qs = _cache4_rows(q)
    given = out
    if out is None:
        out = _dense_like(q)
    else:
        _need(out.shape == shape and out.dtype is q.dtype and out.device == dev and
              out.is_contiguous(), "out must be a dense tensor like q")
    lse = _torch.empty((Hq, T), dtype=_torch.float32, device=dev) if return_lse else None
    _need(ws.device == dev, "ws is on %s, not on %s" % (ws.device, dev))
    _need(ws.dtype is _torch.uint8 and ws.is_contiguous(), "ws must be a tensor that cache4_workspace() made")
    if T:
        _call(dev, s2attn_cache4_attn, q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), ln, cu,
              out.data_ptr(), None if lse is None else lse.data_ptr(), R, T, Hq, Hkv, d, n_pages, P,
              cols, stride, qs, max_new, d ** -0.5 if scale is None else scale, dt, ws.data_ptr(),
              ws.numel())
        _written(given)
    return (out, lse) if return_lse else out
