// The serving calls of the torch layer, from tensors to the C ABI without Python in between: they
// run once per layer and token, where 8 us of checks and marshalling in Python are more than the
// kernels take. A call here handles the plain case (CUDA tensors of the current device, dense channels,
// every argument as documented) and returns None for anything else: the Python layer then goes
// through its own checks and either makes the call or says what is wrong. Otherwise it returns the
// outputs, or the status code of a call that the library refused.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "s2attn.h"

namespace {

using at::Tensor;

const Tensor* tensor(PyObject* x) { return THPVariable_CheckExact(x) ? &THPVariable_Unpack(x) : nullptr; }

// Code of a dtype, or -1.
int code_of(at::ScalarType t) { return t == at::kBFloat16 ? S2_BF16 : t == at::kFloat ? S2_FP32 : -1; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// On the current device.
bool here(const Tensor& t, int device) { return t.is_cuda() && t.get_device() == device; }

bool ints(const Tensor* t, int device, int64_t count) {
  return t && t->scalar_type() == at::kInt && here(*t, device) && t->dim() == 1 && t->is_contiguous() &&
         (count < 0 || t->numel() == count);
}

// A block table of R requests: dense rows that do not overlap or, where they are only read, all the same row.
bool table_ok(const Tensor* t, int device, int64_t R, bool one_row) {
  return t && t->scalar_type() == at::kInt && here(*t, device) && t->dim() == 2 && t->size(0) == R && R > 0 &&
         t->size(1) > 0 && t->size(1) <= INT_MAX && (t->size(1) == 1 || t->stride(1) == 1) &&
         (R == 1 || t->stride(0) >= t->size(1) || (one_row && t->stride(0) == 0));
}
// (The stride of a single row says nothing.)
long long table_stride(const Tensor& t) { return t.size(0) == 1 ? t.size(1) : t.stride(0); }

struct Cache {
  int pages, page, heads, d;
};
bool cache_ok(const Tensor* t, int device, Cache& c) {
  if (!t || t->scalar_type() != at::kByte || !here(*t, device) || t->dim() != 4 || !t->is_contiguous()) return false;
  for (int i = 0; i < 4; i++)
    if (t->size(i) > INT_MAX / 16) return false;
  c = {(int)t->size(0), (int)t->size(2) * 16, (int)t->size(1), (int)t->size(3) / 20};
  return t->size(3) % 20 == 0;
}

// Rows [T, H, d] in 16-byte pieces.
bool rows_ok(const Tensor& t) {
  return t.dim() == 3 && t.stride(2) == 1 && aligned16(t.data_ptr()) &&
         (t.stride(0) * t.element_size()) % 16 == 0 && (t.stride(1) * t.element_size()) % 16 == 0;
}

bool number(PyObject* x, long long& v) {
  if (!PyLong_CheckExact(x)) return false;
  int over = 0;
  v = PyLong_AsLongLongAndOverflow(x, &over);
  return over == 0 && v >= INT_MIN && v <= INT_MAX;
}
bool number(PyObject* x, float& v) {
  if (PyFloat_CheckExact(x)) {
    v = (float)PyFloat_AS_DOUBLE(x);
    return true;
  }
  long long i;
  if (!number(x, i)) return false;
  v = (float)i;
  return true;
}

void* stream(int device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }

// Tells autograd that the library wrote this tensor: a backward pass that saved it before then says so.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject* refused(int status) { return PyLong_FromLong(status); }

PyObject* pair(const Tensor& a, PyObject* b) {
  PyObject* t = PyTuple_New(2);
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

// rope(q, k, positions, freqs, half, mscale, inverse) -> (q', k')
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0]), *k = a[1] == Py_None ? nullptr : tensor(a[1]), *pos = tensor(a[2]), *f = tensor(a[3]);
  float mscale;
  if (!q || (!k && a[1] != Py_None) || !pos || !f || !number(a[5], mscale)) Py_RETURN_NONE;
  const int device = c10::cuda::current_device(), dt = code_of(q->scalar_type());
  const int64_t nd = q->dim();
  if (dt < 0 || !here(*q, device) || !here(*pos, device) || !here(*f, device) || (nd != 3 && nd != 4)) Py_RETURN_NONE;
  const bool wide = pos->scalar_type() == at::kLong;
  if ((!wide && pos->scalar_type() != at::kInt) || f->scalar_type() != at::kDouble || f->dim() != 1 || !f->is_contiguous())
    Py_RETURN_NONE;
  const int64_t B = nd == 4 ? q->size(0) : 1, N = q->size(nd - 3), Hq = q->size(nd - 2), d = q->size(nd - 1);
  if (q->numel() == 0 || B * N > INT_MAX || Hq > INT_MAX || d > 256 || f->numel() > 128) Py_RETURN_NONE;
  long long ps[2];
  if (pos->dim() == 1 && pos->size(0) == N) {
    ps[0] = 0;
    ps[1] = pos->stride(0);
  } else if (pos->dim() == 2 && pos->size(1) == N && (pos->size(0) == 1 || pos->size(0) == B)) {
    ps[0] = pos->size(0) == 1 ? 0 : pos->stride(0);
    ps[1] = pos->stride(1);
  } else {
    Py_RETURN_NONE;
  }
  if (q->stride(nd - 1) != 1 || !aligned16(q->data_ptr())) Py_RETURN_NONE;
  const long long qs[3] = {nd == 4 ? q->stride(0) : 0, q->stride(nd - 3), q->stride(nd - 2)};
  long long ks[3] = {};
  int64_t Hkv = 0;
  if (k) {
    if (k->scalar_type() != q->scalar_type() || !here(*k, device) || k->dim() != nd || k->size(nd - 1) != d ||
        k->size(nd - 3) != N || (nd == 4 && k->size(0) != B) || k->numel() == 0 || k->size(nd - 2) > INT_MAX ||
        k->stride(nd - 1) != 1 || !aligned16(k->data_ptr()))
      Py_RETURN_NONE;
    Hkv = k->size(nd - 2);
    ks[0] = nd == 4 ? k->stride(0) : 0;
    ks[1] = k->stride(nd - 3);
    ks[2] = k->stride(nd - 2);
  }
  const Tensor qo = at::empty(q->sizes(), q->options()), ko = k ? at::empty(k->sizes(), k->options()) : Tensor();
  const int status = s2attn_rope(q->data_ptr(), qo.data_ptr(), k ? k->data_ptr() : nullptr, k ? ko.data_ptr() : nullptr,
                                 pos->data_ptr(), wide, static_cast<const double*>(f->data_ptr()), (int)B, (int)N, (int)Hq,
                                 (int)Hkv, (int)d, 2 * (int)f->numel(), qs, k ? ks : nullptr, ps,
                                 PyObject_IsTrue(a[4]) ? S2_ROPE_HALF : S2_ROPE_INTERLEAVED, PyObject_IsTrue(a[6]), mscale, dt,
                                 stream(device));
  if (status) return refused(status);
  return pair(qo, k ? THPVariable_Wrap(ko) : Py_NewRef(Py_None));
}

// page_plan(cached, new, free, free_count, table, page_size, max_tokens) -> cu_new, lens, positions, slots, free_count, left_out
PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) Py_RETURN_NONE;
  const Tensor *cached = tensor(a[0]), *fresh = tensor(a[1]), *free = tensor(a[2]), *count = tensor(a[3]), *table = tensor(a[4]);
  long long page, T;
  const int device = c10::cuda::current_device();
  if (!ints(cached, device, -1) || !number(a[5], page) || !number(a[6], T) || T < 0 || T > INT_MAX - 4) Py_RETURN_NONE;
  const int64_t R = cached->numel();
  if (R > 4096 || !ints(fresh, device, R) || !ints(free, device, -1) || free->numel() > INT_MAX || !ints(count, device, 1) ||
      !table_ok(table, device, R, false))
    Py_RETURN_NONE;
  const int64_t rows = (T + 3) & ~3LL;  // positions and slots on 16 bytes
  const Tensor out = at::empty({2 * rows + 2 * R + 3}, cached->options());
  int* p = static_cast<int*>(out.data_ptr());
  int* cu = p + 2 * rows;
  const int status = s2attn_page_plan(
      static_cast<const int*>(cached->data_ptr()), static_cast<const int*>(fresh->data_ptr()),
      static_cast<const int*>(free->data_ptr()), static_cast<const int*>(count->data_ptr()),
      static_cast<int*>(table->data_ptr()), cu, cu + R + 1, p, p + rows, cu + 2 * R + 1, (int)R, (int)T, (int)free->numel(),
      (int)table->size(1), table_stride(*table), (int)page, stream(device));
  if (status) return refused(status);
  written(*table);
  at::AutoDispatchBelowADInplaceOrView plain;  // whole numbers: no views to track
  const int64_t at[6] = {2 * rows, 2 * rows + R + 1, 0, rows, 2 * rows + 2 * R + 1, 2 * rows + 2 * R + 2};
  const int64_t len[6] = {R + 1, R, T, T, 1, 1};
  PyObject* t = PyTuple_New(6);
  for (int i = 0; i < 6; i++) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(out.as_strided({len[i]}, {1}, at[i])));
  return t;
}

// append(k, v, cache, slots) -> 0
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) Py_RETURN_NONE;
  const Tensor *k = tensor(a[0]), *v = tensor(a[1]), *cache = tensor(a[2]), *slots = tensor(a[3]);
  const int device = c10::cuda::current_device();
  Cache c;
  if (!k || !v || !cache_ok(cache, device, c) || !here(*k, device) || !here(*v, device)) Py_RETURN_NONE;
  const int dt = code_of(k->scalar_type());
  if (dt < 0 || v->scalar_type() != k->scalar_type() || !rows_ok(*k) || !rows_ok(*v) || !k->sizes().equals(v->sizes()) ||
      k->size(1) != c.heads || k->size(2) != c.d || k->size(0) == 0 || k->size(0) > INT_MAX || !ints(slots, device, k->size(0)))
    Py_RETURN_NONE;
  const long long ks[2] = {k->stride(0), k->stride(1)}, vs[2] = {v->stride(0), v->stride(1)};
  const int status = s2attn_cache4_append(k->data_ptr(), v->data_ptr(), cache->data_ptr(), static_cast<const int*>(slots->data_ptr()),
                                          (int)k->size(0), c.heads, c.d, c.pages, c.page, ks, vs, dt, stream(device));
  if (status == S2_OK) written(*cache);
  return refused(status);
}

// read(cache, slots, code) -> (k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) Py_RETURN_NONE;
  const Tensor *cache = tensor(a[0]), *slots = tensor(a[1]);
  const int device = c10::cuda::current_device();
  Cache c;
  long long dt;
  if (!cache_ok(cache, device, c) || !ints(slots, device, -1) || !number(a[2], dt) || dt < 0 || slots->numel() == 0 ||
      slots->numel() > INT_MAX)
    Py_RETURN_NONE;
  const auto options = cache->options().dtype(dt == S2_BF16 ? at::kBFloat16 : at::kFloat);
  const Tensor k = at::empty({slots->numel(), c.heads, c.d}, options), v = at::empty({slots->numel(), c.heads, c.d}, options);
  const int status = s2attn_cache4_read(cache->data_ptr(), static_cast<const int*>(slots->data_ptr()), k.data_ptr(), v.data_ptr(),
                                        (int)slots->numel(), c.heads, c.d, c.pages, c.page, (int)dt, stream(device));
  return status ? refused(status) : pair(k, THPVariable_Wrap(v));
}

// attention(q, cache, table, lens, cu_new, max_new, scale, ws, out, return_lse) -> o, or (o, lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) Py_RETURN_NONE;
  const Tensor *q = tensor(a[0]), *cache = tensor(a[1]), *table = tensor(a[2]), *lens = tensor(a[3]), *cu = tensor(a[4]),
               *ws = tensor(a[7]), *given = tensor(a[8]);
  const int device = c10::cuda::current_device();
  Cache c;
  long long max_new;
  if (!q || !here(*q, device) || !rows_ok(*q) || !cache_ok(cache, device, c) || !ints(lens, device, -1) || !number(a[5], max_new))
    Py_RETURN_NONE;
  const int64_t R = lens->numel(), T = q->size(0), Hq = q->size(1);
  const int dt = code_of(q->scalar_type());
  float scale = c.d > 0 ? (float)std::pow((double)c.d, -0.5) : 0.f;
  if (dt < 0 || q->size(2) != c.d || T == 0 || T > INT_MAX || Hq > INT_MAX || R > INT_MAX - 1 || !ints(cu, device, R + 1) ||
      !table_ok(table, device, R, true) || (a[6] != Py_None && !number(a[6], scale)) || !ws || !here(*ws, device) || ws->dim() != 1 ||
      ws->scalar_type() != at::kByte || !ws->is_contiguous() ||
      (!given && a[8] != Py_None))
    Py_RETURN_NONE;
  if (given && (!here(*given, device) || given->scalar_type() != q->scalar_type() || !given->sizes().equals(q->sizes()) ||
                !given->is_contiguous()))
    Py_RETURN_NONE;
  const Tensor o = given ? *given : at::empty(q->sizes(), q->options());
  const bool with_lse = PyObject_IsTrue(a[9]);
  const Tensor lse = with_lse ? at::empty({Hq, T}, q->options().dtype(at::kFloat)) : Tensor();
  const long long qs[2] = {q->stride(0), q->stride(1)};
  const int status = s2attn_cache4_attn(
      q->data_ptr(), cache->data_ptr(), static_cast<const int*>(table->data_ptr()), static_cast<const int*>(lens->data_ptr()),
      static_cast<const int*>(cu->data_ptr()), o.data_ptr(), with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, (int)R,
      (int)T, (int)Hq, c.heads, c.d, c.pages, c.page, (int)table->size(1), table_stride(*table), qs, (int)max_new, scale, dt,
      ws->data_ptr(), ws->numel(), stream(device));
  if (status) return refused(status);
  if (given) written(*given);
  PyObject* out = given ? Py_NewRef(a[8]) : THPVariable_Wrap(o);
  if (!with_lse) return out;
  PyObject* t = PyTuple_New(2);
  PyTuple_SET_ITEM(t, 0, out);
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(lse));
  return t;
}

// A C++ exception (torch is out of memory, say) becomes the Python one that torch would raise.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return F(self, a, n);
  END_HANDLE_TH_ERRORS
}

#define CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(rope), CALL(page_plan), CALL(append), CALL(read), CALL(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__serve_calls() { return PyModule_Create(&module); }
