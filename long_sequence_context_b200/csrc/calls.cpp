// calls.cpp -- the ordinary calls of the paged cache without ctypes: the checks,
// the outputs' allocation and the call into libcpattn.so in C++.
//
// A step of one token per request is four or five calls whose kernels take a few
// microseconds each; through ctypes and torch's Python functions the host takes
// 10 to 17 for a call, here 4 to 8.  Every function compares all its arguments
// at once and returns None, having done nothing, when they are not exactly the
// ordinary ones: cpattn.py then goes through its own checks, which name the
// argument that is wrong, and its ctypes calls, which take the rarer ones
// (outputs, workspaces and streams given).  Otherwise it returns the C
// function's status and the outputs.  The library's functions come as addresses
// (bind), so that both ways call the same loaded library.  cpattn.py does without
// this module where it is missing or was built for another torch or Python (tag).
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "cpattn.h"

namespace {

decltype(&cpattn_cache_plan_workspace_bytes) f_plan_ws;
decltype(&cpattn_cache_plan) f_plan;
decltype(&cpattn_cache_append) f_append;
decltype(&cpattn_select_pages) f_select;
decltype(&cpattn_decode_workspace_bytes) f_decode_ws;
decltype(&cpattn_decode) f_decode;

// A contiguous CUDA tensor of the given type and device (any device when dev < 0).
const at::Tensor* plain(PyObject* o, at::ScalarType type, int64_t dims, int dev) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type || t.dim() != dims || !t.is_cuda() || !t.is_contiguous() || t.layout() != at::kStrided)
    return nullptr;
  return dev >= 0 && t.get_device() != dev ? nullptr : &t;
}
bool sized(const at::Tensor* t, std::initializer_list<int64_t> sizes) {
  return t && t->sizes() == c10::IntArrayRef(sizes);
}
bool whole(PyObject* o, long long& x) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  x = PyLong_AsLongLongAndOverflow(o, &over);
  return !over;
}
bool fits_int(long long x) { return x >= 0 && x <= 0x7fffffffLL; }
bool current(int dev) { return c10::cuda::current_device() == dev; }
void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
at::Tensor empty(std::initializer_list<int64_t> sizes, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
}
// `n` elements of one allocation from element `at` on, as a tensor of one dimension.
at::Tensor part(const at::Tensor& all, int64_t at, int64_t n) {
  const int64_t one = 1;
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_sizes_and_strides(c10::IntArrayRef(n), c10::IntArrayRef(one), at);
  return t;
}
PyObject* answer(int status, std::initializer_list<at::Tensor> outputs) {
  PyObject* r = PyTuple_New((Py_ssize_t)outputs.size() + 1);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const at::Tensor& t : outputs) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// The cache's element type: rows' type and code; 8-bit caches need kv_amax.
struct Kind {
  at::ScalarType stored, rows;
  int code, rows_code;
  const float* amax;
};
bool kind_of(PyObject* cache, PyObject* amax, Kind& k) {
  if (!THPVariable_Check(cache)) return false;
  const at::Tensor& t = THPVariable_Unpack(cache);
  k.stored = t.scalar_type();
  k.amax = nullptr;
  if (k.stored == at::kByte) {
    k.rows = at::kBFloat16, k.code = CPATTN_E4M3, k.rows_code = CPATTN_BF16;
    if (!amax) return true;  // not needed for a choice of pages
    if (!t.is_cuda()) return false;
    const at::Tensor* a = plain(amax, at::kFloat, 1, t.get_device());
    if (!sized(a, {2})) return false;
    k.amax = a->const_data_ptr<float>();
    return true;
  }
  if (k.stored != at::kBFloat16 && k.stored != at::kFloat) return false;
  k.rows = k.stored;
  k.code = k.rows_code = k.stored == at::kFloat ? CPATTN_FP32 : CPATTN_BF16;
  return !amax || amax == Py_None;
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return PyErr_Format(PyExc_TypeError, "bind takes six addresses");
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  f_plan_ws = reinterpret_cast<decltype(f_plan_ws)>(p[0]);
  f_plan = reinterpret_cast<decltype(f_plan)>(p[1]);
  f_append = reinterpret_cast<decltype(f_append)>(p[2]);
  f_select = reinterpret_cast<decltype(f_select)>(p[3]);
  f_decode_ws = reinterpret_cast<decltype(f_decode_ws)>(p[4]);
  f_decode = reinterpret_cast<decltype(f_decode)>(p[5]);
  Py_RETURN_NONE;
}

// (lens, delta, block_table, free_ring, free_state, page_size, capacity)
PyObject* cache_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long long page_size, capacity;
  if (n != 7 || !whole(a[5], page_size) || !whole(a[6], capacity) || !fits_int(page_size) || !fits_int(capacity)) Py_RETURN_NONE;
  const at::Tensor* table = plain(a[2], at::kInt, 2, -1);
  if (!table) Py_RETURN_NONE;
  const int dev = table->get_device();
  const int64_t R = table->size(0), width = table->size(1);
  const at::Tensor *lens = plain(a[0], at::kInt, 1, dev), *delta = plain(a[1], at::kInt, 1, dev),
                   *ring = plain(a[3], at::kInt, 1, dev), *state = plain(a[4], at::kInt, 1, dev);
  if (!sized(lens, {R}) || !sized(delta, {R}) || !ring || !sized(state, {2}) || !fits_int(R) || !fits_int(width) ||
      !fits_int(ring->size(0)) || !current(dev))
    Py_RETURN_NONE;
  // the small outputs are one allocation: five take 1 us longer
  const int64_t stretch = (R + 4) / 4 * 4;  // of R + 1 elements, 16-byte aligned
  const at::Tensor small = empty({2 * stretch + 8}, at::kInt, dev), slots = empty({capacity}, at::kLong, dev);
  const at::Tensor lens_out = part(small, 0, R), cu = part(small, stretch, R + 1), state_out = part(small, 2 * stretch, 2),
                   verdict = part(small, 2 * stretch + 4, 1);
  const size_t need = f_plan_ws((int)R, (long)capacity);
  at::Tensor ws;
  if (need) ws = empty({(int64_t)need}, at::kByte, dev);
  void* stream = stream_of(dev);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f_plan(lens->const_data_ptr<int>(), delta->const_data_ptr<int>(), table->mutable_data_ptr<int>(), (int)R,
                  (int)width, (int)page_size, ring->mutable_data_ptr<int>(), state->const_data_ptr<int>(),
                  (int)ring->size(0), lens_out.mutable_data_ptr<int>(), state_out.mutable_data_ptr<int>(),
                  cu.mutable_data_ptr<int>(), slots.mutable_data_ptr<int64_t>(), (long)capacity,
                  verdict.mutable_data_ptr<int>(), need ? ws.mutable_data_ptr() : nullptr, need, stream);
  Py_END_ALLOW_THREADS
  return answer(status, {lens_out, state_out, cu, slots, verdict});
  END_HANDLE_TH_ERRORS
}

// (k_new, v_new, slots, k_cache, v_cache, k_bounds, kv_amax)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Kind kind;
  if (n != 7 || !kind_of(a[3], a[6], kind)) Py_RETURN_NONE;
  const at::Tensor* kc = plain(a[3], kind.stored, 4, -1);
  if (!kc || kc->numel() == 0) Py_RETURN_NONE;
  const int dev = kc->get_device();
  const at::Tensor *vc = plain(a[4], kind.stored, 4, dev), *slots = plain(a[2], at::kLong, 1, dev), *bounds = nullptr;
  if (!vc || vc->sizes() != kc->sizes() || !slots || !THPVariable_Check(a[0]) || !THPVariable_Check(a[1])) Py_RETURN_NONE;
  const int64_t pages = kc->size(0), heads = kc->size(1), P = kc->size(2), D = kc->size(3), N = slots->size(0);
  if (a[5] != Py_None && !sized(bounds = plain(a[5], kind.stored, 4, dev), {pages, heads, 2, D})) Py_RETURN_NONE;
  const at::Tensor &k = THPVariable_Unpack(a[0]), &v = THPVariable_Unpack(a[1]);
  for (const at::Tensor* t : {&k, &v})
    if (t->scalar_type() != kind.rows || !t->is_cuda() || t->get_device() != dev || t->layout() != at::kStrided ||
        t->sizes() != c10::IntArrayRef({N, heads, D}) || t->stride(2) != 1)
      Py_RETURN_NONE;
  if (!fits_int(pages) || !fits_int(heads) || !fits_int(P) || !current(dev)) Py_RETURN_NONE;
  void* stream = stream_of(dev);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f_append(k.const_data_ptr(), v.const_data_ptr(), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                    slots->const_data_ptr<int64_t>(), N, kc->mutable_data_ptr(), vc->mutable_data_ptr(),
                    bounds ? bounds->mutable_data_ptr() : nullptr, (int)heads, (int)D, (int)P, (int)pages, kind.amax,
                    kind.rows_code, kind.code, stream);
  Py_END_ALLOW_THREADS
  return answer(status, {});
  END_HANDLE_TH_ERRORS
}

// (q, k_bounds, block_table, lens, page_size, budget, keep_first)
PyObject* select_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long long page_size, budget, keep;
  Kind kind;
  if (n != 7 || !whole(a[4], page_size) || !whole(a[5], budget) || !whole(a[6], keep) || !kind_of(a[1], nullptr, kind) ||
      !fits_int(page_size) || !fits_int(budget) || keep < 0 || keep >= budget)
    Py_RETURN_NONE;
  const at::Tensor* b = plain(a[1], kind.stored, 4, -1);
  if (!b || b->numel() == 0 || b->size(2) != 2) Py_RETURN_NONE;
  const int dev = b->get_device();
  const at::Tensor *q = plain(a[0], kind.rows, 3, dev), *table = plain(a[2], at::kInt, 2, dev), *lens = plain(a[3], at::kInt, 1, dev);
  const int64_t pages = b->size(0), heads = b->size(1), D = b->size(3);
  if (!q || !table || !lens) Py_RETURN_NONE;
  const int64_t R = table->size(0), width = table->size(1), Hq = q->size(1);
  if (!sized(q, {R, Hq, D}) || !sized(lens, {R}) || Hq % heads != 0 || !fits_int(R) || !fits_int(width) || !fits_int(pages) ||
      !fits_int(Hq) || !current(dev))
    Py_RETURN_NONE;
  const at::Tensor out = empty({R, heads, budget}, at::kInt, dev);
  void* stream = stream_of(dev);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f_select(q->const_data_ptr(), b->const_data_ptr(), table->const_data_ptr<int>(), lens->const_data_ptr<int>(),
                    out.mutable_data_ptr<int>(), (int)R, (int)Hq, (int)heads, (int)D, (int)page_size, (int)width, (int)pages,
                    (int)budget, (int)keep, kind.rows_code, kind.code, stream);
  Py_END_ALLOW_THREADS
  return answer(status, {out});
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, block_table, lens, pages, kv_amax, scale)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Kind kind;
  if (n != 8 || !kind_of(a[1], a[6], kind)) Py_RETURN_NONE;
  const at::Tensor* kc = plain(a[1], kind.stored, 4, -1);
  if (!kc || kc->numel() == 0) Py_RETURN_NONE;
  const int dev = kc->get_device();
  const at::Tensor *vc = plain(a[2], kind.stored, 4, dev), *q = plain(a[0], kind.rows, 3, dev),
                   *table = plain(a[3], at::kInt, 2, dev), *lens = plain(a[4], at::kInt, 1, dev), *list = nullptr;
  if (!vc || vc->sizes() != kc->sizes() || !q || !table || !lens) Py_RETURN_NONE;
  const int64_t pages = kc->size(0), heads = kc->size(1), P = kc->size(2), D = kc->size(3);
  const int64_t R = table->size(0), width = table->size(1), Hq = q->size(1);
  if (!sized(q, {R, Hq, D}) || !sized(lens, {R}) || Hq % heads != 0) Py_RETURN_NONE;
  if (a[5] != Py_None &&
      (!(list = plain(a[5], at::kInt, 3, dev)) || list->size(0) != R || list->size(1) != heads || list->size(2) < 1))
    Py_RETURN_NONE;
  const int64_t budget = list ? list->size(2) : 0;
  double scale;
  if (a[7] == Py_None) scale = 1.0 / std::sqrt((double)D);
  else if (PyFloat_CheckExact(a[7])) scale = PyFloat_AS_DOUBLE(a[7]);
  else Py_RETURN_NONE;
  if (!fits_int(pages) || !fits_int(heads) || !fits_int(P) || !fits_int(R) || !fits_int(width) || !fits_int(Hq) ||
      !fits_int(budget) || !current(dev))
    Py_RETURN_NONE;
  const at::Tensor o = empty({R, Hq, D}, kind.rows, dev), lse = empty({R, Hq}, at::kFloat, dev);
  const size_t need = f_decode_ws((int)R, (int)Hq, (int)heads, (int)D);
  const at::Tensor ws = empty({(int64_t)need}, at::kByte, dev);
  void* stream = stream_of(dev);
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f_decode(q->const_data_ptr(), kc->const_data_ptr(), vc->const_data_ptr(), table->const_data_ptr<int>(),
                    lens->const_data_ptr<int>(), list ? list->const_data_ptr<int>() : nullptr, o.mutable_data_ptr(),
                    lse.mutable_data_ptr<float>(), (int)R, (int)Hq, (int)heads, (int)D, (int)P, (int)width, (int)pages,
                    (int)budget, (float)scale, kind.amax, ws.mutable_data_ptr(), need, kind.rows_code, kind.code,
                    kind.rows_code, stream);
  Py_END_ALLOW_THREADS
  return answer(status, {o, lse});
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"cache_plan", (PyCFunction)(void (*)(void))cache_plan, METH_FASTCALL, nullptr},
    {"cache_append", (PyCFunction)(void (*)(void))cache_append, METH_FASTCALL, nullptr},
    {"select_pages", (PyCFunction)(void (*)(void))select_pages, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void (*)(void))decode, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "tag", CALLS_TAG) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
