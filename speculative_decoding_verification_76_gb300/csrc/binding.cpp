// The host side of extend_tables, release_pages, append_tokens and decode_attn: checks
// the tensors, allocates the outputs and calls the C ABI on the tensors' device and its
// current stream.  These calls run once per drafted token, where a few microseconds of
// kernels sit behind a dozen tensor arguments: checked in Python and marshalled with
// ctypes they cost 11 us of host time each beside the launch, here 2.
//
// Every entry point catches what is thrown: a refused argument is a ValueError, a status
// other than SPEC_OK a SpecError, PyTorch's own errors are passed on.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <sstream>

#include "../../include/spec_verify.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {  // -> ValueError
  std::string what;
};
struct Failed {  // -> SpecError
  const char* fn;
  spec_status code;
};

template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused{s.str()};
}

void check(const char* fn, spec_status code) {
  if (code != SPEC_OK) throw Failed{fn, code};
}

const Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    refuse(name, " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

const Tensor& tensor_on(PyObject* o, const char* name, c10::Device dev) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).device() != dev)
    refuse(name, " must be a tensor on ", dev);
  return THPVariable_Unpack(o);
}

// The address of a contiguous tensor of this type and shape on `dev`.
template <typename T = int32_t>
T* plain(PyObject* o, const char* name, c10::Device dev, ScalarType type, at::IntArrayRef shape) {
  const Tensor& t = tensor_on(o, name, dev);
  if (t.scalar_type() != type) refuse(name, " must be ", type, ", got ", t.scalar_type());
  if (t.sizes() != shape) refuse(name, " has shape ", t.sizes(), ", expected ", shape);
  if (!t.is_contiguous()) refuse(name, " must be contiguous");
  return static_cast<T*>(t.data_ptr());
}

bool given(PyObject* o) { return o != Py_None; }

int64_t whole(PyObject* o, const char* name, int64_t least) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < least || v > INT_MAX) refuse(name, " must be from ", least, " to 2^31 - 1, got ", v);
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

Tensor empty(at::IntArrayRef shape, ScalarType type, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

spec_dtype code_of(ScalarType t) {
  return t == at::kFloat ? SPEC_F32 : t == at::kBFloat16 ? SPEC_BF16
         : t == at::kHalf ? SPEC_F16 : SPEC_E4M3;
}

struct Caches {
  void *k, *v;
  spec_dtype type;
  int pages, P, Hkv, D;
  int64_t page, token, head;  // strides
};

Caches caches(PyObject* ko, PyObject* vo, c10::Device dev, ScalarType rows) {
  const Tensor& k = tensor_on(ko, "k_cache", dev);
  const Tensor& v = tensor_on(vo, "v_cache", dev);
  if (k.dim() != 4 || v.sizes() != k.sizes())
    refuse("caches must be [pages, page_size, Hkv, D], both alike");
  if (v.scalar_type() != k.scalar_type()) refuse("k_cache and v_cache must have one dtype");
  if (k.scalar_type() != rows &&
      (k.scalar_type() != at::kFloat8_e4m3fn || rows == at::kFloat))
    refuse("caches must be ", rows, rows == at::kFloat ? "" : " or Float8_e4m3fn");
  if (k.stride(3) != 1 || v.strides() != k.strides())
    refuse("caches must have the same strides, 1 over D");
  if (k.size(0) > INT_MAX || k.size(1) > INT_MAX || k.size(2) > INT_MAX || k.size(3) > INT_MAX)
    refuse("cache sizes must be below 2^31");
  return {k.data_ptr(), v.data_ptr(), code_of(k.scalar_type()), (int)k.size(0), (int)k.size(1),
          (int)k.size(2), (int)k.size(3), k.stride(0), k.stride(1), k.stride(2)};
}

const float* scale(PyObject* o, const char* name, const Caches& c, c10::Device dev) {
  if (!given(o)) return nullptr;
  if (c.type != SPEC_E4M3) refuse("scales belong to Float8_e4m3fn caches");
  return plain<float>(o, name, dev, at::kFloat, {c.Hkv});
}

// [T, heads, D] rows whose heads lie side by side; *stride: from row to row.
void* rows(PyObject* o, const char* name, c10::Device dev, ScalarType type, int64_t T,
           int64_t heads, int64_t D, int64_t* stride) {
  const Tensor& t = tensor_on(o, name, dev);
  if (t.scalar_type() != type) refuse(name, " must be ", type, ", got ", t.scalar_type());
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != D)
    refuse(name, " must be [tokens, ", heads, ", ", D, "], got ", t.sizes());
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D))
    refuse(name, ": a row's heads must lie side by side");
  if (t.size(0) != T) refuse(name, ": all must have the same rows");
  *stride = t.stride(0);
  return t.data_ptr();
}

// ------------------------------------------------------------------ the four calls
PyObject* extend_tables(PyObject* const* a) {
  const Tensor& ctx = cuda_tensor(a[0], "ctx_len");
  const auto dev = ctx.device();
  const c10::cuda::CUDAGuard guard(dev);
  const auto i32 = at::kInt;
  const Tensor& tab = tensor_on(a[2], "block_table", dev);
  const Tensor& lst = tensor_on(a[3], "free_list", dev);
  if (ctx.dim() != 1 || tab.dim() != 2 || lst.dim() != 1)
    refuse("ctx_len [B], block_table [B, max_pages], free_list [num_pages]");
  const int64_t B = ctx.size(0), width = tab.size(1), n = lst.size(0);
  const int64_t P = whole(a[5], "page_size", 1), cap = whole(a[6], "max_tokens", 0);
  if (B > INT_MAX || width > INT_MAX || n > INT_MAX) refuse("sizes must be below 2^31");
  const int32_t* c = plain(a[0], "ctx_len", dev, i32, {B});
  const int32_t* add = plain(a[1], "add_len", dev, i32, {B});
  int32_t* table = plain(a[2], "block_table", dev, i32, {B, width});
  const int32_t* list = plain(a[3], "free_list", dev, i32, {n});
  const int32_t* count = plain(a[4], "free_count", dev, i32, {1});
  static const char* const names[6] = {"slot_map", "positions", "cu_len",
                                       "new_len",  "free_count", "status"};
  const int64_t sizes[6] = {cap, cap, B + 1, B, 1, B};
  THPObjectPtr made;
  PyObject* out = a[7];
  if (!given(out)) {
    made = PyDict_New();
    if (!made) throw python_error();
    for (int i = 0; i < 6; ++i) {
      THPObjectPtr t(THPVariable_Wrap(empty({sizes[i]}, i == 0 ? at::kLong : i32, dev)));
      if (!t || PyDict_SetItemString(made.get(), names[i], t.get())) throw python_error();
    }
    out = made.get();
  } else if (!PyDict_Check(out)) {
    refuse("out must be the dict of an earlier call");
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    PyObject* o = PyDict_GetItemString(out, names[i]);
    if (!o) refuse("out has no ", names[i]);
    p[i] = plain<void>(o, names[i], dev, i == 0 ? at::kLong : i32, {sizes[i]});
  }
  check("spec_extend_tables",
        spec_extend_tables(c, add, (int)B, (int)P, table, (int)width, list, (int)n, count,
                           (int)cap, static_cast<int64_t*>(p[0]), static_cast<int32_t*>(p[1]),
                           static_cast<int32_t*>(p[2]), static_cast<int32_t*>(p[3]),
                           static_cast<int32_t*>(p[4]), static_cast<int32_t*>(p[5]),
                           stream_of(dev)));
  Py_INCREF(out);
  return out;
}

PyObject* release_pages(PyObject* const* a) {
  const Tensor& len = cuda_tensor(a[1], "length");
  const auto dev = len.device();
  const c10::cuda::CUDAGuard guard(dev);
  const auto i32 = at::kInt;
  const Tensor& tab = tensor_on(a[0], "block_table", dev);
  const Tensor& lst = tensor_on(a[3], "free_list", dev);
  if (len.dim() != 1 || tab.dim() != 2 || lst.dim() != 1)
    refuse("length [B], block_table [B, max_pages], free_list [num_pages]");
  const int64_t B = len.size(0), width = tab.size(1), n = lst.size(0);
  const int64_t P = whole(a[5], "page_size", 1);
  if (B > INT_MAX || width > INT_MAX || n > INT_MAX) refuse("sizes must be below 2^31");
  const int32_t* table = plain(a[0], "block_table", dev, i32, {B, width});
  const int32_t* held = plain(a[1], "length", dev, i32, {B});
  const int32_t* keep = plain(a[2], "keep_pages", dev, i32, {B});
  int32_t* list = plain(a[3], "free_list", dev, i32, {n});
  const int32_t* count = plain(a[4], "free_count", dev, i32, {1});
  THPObjectPtr made[2];
  PyObject* out[2] = {a[6], a[7]};
  for (int i = 0; i < 2; ++i)
    if (!given(out[i])) {
      made[i] = THPVariable_Wrap(empty({i ? B : 1}, i32, dev));
      if (!made[i]) throw python_error();
      out[i] = made[i].get();
    }
  check("spec_release_pages",
        spec_release_pages(table, (int)width, held, keep, (int)B, (int)P, list, (int)n, count,
                           plain(out[0], "total", dev, i32, {1}),
                           plain(out[1], "status", dev, i32, {B}), stream_of(dev)));
  return PyTuple_Pack(2, out[0], out[1]);
}

PyObject* append_tokens(PyObject* const* a) {
  const Tensor& kn = cuda_tensor(a[0], "k_new");
  const auto dev = kn.device();
  const c10::cuda::CUDAGuard guard(dev);
  const auto type = kn.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
    refuse("k_new must be bf16, fp16 or fp32");
  const Caches c = caches(a[2], a[3], dev, type);
  if (kn.dim() != 3) refuse("k_new must be [tokens, ", c.Hkv, ", ", c.D, "]");
  const int64_t T = kn.size(0);
  if (T > INT_MAX) refuse("tokens must be below 2^31");
  int64_t ks, vs, qs = 0, os = 0;
  const void* k = rows(a[0], "k_new", dev, type, T, c.Hkv, c.D, &ks);
  const void* v = rows(a[1], "v_new", dev, type, T, c.Hkv, c.D, &vs);
  const int64_t* slots = plain<int64_t>(a[4], "slot_map", dev, at::kLong, {T});
  const double base = number(a[8]);
  const int32_t* pos = nullptr;
  if (given(a[5]))
    pos = plain(a[5], "positions", dev, at::kInt, {T});
  else if (base != 0.0)
    refuse("positions are needed to rotate (rope_base 0: no rotation)");
  int64_t Hq = 0;
  const void* q = nullptr;
  void* qo = nullptr;
  PyObject* out = a[7];
  THPObjectPtr made;
  if (given(a[6])) {
    const Tensor& qt = tensor_on(a[6], "q", dev);
    if (qt.dim() != 3 || qt.size(0) != T) refuse("q must be [tokens, Hq, D]");
    Hq = qt.size(1);
    if (Hq > INT_MAX) refuse("heads must be below 2^31");
    q = rows(a[6], "q", dev, type, T, Hq, c.D, &qs);
    if (!given(out)) {
      made = THPVariable_Wrap(
          at::zeros({T, Hq, c.D}, at::TensorOptions().dtype(type).device(dev)));
      if (!made) throw python_error();
      out = made.get();
    }
    qo = rows(out, "q_out", dev, type, T, Hq, c.D, &os);
  } else if (given(out)) {
    refuse("q_out without q");
  }
  const float* sk = scale(a[9], "k_scale", c, dev);
  const float* sv = scale(a[10], "v_scale", c, dev);
  check("spec_append_tokens",
        spec_append_tokens(k, ks, v, vs, q, qs, qo, os, code_of(type), c.k, c.v, c.type, sk, sv,
                           c.pages, c.P, c.page, c.token, c.head, slots, pos, (int)T, (int)Hq,
                           c.Hkv, c.D, base, stream_of(dev)));
  Py_INCREF(out);
  return out;
}

PyObject* decode_attn(PyObject* const* a) {
  const Tensor& q = cuda_tensor(a[0], "q");
  const auto dev = q.device();
  const c10::cuda::CUDAGuard guard(dev);
  const auto type = q.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf) refuse("q must be bf16 or fp16");
  if (q.dim() != 3 || q.stride(2) != 1) refuse("q must be [B, Hq, D], contiguous over D");
  const Caches c = caches(a[1], a[2], dev, type);
  const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
  if (D != c.D) refuse("head_dim mismatch");
  const Tensor& tab = tensor_on(a[3], "block_table", dev);
  if (tab.dim() != 2) refuse("block_table must be [B, max_pages]");
  const int64_t width = tab.size(1);
  if (B > INT_MAX || Hq > INT_MAX || width > INT_MAX) refuse("sizes must be below 2^31");
  const int32_t* table = plain(a[3], "block_table", dev, at::kInt, {B, width});
  const int32_t* lens = plain(a[4], "seq_len", dev, at::kInt, {B});
  const double sm_scale = number(a[5]);
  const int64_t window = whole(a[6], "window", 0);
  const float* sk = scale(a[7], "k_scale", c, dev);
  const float* sv = scale(a[8], "v_scale", c, dev);
  Tensor ws;
  if (given(a[9])) {
    if (!THPVariable_Check(a[9]) || THPVariable_Unpack(a[9]).device() != dev ||
        THPVariable_Unpack(a[9]).scalar_type() != at::kByte ||
        !THPVariable_Unpack(a[9]).is_contiguous())
      refuse("workspace must come from new_workspace on q's device");
    ws = THPVariable_Unpack(a[9]);
  } else {
    const size_t need = spec_decode_attn_workspace_size((int)B, (int)Hq, c.Hkv, (int)D);
    ws = at::zeros({(int64_t)(need < 256 ? 256 : need)},
                   at::TensorOptions().dtype(at::kByte).device(dev));
  }
  THPObjectPtr made[2];
  PyObject* out[2] = {a[10], a[11]};
  for (int i = 0; i < 2; ++i)
    if (!given(out[i])) {
      made[i] = THPVariable_Wrap(i ? empty({B, Hq}, at::kFloat, dev) : empty({B, Hq, D}, type, dev));
      if (!made[i]) throw python_error();
      out[i] = made[i].get();
    }
  void* o = plain<void>(out[0], "out", dev, type, {B, Hq, D});
  float* lse = plain<float>(out[1], "lse", dev, at::kFloat, {B, Hq});
  check("spec_decode_attn",
        spec_decode_attn(q.data_ptr(), q.stride(0), q.stride(1), code_of(type), c.k, c.v, c.type,
                         sk, sv, c.pages, c.P, c.page, c.token, c.head, table, (int)width, lens,
                         (int)B, (int)Hq, c.Hkv, (int)D, (int)window, (float)sm_scale,
                         ws.data_ptr(), (size_t)ws.numel(), o, lse, stream_of(dev)));
  return PyTuple_Pack(2, out[0], out[1]);
}

// ------------------------------------------------------------------ the module
PyObject* g_spec_error = nullptr;  // the package's SpecError

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const Failed& e) {
    PyObject* x = g_spec_error ? PyObject_CallFunction(g_spec_error, "sis", e.fn, (int)e.code,
                                                       spec_status_str(e.code))
                               : nullptr;
    if (x) {
      PyErr_SetObject(g_spec_error, x);
      Py_DECREF(x);
    } else if (!PyErr_Occurred()) {
      PyErr_Format(PyExc_RuntimeError, "%s failed: %s", e.fn, spec_status_str(e.code));
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_spec_error);
  g_spec_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyModuleDef* module_def() {
  static PyMethodDef methods[] = {method<extend_tables, 8>("extend_tables"),
                                  method<release_pages, 8>("release_pages"),
                                  method<append_tokens, 11>("append_tokens"),
                                  method<decode_attn, 12>("decode_attn"),
                                  {"set_error", set_error, METH_O, nullptr},
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1,     methods,
                            nullptr,               nullptr,   nullptr, nullptr};
  return &def;
}

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(module_def()); }
