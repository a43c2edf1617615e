// The host side of the calls of a serving step (tables, appends, rotation, scaled caches,
// one-token and scaled-cache attention, served logits): checks
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
#include <vector>

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

// ------------------------------------------------------------------ scaled caches and their step
struct Rope {  // a Python Rope as the C struct, and its own frequencies
  spec_rope c{};
  std::vector<double> freqs;
};

const spec_rope* rope_of(PyObject* o, Rope* r) {
  if (!given(o)) return nullptr;
  // Rope keeps its numbers as one tuple, in spec_rope's order (attributes one by one cost 1 us)
  THPObjectPtr t(PyObject_GetAttrString(o, "_c"));
  if (!t || !PyTuple_Check(t.get()) || PyTuple_GET_SIZE(t.get()) != 10) {
    PyErr_Clear();
    refuse("rope must be a Rope");
  }
  auto item = [&](int i) { return PyTuple_GET_ITEM(t.get(), i); };
  r->c.dim = (int32_t)whole(item(0), "rope.dim", 0);
  r->c.interleaved = (int32_t)whole(item(1), "rope.interleaved", 0);
  r->c.scaling = (int32_t)whole(item(2), "rope.scaling", 0);
  double* to[6] = {&r->c.base, &r->c.factor, &r->c.original_len,
                   &r->c.low,  &r->c.high,   &r->c.magnitude};
  for (int i = 0; i < 6; ++i) *to[i] = number(item(3 + i));
  if (given(item(9))) {
    PyObject* f = item(9);
    if (!PyTuple_Check(f) || PyTuple_GET_SIZE(f) != r->c.dim / 2)
      refuse("rope.freqs must hold dim / 2 numbers");
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(f); ++i)
      r->freqs.push_back(number(PyTuple_GET_ITEM(f, i)));
    r->c.freqs = r->freqs.data();
  }
  return &r->c;
}

// Bytes that a tensor spans, for outputs that must not lie over inputs.
struct Span {
  uintptr_t from = 0, to = 0;
  Span() = default;
  explicit Span(const Tensor& t) : from((uintptr_t)t.data_ptr()), to(from) {
    if (t.numel() == 0) return;
    int64_t last = 0;
    for (int64_t i = 0; i < t.dim(); ++i) last += (t.size(i) - 1) * t.stride(i);
    to = from + (last + 1) * t.element_size();
  }
  bool meets(const Span& o) const { return from < o.to && o.from < to; }
};

void apart(PyObject* out, const char* name, std::initializer_list<PyObject*> ins) {
  const Span a(THPVariable_Unpack(out));
  for (PyObject* o : ins)
    if (given(o) && THPVariable_Check(o) && a.meets(Span(THPVariable_Unpack(o))))
      refuse(name, " must not share memory with an input");
}

// Out may be the input itself; otherwise the two are apart (rows may interleave: slices of one
// projection lie between one another, which the spans of a single row settle).
bool rows_meet(const Tensor& a, const Tensor& b) {
  if (!Span(a).meets(Span(b))) return false;
  if (a.dim() != 3 || b.dim() != 3 || a.size(0) < 2 || b.size(0) < 2) return true;
  const int64_t s = a.stride(0) * (int64_t)a.element_size();
  if (s <= 0 || s != b.stride(0) * (int64_t)b.element_size()) return true;
  // rows of both repeat every s bytes: compare one period
  const int64_t na = a.size(1) * a.size(2) * (int64_t)a.element_size();
  const int64_t nb = b.size(1) * b.size(2) * (int64_t)b.element_size();
  int64_t d = ((int64_t)((uintptr_t)b.data_ptr() - (uintptr_t)a.data_ptr()) % s + s) % s;
  return d < na || d + nb > s;
}

void out_apart(PyObject* out, const char* name, PyObject* same, std::initializer_list<PyObject*> ins) {
  const Tensor& t = THPVariable_Unpack(out);
  for (PyObject* o : ins) {
    if (!given(o) || !THPVariable_Check(o)) continue;
    const Tensor& u = THPVariable_Unpack(o);
    if (o == same && u.data_ptr() == t.data_ptr() && u.strides() == t.strides()) continue;  // in place
    if (rows_meet(t, u)) refuse(name, " must not share memory with another argument");
  }
}

PyObject* rotate(PyObject* const* a) {  // q, positions, rope, k, q_out, k_out
  const Tensor& q = cuda_tensor(a[0], "q");
  const auto dev = q.device();
  const c10::cuda::CUDAGuard guard(dev);
  const auto type = q.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
    refuse("q must be bf16, fp16 or fp32");
  if (q.dim() != 3) refuse("q must be [tokens, Hq, D]");
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
  if (T > INT_MAX || Hq > INT_MAX || D > INT_MAX) refuse("sizes must be below 2^31");
  int64_t qs, ks = 0, qos, kos = 0, Hkv = 0;
  const void* qp = rows(a[0], "q", dev, type, T, Hq, D, &qs);
  const int32_t* pos = plain(a[1], "positions", dev, at::kInt, {T});
  Rope rope;
  if (!given(a[2])) refuse("rope is needed");
  const spec_rope* rp = rope_of(a[2], &rope);
  const void* kp = nullptr;
  if (given(a[3])) {
    const Tensor& k = tensor_on(a[3], "k", dev);
    if (k.dim() != 3) refuse("k must be [tokens, Hkv, D]");
    Hkv = k.size(1);
    if (Hkv < 1 || Hkv > INT_MAX) refuse("k must have heads");
    kp = rows(a[3], "k", dev, type, T, Hkv, D, &ks);
  } else if (given(a[5])) {
    refuse("k_out without k");
  }
  THPObjectPtr made[2];
  PyObject* out[2] = {a[4], a[5]};
  for (int i = 0; i < 2; ++i)
    if (!given(out[i]) && (i == 0 || kp)) {
      made[i] = THPVariable_Wrap(at::zeros({T, i ? Hkv : Hq, D},
                                           at::TensorOptions().dtype(type).device(dev)));
      if (!made[i]) throw python_error();
      out[i] = made[i].get();
    }
  void* qo = rows(out[0], "q_out", dev, type, T, Hq, D, &qos);
  void* ko = kp ? rows(out[1], "k_out", dev, type, T, Hkv, D, &kos) : nullptr;
  if (!made[0]) out_apart(out[0], "q_out", a[0], {a[0], a[1], a[3], made[1] || !kp ? Py_None : out[1]});
  if (kp && !made[1]) out_apart(out[1], "k_out", a[3], {a[0], a[1], a[3]});
  check("spec_rotate", spec_rotate(qp, qs, qo, qos, kp, ks, ko, kos, code_of(type), pos, (int)T,
                                   (int)Hq, (int)Hkv, (int)D, rp, stream_of(dev)));
  return PyTuple_Pack(2, out[0], out[1]);
}

struct Scaled : Caches {
  float *ks, *vs;
  int block;
};

Scaled scaled_cache(PyObject* const* a, c10::Device dev) {  // k_cache, v_cache, k_scale, v_scale
  const Tensor& k = tensor_on(a[0], "k_cache", dev);
  if (k.scalar_type() != at::kFloat8_e4m3fn) refuse("a scaled cache is Float8_e4m3fn");
  Scaled c{caches(a[0], a[1], dev, at::kHalf), nullptr, nullptr, 0};
  const Tensor& s = tensor_on(a[2], "k_scale", dev);
  if (s.dim() != 3 || s.size(1) < 1 || c.P % s.size(1))
    refuse("k_scale must be [pages, page_size / block, Hkv]");
  c.block = (int)(c.P / s.size(1));
  c.ks = plain<float>(a[2], "k_scale", dev, at::kFloat, {c.pages, s.size(1), c.Hkv});
  c.vs = plain<float>(a[3], "v_scale", dev, at::kFloat, {c.pages, s.size(1), c.Hkv});
  return c;
}

// k_new, v_new, k_cache, v_cache, k_scale, v_scale, slot_map, positions, q, q_out, rope
PyObject* append_scaled(PyObject* const* a) {
  const Tensor& kn = cuda_tensor(a[0], "k_new");
  const auto dev = kn.device();
  const c10::cuda::CUDAGuard guard(dev);
  const auto type = kn.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf) refuse("k_new must be bf16 or fp16");
  const Scaled c = scaled_cache(a + 2, dev);
  if (kn.dim() != 3) refuse("k_new must be [tokens, ", c.Hkv, ", ", c.D, "]");
  const int64_t T = kn.size(0);
  if (T > INT_MAX) refuse("tokens must be below 2^31");
  int64_t ks, vs, qs = 0, os = 0, Hq = 0;
  const void* k = rows(a[0], "k_new", dev, type, T, c.Hkv, c.D, &ks);
  const void* v = rows(a[1], "v_new", dev, type, T, c.Hkv, c.D, &vs);
  const int64_t* slots = plain<int64_t>(a[6], "slot_map", dev, at::kLong, {T});
  Rope rope;
  const spec_rope* rp = rope_of(a[10], &rope);
  const int32_t* pos = nullptr;
  if (given(a[7]))
    pos = plain(a[7], "positions", dev, at::kInt, {T});
  else if (rp)
    refuse("positions are needed to rotate");
  const void* q = nullptr;
  void* qo = nullptr;
  PyObject* out = a[9];
  THPObjectPtr made;
  if (given(a[8])) {
    const Tensor& qt = tensor_on(a[8], "q", dev);
    if (qt.dim() != 3 || qt.size(0) != T) refuse("q must be [tokens, Hq, D]");
    Hq = qt.size(1);
    if (Hq > INT_MAX) refuse("heads must be below 2^31");
    q = rows(a[8], "q", dev, type, T, Hq, c.D, &qs);
    if (!given(out)) {
      made = THPVariable_Wrap(
          at::zeros({T, Hq, c.D}, at::TensorOptions().dtype(type).device(dev)));
      if (!made) throw python_error();
      out = made.get();
    }
    qo = rows(out, "q_out", dev, type, T, Hq, c.D, &os);
    if (!made) out_apart(out, "q_out", a[8], {a[8], a[0], a[1]});
  } else if (given(out)) {
    refuse("q_out without q");
  }
  // What is written: caches and scales share memory with nothing else (K's and V's caches may lie
  // between one another), q_out with none of them nor with slots and positions.
  Span span[9];
  for (int i = 0; i < 9; ++i)
    if (given(a[i])) span[i] = Span(THPVariable_Unpack(a[i]));
  static const char* const names[4] = {"k_cache", "v_cache", "k_scale", "v_scale"};
  for (int i = 2; i < 6; ++i)
    for (int j = 0; j < 9; ++j)
      if (j != i && !(i < 4 && (j == 2 || j == 3)) && span[i].meets(span[j]))
        refuse(names[i - 2], " must not share memory with another argument");
  if (c.k == c.v) refuse("k_cache must not share memory with v_cache");
  if (qo && !made) {
    const Span o(THPVariable_Unpack(out));
    for (int j = 2; j < 8; ++j)
      if (o.meets(span[j])) refuse("q_out must not share memory with another argument");
  }
  check("spec_append_scaled",
        spec_append_scaled(k, ks, v, vs, q, qs, qo, os, code_of(type), c.k, c.v, c.ks, c.vs,
                           c.pages, c.P, c.block, c.page, c.token, c.head, slots, pos, (int)T,
                           (int)Hq, c.Hkv, c.D, rp, stream_of(dev)));
  Py_INCREF(out);
  return out;
}

// k_cache, v_cache, k_scale, v_scale, slot_map, k_out, v_out
PyObject* read_scaled(PyObject* const* a) {
  const Tensor& kc = cuda_tensor(a[0], "k_cache");
  const auto dev = kc.device();
  const c10::cuda::CUDAGuard guard(dev);
  const Scaled c = scaled_cache(a, dev);
  const Tensor& sl = tensor_on(a[4], "slot_map", dev);
  if (sl.dim() != 1 || sl.size(0) > INT_MAX) refuse("slot_map must be [tokens]");
  const int64_t T = sl.size(0);
  const int64_t* slots = plain<int64_t>(a[4], "slot_map", dev, at::kLong, {T});
  auto type = at::kBFloat16;
  for (int i = 5; i < 7; ++i)
    if (given(a[i])) type = tensor_on(a[i], "an output", dev).scalar_type();
  if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
    refuse("outputs must be bf16, fp16 or fp32");
  THPObjectPtr made[2];
  PyObject* out[2] = {a[5], a[6]};
  int64_t st[2];
  void* p[2];
  for (int i = 0; i < 2; ++i) {
    if (!given(out[i])) {
      made[i] = THPVariable_Wrap(
          at::zeros({T, c.Hkv, c.D}, at::TensorOptions().dtype(type).device(dev)));
      if (!made[i]) throw python_error();
      out[i] = made[i].get();
    }
    p[i] = rows(out[i], i ? "v_out" : "k_out", dev, type, T, c.Hkv, c.D, &st[i]);
  }
  if (!made[0]) out_apart(out[0], "k_out", nullptr, {a[0], a[1], a[2], a[3], a[4], out[1]});
  if (!made[1]) out_apart(out[1], "v_out", nullptr, {a[0], a[1], a[2], a[3], a[4], out[0]});
  check("spec_read_scaled",
        spec_read_scaled(c.k, c.v, c.ks, c.vs, c.pages, c.P, c.block, c.page, c.token, c.head,
                         slots, (int)T, c.Hkv, c.D, p[0], st[0], p[1], st[1], code_of(type),
                         stream_of(dev)));
  return PyTuple_Pack(2, out[0], out[1]);
}

// q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_len, anc_mask, scale, window, workspace,
// out, lse
PyObject* verify_attn_scaled(PyObject* const* a) {
  const Tensor& q = cuda_tensor(a[0], "q");
  const auto dev = q.device();
  const c10::cuda::CUDAGuard guard(dev);
  const auto type = q.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf) refuse("q must be bf16 or fp16");
  if (q.dim() != 4 || q.stride(3) != 1) refuse("q must be [B, R, Hq, D], contiguous over D");
  const Scaled c = scaled_cache(a + 1, dev);
  const int64_t B = q.size(0), R = q.size(1), Hq = q.size(2), D = q.size(3);
  if (D != c.D) refuse("head_dim mismatch");
  const Tensor& tab = tensor_on(a[5], "block_table", dev);
  if (tab.dim() != 2) refuse("block_table must be [B, max_pages]");
  const int64_t width = tab.size(1);
  if (B > INT_MAX || R > INT_MAX || Hq > INT_MAX || width > INT_MAX)
    refuse("sizes must be below 2^31");
  const int32_t* table = plain(a[5], "block_table", dev, at::kInt, {B, width});
  const int32_t* ctx = plain(a[6], "ctx_len", dev, at::kInt, {B});
  const uint64_t* mask = nullptr;
  if (given(a[7])) mask = plain<uint64_t>(a[7], "anc_mask", dev, at::kLong, {B, R});
  const double sm_scale = number(a[8]);
  const int64_t window = whole(a[9], "window", 0);
  Tensor ws;
  if (given(a[10])) {
    if (!THPVariable_Check(a[10]) || THPVariable_Unpack(a[10]).device() != dev ||
        THPVariable_Unpack(a[10]).scalar_type() != at::kByte ||
        !THPVariable_Unpack(a[10]).is_contiguous())
      refuse("workspace must come from new_workspace on q's device");
    ws = THPVariable_Unpack(a[10]);
  } else {
    const size_t need = spec_verify_attn_scaled_workspace_size((int)B, (int)R, (int)Hq, c.Hkv, (int)D);
    ws = at::zeros({(int64_t)(need < 256 ? 256 : need)},
                   at::TensorOptions().dtype(at::kByte).device(dev));
  }
  THPObjectPtr made[2];
  PyObject* out[2] = {a[11], a[12]};
  for (int i = 0; i < 2; ++i)
    if (!given(out[i])) {
      made[i] = THPVariable_Wrap(i ? empty({B, R, Hq}, at::kFloat, dev)
                                   : empty({B, R, Hq, D}, type, dev));
      if (!made[i]) throw python_error();
      out[i] = made[i].get();
    }
  void* o = plain<void>(out[0], "out", dev, type, {B, R, Hq, D});
  float* lse = plain<float>(out[1], "lse", dev, at::kFloat, {B, R, Hq});
  for (int i = 0; i < 2; ++i)
    if (!made[i])
      apart(out[i], i ? "lse" : "out",
            {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[10], i ? out[0] : Py_None});
  check("spec_verify_attn_scaled",
        spec_verify_attn_scaled(q.data_ptr(), q.stride(0), q.stride(1), q.stride(2), code_of(type),
                                c.k, c.v, c.ks, c.vs, c.pages, c.P, c.block, c.page, c.token,
                                c.head, table, (int)width, ctx, mask, (int)B, (int)R, (int)Hq,
                                c.Hkv, (int)D, (int)window, (float)sm_scale, ws.data_ptr(),
                                (size_t)ws.numel(), o, lse, stream_of(dev)));
  return PyTuple_Pack(2, out[0], out[1]);
}

// logits, out, history, prompt_len, block_tokens, parent, repetition, frequency, presence,
// bias_ids, bias, mask, mask_row
PyObject* logits_process(PyObject* const* a) {
  const Tensor& x = cuda_tensor(a[0], "logits");
  const auto dev = x.device();
  const c10::cuda::CUDAGuard guard(dev);
  const auto type = x.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
    refuse("logits must be bf16, fp16 or fp32");
  if (x.dim() != 3) refuse("logits must be [B, R, V]");
  const int64_t B = x.size(0), R = x.size(1), V = x.size(2);
  if (B > INT_MAX || R > INT_MAX || V > INT_MAX) refuse("sizes must be below 2^31");
  // (one row per sequence: the distance from row to row is the batch's, whatever stands in between)
  if ((V > 1 && x.stride(2) != 1) || (B > 1 && R > 1 && x.stride(0) != R * x.stride(1)))
    refuse("logits: rows must be equally far apart, contiguous over V");
  const int64_t stride = R > 1 ? x.stride(1) : B > 1 ? x.stride(0) : V;
  auto width = [&](int i, const char* name) -> int64_t {  // of a [B, n] array; 0: not given
    if (!given(a[i])) return 0;
    const Tensor& t = tensor_on(a[i], name, dev);
    if (t.dim() != 2 || t.size(1) > INT_MAX) refuse(name, " must have two dimensions");
    return t.size(1);
  };
  auto ints = [&](int i, const char* name, at::IntArrayRef shape) -> const int32_t* {
    return given(a[i]) ? plain(a[i], name, dev, at::kInt, shape) : nullptr;
  };
  auto floats = [&](int i, const char* name, at::IntArrayRef shape) -> const float* {
    return given(a[i]) ? plain<float>(a[i], name, dev, at::kFloat, shape) : nullptr;
  };
  const int64_t H = width(2, "history"), n = width(9, "bias_ids");
  const int32_t* history = ints(2, "history", {B, H});
  const int32_t* prompt = ints(3, "prompt_len", {B});
  if (prompt && !history) refuse("prompt_len without history");
  const int32_t* parent = ints(5, "parent", {B, R});
  if (parent && !given(a[4])) refuse("parent without block_tokens");
  const int32_t* tokens = ints(4, "block_tokens", {B, parent ? R : R - 1});
  const float* rep = floats(6, "repetition", {B});
  const float* fr = floats(7, "frequency", {B});
  const float* pr = floats(8, "presence", {B});
  if (given(a[9]) != given(a[10])) refuse("bias_ids and bias come together");
  const int32_t* ids = ints(9, "bias_ids", {B, n});
  const float* bias = floats(10, "bias", {B, n});
  int64_t masks = 0;
  const int32_t* mask = nullptr;
  if (given(a[11])) {
    width(11, "mask");
    masks = THPVariable_Unpack(a[11]).size(0);
    if (masks > INT_MAX) refuse("masks must be below 2^31");
    mask = ints(11, "mask", {masks, (V + 31) / 32});
    if (!given(a[12]) && masks != B * R) refuse("mask must have B * R rows without mask_row");
  } else if (given(a[12])) {
    refuse("mask_row without mask");
  }
  const int32_t* row = ints(12, "mask_row", {B, R});
  THPObjectPtr made;
  PyObject* out = a[1];
  if (!given(out)) {
    made = THPVariable_Wrap(empty({B, R, V}, at::kFloat, dev));
    if (!made) throw python_error();
    out = made.get();
  }
  float* o = plain<float>(out, "out", dev, at::kFloat, {B, R, V});
  if (!made) {
    if (o != x.data_ptr() || type != at::kFloat || !x.is_contiguous()) apart(out, "out", {a[0]});
    apart(out, "out", {a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12]});
  }
  check("spec_logits_process",
        spec_logits_process(x.data_ptr(), stride, code_of(type), o, (int)B, (int)R, (int)V,
                            history, (int)H, prompt, tokens, parent, rep, fr, pr, ids, bias,
                            (int)n, mask, (int)masks, row, stream_of(dev)));
  Py_INCREF(out);
  return out;
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
                                  method<rotate, 6>("rotate"),
                                  method<append_scaled, 11>("append_scaled"),
                                  method<read_scaled, 7>("read_scaled"),
                                  method<verify_attn_scaled, 13>("verify_attn_scaled"),
                                  method<logits_process, 13>("logits_process"),
                                  {"set_error", set_error, METH_O, nullptr},
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1,     methods,
                            nullptr,               nullptr,   nullptr, nullptr};
  return &def;
}

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(module_def()); }
