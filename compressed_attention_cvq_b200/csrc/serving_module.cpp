// Python module _serving: the argument checks, outputs and calls of serving.py in native code.
// A decode step makes these calls one after another, and checked in Python they took 25 us of
// host time each where the kernels take 3 to 20.
//
// The library's functions are handed in by address (bind), so that the module serves whichever
// build of the library the binding has loaded.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cuda_runtime_api.h>

#include <algorithm>
#include <cstring>
#include <initializer_list>
#include <string>

#include "cvq.h"

namespace {

struct Api {
  decltype(&cvq_prefix_workspace_bytes) prefix_workspace_bytes;
  decltype(&cvq_prefix_suggest_splits) prefix_suggest_splits;
  decltype(&cvq_prefix_attend) prefix_attend;
  decltype(&cvq_paged_append) paged_append;
  decltype(&cvq_paged_workspace_bytes) paged_workspace_bytes;
  decltype(&cvq_paged_suggest_splits) paged_suggest_splits;
  decltype(&cvq_paged_attend) paged_attend;
} api;
PyObject* check_status = nullptr;      // check(status, name): raises unless the status is CVQ_OK

using Shape = std::initializer_list<int64_t>;

[[noreturn]] void bad(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw python_error();
}

template <typename Sizes>
std::string show(const Sizes& s) {
  std::string r = "(";
  size_t i = 0;
  for (int64_t x : s) {
    if (i++) r += ", ";
    r += std::to_string(x);
  }
  return r + (s.size() == 1 ? ",)" : ")");
}

std::string dtype_name(at::ScalarType t) {
  const char* n = t == at::kFloat ? "float32" : t == at::kHalf ? "float16" : t == at::kBFloat16 ? "bfloat16"
                  : t == at::kInt ? "int32" : t == at::kByte ? "uint8" : c10::toString(t);
  return std::string("torch.") + n;
}

int dtype_code(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return CVQ_F32;
  if (t == at::kBFloat16) return CVQ_BF16;
  if (t == at::kHalf) return CVQ_F16;
  bad(std::string(name) + " must be float32, bfloat16 or float16, got " + dtype_name(t));
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw python_error();
  }
  return THPVariable_Unpack(o);
}

// an empty tensor has no address
template <typename T = void>
T* ptr(const at::Tensor& t) {
  return t.numel() == 0 ? nullptr : static_cast<T*>(t.data_ptr());
}

bool same(at::IntArrayRef a, Shape b) { return a.size() == b.size() && std::equal(b.begin(), b.end(), a.begin()); }

// a dense tensor of this device, type and shape
void check(const at::Tensor& t, const char* name, c10::Device dev, at::ScalarType dtype, Shape shape) {
  if (t.device() != dev) bad(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
  if (t.scalar_type() != dtype) bad(std::string(name) + " has dtype " + dtype_name(t.scalar_type()) + ", expected " + dtype_name(dtype));
  if (!same(t.sizes(), shape)) bad(std::string(name) + " has shape " + show(t.sizes()) + ", expected " + show(shape));
  if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
}

c10::Device cuda_device(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) bad(std::string(name) + " must be a CUDA tensor");
  return t.device();
}

// The tensors' device is current, and so is the stream that a call was given: for as long as this
// lives.  The library launches on the current device; what the call allocates, and clears, for itself
// is then ordered with its kernels, and the allocator hands it on in the order of the same stream.
struct On {
  On(c10::Device dev, PyObject* given) {
    if (given == Py_None) {
      if (c10::cuda::current_device() != dev.index()) device.set_index(dev.index());
    } else {
      void* p = PyLong_AsVoidPtr(given);
      if (p == nullptr && PyErr_Occurred()) throw python_error();
      current.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), dev.index()));
    }
    stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  }
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard current;
  void* stream;
};

int sm_count(c10::Device dev) {
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev.index()) != cudaSuccess) bad("no SM count for " + dev.str());
  return n;
}

int int_of(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < INT32_MIN || v > INT32_MAX) bad("n_splits out of range");
  return static_cast<int>(v);
}

template <typename T>
const T* struct_at(PyObject* address) {
  const T* p = static_cast<const T*>(PyLong_AsVoidPtr(address));
  if (p == nullptr) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no shape");
    throw python_error();
  }
  return p;
}

void raise_for(cvq_status st, const char* name) {
  if (st == CVQ_OK) return;
  PyObject* r = PyObject_CallFunction(check_status, "is", static_cast<int>(st), name);
  Py_XDECREF(r);
  if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, name);
  throw python_error();
}

// clear: whether the call takes what the workspace holds
at::Tensor workspace_of(PyObject* o, size_t need, c10::Device dev, const char* what, bool clear) {
  if (need == 0) bad(std::string("invalid shape or n_splits for ") + what);
  if (o == Py_None) {
    const auto bytes = at::TensorOptions().dtype(at::kByte).device(dev);
    return clear ? at::zeros({static_cast<int64_t>(need)}, bytes) : at::empty({static_cast<int64_t>(need)}, bytes);
  }
  const at::Tensor& ws = tensor(o, "workspace");
  if (ws.device() != dev || static_cast<size_t>(ws.numel()) * ws.element_size() < need || !ws.is_contiguous())
    bad("workspace must be " + std::to_string(need) + " dense bytes on " + dev.str());
  return ws;
}

struct Outputs {
  at::Tensor out, lse;
};
Outputs outputs_of(PyObject* out, PyObject* lse, PyObject* out_dtype, at::ScalarType otherwise, int64_t B, int64_t Hq, c10::Device dev) {
  Outputs r;
  if (out_dtype != Py_None && !THPDtype_Check(out_dtype)) {
    PyErr_SetString(PyExc_TypeError, "out_dtype must be a torch.dtype");
    throw python_error();
  }
  const at::ScalarType want = out_dtype != Py_None ? reinterpret_cast<THPDtype*>(out_dtype)->scalar_type : otherwise;
  if (out == Py_None) {
    dtype_code(want, "out");
    r.out = at::empty({B, Hq, 128}, at::TensorOptions().dtype(want).device(dev));
  } else {
    r.out = tensor(out, "out");
    if (out_dtype != Py_None && r.out.scalar_type() != want)
      bad("out has dtype " + dtype_name(r.out.scalar_type()) + ", expected " + dtype_name(want));
    check(r.out, "out", dev, r.out.scalar_type(), {B, Hq, 128});
  }
  if (lse == Py_None) {
    r.lse = at::empty({B, Hq}, at::TensorOptions().dtype(at::kFloat).device(dev));
  } else {
    r.lse = tensor(lse, "lse");
    check(r.lse, "lse", dev, at::kFloat, {B, Hq});
  }
  return r;
}

// (out, lse), the caller's own objects where it gave them
PyObject* result(const Outputs& o, PyObject* out, PyObject* lse) {
  PyObject* a = out == Py_None ? THPVariable_Wrap(o.out) : Py_NewRef(out);
  PyObject* b = lse == Py_None ? THPVariable_Wrap(o.lse) : Py_NewRef(lse);
  PyObject* r = a != nullptr && b != nullptr ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  if (r == nullptr) throw python_error();
  return r;
}

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    throw python_error();
  }
  if (check_status == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    throw python_error();
  }
}

// floats between the heads of a codebook [(Hkv,) groups, R, entries, ...]
int64_t codebook_stride(const at::Tensor& cb, const char* name, c10::Device dev, const cvq_shape* s, bool key) {
  const bool wide = s->group_dim == 64;
  const int64_t groups = wide ? 2 : 16, entries = wide ? 64 : 256, d = wide ? 64 : 8, H = s->n_kv_heads;
  const bool per_head = cb.dim() == (key ? 6 : 5);
  if (key) {
    if (per_head) check(cb, name, dev, at::kFloat, {H, groups, s->R, entries, d / 2, 2});
    else check(cb, name, dev, at::kFloat, {groups, s->R, entries, d / 2, 2});
  } else {
    if (per_head) check(cb, name, dev, at::kFloat, {H, groups, s->R, entries, d});
    else check(cb, name, dev, at::kFloat, {groups, s->R, entries, d});
  }
  return per_head ? groups * s->R * entries * d : 0;
}

void check_codes(const at::Tensor& t, const char* name, c10::Device dev, const cvq_shape* s) {
  const int64_t H = s->n_kv_heads, R = s->R, T = s->t_cap;
  const bool one = t.dim() == 5;
  if (s->group_dim == 64) {
    const int64_t row = s->code_bits == 6 ? T * 3 / 4 : T;
    if (one) check(t, name, dev, at::kByte, {1, H, 2, R, row});
    else check(t, name, dev, at::kByte, {H, 2, R, row});
  } else {
    if (one) check(t, name, dev, at::kByte, {1, H, T, R, 16});
    else check(t, name, dev, at::kByte, {H, T, R, 16});
  }
}

// shape, q, key_cb, key_codes, val_codes, prefix_len, val_cb, n_splits, workspace, out, lse,
// out_dtype, stream
PyObject* prefix_attend(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 13);
  const cvq_shape* s = struct_at<cvq_shape>(p[0]);
  const at::Tensor &q = tensor(p[1], "q"), &kcb = tensor(p[2], "key_cb"), &kc = tensor(p[3], "key_codes"),
                   &vc = tensor(p[4], "val_codes"), &len = tensor(p[5], "prefix_len"), &vcb = tensor(p[6], "val_cb");
  const c10::Device dev = cuda_device(q, "q");
  check(q, "q", dev, q.scalar_type(), {s->batch, s->n_q_heads, 128});
  check_codes(kc, "key_codes", dev, s);
  check_codes(vc, "val_codes", dev, s);
  check(len, "prefix_len", dev, at::kInt, {1});
  const int64_t ks = codebook_stride(kcb, "key_cb", dev, s, true), vs = codebook_stride(vcb, "val_cb", dev, s, false);
  const int qd = dtype_code(q.scalar_type(), "q");
  const On on(dev, p[12]);
  const int splits = p[7] == Py_None ? api.prefix_suggest_splits(s, qd, sm_count(dev)) : int_of(p[7]);
  const at::Tensor ws = workspace_of(p[8], api.prefix_workspace_bytes(s, splits), dev, "cvq_prefix_workspace_bytes", false);
  const Outputs o = outputs_of(p[9], p[10], p[11], q.scalar_type(), s->batch, s->n_q_heads, dev);
  raise_for(api.prefix_attend(s, ptr(q), qd, ptr<float>(kcb), ks, ptr<uint8_t>(kc), ptr<uint8_t>(vc),
                              ptr<int32_t>(len), ptr<float>(vcb), vs, splits, ptr(ws), ptr(o.out),
                              dtype_code(o.out.scalar_type(), "out"), ptr<float>(o.lse), on.stream),
            "cvq_prefix_attend");
  return result(o, p[9], p[10]);
  END_HANDLE_TH_ERRORS
}

void check_pool(const at::Tensor& t, const char* name, c10::Device dev, const cvq_paged* g) {
  if (t.device() != dev) bad(std::string(name) + " is on " + t.device().str() + ", expected " + dev.str());
  if (t.scalar_type() != (g->kv_dtype == CVQ_BF16 ? at::kBFloat16 : at::kHalf))
    bad(std::string(name) + " has dtype " + dtype_name(t.scalar_type()) + ", not the cache's");
  const int64_t rows = static_cast<int64_t>(g->page_size) * 128, dense = g->n_kv_heads * rows;
  const int64_t sizes[4] = {g->n_pages, g->n_kv_heads, g->page_size, 128};
  const int64_t strides[4] = {g->page_stride != 0 ? g->page_stride : dense, rows, 128, 1};
  bool ok = t.dim() == 4;
  for (int i = 0; ok && i < 4; ++i) ok = t.size(i) == sizes[i] && (sizes[i] == 1 || t.stride(i) == strides[i]);
  if (!ok)
    bad(std::string(name) + " must be " + show(at::IntArrayRef(sizes, 4)) + " with strides " + show(at::IntArrayRef(strides, 4)) +
        ", got " + show(t.sizes()) + " with " + show(t.strides()));
}

void check_pages(const cvq_paged* g, const at::Tensor& kp, const at::Tensor& vp, const at::Tensor& table, const at::Tensor& lens, c10::Device dev) {
  check_pool(kp, "k_pages", dev, g);
  check_pool(vp, "v_pages", dev, g);
  check(table, "page_table", dev, at::kInt, {g->batch, g->max_pages});
  check(lens, "seq_lens", dev, at::kInt, {g->batch});
}

// token stride of [n, heads, 128] whose heads are dense (tokens may be strided; a single one has no
// stride, whatever the tensor says)
int64_t token_stride(const at::Tensor& t, const char* name, c10::Device dev, at::ScalarType dtype, int64_t n, int64_t heads) {
  if (t.device() != dev || t.scalar_type() != dtype) bad(std::string(name) + " must be " + dtype_name(dtype) + " on " + dev.str());
  if (!same(t.sizes(), {n, heads, 128}) || t.stride(2) != 1 || (heads > 1 && t.stride(1) != 128))
    bad(std::string(name) + " must be [" + std::to_string(n) + ", " + std::to_string(heads) + ", 128] with dense heads");
  return n > 1 ? t.stride(0) : heads * 128;
}

// paged, k, v, tok_offsets, seq_lens, page_table, k_pages, v_pages, q, q_out, pos_offsets, stream
PyObject* paged_append(PyObject*, PyObject* const* p, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  need_args(n_args, 12);
  const cvq_paged* g = struct_at<cvq_paged>(p[0]);
  const at::Tensor &k = tensor(p[1], "k"), &v = tensor(p[2], "v"), &off = tensor(p[3], "tok_offsets"), &lens = tensor(p[4], "seq_lens"),
                   &table = tensor(p[5], "page_table"), &kp = tensor(p[6], "k_pages"), &vp = tensor(p[7], "v_pages");
  const c10::Device dev = cuda_device(k, "k");
  const On on(dev, p[11]);
  if (k.dim() != 3 || k.size(0) > INT32_MAX) bad("k must be [tokens, KV heads, 128]");
  const int64_t n = k.size(0);
  const at::ScalarType dt = k.scalar_type();
  check_pages(g, kp, vp, table, lens, dev);
  const int64_t ks = token_stride(k, "k", dev, dt, n, g->n_kv_heads), vs = token_stride(v, "v", dev, dt, n, g->n_kv_heads);
  check(off, "tok_offsets", dev, at::kInt, {static_cast<int64_t>(g->batch) + 1});
  const int32_t* pos = nullptr;
  if (p[10] != Py_None) {
    const at::Tensor& t = tensor(p[10], "pos_offsets");
    check(t, "pos_offsets", dev, at::kInt, {g->batch});
    pos = ptr<int32_t>(t);
  }
  int64_t qs = 0;
  const void* q = nullptr;
  at::Tensor qo;
  if (p[8] != Py_None) {
    const at::Tensor& t = tensor(p[8], "q");
    qs = token_stride(t, "q", dev, dt, n, g->n_q_heads);
    q = ptr(t);
    if (p[9] == Py_None) {
      qo = at::empty({n, g->n_q_heads, 128}, t.options());
    } else {
      qo = tensor(p[9], "q_out");
      check(qo, "q_out", dev, dt, {n, g->n_q_heads, 128});
    }
  } else if (p[9] != Py_None) {
    bad("q_out without q");
  }
  const int code = dtype_code(dt, "k");
  if (n > 0) {
    raise_for(api.paged_append(g, static_cast<int32_t>(n), q, qs, ptr(k), ks, ptr(v), vs, code, ptr<int32_t>(off),
                               ptr<int32_t>(lens), pos, ptr<int32_t>(table), ptr(kp), ptr(vp),
                               q != nullptr ? ptr(qo) : nullptr, on.stream),
              "cvq_paged_append");
  }
  if (p[9] != Py_None || p[8] == Py_None) return Py_NewRef(p[9]);
  return THPVariable_Wrap(qo);
  END_HANDLE_TH_ERRORS
}

// paged, q, k_pages, v_pages, page_table, seq_lens, n_splits, workspace, prev_out, prev_lse, out,
// lse, out_dtype, stream
PyObject* paged_attend(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 14);
  const cvq_paged* g = struct_at<cvq_paged>(p[0]);
  const at::Tensor &q = tensor(p[1], "q"), &kp = tensor(p[2], "k_pages"), &vp = tensor(p[3], "v_pages"),
                   &table = tensor(p[4], "page_table"), &lens = tensor(p[5], "seq_lens");
  const c10::Device dev = cuda_device(q, "q");
  check(q, "q", dev, q.scalar_type(), {g->batch, g->n_q_heads, 128});
  check_pages(g, kp, vp, table, lens, dev);
  const float *po = nullptr, *pl = nullptr;
  if (p[8] != Py_None || p[9] != Py_None) {
    const at::Tensor &a = tensor(p[8], "prev out"), &b = tensor(p[9], "prev lse");
    check(a, "prev out", dev, at::kFloat, {g->batch, g->n_q_heads, 128});
    check(b, "prev lse", dev, at::kFloat, {g->batch, g->n_q_heads});
    po = ptr<float>(a);
    pl = ptr<float>(b);
  }
  const int qd = dtype_code(q.scalar_type(), "q");
  const On on(dev, p[13]);
  const int splits = p[6] == Py_None ? api.paged_suggest_splits(g, sm_count(dev)) : int_of(p[6]);
  const at::Tensor ws = workspace_of(p[7], api.paged_workspace_bytes(g, splits), dev, "cvq_paged_workspace_bytes", true);
  const Outputs o = outputs_of(p[10], p[11], p[12], q.scalar_type(), g->batch, g->n_q_heads, dev);
  raise_for(api.paged_attend(g, ptr(q), qd, ptr(kp), ptr(vp), ptr<int32_t>(table), ptr<int32_t>(lens),
                             splits, ptr(ws), po, pl, ptr(o.out), dtype_code(o.out.scalar_type(), "out"),
                             ptr<float>(o.lse), on.stream),
            "cvq_paged_attend");
  return result(o, p[10], p[11]);
  END_HANDLE_TH_ERRORS
}

// bind(check, addresses of the seven functions in Api's order)
PyObject* bind(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  constexpr Py_ssize_t kFns = sizeof(Api) / sizeof(void*);
  if (n != 1 + kFns) bad("bind takes the status check and seven addresses");
  void* at[kFns];
  for (Py_ssize_t i = 0; i < kFns; ++i) {
    at[i] = PyLong_AsVoidPtr(p[1 + i]);
    if (PyErr_Occurred()) throw python_error();
  }
  static_assert(sizeof(at) == sizeof(api));
  std::memcpy(&api, at, sizeof(api));
  Py_XSETREF(check_status, Py_NewRef(p[0]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"prefix_attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_attend)), METH_FASTCALL, nullptr},
    {"paged_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_append)), METH_FASTCALL, nullptr},
    {"paged_attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attend)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", "Checks and calls of the serving operators.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
