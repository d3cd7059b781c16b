// The Python calls of the head norms / rotation and of the byte cache, from torch tensors to the C ABI.
//
// A decode step makes these calls once per layer on tensors of a few hundred kilobytes, where the call
// costs more than the kernel: checked and marshalled in Python through ctypes a call took the host 18-20 us
// (Grace), here 5-9.  This file only checks tensors, allocates outputs and workspaces through torch (on
// the current stream, so their memory belongs to it) and fills the ABI's structs; what the library refuses
// becomes its TQError.  Arguments come by position from byte_cache.py, which documents them.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "tq.h"

namespace {

PyObject* g_error = nullptr;  // TQError

struct Refused : std::exception {
  std::string msg;
  explicit Refused(std::string m) : msg(std::move(m)) {}
  const char* what() const noexcept override { return msg.c_str(); }
};
struct Failed : std::exception {};  // the Python error is set

std::string shape_text(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

bool given(PyObject* o) { return o != Py_None; }
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

tq_dtype dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return TQ_F32;
    case at::kBFloat16: return TQ_BF16;
    case at::kHalf: return TQ_F16;
    default: throw Refused(std::string("unsupported dtype ") + c10::toString(t) + ": float32, bfloat16 or float16");
  }
}
tq_dtype dtype_of(const at::Tensor& t) { return dtype_code(t.scalar_type()); }

void same_kind(const at::Tensor& t, const char* name, at::ScalarType dt, int device) {
  if (t.scalar_type() != dt || t.get_device() != device)
    throw Refused(std::string(name) + " must be a " + c10::toString(dt) + " tensor on cuda:" + std::to_string(device) + ", not " +
                  c10::toString(t.scalar_type()) + " on " + t.device().str());
}

// An input or output of numbers: no gradient passes through the calls, and memory is read as it is.
void plain(const at::Tensor& t, const char* name) {
  if (t.requires_grad() && at::GradMode::is_enabled())
    throw Refused(std::string(name) + " requires a gradient, which is not computed here: call under torch.no_grad(), or detach it");
  if (t.is_neg()) throw Refused(std::string(name) + " is a view with a pending negation: resolve_neg() it");
}

void has_shape(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) {
    std::string want = "[";
    for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
    throw Refused(std::string(name) + " must have shape " + want + "], not " + shape_text(t));
  }
}

// Rows of a 4-d view whose dims b, n, h are batch, token and head.
tq_heads heads(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dt, int device, int b, int n, int h) {
  same_kind(t, name, dt, device);
  plain(t, name);
  has_shape(t, name, shape);
  if (t.stride(3) != 1 && t.size(3) > 1) throw Refused(std::string(name) + ": the head dimension must be contiguous");
  return tq_heads{t.const_data_ptr(), t.stride(b), t.stride(n), t.stride(h), (int32_t)t.size(h)};
}

const int32_t* ints(PyObject* o, const char* name, at::IntArrayRef shape, int device) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor(o, name);
  same_kind(t, name, at::kInt, device);
  has_shape(t, name, shape);
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  return (const int32_t*)t.const_data_ptr();
}

const void* weight(PyObject* o, const char* name, int64_t d, at::ScalarType dt, int device) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor(o, name);
  same_kind(t, name, dt, device);
  plain(t, name);
  has_shape(t, name, {d});
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  return t.const_data_ptr();
}

// The caller's output, checked, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dt, int device) {
  if (!given(o)) return at::empty(shape, at::TensorOptions().dtype(dt).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)device)));
  const at::Tensor& t = tensor(o, name);
  same_kind(t, name, dt, device);
  plain(t, name);
  has_shape(t, name, shape);
  if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  return t;
}

long long item(PyObject* tuple, int i) { return PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i)); }

// Rotary._args: (table, rotary_dim, interleaved, num_axes)
std::optional<tq_rotary> rotary(PyObject* o, int device) {
  if (!given(o)) return std::nullopt;
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) throw Refused("bad rotary");
  const at::Tensor& t = tensor(PyTuple_GET_ITEM(o, 0), "the rotary table");
  if (t.get_device() != device) throw Refused("the rotary table must be on cuda:" + std::to_string(device));
  if (t.numel() != item(o, 1) / 2 || !t.is_contiguous()) throw Refused("the rotary table was resized");
  return tq_rotary{(const uint64_t*)t.const_data_ptr(), (int32_t)item(o, 1), (int32_t)item(o, 2), (int32_t)item(o, 3)};
}

// PagedByteCache._args: (head_dim, q heads, kv heads, num_pages, max_blocks, pool, error)
struct Cache {
  tq_byte_config cfg;
  int32_t pages, blocks;
  void* pool;
  int32_t* error;
  int device;
};
Cache cache(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 7) throw Refused("bad cache");
  const at::Tensor &pool = tensor(PyTuple_GET_ITEM(o, 5), "pool"), &error = tensor(PyTuple_GET_ITEM(o, 6), "error");
  const tq_byte_config cfg = {(int32_t)item(o, 0), (int32_t)item(o, 1), (int32_t)item(o, 2)};
  const int32_t pages = (int32_t)item(o, 3);
  if (pool.numel() != (int64_t)tq_byte_pool_bytes(&cfg, pages) || !pool.is_contiguous() || error.numel() != 1 ||
      error.get_device() != pool.get_device())
    throw Refused("the pool or its error word was resized or moved");
  return Cache{cfg, pages, (int32_t)item(o, 4), pool.data_ptr(), (int32_t*)error.data_ptr(), pool.get_device()};
}
tq_page_table page_table(PyObject* o, const Cache& c, int64_t* batch) {
  const at::Tensor& t = tensor(o, "block_table");
  same_kind(t, "block_table", at::kInt, c.device);
  if (t.dim() != 2 || t.size(1) != c.blocks || !t.is_contiguous())
    throw Refused("block_table must be a contiguous tensor [batch][" + std::to_string(c.blocks) + "], not " + shape_text(t));
  *batch = t.size(0);
  return tq_page_table{(const int32_t*)t.const_data_ptr(), c.blocks, c.pages};
}

void check(tq_status s) {
  if (s == TQ_OK) return;
  const char* msg = tq_last_error();
  PyObject* args = Py_BuildValue("is", (int)s, *msg ? msg : tq_status_string(s));
  PyObject* e = args ? PyObject_CallObject(g_error, args) : nullptr;
  Py_XDECREF(args);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Failed();
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed();
  return (float)v;
}

// The device's guard (only where another one is current) and its current stream.
struct On {
  std::optional<c10::cuda::CUDAGuard> guard;
  tq_stream stream = nullptr;
  explicit On(int device) {
    if (device < 0) throw Refused("tensors must be on a CUDA device");
    if (c10::cuda::current_device() != device) guard.emplace((c10::DeviceIndex)device);
    stream = (tq_stream)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  }
};

int32_t narrow(int64_t v, const char* what) {
  if (v < 0 || v > INT32_MAX) throw Refused(std::string(what) + " is too large");
  return (int32_t)v;
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Failed&) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "call failed");
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {  // of an output or a workspace: torch's own type, which callers catch
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
bool count_args(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// norm_rotate(q, k, rotary, positions, start, q_weight, k_weight, eps, float32_out, q_out, k_out) -> (q, k)
PyObject* norm_rotate(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_args(n_args, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    const bool has_q = given(a[0]), has_k = given(a[1]);
    if (!has_q && !has_k) throw Refused("neither q nor k given");
    const at::Tensor& x = has_q ? tensor(a[0], "q") : tensor(a[1], "k");
    if (x.dim() != 4 || !x.is_cuda()) throw Refused("q and k must be CUDA tensors of 4 dims");
    const tq_dtype code = dtype_of(x);
    const at::ScalarType dt = x.scalar_type(), odt = given(a[8]) && PyObject_IsTrue(a[8]) ? at::kFloat : dt;
    const int device = x.get_device();
    const int64_t B = x.size(0), n = x.size(has_q ? 1 : 2), d = x.size(3);
    const auto rot = rotary(a[2], device);
    tq_heads qh, kh;
    int64_t qs[4] = {B, n, has_q ? x.size(2) : 0, d}, ks[4] = {B, 0, n, d};
    if (has_q) qh = heads(x, "q", qs, dt, device, 0, 1, 2);
    if (has_k) {
      const at::Tensor& k = tensor(a[1], "k");
      if (k.dim() == 4) ks[1] = k.size(1);
      kh = heads(k, "k", ks, dt, device, 0, 2, 1);
    }
    const int32_t* pos = ints(a[3], "positions", {rot ? rot->num_axes : 1, B, n}, device);
    const int32_t* start = ints(a[4], "start", {B}, device);
    const void* wq = weight(a[5], "q_weight", d, dt, device);
    const void* wk = weight(a[6], "k_weight", d, dt, device);
    const float eps = number(a[7]);
    const On on(device);
    at::Tensor qo, ko;
    if (has_q) qo = output(a[9], "q_out", qs, odt, device);
    if (has_k) ko = output(a[10], "k_out", ks, odt, device);
    if (B > 0 && n > 0)
      check(tq_norm_rotate(narrow(d, "head_dim"), code, odt == at::kFloat ? TQ_F32 : code, narrow(B, "batch"), narrow(n, "n"),
                           has_q ? &qh : nullptr, wq, has_q ? qo.data_ptr() : nullptr, has_k ? &kh : nullptr, wk,
                           has_k ? ko.data_ptr() : nullptr, eps, rot ? &*rot : nullptr, pos, start, on.stream));
    PyObject* out = PyTuple_New(2);
    if (!out) throw Failed();
    PyTuple_SET_ITEM(out, 0, has_q ? THPVariable_Wrap(qo) : Py_NewRef(Py_None));
    PyTuple_SET_ITEM(out, 1, has_k ? THPVariable_Wrap(ko) : Py_NewRef(Py_None));
    return out;
  });
}

// append(cache, k, v, start, block_table, count, rotary, positions, k_weight, q, q_weight, eps, q_out) -> q_out or None
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_args(n_args, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache(a[0]);
    int64_t B;
    const tq_page_table pt = page_table(a[4], c, &B);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const tq_dtype code = dtype_of(k);
    const at::ScalarType dt = k.scalar_type();
    const int64_t n = k.dim() == 4 ? k.size(2) : 0, d = c.cfg.head_dim;
    const int64_t shape[4] = {B, c.cfg.num_kv_heads, n, d};
    const tq_heads kh = heads(k, "k", shape, dt, c.device, 0, 2, 1), vh = heads(v, "v", shape, dt, c.device, 0, 2, 1);
    const auto rot = rotary(a[6], c.device);
    if (!given(a[3])) throw Refused("start must be given");
    const int32_t* start = ints(a[3], "start", {B}, c.device);
    const int32_t* count = ints(a[5], "count", {B}, c.device);
    const int32_t* pos = ints(a[7], "positions", {rot ? rot->num_axes : 1, B, n}, c.device);
    const void* wk = weight(a[8], "k_weight", d, dt, c.device);
    const void* wq = weight(a[10], "q_weight", d, dt, c.device);
    const bool has_q = given(a[9]);
    const int64_t qs[4] = {B, n, c.cfg.num_q_heads, d};
    tq_heads qh;
    if (has_q) qh = heads(tensor(a[9], "q"), "q", qs, dt, c.device, 0, 1, 2);
    const float eps = number(a[11]);
    const On on(c.device);
    at::Tensor qo;
    if (has_q) qo = output(a[12], "q_out", qs, dt, c.device);
    if (B > 0 && n > 0)
      check(tq_byte_append_paged(&c.cfg, c.pool, &pt, narrow(B, "batch"), narrow(n, "n"), code, &kh, &vh, start, count, wk, eps,
                                 rot ? &*rot : nullptr, pos, has_q ? &qh : nullptr, wq, has_q ? qo.data_ptr() : nullptr, c.error,
                                 on.stream));
    return has_q ? THPVariable_Wrap(qo) : Py_NewRef(Py_None);
  });
}

// attention(cache, q, seq_len, block_table, count, scale, out, tree) -> out
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_args(n_args, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache(a[0]);
    int64_t B;
    const tq_page_table pt = page_table(a[3], c, &B);
    const at::Tensor& q = tensor(a[1], "q");
    const tq_dtype code = dtype_of(q);
    const at::ScalarType dt = q.scalar_type();
    const int64_t d = c.cfg.head_dim, nq = q.dim() == 4 ? q.size(1) : 1;
    tq_heads qh;
    if (q.dim() == 3) {  // one query per entry
      same_kind(q, "q", dt, c.device);
      plain(q, "q");
      has_shape(q, "q", {B, c.cfg.num_q_heads, d});
      if (q.stride(2) != 1) throw Refused("q: the head dimension must be contiguous");
      qh = tq_heads{q.const_data_ptr(), q.stride(0), 0, q.stride(1), c.cfg.num_q_heads};
    } else {
      qh = heads(q, "q", {B, nq, c.cfg.num_q_heads, d}, dt, c.device, 0, 1, 2);
    }
    if (!given(a[2])) throw Refused("seq_len must be given");
    const int32_t* seq = ints(a[2], "seq_len", {B}, c.device);
    const int32_t* count = ints(a[4], "count", {B}, c.device);
    const float scale = number(a[5]);
    const int32_t* tree = ints(a[7], "tree", {B, nq, (nq + 31) / 32}, c.device);
    const On on(c.device);
    at::Tensor out = output(a[6], "out", q.sizes(), dt, c.device);
    if (B > 0 && nq > 0) {
      const size_t need = tree ? tq_byte_tree_attention_workspace_bytes(&c.cfg, narrow(B, "batch"), narrow(nq, "nq"), code)
                               : tq_byte_attention_workspace_bytes(&c.cfg, &pt, narrow(B, "batch"), narrow(nq, "nq"), code);
      at::Tensor ws;
      if (need) ws = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(out.device()));
      void* w = need ? ws.data_ptr() : nullptr;
      check(tree ? tq_byte_tree_attention_paged(&c.cfg, c.pool, &pt, (int32_t)B, (int32_t)nq, code, &qh, seq, count, tree, scale,
                                                out.data_ptr(), w, need, c.error, on.stream)
                 : tq_byte_attention_paged(&c.cfg, c.pool, &pt, (int32_t)B, (int32_t)nq, code, &qh, seq, count, scale,
                                           out.data_ptr(), w, need, c.error, on.stream));
    }
    return THPVariable_Wrap(out);
  });
}

// draft_tree(parents, start, count, masks, positions) -> (masks, positions)
PyObject* draft_tree(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_args(n_args, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& p = tensor(a[0], "parents");
    if (p.dim() != 2 || !p.is_cuda()) throw Refused("parents must be a CUDA tensor [batch][n], not " + shape_text(p));
    const int device = p.get_device();
    const int64_t B = p.size(0), n = p.size(1);
    const int32_t* parents = ints(a[0], "parents", {B, n}, device);
    const int32_t* start = ints(a[1], "start", {B}, device);
    const int32_t* count = ints(a[2], "count", {B}, device);
    const On on(device);
    at::Tensor masks = output(a[3], "masks", {B, n, (n + 31) / 32}, at::kInt, device);
    at::Tensor positions = output(a[4], "positions", {1, B, n}, at::kInt, device);
    if (B > 0 && n > 0)
      check(tq_draft_tree(narrow(B, "batch"), narrow(n, "n"), parents, start, count, (int32_t*)masks.data_ptr(),
                          (int32_t*)positions.data_ptr(), on.stream));
    PyObject* out = PyTuple_New(2);
    if (!out) throw Failed();
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(masks));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(positions));
    return out;
  });
}

// keep(cache, path, start, block_table, count, seq_len) -> seq_len
PyObject* keep(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_args(n_args, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache(a[0]);
    int64_t B;
    const tq_page_table pt = page_table(a[3], c, &B);
    const at::Tensor& p = tensor(a[1], "path");
    if (p.dim() != 2) throw Refused("path must be a tensor [batch][n], not " + shape_text(p));
    const int64_t n = p.size(1);
    const int32_t* path = ints(a[1], "path", {B, n}, c.device);
    if (!given(a[2])) throw Refused("start must be given");
    const int32_t* start = ints(a[2], "start", {B}, c.device);
    const int32_t* count = ints(a[4], "count", {B}, c.device);
    const On on(c.device);
    at::Tensor len = output(a[5], "seq_len", {B}, at::kInt, c.device);
    if (B > 0)
      check(tq_byte_keep_paged(&c.cfg, c.pool, &pt, narrow(B, "batch"), narrow(n, "n"), path, start, count,
                               (int32_t*)len.data_ptr(), c.error, on.stream));
    return THPVariable_Wrap(len);
  });
}

// read(cache, start, block_table, n, count, dtype, k_out, v_out) -> (k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_args(n_args, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Cache c = cache(a[0]);
    int64_t B;
    const tq_page_table pt = page_table(a[2], c, &B);
    if (!given(a[1])) throw Refused("start must be given");
    const int32_t* start = ints(a[1], "start", {B}, c.device);
    const long long n = PyLong_AsLongLong(a[3]);
    if (n == -1 && PyErr_Occurred()) throw Failed();
    const int32_t* count = ints(a[4], "count", {B}, c.device);
    if (!THPDtype_Check(a[5])) throw Refused("dtype must be a torch.dtype");
    const at::ScalarType dt = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    const tq_dtype code = dtype_code(dt);
    if (n < 0) throw Refused("n must be >= 0");
    narrow(n, "n");
    const On on(c.device);
    const int64_t shape[4] = {B, c.cfg.num_kv_heads, n, c.cfg.head_dim};
    at::Tensor k = output(a[6], "k_out", shape, dt, c.device), v = output(a[7], "v_out", shape, dt, c.device);
    if (B > 0 && n > 0)
      check(tq_byte_read_paged(&c.cfg, c.pool, &pt, narrow(B, "batch"), (int32_t)n, code, start, count, k.data_ptr(), v.data_ptr(),
                               c.error, on.stream));
    PyObject* out = PyTuple_New(2);
    if (!out) throw Failed();
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(v));
    return out;
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"norm_rotate", (PyCFunction)(void (*)(void))norm_rotate, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
    {"draft_tree", (PyCFunction)(void (*)(void))draft_tree, METH_FASTCALL, nullptr},
    {"keep", (PyCFunction)(void (*)(void))keep, METH_FASTCALL, nullptr},
    {"read", (PyCFunction)(void (*)(void))read, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tq_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tq_torch(void) { return PyModule_Create(&kModule); }
