// pd_bind.cpp -- the Python side of the calls that a serving step makes once a
// layer: checks torch tensors and passes their addresses on to the C ABI.
//
// A step of one token per request is a few microseconds of GPU work, and reading
// a tensor's attributes one by one from Python takes longer than that. This
// module does the same reading in C++: per call it takes what the functions of
// the package's __init__.py have, checks it, and calls the library through the
// addresses that init() was given, so it links against no part of it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/pd.h"

namespace {

PyObject* g_error = nullptr;  // the package's PdError
decltype(&pd_batch_tables) g_batch_tables = nullptr;
decltype(&pd_qk_norm_rope) g_norm_rope = nullptr;
decltype(&pd_qk_norm_rope_append) g_norm_rope_append = nullptr;
decltype(&pd_attn_chunk) g_attn_chunk = nullptr;
decltype(&pd_attn_chunk_workspace_size) g_chunk_workspace = nullptr;

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(const char* format, ...) {
  char text[256];
  va_list args;
  va_start(args, format);
  vsnprintf(text, sizeof(text), format, args);
  va_end(args);
  PyErr_SetString(g_error, text);
  throw Refused{};
}

// A call's tensors, all on one device.
struct Args {
  int device = -1;

  // The tensor, or null for None.
  const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
    if (o == Py_None) {
      if (optional) return nullptr;
      refuse("%s is missing", name);
    }
    if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    const int d = t.get_device();
    if (device >= 0 && d != device) refuse("%s is on device %d, the arguments before it on device %d", name, d, device);
    device = d;
    return &t;
  }

  // Address of a contiguous tensor of a type with at least n entries.
  template <typename T>
  T* vector(PyObject* o, const char* name, at::ScalarType type, int64_t n = 0, bool optional = false) {
    const at::Tensor* t = tensor(o, name, optional);
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != type || !t->is_contiguous())
      refuse("%s must be a contiguous %s tensor", name, c10::toString(type));
    if (t->numel() < n) refuse("%s has %lld entries, %lld are needed", name, (long long)t->numel(), (long long)n);
    return static_cast<T*>(t->data_ptr());
  }
};

constexpr at::ScalarType kI32 = at::ScalarType::Int, kI64 = at::ScalarType::Long, kF32 = at::ScalarType::Float;

int dtype_code(at::ScalarType t, const char* name) {
  if (t == at::ScalarType::Float) return PD_F32;
  if (t == at::ScalarType::BFloat16) return PD_BF16;
  refuse("%s: unsupported dtype %s", name, c10::toString(t));
}

// A [tokens][heads][dim] tensor whose heads lie one after another: its token stride.
int64_t rows(const at::Tensor& t, const char* name) {
  if (t.dim() != 3 || t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2)))
    refuse("%s must be [tokens][heads][dim] with contiguous heads", name);
  // (a stride of 0 says "contiguous" to the library)
  if (t.size(0) > 1 && t.stride(0) == 0 && t.numel() > 0) refuse("the tokens of %s are one row", name);
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

int64_t same_rows(const at::Tensor& t, const at::Tensor& like, const char* name) {
  if (t.dim() != 3 || t.sizes() != like.sizes()) refuse("%s has another shape than it should have", name);
  if (t.scalar_type() != like.scalar_type()) refuse("%s has another dtype than its input", name);
  return rows(t, name);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

int32_t int32(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse("%s is out of range", name);
  return (int32_t)v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v == 1;
}

void* stream_of(PyObject* o) { return reinterpret_cast<void*>(integer(o)); }

struct Pools {
  const at::Tensor *k, *v;
  int32_t num_pages, heads, page, dim;
};

// Two contiguous 4-D pools of the same shape, HND (0) or NHD (1).
Pools pools(Args& a, PyObject* k, PyObject* v, int layout) {
  Pools p{a.tensor(k, "k_pool"), a.tensor(v, "v_pool"), 0, 0, 0, 0};
  if (p.k->dim() != 4 || p.k->sizes() != p.v->sizes() || !p.k->is_contiguous() || !p.v->is_contiguous())
    refuse("k_pool and v_pool must be contiguous pools of the same shape");
  if (p.k->scalar_type() != p.v->scalar_type()) refuse("k_pool and v_pool differ in dtype");
  p.num_pages = (int32_t)p.k->size(0);
  p.heads = (int32_t)p.k->size(layout == PD_LAYOUT_HND ? 1 : 2);
  p.page = (int32_t)p.k->size(layout == PD_LAYOUT_HND ? 2 : 1);
  p.dim = (int32_t)p.k->size(3);
  return p;
}

// (device, status): every entry returns them; the caller makes another device
// current and calls again when `device` is not the one it passed as current.
PyObject* done(int device, int status) {
  if (status == PD_OK) Py_RETURN_NONE;
  return Py_BuildValue("(ii)", device, status);
}
constexpr int kOtherDevice = 1;  // not a pd_status

// Calls the library without the interpreter's lock, as ctypes does: a launch on a full
// queue blocks, and no other thread of the program has to wait with it.
template <typename... P, typename... A>
int unlocked(int (*call)(P...), A... args) {
  PyThreadState* state = PyEval_SaveThread();
  const int rc = call(args...);
  PyEval_RestoreThread(state);
  return rc;
}

// batch_tables(current device, stream or None, new_len, cached_len, block_table, rows, free_pages, free_count,
//   free_count_out, qo_indptr, kv_len, page_indptr, page_indices, positions, slot_map, dev_status, page_size, num_pages,
//   total_qo, max_page_indices)
PyObject* batch_tables(PyObject* const* o) {
  Args a;
  const at::Tensor* fresh = a.tensor(o[2], "new_len");
  if (a.device != integer(o[0])) return done(a.device, kOtherDevice);
  const int64_t B = fresh->numel();
  pd_tables_desc d{};
  d.batch_size = (int32_t)B;
  d.page_size = int32(o[16], "page_size");
  d.num_pages = int32(o[17], "num_pages");
  d.total_qo = int32(o[18], "total_qo");
  d.max_page_indices = int32(o[19], "max_page_indices");
  const auto* new_len = a.vector<int32_t>(o[2], "new_len", kI32);
  const auto* cached = a.vector<int32_t>(o[3], "cached_len", kI32, B);
  const at::Tensor* table = a.tensor(o[4], "block_table");
  if (table->dim() != 2) refuse("block_table must be [rows][pages]");
  auto* block_table = a.vector<int32_t>(o[4], "block_table", kI32);
  if (table->size(0) > INT32_MAX || table->size(1) > INT32_MAX) refuse("block_table is too large");
  d.table_rows = (int32_t)table->size(0);
  d.table_cols = (int32_t)table->size(1);
  const auto* row = a.vector<int32_t>(o[5], "rows", kI32, B, true);
  const auto* free_pages = a.vector<int32_t>(o[6], "free_pages", kI32, 0, true);
  const auto* count = a.vector<int32_t>(o[7], "free_count", kI32, 1, free_pages == nullptr);
  auto* left = a.vector<int32_t>(o[8], "free_count_out", kI32, 1, free_pages == nullptr);
  if (free_pages != nullptr) d.free_capacity = (int32_t)THPVariable_Unpack(o[6]).numel();
  auto* qo = a.vector<int32_t>(o[9], "qo_indptr", kI32, B + 1);
  auto* kv = a.vector<int32_t>(o[10], "kv_len", kI32, B);
  auto* pp = a.vector<int32_t>(o[11], "page_indptr", kI32, B + 1);
  auto* px = a.vector<int32_t>(o[12], "page_indices", kI32, d.max_page_indices);
  auto* pos = a.vector<int32_t>(o[13], "positions", kI32, d.total_qo);
  auto* slot = a.vector<int64_t>(o[14], "slot_map", kI64, d.total_qo);
  auto* status = a.vector<int32_t>(o[15], "dev_status", kI32, 1, true);
  return done(a.device, unlocked(g_batch_tables, &d, row, cached, new_len, block_table, free_pages, count, left, qo, kv,
                                 pp, px, pos, slot, status, stream_of(o[1])));
}

// What both forms of the norm and rotation share: q, k, weights, frequencies and positions at o[2..7].
struct NormRope {
  const at::Tensor *q, *k;
  const void *qw, *kw;
  const float* freq;
  const int32_t* pos;
  pd_norm_rope_desc d{};
  int32_t tokens;

  NormRope(Args& a, PyObject* const* o, PyObject* eps, PyObject* interleaved) {
    q = a.tensor(o[2], "q");
    k = a.tensor(o[3], "k");
    d.q_stride = rows(*q, "q");
    d.k_stride = rows(*k, "k");
    const at::ScalarType dt = q->scalar_type();
    if (k->scalar_type() != dt || k->size(2) != q->size(2) || k->size(0) != q->size(0))
      refuse("q and k differ in dtype, head_dim or tokens");
    if (q->size(0) > INT32_MAX) refuse("too many tokens");
    tokens = (int32_t)q->size(0);
    d.num_qo_heads = (int32_t)q->size(1);
    d.num_kv_heads = (int32_t)k->size(1);
    d.head_dim = (int32_t)q->size(2);
    d.dtype = dtype_code(dt, "q");
    qw = a.vector<void>(o[4], "q_weight", dt, d.head_dim, true);
    kw = a.vector<void>(o[5], "k_weight", dt, d.head_dim, true);
    freq = a.vector<float>(o[6], "inv_freq", kF32, 0, true);
    pos = a.vector<int32_t>(o[7], "positions", kI32, freq != nullptr ? tokens : 0, freq == nullptr);
    d.rope_dim = freq != nullptr ? 2 * (int32_t)THPVariable_Unpack(o[6]).numel() : 0;
    d.eps = (float)real(eps);
    d.interleaved = truth(interleaved);
  }
};

// norm_rope(current device, stream, q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out, eps, interleaved)
PyObject* norm_rope(PyObject* const* o) {
  Args a;
  a.tensor(o[2], "q");
  if (a.device != integer(o[0])) return done(a.device, kOtherDevice);
  NormRope n(a, o, o[10], o[11]);
  const at::Tensor *qo = a.tensor(o[8], "q_out"), *ko = a.tensor(o[9], "k_out");
  n.d.q_out_stride = same_rows(*qo, *n.q, "q_out");
  n.d.k_out_stride = same_rows(*ko, *n.k, "k_out");
  return done(a.device, unlocked(g_norm_rope, &n.d, n.tokens, n.q->data_ptr(), n.k->data_ptr(), n.qw, n.kw, n.freq,
                                 n.pos, qo->data_ptr(), ko->data_ptr(), stream_of(o[1])));
}

// norm_rope_append(current device, stream, q, k, q_weight, k_weight, inv_freq, positions, v, slot_map, k_pool, v_pool,
//   q_out, dev_status, eps, interleaved, layout)
PyObject* norm_rope_append(PyObject* const* o) {
  Args a;
  a.tensor(o[2], "q");
  if (a.device != integer(o[0])) return done(a.device, kOtherDevice);
  NormRope n(a, o, o[14], o[15]);
  const at::Tensor* v = a.tensor(o[8], "v");
  n.d.v_stride = same_rows(*v, *n.k, "v");
  const auto* slot = a.vector<int64_t>(o[9], "slot_map", kI64, n.tokens);
  n.d.layout = int32(o[16], "layout");
  const Pools p = pools(a, o[10], o[11], n.d.layout);
  if (p.heads != n.d.num_kv_heads || p.dim != n.d.head_dim || p.k->scalar_type() != n.q->scalar_type())
    refuse("the pools' heads, head_dim or dtype are not those of k");
  n.d.page_size = p.page;
  n.d.num_pages = p.num_pages;
  const at::Tensor* qo = a.tensor(o[12], "q_out");
  n.d.q_out_stride = same_rows(*qo, *n.q, "q_out");
  auto* status = a.vector<int32_t>(o[13], "dev_status", kI32, 1, true);
  return done(a.device, unlocked(g_norm_rope_append, &n.d, n.tokens, n.q->data_ptr(), n.k->data_ptr(), v->data_ptr(),
                                 n.qw, n.kw, n.freq, n.pos, slot, qo->data_ptr(), p.k->data_ptr(), p.v->data_ptr(),
                                 status, stream_of(o[1])));
}

// attn_chunk(current device, stream, q, k_pool, v_pool, kv_len, page_indptr, page_indices, qo_indptr, o, lse, workspace,
//   dev_status, causal, window_left, sm_scale, max_qo_len, max_kv_len, layout); a workspace that is missing or too small
//   gives (the bytes needed, PD_ERR_WORKSPACE)
PyObject* attn_chunk(PyObject* const* o) {
  Args a;
  const at::Tensor* q = a.tensor(o[2], "q");
  if (a.device != integer(o[0])) return done(a.device, kOtherDevice);
  pd_attn_desc d{};
  d.layout = int32(o[18], "layout");
  const Pools p = pools(a, o[3], o[4], d.layout);
  if (p.k->scalar_type() != q->scalar_type()) refuse("q and the pools differ in dtype");
  const int64_t stride = rows(*q, "q");
  if (q->size(2) != p.dim) refuse("q and the pools differ in head_dim");
  if (q->size(0) > INT32_MAX) refuse("too many rows");
  pd_batch b{};
  b.kv_len = a.vector<int32_t>(o[5], "kv_len", kI32);
  const int64_t B = THPVariable_Unpack(o[5]).numel();
  b.batch_size = (int32_t)B;
  b.page_indptr = a.vector<int32_t>(o[6], "page_indptr", kI32, B + 1);
  b.page_indices = a.vector<int32_t>(o[7], "page_indices", kI32);
  b.qo_indptr = a.vector<int32_t>(o[8], "qo_indptr", kI32, B + 1);
  b.num_pages = p.num_pages;
  b.total_qo = (int32_t)q->size(0);
  b.max_qo_len = int32(o[16], "max_qo_len");
  b.max_kv_len = int32(o[17], "max_kv_len");
  const at::Tensor* out = a.tensor(o[9], "o");
  if (out->sizes() != q->sizes() || !out->is_contiguous()) refuse("o must be contiguous and shaped like q");
  auto* lse = a.vector<float>(o[10], "lse", kF32, q->size(0) * q->size(1), true);
  const at::Tensor* ws = a.tensor(o[11], "workspace", true);
  if (ws != nullptr && !ws->is_contiguous()) refuse("workspace must be contiguous");
  auto* status = a.vector<int32_t>(o[12], "dev_status", kI32, 1, true);
  d.num_qo_heads = (int32_t)q->size(1);
  d.num_kv_heads = p.heads;
  d.head_dim = p.dim;
  d.page_size = p.page;
  d.kv_dtype = dtype_code(q->scalar_type(), "q");
  d.o_dtype = dtype_code(out->scalar_type(), "o");
  d.causal = truth(o[13]);
  d.sm_scale = o[15] == Py_None ? 0.f : (float)real(o[15]);
  const int32_t window = o[14] == Py_None ? -1 : int32(o[14], "window_left");
  int rc = PD_ERR_WORKSPACE;
  if (ws != nullptr)
    rc = unlocked(g_attn_chunk, &d, &b, window, stride, q->data_ptr(), p.k->data_ptr(), p.v->data_ptr(),
                  out->data_ptr(), lse, ws->data_ptr(), ws->numel() * ws->element_size(), status, stream_of(o[1]));
  if (rc != PD_ERR_WORKSPACE) return done(a.device, rc);
  return Py_BuildValue("(Ki)", (unsigned long long)g_chunk_workspace(&d, &b), rc);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(g_error, e.what());
    return nullptr;
  }
}

// init(PdError, addresses of the entry points in the order below)
PyObject* init(PyObject* const* o) {
  Py_INCREF(o[0]);
  Py_XDECREF(g_error);
  g_error = o[0];
  g_batch_tables = reinterpret_cast<decltype(g_batch_tables)>(integer(o[1]));
  g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(integer(o[2]));
  g_norm_rope_append = reinterpret_cast<decltype(g_norm_rope_append)>(integer(o[3]));
  g_attn_chunk = reinterpret_cast<decltype(g_attn_chunk)>(integer(o[4]));
  g_chunk_workspace = reinterpret_cast<decltype(g_chunk_workspace)>(integer(o[5]));
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<init, 6>("init"),
                           method<batch_tables, 20>("batch_tables"),
                           method<norm_rope, 12>("norm_rope"),
                           method<norm_rope_append, 17>("norm_rope_append"),
                           method<attn_chunk, 19>("attn_chunk"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pd_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// PD_TORCH: the version of the torch whose headers this was compiled with.
PyMODINIT_FUNC PyInit__pd_bind() {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", PD_TORCH) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
