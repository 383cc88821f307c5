// The paged cache's calls for Python (include/mf.h: mf_paged_decode, mf_kv_append, mf_kv_evict,
// mf_map_key_scores): checks of the tensors, descriptors, workspaces, streams.  The same checks
// took 9 to 12 us a call in Python, twice the launches of a small decode step; here they take
// less than one.  libmf.so itself is reached through the addresses that `attach` gets, so the
// package loads one library whatever MF_LIBRARY names.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <array>
#include <optional>
#include <sstream>
#include <string>

#include "mf.h"

namespace {

struct Api {
  decltype(&mf_paged_decode) decode;
  decltype(&mf_paged_decode_workspace_size) decode_ws;
  decltype(&mf_kv_append) append;
  decltype(&mf_kv_evict) evict;
  decltype(&mf_kv_evict_workspace_size) evict_ws;
  decltype(&mf_map_key_scores) scores;
  decltype(&mf_map_key_scores_workspace_size) scores_ws;
} api{};
PyObject* raise_status = nullptr;  // Python: raises the error of a status

// a refused argument: the Python exception that says so
struct Refusal {
  PyObject* type;
  std::string what;
};
// a Python exception is set already
struct Raised {};

[[noreturn]] void refuse(const std::string& what, PyObject* type = PyExc_ValueError) { throw Refusal{type, what}; }

std::string show(at::IntArrayRef sizes) {
  std::ostringstream s;
  s << sizes;
  return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) refuse(std::string(what) + " must be a CUDA tensor");
  return t;
}

const at::Tensor& tensor(PyObject* o, const char* what, int64_t dims) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != dims)
    refuse(std::string(what) + " has shape " + show(t.sizes()) + ", expected " + std::to_string(dims) + " dimensions");
  return t;
}

// address of a tensor that is as the call needs it
void* at_address(const at::Tensor& t, const char* what, at::ScalarType dtype, at::IntArrayRef shape, int index,
                 bool dense = true) {
  if (t.scalar_type() != dtype)
    refuse(std::string(what) + " must be " + c10::toString(dtype) + ", not " + c10::toString(t.scalar_type()));
  if (t.get_device() != index)
    refuse(std::string(what) + " is on " + t.device().str() + ", the call's other tensors on cuda:" + std::to_string(index));
  if (t.sizes() != shape) refuse(std::string(what) + " has shape " + show(t.sizes()) + ", expected " + show(shape));
  if (dense && !t.is_contiguous()) refuse(std::string(what) + " must be contiguous");
  return t.data_ptr();
}
template <class P = void>
P* at_address(PyObject* o, const char* what, at::ScalarType dtype, at::IntArrayRef shape, int index) {
  return o == Py_None ? nullptr : static_cast<P*>(at_address(tensor(o, what), what, dtype, shape, index));
}
template <class P = void>
P* required(PyObject* o, const char* what, at::ScalarType dtype, at::IntArrayRef shape, int index) {
  return static_cast<P*>(at_address(tensor(o, what), what, dtype, shape, index));
}

mf_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return MF_F32;
  if (t.scalar_type() == at::kBFloat16) return MF_BF16;
  refuse(std::string("unsupported dtype ") + c10::toString(t.scalar_type()), PyExc_TypeError);
}

// Elements between the rows (dim 0) of one or two tensors, which must agree; their other dims must
// be dense.  0 for dense rows, as the C calls take it: rows of an expanded tensor, which are 0 apart,
// are refused, as all are that begin inside the row before them.
int64_t row_stride(const at::Tensor& a, const at::Tensor& b, const char* what) {
  if (a.is_contiguous() && b.is_contiguous()) return 0;
  for (const at::Tensor* t : {&a, &b}) {
    int64_t step = 1;
    for (int64_t k = t->dim() - 1; k > 0; --k) {
      if (t->size(k) != 1 && t->stride(k) != step) refuse(std::string(what) + ": the dims after the first must be dense");
      step *= t->size(k);
    }
    if (t->size(0) > 1 && t->stride(0) < step)
      refuse(std::string(what) + " overlap: " + std::to_string(t->stride(0)) + " elements apart, " + std::to_string(step) +
             " long (an expanded tensor has to be copied first)");
  }
  if (a.size(0) <= 1 || a.numel() == 0) return 0;
  if (a.stride(0) != b.stride(0)) refuse(std::string(what) + " must have the same stride");
  return a.stride(0);
}

int32_t i32(PyObject* o, const char* what) {
  THPObjectPtr n(PyNumber_Index(o));
  if (!n) throw Raised{};
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(n.get(), &overflow);
  if (overflow || v < INT32_MIN || v > INT32_MAX) refuse(std::string(what) + " does not fit 32 bits");
  return (int32_t)v;
}
int32_t i32(int64_t v, const char* what) {
  if (v > INT32_MAX) refuse(std::string(what) + " does not fit 32 bits");
  return (int32_t)v;
}

struct Names {
  PyObject *K, *V, *block_table, *seq_lens, *max_len, *row_ptr, *col_idx, *values, *stream_id, *device_index,
      *device_type;
} names{};

THPObjectPtr attribute(PyObject* o, PyObject* name) {
  THPObjectPtr v(PyObject_GetAttr(o, name));
  if (!v) throw Raised{};
  return v;
}

// a PagedKV, checked; holds on to its tensors while the call is enqueued
struct Kv {
  THPObjectPtr K, V, table, lens;
  mf_paged_kv d{};
  int index;
  at::ScalarType dtype;
  int64_t nseq, h_kv, dim;

  explicit Kv(PyObject* kv)
      : K(attribute(kv, names.K)), V(attribute(kv, names.V)), table(attribute(kv, names.block_table)),
        lens(attribute(kv, names.seq_lens)) {
    THPObjectPtr top = attribute(kv, names.max_len);
    if (THPVariable_Check(K.get())) dtype_of(THPVariable_Unpack(K.get()));
    const at::Tensor &k = tensor(K.get(), "K", 4), &v = tensor(V.get(), "V", 4), &t = tensor(table.get(), "block_table", 2);
    d.dtype = dtype_of(k);
    dtype = k.scalar_type();
    index = k.get_device();
    d.K = k.data_ptr();
    d.V = at_address(v, "V", dtype, k.sizes(), index, false);
    d.page_stride = row_stride(k, v, "pages of K and V");
    d.n_pages = i32(k.size(0), "n_pages");
    d.page_size = i32(k.size(1), "page_size");
    d.h_kv = i32(h_kv = k.size(2), "h_kv");
    d.d = i32(dim = k.size(3), "d");
    d.nseq = i32(nseq = t.size(0), "nseq");
    d.max_pages = i32(t.size(1), "max_pages");
    d.block_table = static_cast<int32_t*>(at_address(t, "block_table", at::kInt, t.sizes(), index));
    d.seq_lens = required<int32_t>(lens.get(), "seq_lens", at::kInt, {nseq}, index);
    d.max_len = i32(top.get(), "max_len");
  }
};

// The device and stream of a call: the given stream, or the current one of the tensors' device.
// Tensors that the call allocates come from that stream's pool.
class Where {
 public:
  Where(int index, PyObject* stream) : device_(index), stream_(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index)) {
    if (stream == Py_None) return;
    const long long id = number(stream, names.stream_id), at = number(stream, names.device_index),
                    type = number(stream, names.device_type);
    if (at != index) refuse("stream is on cuda:" + std::to_string(at) + ", the call's tensors on cuda:" + std::to_string(index));
    stream_ = c10::cuda::CUDAStream::unpack3(id, (c10::DeviceIndex)at, (c10::DeviceType)type);
    guard_.emplace(stream_);
  }
  void* handle() const { return stream_.stream(); }

 private:
  static long long number(PyObject* stream, PyObject* name) {
    const long long v = PyLong_AsLongLong(attribute(stream, name).get());
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
  }
  c10::cuda::CUDAGuard device_;
  c10::cuda::CUDAStream stream_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

at::TensorOptions on(int index, at::ScalarType dtype) {
  return at::TensorOptions().dtype(dtype).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)index));
}

void check(int status) {
  if (status == MF_OK) return;
  THPObjectPtr r(PyObject_CallFunction(raise_status, "i", status));
  if (r) PyErr_SetString(PyExc_RuntimeError, "mf call failed");
  throw Raised{};
}

// enqueues without the interpreter lock, as a call through ctypes does
template <class F> void enqueue(F&& f) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(state);
  check(status);
}

// the caller's workspace, or one from the stream's pool
struct Scratch {
  at::Tensor own;
  void* p;
  size_t bytes;
  template <class Size> Scratch(PyObject* given, int index, Size&& size) {
    if (given != Py_None) {
      const at::Tensor& t = tensor(given, "workspace");
      if (t.get_device() != index || !t.is_contiguous()) refuse("workspace must be a contiguous tensor on cuda:" + std::to_string(index));
      p = t.data_ptr();
      bytes = t.nbytes();
      return;
    }
    size_t need = 0;
    check(size(&need));
    own = at::empty({(int64_t)std::max<size_t>(need, 1)}, on(index, at::kByte));
    p = own.data_ptr();
    bytes = need;
  }
};

template <class F> PyObject* call(Py_ssize_t have, Py_ssize_t want, F&& f) {
  HANDLE_TH_ERRORS
  try {
    if (have != want) refuse("expected " + std::to_string(want) + " arguments", PyExc_TypeError);
    return f();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const Raised&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// kv, Q, O, scale, lse, score, score_out, o_f32, workspace, stream
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> PyObject* {
    Kv kv(a[0]);
    const Where where(kv.index, a[9]);
    const at::Tensor& Q = tensor(a[1], "Q", 3);
    const int64_t h_r = Q.size(1);
    const int wide_o = PyObject_IsTrue(a[7]);
    if (wide_o < 0) throw Raised{};
    const at::ScalarType o_type = wide_o ? at::kFloat : kv.dtype;
    mf_paged_decode_desc d{};
    d.kv = kv.d;
    d.Q = at_address(Q, "Q", kv.dtype, {kv.nseq, h_r, kv.dim}, kv.index, false);
    d.q_stride = row_stride(Q, Q, "rows of Q");
    d.h_r = i32(h_r, "h_r");
    const double scale = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw Raised{};
    d.scale = (float)scale;
    if (scale != 0.0 && d.scale == 0.0f) refuse("scale is too small for a float32 (0 would mean 1 / sqrt(d))");
    const at::Tensor O = a[2] == Py_None ? at::empty({kv.nseq, h_r, kv.dim}, on(kv.index, o_type)) : tensor(a[2], "O");
    d.O = at_address(O, "O", o_type, {kv.nseq, h_r, kv.dim}, kv.index);
    d.lse = at_address<float>(a[4], "lse", at::kFloat, {kv.nseq, h_r}, kv.index);
    if (a[5] != Py_None || a[6] != Py_None) {
      const int64_t wide = a[5] != Py_None ? tensor(a[5], "score", 3).size(2) : tensor(a[6], "score_out", 3).size(2);
      d.score_in = at_address<float>(a[5], "score", at::kFloat, {kv.nseq, kv.h_kv, wide}, kv.index);
      d.score_out = at_address<float>(a[6], "score_out", at::kFloat, {kv.nseq, kv.h_kv, wide}, kv.index);
      if (a[6] == Py_None) d.score_out = const_cast<float*>(d.score_in);
      d.score_stride = wide;
    }
    d.flags = wide_o ? MF_DECODE_O_F32 : 0;
    const Scratch ws(a[8], kv.index, [&](size_t* need) { return api.decode_ws(&d, need); });
    enqueue([&] { return api.decode(&d, ws.p, ws.bytes, where.handle()); });
    return a[2] == Py_None ? THPVariable_Wrap(O) : Py_NewRef(a[2]);
  });
}

// kv, K_new, V_new, cu_seqlens_new, max_new, n_seen, score, pos, stream
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&]() -> PyObject* {
    Kv kv(a[0]);
    const Where where(kv.index, a[8]);
    const at::Tensor &K = tensor(a[1], "K_new", 3), &V = tensor(a[2], "V_new", 3);
    mf_kv_append_desc d{};
    d.kv = kv.d;
    d.total_new = K.size(0);
    d.K_new = at_address(K, "K_new", kv.dtype, {d.total_new, kv.h_kv, kv.dim}, kv.index, false);
    d.V_new = at_address(V, "V_new", kv.dtype, {d.total_new, kv.h_kv, kv.dim}, kv.index, false);
    d.new_stride = row_stride(K, V, "rows of K_new and V_new");
    d.cu_seqlens_new = required<int32_t>(a[3], "cu_seqlens_new", at::kInt, {kv.nseq + 1}, kv.index);
    d.max_new = i32(a[4], "max_new");
    d.n_seen = at_address<int32_t>(a[5], "n_seen", at::kInt, {kv.nseq}, kv.index);
    if (a[6] != Py_None || a[7] != Py_None) {
      const int64_t wide = a[6] != Py_None ? tensor(a[6], "score", 3).size(2) : tensor(a[7], "pos", 3).size(2);
      d.score = at_address<float>(a[6], "score", at::kFloat, {kv.nseq, kv.h_kv, wide}, kv.index);
      d.pos = at_address<int32_t>(a[7], "pos", at::kInt, {kv.nseq, kv.h_kv, wide}, kv.index);
      d.score_stride = wide;
    }
    enqueue([&] { return api.append(&d, where.handle()); });
    Py_RETURN_NONE;
  });
}

// kv, score, pos, budget, sink, window, n_seen, score_out, pos_out, seq_lens_out, workspace, stream
PyObject* kv_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&]() -> PyObject* {
    Kv kv(a[0]);
    const Where where(kv.index, a[11]);
    const int64_t wide = tensor(a[1], "score", 3).size(2);
    const std::array<int64_t, 3> shape{kv.nseq, kv.h_kv, wide};
    mf_kv_evict_desc d{};
    d.kv = kv.d;
    float* s = required<float>(a[1], "score", at::kFloat, shape, kv.index);
    int32_t* p = required<int32_t>(a[2], "pos", at::kInt, shape, kv.index);
    d.score_in = s;
    d.pos_in = p;
    d.score_out = a[7] == Py_None ? s : required<float>(a[7], "score_out", at::kFloat, shape, kv.index);
    d.pos_out = a[8] == Py_None ? p : required<int32_t>(a[8], "pos_out", at::kInt, shape, kv.index);
    d.score_stride = wide;
    d.n_seen = at_address<int32_t>(a[6], "n_seen", at::kInt, {kv.nseq}, kv.index);
    d.budget = i32(a[3], "budget");
    d.sink = i32(a[4], "sink");
    d.window = i32(a[5], "window");
    PyObject* out = a[9] == Py_None ? kv.lens.get() : a[9];
    d.seq_lens_out = required<int32_t>(out, "seq_lens_out", at::kInt, {kv.nseq}, kv.index);
    const Scratch ws(a[10], kv.index, [&](size_t* need) { return api.evict_ws(&d, need); });
    enqueue([&] { return api.evict(&d, ws.p, ws.bytes, where.handle()); });
    return Py_NewRef(out);
  });
}

// bsr, W, cu_seqlens, qblock_base, max_seqlen, h_kv, score, workspace, stream
PyObject* map_key_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 9, [&]() -> PyObject* {
    THPObjectPtr row_ptr = attribute(a[0], names.row_ptr), col_idx = attribute(a[0], names.col_idx),
                       vals = attribute(a[0], names.values);
    const at::Tensor& values = tensor(vals.get(), "values", 4);
    mf_key_scores_desc d{};
    d.map_dtype = dtype_of(values);
    const int index = values.get_device();
    const Where where(index, a[8]);
    const at::Tensor &rows = tensor(row_ptr.get(), "row_ptr", 1), &kept = tensor(col_idx.get(), "col_idx", 1),
                     &W = tensor(a[1], "W", 2), &cu = tensor(a[2], "cu_seqlens", 1);
    const int64_t cap = values.size(0), h_s = values.size(1), B = values.size(2), nseq = cu.size(0) - 1;
    if (values.size(3) != B || kept.size(0) < cap || rows.size(0) < 1)
      refuse("values must be [capacity, h_s, B, B], col_idx [capacity], row_ptr [rows + 1]");
    if (nseq < 0) refuse("cu_seqlens must have nseq + 1 entries");
    d.bsr.values = at_address(values, "values", values.scalar_type(), values.sizes(), index);
    d.bsr.row_ptr = static_cast<int32_t*>(at_address(rows, "row_ptr", at::kInt, rows.sizes(), index));
    d.bsr.col_idx = static_cast<int32_t*>(at_address(kept, "col_idx", at::kInt, kept.sizes(), index));
    d.bsr.capacity_blocks = cap;
    d.n_rows = rows.size(0) - 1;
    d.h_s = i32(h_s, "h_s");
    d.B = i32(B, "B");
    d.W = static_cast<float*>(at_address(W, "W", at::kFloat, {W.size(0), h_s}, index));
    d.h_r = i32(W.size(0), "h_r");
    d.h_kv = i32(a[5], "h_kv");
    d.cu_seqlens = static_cast<int32_t*>(at_address(cu, "cu_seqlens", at::kInt, {nseq + 1}, index));
    d.qblock_base = required<int32_t>(a[3], "qblock_base", at::kInt, {nseq}, index);
    d.nseq = i32(nseq, "nseq");
    d.max_seqlen = i32(a[4], "max_seqlen");
    if (d.h_kv < 1) refuse("h_kv must be >= 1");
    const at::Tensor score = a[6] == Py_None
        ? at::zeros({nseq, d.h_kv, std::max<int64_t>(d.max_seqlen, 1)}, on(index, at::kFloat))
        : tensor(a[6], "score", 3);
    d.score_stride = score.size(2);
    d.score = static_cast<float*>(at_address(score, "score", at::kFloat, {nseq, d.h_kv, d.score_stride}, index));
    const Scratch ws(a[7], index, [&](size_t* need) { return api.scores_ws(&d, need); });
    enqueue([&] { return api.scores(&d, ws.p, ws.bytes, where.handle()); });
    return a[6] == Py_None ? THPVariable_Wrap(score) : Py_NewRef(a[6]);
  });
}

// the mf_paged_kv of a PagedKV, as bytes
PyObject* paged_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 1, [&]() -> PyObject* {
    Kv kv(a[0]);
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&kv.d), sizeof(kv.d));
  });
}

// addresses of libmf's functions by name, and the function that raises a status
PyObject* attach(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 2, [&]() -> PyObject* {
    auto find = [&](const char* name) -> void* {
      PyObject* v = PyDict_GetItemString(a[0], name);
      void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
      if (!p) refuse(std::string("no address of ") + name);
      return p;
    };
    Api f;
    f.decode = reinterpret_cast<decltype(f.decode)>(find("mf_paged_decode"));
    f.decode_ws = reinterpret_cast<decltype(f.decode_ws)>(find("mf_paged_decode_workspace_size"));
    f.append = reinterpret_cast<decltype(f.append)>(find("mf_kv_append"));
    f.evict = reinterpret_cast<decltype(f.evict)>(find("mf_kv_evict"));
    f.evict_ws = reinterpret_cast<decltype(f.evict_ws)>(find("mf_kv_evict_workspace_size"));
    f.scores = reinterpret_cast<decltype(f.scores)>(find("mf_map_key_scores"));
    f.scores_ws = reinterpret_cast<decltype(f.scores_ws)>(find("mf_map_key_scores_workspace_size"));
    api = f;
    raise_status = Py_NewRef(a[1]);
    Py_RETURN_NONE;
  });
}

#define MF_CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MF_CALL(paged_decode), MF_CALL(kv_append), MF_CALL(kv_evict), MF_CALL(map_key_scores),
                         MF_CALL(paged_kv), MF_CALL(attach), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mf_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mf_bind() {
  PyObject** const at[] = {&names.K, &names.V, &names.block_table, &names.seq_lens, &names.max_len, &names.row_ptr,
                           &names.col_idx, &names.values, &names.stream_id, &names.device_index, &names.device_type};
  const char* const text[] = {"K", "V", "block_table", "seq_lens", "max_len", "row_ptr",
                              "col_idx", "values", "stream_id", "device_index", "device_type"};
  for (size_t i = 0; i < sizeof(text) / sizeof(text[0]); ++i)
    if (!(*at[i] = PyUnicode_InternFromString(text[i]))) return nullptr;
  return PyModule_Create(&module);
}
