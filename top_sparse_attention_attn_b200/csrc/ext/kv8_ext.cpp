// kv8_ext.cpp -- the CPython side of kv8.py: checks torch tensors, allocates outputs and
// the workspace, fills the C ABI's structs and calls sa_page_plan / sa_kv8_write /
// sa_kv8_fwd.  A decode step's kernels take a few microseconds; the same marshalling in
// Python took 10 to 20 per call.
//
// Each function takes positional arguments (kv8.py names and documents them), raises
// TypeError / ValueError on tensors that do not fit, and returns the sa_status as an int
// where the library refuses the call.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <string>

#include "../../../include/sparse_attn.h"

namespace {

struct Refusal {
  PyObject* type;
  std::string what;
};
[[noreturn]] void type_error(const std::string& s) { throw Refusal{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refusal{PyExc_ValueError, s}; }

std::string shape_text(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " is not a tensor");
  return THPVariable_Unpack(o);
}

// Device index of a tensor, -1 on the CPU.
int index_of(const at::Tensor& t) { return t.is_cuda() ? (int)t.get_device() : -1; }

void check_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    type_error(std::string(name) + " is " + c10::toString(t.scalar_type()) + ": " + c10::toString(type) + " expected");
}
void check_device(const at::Tensor& t, const char* name, int index) {
  if (index_of(t) != index)
    value_error(std::string(name) + " is on " + t.device().str() + ": " +
                (index < 0 ? std::string("the CPU") : "cuda:" + std::to_string(index)) + " expected");
}

// Pointer of a contiguous tensor of this type, device and shape.
void* need(PyObject* o, const char* name, at::ScalarType type, int index, c10::IntArrayRef shape) {
  const at::Tensor& t = tensor(o, name);
  check_type(t, name, type);
  check_device(t, name, index);
  if (t.sizes() != shape)
    value_error(std::string(name) + " has shape " + shape_text(t.sizes()) + ": " + shape_text(shape) + " expected");
  if (!t.is_contiguous()) value_error(std::string(name) + " is not contiguous");
  return t.data_ptr();
}
int32_t* need_i32(PyObject* o, const char* name, int index, int64_t n) {
  return static_cast<int32_t*>(need(o, name, at::kInt, index, {n}));
}

int32_t dtype_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return SA_DTYPE_BF16;
  if (t.scalar_type() == at::kHalf) return SA_DTYPE_FP16;
  type_error(std::string(name) + " is " + c10::toString(t.scalar_type()) + ": bfloat16 or float16 expected");
}

struct Table {
  int32_t* ptr;
  int64_t rows, pages, stride;
};
Table table_of(PyObject* o, int index) {
  const at::Tensor& t = tensor(o, "block_table");
  if (t.scalar_type() != at::kInt || t.dim() != 2) type_error("block_table: int32 [B, max_pages] expected");
  check_device(t, "block_table", index);
  if (t.numel() == 0) return {static_cast<int32_t*>(t.data_ptr()), t.size(0), t.size(1), t.size(1)};
  if (t.size(1) > 1 && t.stride(1) != 1) value_error("block_table rows are not contiguous");
  const int64_t row = t.size(0) > 1 ? t.stride(0) : t.size(1);
  if (row < t.size(1)) value_error("block_table rows overlap");
  return {static_cast<int32_t*>(t.data_ptr()), t.size(0), t.size(1), row};
}

// Elements from token to token of [T, heads, d] or [B, s, heads, d] whose tokens lie
// evenly apart and whose token rows are contiguous.
int64_t token_step(const at::Tensor& t, const char* name, int64_t heads, int64_t d, int index) {
  check_device(t, name, index);
  const int64_t n = t.dim();
  if ((n != 3 && n != 4) || t.size(n - 2) != heads || t.size(n - 1) != d)
    value_error(std::string(name) + " has shape " + shape_text(t.sizes()) + ": [T, " + std::to_string(heads) + ", " +
                std::to_string(d) + "] or [B, s, " + std::to_string(heads) + ", " + std::to_string(d) + "] expected");
  int64_t step = heads * d;
  if (t.numel() == 0) return step;  // no element lies anywhere
  if ((d > 1 && t.stride(n - 1) != 1) || (heads > 1 && t.stride(n - 2) != d))
    value_error(std::string(name) + ": a token's rows are not contiguous");
  if (n == 3) {
    if (t.size(0) > 1) step = t.stride(0);
  } else if (t.size(1) > 1) {
    step = t.stride(1);
    if (t.size(0) > 1 && t.stride(0) != step * t.size(1)) value_error(std::string(name) + ": tokens do not lie evenly apart");
  } else if (t.size(0) > 1) {
    step = t.stride(0);
  }
  return step;
}

// n elements of `type` in the memory of `all`, from element `from` on (a view would cost as much as an
// allocation).
at::Tensor part_of(const at::Tensor& all, at::ScalarType type, int64_t from, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                          c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(from);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

int32_t to_i32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}
int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + ": an integer expected");
  }
  return v;
}

// Makes the device and the call's stream (a cudaStream_t as an integer, None for the current
// one) current, so that what the call allocates belongs to that stream.
class OnStream {
 public:
  OnStream(PyObject* o, int index) {
    if (index < 0) value_error("the tensors are on the CPU: a CUDA device expected");
    if (o == Py_None) {
      device_.set_index((c10::DeviceIndex)index);
    } else {
      const auto raw = reinterpret_cast<cudaStream_t>((uintptr_t)integer(o, "stream"));
      stream_.reset_stream(raw ? c10::cuda::getStreamFromExternal(raw, (c10::DeviceIndex)index)
                               : c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)index));
    }
    raw_ = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  }
  void* get() const { return raw_; }

 private:
  c10::cuda::OptionalCUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard stream_;
  void* raw_ = nullptr;
};

// The cache (a bytes object that holds its sa_kv8_cache, and its device index) with a
// step's tokens in it.
sa_kv8_cache step_of(PyObject* bytes, int index, const at::Tensor& x, const char* name, PyObject* table, PyObject* lens,
                     PyObject* cu) {
  sa_kv8_cache c;
  if (!PyBytes_Check(bytes) || PyBytes_GET_SIZE(bytes) != (Py_ssize_t)sizeof(c)) type_error("not a cache");
  memcpy(&c, PyBytes_AS_STRING(bytes), sizeof(c));
  const Table t = table_of(table, index);
  c.block_table = t.ptr;
  c.batch = to_i32(t.rows, "B");
  c.max_pages = to_i32(t.pages, "max_pages");
  c.table_stride = t.stride;
  c.seq_lens = need_i32(lens, "seq_lens", index, t.rows);
  if (cu != Py_None) {
    if (x.dim() != 3) value_error(std::string(name) + " is [T, heads, d] where cu_seqlens_q is given");
    c.layout = SA_LAYOUT_TND;
    c.t_q = to_i32(x.size(0), "T");
    c.cu_seqlens_q = need_i32(cu, "cu_seqlens_q", index, t.rows + 1);
  } else {
    if (x.dim() != 4 || x.size(0) != t.rows) value_error(std::string(name) + " is [B, s, heads, d] where cu_seqlens_q is not given");
    c.layout = SA_LAYOUT_BSND;
    c.s_q = to_i32(x.size(1), "s");
  }
  return c;
}

#define KV8_BEGIN(n, where)                                                          \
  HANDLE_TH_ERRORS                                                                   \
  if (nargs != (n)) return PyErr_Format(PyExc_TypeError, where ": %d arguments", n); \
  try {
#define KV8_END                                         \
  }                                                     \
  catch (const Refusal& r) {                            \
    PyErr_SetString(r.type, r.what.c_str());            \
    return nullptr;                                     \
  }                                                     \
  END_HANDLE_TH_ERRORS

// plan(old_lens, new_lens, block_table, free_pages, n_free, page_size, n_tokens, stream)
PyObject* kv8_plan(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  KV8_BEGIN(8, "plan")
  const at::Tensor& old = tensor(v[0], "old_lens");
  if (old.dim() != 1) value_error("old_lens is [B]");
  const int index = index_of(old);
  const int64_t B = old.size(0);
  sa_page_plan_args a = {};
  a.batch = to_i32(B, "B");
  a.old_lens = need_i32(v[0], "old_lens", index, B);
  a.new_lens = need_i32(v[1], "new_lens", index, B);
  const Table t = table_of(v[2], index);
  if (t.rows != B) value_error("block_table has " + std::to_string(t.rows) + " rows: " + std::to_string(B) + " expected");
  a.block_table = t.ptr;
  a.max_pages = to_i32(t.pages, "max_pages");
  a.table_stride = t.stride;
  const at::Tensor& free = tensor(v[3], "free_pages");
  if (free.dim() != 1) value_error("free_pages is [n]");
  a.free_capacity = to_i32(free.size(0), "free_pages");
  a.free_pages = need_i32(v[3], "free_pages", index, free.size(0));
  a.n_free = need_i32(v[4], "n_free", index, 1);
  a.page_size = to_i32(integer(v[5], "page_size"), "page_size");
  a.n_tokens = to_i32(integer(v[6], "n_tokens"), "n_tokens");
  const OnStream st(v[7], index);
  // one allocation: slots, then the int32 outputs
  const int64_t T = a.n_tokens > 0 ? a.n_tokens : 0;
  const at::Tensor all = at::empty({T + B + 2}, old.options().dtype(at::kLong));
  const at::Tensor slots = part_of(all, at::kLong, 0, T), lens = part_of(all, at::kInt, 2 * T, B),
                   cu = part_of(all, at::kInt, 2 * T + B, B + 1), left = part_of(all, at::kInt, 2 * T + 2 * B + 1, 1),
                   served = part_of(all, at::kInt, 2 * T + 2 * B + 2, 1);
  a.seq_lens = static_cast<int32_t*>(lens.data_ptr());
  a.cu_seqlens_q = static_cast<int32_t*>(cu.data_ptr());
  a.n_free_out = static_cast<int32_t*>(left.data_ptr());
  a.n_served = static_cast<int32_t*>(served.data_ptr());
  a.slots = static_cast<int64_t*>(slots.data_ptr());
  const sa_status status = sa_page_plan(&a, st.get());
  if (status != SA_OK) return PyLong_FromLong(status);
  PyObject* r = PyTuple_New(5);
  if (!r) return nullptr;
  const at::Tensor* outs[5] = {&lens, &cu, &slots, &left, &served};
  for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(*outs[i]));
  return r;
  KV8_END
}

// write(cache, index, k, v, block_table, seq_lens, cu_seqlens_q, stream)
PyObject* kv8_write(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  KV8_BEGIN(8, "write")
  const int index = (int)integer(v[1], "index");
  const at::Tensor& k = tensor(v[2], "k");
  sa_kv8_rows r = {};
  r.dtype = dtype_of(k, "k");
  const sa_kv8_cache c = step_of(v[0], index, k, "k", v[4], v[5], v[6]);
  if ((v[3] == Py_None) != (c.kv_shared != 0)) value_error("v goes with a cache of separate K and V");
  r.k_stride = token_step(k, "k", c.n_heads_kv, c.d_qk, index);
  r.k = k.data_ptr();
  if (v[3] != Py_None) {
    const at::Tensor& x = tensor(v[3], "v");
    if (x.scalar_type() != k.scalar_type() || x.dim() != k.dim() || x.sizes().slice(0, x.dim() - 1) != k.sizes().slice(0, k.dim() - 1))
      type_error("v " + shape_text(x.sizes()) + " does not go with k " + shape_text(k.sizes()));
    r.v_stride = token_step(x, "v", c.n_heads_kv, c.d_v, index);
    r.v = x.data_ptr();
  }
  const OnStream st(v[7], index);
  return PyLong_FromLong(sa_kv8_write(&c, &r, st.get()));
  KV8_END
}

// attend(cache, index, q, block_table, seq_lens, cu_seqlens_q, idx, block_size, topk_len, win_left, sinks, scale,
//        o, lse, stream)
PyObject* kv8_attend(PyObject*, PyObject* const* v, Py_ssize_t nargs) {
  KV8_BEGIN(15, "attend")
  const int index = (int)integer(v[1], "index");
  const at::Tensor& q = tensor(v[2], "q");
  sa_kv8_query a = {};
  a.dtype = dtype_of(q, "q");
  const sa_kv8_cache c = step_of(v[0], index, q, "q", v[3], v[4], v[5]);
  const int64_t n = q.dim(), Hq = q.size(n - 2);
  a.n_heads_q = to_i32(Hq, "Hq");
  a.q_stride = token_step(q, "q", Hq, c.d_qk, index);
  a.q = q.data_ptr();
  at::DimVector shape(q.sizes().begin(), q.sizes().end());  // [.., x, y] with the last two replaced as needed
  a.block_size = to_i32(integer(v[7], "block_size"), "block_size");
  if (v[6] != Py_None) {
    const at::Tensor& idx = tensor(v[6], "idx");
    const int64_t topk = idx.dim() ? idx.size(idx.dim() - 1) : 0;
    if (topk == 0) value_error("idx has no slots");
    shape[n - 2] = c.n_heads_kv;
    shape[n - 1] = topk;
    a.idx = static_cast<int32_t*>(need(v[6], "idx", at::kInt, index, shape));
    a.topk = to_i32(topk, "topk");
    if (v[8] != Py_None)
      a.topk_len = static_cast<int32_t*>(need(v[8], "topk_len", at::kInt, index, c10::IntArrayRef(shape).slice(0, n - 1)));
  } else if (v[8] != Py_None) {
    value_error("topk_len goes with idx");
  }
  a.win_left = -1;
  if (v[9] != Py_None) {
    a.win_left = integer(v[9], "window");
    if (a.win_left < 0) value_error("window is the rows before a token's own that it sees: 0 or more");
  }
  if (v[10] != Py_None) a.sinks = static_cast<float*>(need(v[10], "sinks", at::kFloat, index, {Hq}));
  const double scale = PyFloat_AsDouble(v[11]);
  if (scale == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("scale: a number expected");
  }
  a.scale = (float)scale;
  shape[n - 2] = Hq;
  shape[n - 1] = c.d_v;
  const c10::IntArrayRef o_shape(shape), lse_shape = o_shape.slice(0, n - 1);
  if (v[12] != Py_None) a.o = need(v[12], "o", q.scalar_type(), index, o_shape);
  if (v[13] != Py_None) a.lse = static_cast<float*>(need(v[13], "lse", at::kFloat, index, lse_shape));
  const OnStream st(v[14], index);
  at::Tensor o, lse;
  if (v[12] == Py_None) {
    o = at::empty(o_shape, q.options());
    a.o = o.data_ptr();
  }
  if (v[13] == Py_None) {
    lse = at::empty(lse_shape, q.options().dtype(at::kFloat));
    a.lse = static_cast<float*>(lse.data_ptr());
  }
  size_t bytes = 0;
  sa_status status = sa_kv8_fwd_get_workspace_size(&c, &a, &bytes);
  if (status != SA_OK) return PyLong_FromLong(status);
  const c10::DataPtr ws = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
  status = sa_kv8_fwd(&c, &a, ws.get(), bytes, st.get());
  if (status != SA_OK) return PyLong_FromLong(status);
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyObject* out[2] = {v[12], v[13]};
  for (int i = 0; i < 2; ++i) {
    if (out[i] != Py_None) Py_INCREF(out[i]);
    else out[i] = THPVariable_Wrap(i ? lse : o);
    PyTuple_SET_ITEM(r, i, out[i]);
  }
  return r;
  KV8_END
}

PyMethodDef methods[] = {
    {"plan", (PyCFunction)(void*)kv8_plan, METH_FASTCALL, nullptr},
    {"write", (PyCFunction)(void*)kv8_write, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void*)kv8_attend, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv8_ext", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__kv8_ext(void) { return PyModule_Create(&module); }
