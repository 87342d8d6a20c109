// attention_torch.cpp — the PyTorch side of the attention calls: checks of the
// tensors, outputs and workspace from PyTorch's allocator, the C entry point.
//
// What the calls of a decode step do on the GPU takes 4 to 12 us with few rows; a
// binding written in Python needs 20 to 30 us a call to check and pass on some
// fifteen tensors. Here a call takes 8 to 12 us: about 1 us of checks, 1.5 for
// letting go of the interpreter lock, the rest allocations and launches.
// The entry points' addresses come from the loaded library (normal or
// bounds-checked) and change when another one is loaded; nothing else is kept
// between calls.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "moe.h"

namespace {

decltype(&moe_qkv_append) qkv_append = nullptr;
decltype(&moe_attend_paged_workspace) attend_paged_workspace = nullptr;
decltype(&moe_attend_paged) attend_paged = nullptr;
decltype(&moe_attend_prompt_workspace) attend_prompt_workspace = nullptr;
decltype(&moe_attend_prompt) attend_prompt = nullptr;

struct Refused : std::runtime_error {  // becomes a ValueError
  using std::runtime_error::runtime_error;
};
struct Raised {};  // a Python error is set

// While allocating and launching, which may wait for the GPU, other Python threads run.
struct WithoutGil {
  PyThreadState *state = PyEval_SaveThread();
  WithoutGil() = default;
  WithoutGil(const WithoutGil &) = delete;
  ~WithoutGil() { PyEval_RestoreThread(state); }
};

[[noreturn]] void refuse(const std::string &what) { throw Refused(what); }

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(name) + " must be a tensor");  // a TypeError
  return THPVariable_Unpack(o);
}

const at::Tensor *optional_tensor(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

bool flag(PyObject *o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw Raised();
  return r != 0;
}

double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

int32_t size32(int64_t v, const char *name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return int32_t(v);
}

// The calls have no backward pass: a result without a gradient must not come of an input that wants one.
void no_gradients(std::initializer_list<const at::Tensor *> inputs) {
  if (!at::GradMode::is_enabled()) return;
  for (const at::Tensor *t : inputs)
    if (t && t->requires_grad())
      refuse("an input requires a gradient, and the call has no backward pass: make it under torch.no_grad()");
}

// A tensor that a call has written: autograd may hold it for a backward pass, which then has to see that.
void written(const at::Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Device and type of q, which the other tensors share.
struct Kind {
  at::Device device = at::Device(at::kCPU);
  at::ScalarType type = at::kBFloat16;

  explicit Kind(const at::Tensor &q) : device(q.device()), type(q.scalar_type()) {
    if (q.dim() != 3) refuse("q must have 3 dimensions");
    if (!device.is_cuda() || (type != at::kBFloat16 && type != at::kHalf)) refuse("q must be a CUDA tensor in bf16 or fp16");
  }
  uint32_t code() const { return type == at::kHalf ? MOE_DTYPE_F16 : MOE_DTYPE_BF16; }
};

// Row stride of a [rows][heads][dim] tensor whose rows are contiguous, on the device and in the type of q.
int64_t rows(const at::Tensor &t, const char *name, const Kind &kind) {
  if (t.dim() != 3) refuse(std::string(name) + " must have 3 dimensions");
  if (t.device() != kind.device || t.scalar_type() != kind.type)
    refuse(std::string(name) + " must have the device and type of q");
  const int64_t heads = t.size(1), dim = t.size(2);
  if (t.numel() && ((dim > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != dim)))
    refuse("the heads of a row of " + std::string(name) + " must be contiguous");
  return t.size(0) > 1 && t.numel() ? t.stride(0) : heads * dim;
}

// Address of a contiguous vector of n.
template <class P>
P *vector(const at::Tensor &t, const char *name, at::ScalarType type, int64_t n, const Kind &kind) {
  if (t.scalar_type() != type || t.device() != kind.device || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " vector of " + std::to_string(n) +
           " on q's device");
  return static_cast<P *>(t.data_ptr());
}

int32_t *status_word(const at::Tensor *t, const Kind &kind) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->device() != kind.device || t->numel() < 1)
    refuse("d_status must be an int32 tensor on q's device");
  return static_cast<int32_t *>(t->data_ptr());
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const Kind &kind) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(kind.device));
}

// The output, given or new, and its row stride.
at::Tensor output(const at::Tensor *out, const at::Tensor &q, const Kind &kind, int64_t &stride) {
  if (!out) {
    stride = q.size(1) * q.size(2);
    return make(q.sizes(), kind.type, kind);
  }
  if (out->sizes() != q.sizes()) refuse("out must have the shape of q");
  stride = rows(*out, "out", kind);
  return *out;
}

// The parts of a KVCacheMXFP4, which were checked when it was made. append: they are about to be written.
moe_kv_cache_t kv_cache(PyObject *cache, at::Device &device, bool append) {
  PyObject *parts = PyObject_GetAttrString(cache, "_parts");
  if (!parts) throw Raised();
  bool good = PyTuple_Check(parts) && PyTuple_GET_SIZE(parts) == 4;
  for (int i = 0; good && i < 4; ++i) good = THPVariable_Check(PyTuple_GET_ITEM(parts, i));
  if (!good) {
    Py_DECREF(parts);
    refuse("cache must be a KVCacheMXFP4");
  }
  const at::Tensor &k = THPVariable_Unpack(PyTuple_GET_ITEM(parts, 0));
  moe_kv_cache_t c = {};
  uint8_t **at[4] = {&c.k_codes, &c.k_scales, &c.v_codes, &c.v_scales};
  for (int i = 0; i < 4; ++i) *at[i] = static_cast<uint8_t *>(THPVariable_Unpack(PyTuple_GET_ITEM(parts, i)).data_ptr());
  device = k.device();
  c.num_pages = int32_t(k.size(0));
  c.num_kv_heads = int32_t(k.size(1));
  c.page_size = int32_t(k.size(2));
  c.head_dim = int32_t(2 * k.size(3));
  if (append)
    for (int i = 0; i < 4; ++i) written(THPVariable_Unpack(PyTuple_GET_ITEM(parts, i)));
  Py_DECREF(parts);  // the cache, which the caller holds, holds them
  return c;
}

void *stream_of(const Kind &kind) { return c10::cuda::getCurrentCUDAStream(kind.device.index()).stream(); }

void put(PyObject *dict, const char *key, const at::Tensor &t) {
  PyObject *o = THPVariable_Wrap(t);
  const int r = o ? PyDict_SetItemString(dict, key, o) : -1;
  Py_XDECREF(o);
  if (r) {
    Py_DECREF(dict);
    throw Raised();
  }
}

// The result of a call: what it returns, or the status that it failed with.
PyObject *outputs(const at::Tensor &out, const at::Tensor &lse) {
  PyObject *o = THPVariable_Wrap(out);
  if (!o || !lse.defined()) return o;
  PyObject *z = THPVariable_Wrap(lse);
  PyObject *both = z ? PyTuple_Pack(2, o, z) : nullptr;
  Py_DECREF(o);
  Py_XDECREF(z);
  return both;
}

template <class F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t expect, F f) {
  HANDLE_TH_ERRORS  // PyTorch's own errors, an exhausted device among them, keep their Python types
  try {
    if (n != expect) throw std::invalid_argument("wrong number of arguments");
    return f();
  } catch (const Raised &) {
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::invalid_argument &e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

// bind(addresses of the five entry points)
PyObject *py_bind(PyObject *, PyObject *const *arg, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    void *p[5];
    for (int i = 0; i < 5; ++i) {
      p[i] = PyLong_AsVoidPtr(arg[i]);
      if (!p[i]) throw std::runtime_error("no address");
    }
    qkv_append = reinterpret_cast<decltype(qkv_append)>(p[0]);
    attend_paged_workspace = reinterpret_cast<decltype(attend_paged_workspace)>(p[1]);
    attend_paged = reinterpret_cast<decltype(attend_paged)>(p[2]);
    attend_prompt_workspace = reinterpret_cast<decltype(attend_prompt_workspace)>(p[3]);
    attend_prompt = reinterpret_cast<decltype(attend_prompt)>(p[4]);
    Py_RETURN_NONE;
  });
}

// check_cache(k_codes, k_scales, v_codes, v_scales)
PyObject *py_check_cache(PyObject *, PyObject *const *arg, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject * {
    static const char *const names[4] = {"k_codes", "k_scales", "v_codes", "v_scales"};
    const at::Tensor &k = tensor(arg[0], names[0]);
    if (k.dim() != 4) refuse("k_codes must have 4 dimensions");
    for (int i = 0; i < 4; ++i) {
      const at::Tensor &t = tensor(arg[i], names[i]);
      const std::string name = names[i];
      if (t.scalar_type() != at::kByte || !t.is_cuda() || t.device() != k.device() || !t.is_contiguous())
        refuse(name + " must be a contiguous uint8 CUDA tensor on the cache's device");
      const int64_t want[4] = {k.size(0), k.size(1), k.size(2), i % 2 ? k.size(3) / 16 : k.size(3)};
      if (t.sizes() != at::IntArrayRef(want, 4)) refuse(name + " must have the shape that k_codes asks for");
    }
    for (int i = 0; i < 4; ++i) size32(2 * k.size(i), "k_codes");
    Py_RETURN_NONE;
  });
}

// append(q, k, v, positions, rope, interleaved, q_norm, k_norm, eps, cache, slots, q_out, rotated_keys, cached_values,
// d_status)
PyObject *py_append(PyObject *, PyObject *const *arg, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject * {
    const at::Tensor &q = tensor(arg[0], "q"), &k = tensor(arg[1], "k"), &v = tensor(arg[2], "v");
    no_gradients({&q, &k, &v, optional_tensor(arg[4], "rope"), optional_tensor(arg[6], "q_norm"),
                  optional_tensor(arg[7], "k_norm"), optional_tensor(arg[11], "q_out")});
    const Kind kind(q);
    moe_qkv_append_io_t io = {};
    io.q_stride = rows(q, "q", kind);
    io.k_stride = rows(k, "k", kind);
    io.v_stride = rows(v, "v", kind);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), K = k.size(1);
    if (k.size(0) != T || k.size(2) != D || v.sizes() != k.sizes())
      refuse("k and v must be [T][kv heads][D] with the T and D of q");
    const at::Tensor *positions = optional_tensor(arg[3], "positions"), *rope = optional_tensor(arg[4], "rope");
    if ((rope == nullptr) != (positions == nullptr)) refuse("rope and positions go together");
    if (rope) {
      if (rope->dim() != 2) refuse("rope must have 2 dimensions");
      if (rope->scalar_type() != at::kFloat || rope->device() != kind.device || !rope->is_contiguous())
        refuse("rope must be a contiguous fp32 tensor on q's device");
      io.rope = static_cast<const float *>(rope->data_ptr());
      io.rope_positions = size32(rope->size(0), "rope");
      io.rotary_dim = size32(rope->size(1), "rope");
      io.positions = vector<int32_t>(*positions, "positions", at::kInt, T, kind);
    }
    io.interleaved = flag(arg[5]);
    if (const at::Tensor *w = optional_tensor(arg[6], "q_norm")) io.q_norm = vector<void>(*w, "q_norm", kind.type, D, kind);
    if (const at::Tensor *w = optional_tensor(arg[7], "k_norm")) io.k_norm = vector<void>(*w, "k_norm", kind.type, D, kind);
    io.norm_eps = float(number(arg[8]));
    const at::Tensor *slots = optional_tensor(arg[10], "slots");
    if ((arg[9] == Py_None) != (slots == nullptr)) refuse("cache and slots go together");
    moe_kv_cache_t cache = {};
    if (slots) {
      at::Device device(at::kCPU);
      cache = kv_cache(arg[9], device, true);
      if (device != kind.device || cache.num_kv_heads != K || cache.head_dim != D)
        refuse("the cache must be on q's device, with the kv heads and head size of k");
      io.slots = vector<int64_t>(*slots, "slots", at::kLong, T, kind);
    }
    int32_t *const word = status_word(optional_tensor(arg[14], "d_status"), kind);
    const at::Tensor *given = optional_tensor(arg[11], "q_out");
    if (given && (given->sizes() != q.sizes() || given->scalar_type() != kind.type || given->device() != kind.device ||
                  !given->is_contiguous()))
      refuse("q_out must be contiguous, with the shape, type and device of q");
    const bool rotated_keys = flag(arg[12]), cached_values = flag(arg[13]);
    io.num_tokens = size32(T, "q");
    io.num_heads = size32(H, "q");
    io.num_kv_heads = size32(K, "k");
    io.head_dim = size32(D, "q");
    io.dtype = kind.code();
    at::Tensor q_out, k_out, k_cached, v_cached;
    moe_status_t s;
    {
      const WithoutGil free;
      const c10::cuda::CUDAGuard guard(kind.device);
      q_out = given ? *given : make(q.sizes(), kind.type, kind);
      if (rotated_keys) {
        k_out = make(k.sizes(), kind.type, kind);
        io.k_out = k_out.data_ptr();
      }
      if (cached_values) {
        k_cached = make(k.sizes(), kind.type, kind);
        v_cached = make(k.sizes(), kind.type, kind);
        io.k_cached = k_cached.data_ptr();
        io.v_cached = v_cached.data_ptr();
      }
      io.q = q.data_ptr(), io.k = k.data_ptr(), io.v = v.data_ptr(), io.q_out = q_out.data_ptr();
      s = qkv_append(&io, slots ? &cache : nullptr, word, stream_of(kind));
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    if (given) written(*given);
    PyObject *dict = PyDict_New();
    if (!dict) return nullptr;
    put(dict, "q", q_out);
    if (k_out.defined()) put(dict, "k", k_out);
    if (k_cached.defined()) {
      put(dict, "k_cached", k_cached);
      put(dict, "v_cached", v_cached);
    }
    return dict;
  });
}

// paged(q, cache, page_table, lengths, cu_rows, max_rows, scale or None, out, return_lse, d_status)
PyObject *py_paged(PyObject *, PyObject *const *arg, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    const at::Tensor &q = tensor(arg[0], "q"), &table = tensor(arg[2], "page_table");
    const at::Tensor &lengths = tensor(arg[3], "lengths"), &cu_rows = tensor(arg[4], "cu_rows");
    no_gradients({&q, optional_tensor(arg[7], "out")});
    const Kind kind(q);
    moe_attend_paged_io_t io = {};
    io.q_stride = rows(q, "q", kind);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2), B = lengths.dim() == 1 ? lengths.size(0) : -1;
    io.lengths = vector<int32_t>(lengths, "lengths", at::kInt, B, kind);
    io.cu_rows = vector<int32_t>(cu_rows, "cu_rows", at::kInt, B + 1, kind);
    if (table.dim() != 2 || table.scalar_type() != at::kInt || table.device() != kind.device || table.size(0) != B ||
        !table.is_contiguous())
      refuse("page_table must be a contiguous int32 [sequences][pages] tensor on q's device");
    at::Device device(at::kCPU);
    const moe_kv_cache_t cache = kv_cache(arg[1], device, false);
    if (device != kind.device || cache.head_dim != D) refuse("the cache must be on q's device, with q's head size");
    const int64_t max_rows = PyLong_AsLongLong(arg[5]);
    if (max_rows == -1 && PyErr_Occurred()) return nullptr;
    int32_t *const word = status_word(optional_tensor(arg[9], "d_status"), kind);
    io.num_seqs = size32(B, "lengths");
    io.num_rows = size32(T, "q");
    io.max_pages = size32(table.size(1), "page_table");
    io.max_rows = size32(max_rows, "max_rows");
    io.num_heads = size32(H, "q");
    io.dtype = kind.code();
    io.scale = arg[6] == Py_None ? float(1.0 / std::sqrt(double(D))) : float(number(arg[6]));
    const at::Tensor *given = optional_tensor(arg[7], "out");
    const bool return_lse = flag(arg[8]);
    at::Tensor out, lse, workspace;
    moe_status_t s;
    {
      const WithoutGil free;
      const c10::cuda::CUDAGuard guard(kind.device);
      int64_t bytes = 0;
      s = attend_paged_workspace(&io, &cache, &bytes);
      if (s == MOE_OK) {
        out = output(given, q, kind, io.out_stride);
        if (return_lse) {
          lse = make({T, H}, at::kFloat, kind);
          io.lse = static_cast<float *>(lse.data_ptr());
        }
        workspace = make({bytes}, at::kByte, kind);
        io.q = q.data_ptr();
        io.out = out.data_ptr();
        io.page_table = static_cast<const int32_t *>(table.data_ptr());
        s = attend_paged(&io, &cache, workspace.data_ptr(), bytes, word, stream_of(kind));
      }
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    if (given) written(*given);
    return outputs(out, lse);
  });
}

// prompt(q, k, v, cu_rows, cu_keys, causal, scale or None, out, return_lse, d_status)
PyObject *py_prompt(PyObject *, PyObject *const *arg, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    const at::Tensor &q = tensor(arg[0], "q"), &k = tensor(arg[1], "k"), &v = tensor(arg[2], "v");
    const at::Tensor &cu_rows = tensor(arg[3], "cu_rows"), &cu_keys = tensor(arg[4], "cu_keys");
    no_gradients({&q, &k, &v, optional_tensor(arg[7], "out")});
    const Kind kind(q);
    moe_attend_prompt_io_t io = {};
    io.q_stride = rows(q, "q", kind);
    io.k_stride = rows(k, "k", kind);
    io.v_stride = rows(v, "v", kind);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    if (k.size(2) != D || v.sizes() != k.sizes()) refuse("k and v must be [keys][kv heads][D] with the D of q");
    const int64_t ends = cu_rows.dim() == 1 ? cu_rows.size(0) : 0;
    if (ends < 1) refuse("cu_rows needs an entry for each sequence and one for the end");
    io.cu_rows = vector<int32_t>(cu_rows, "cu_rows", at::kInt, ends, kind);
    io.cu_keys = vector<int32_t>(cu_keys, "cu_keys", at::kInt, ends, kind);
    int32_t *const word = status_word(optional_tensor(arg[9], "d_status"), kind);
    io.num_seqs = size32(ends - 1, "cu_rows");
    io.num_rows = size32(T, "q");
    io.num_keys = size32(k.size(0), "k");
    io.num_heads = size32(H, "q");
    io.num_kv_heads = size32(k.size(1), "k");
    io.head_dim = size32(D, "q");
    io.dtype = kind.code();
    io.causal = flag(arg[5]);
    io.scale = arg[6] == Py_None ? float(1.0 / std::sqrt(double(D))) : float(number(arg[6]));
    const at::Tensor *given = optional_tensor(arg[7], "out");
    const bool return_lse = flag(arg[8]);
    at::Tensor out, lse, workspace;
    moe_status_t s;
    {
      const WithoutGil free;
      const c10::cuda::CUDAGuard guard(kind.device);
      s = attend_prompt_workspace(&io, &io.workspace_bytes);
      if (s == MOE_OK) {
        out = output(given, q, kind, io.out_stride);
        if (return_lse) {
          lse = make({T, H}, at::kFloat, kind);
          io.lse = static_cast<float *>(lse.data_ptr());
        }
        if (io.workspace_bytes > 0) {
          workspace = make({io.workspace_bytes}, at::kByte, kind);
          io.workspace = workspace.data_ptr();
        }
        io.q = q.data_ptr(), io.k = k.data_ptr(), io.v = v.data_ptr(), io.out = out.data_ptr();
        s = attend_prompt(&io, word, stream_of(kind));
      }
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    if (given) written(*given);
    return outputs(out, lse);
  });
}

template <class F>
PyCFunction fast(F *f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {
    {"bind", fast(py_bind), METH_FASTCALL, nullptr},         {"check_cache", fast(py_check_cache), METH_FASTCALL, nullptr},
    {"append", fast(py_append), METH_FASTCALL, nullptr},     {"paged", fast(py_paged), METH_FASTCALL, nullptr},
    {"prompt", fast(py_prompt), METH_FASTCALL, nullptr},     {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "attention_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attention_torch() { return PyModule_Create(&module); }
