// The short host path of the layer's operators.  Their kernels take a few microseconds, reading a dozen tensors'
// attributes, building the C structures and allocating the results in Python ten: here the same is done on the tensors
// themselves.  A call that is not plain (another device or stream, a wrong shape or type, nothing to do, an error) is
// left to the Python form, which checks it anew and says what is wrong: every function returns None then.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty_cuda_dispatch.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <limits>

#include "dsa_indexer.h"

namespace {

// The library's functions, by address: the library is the one that _lib loaded.
struct Library {
  decltype(&dsa_rmsnorm_fp8) rmsnorm = nullptr;
  decltype(&dsa_latent_append_rope) append = nullptr;
  decltype(&dsa_sparse_attention) sparse = nullptr;
  decltype(&dsa_sparse_attention_workspace_bytes) sparse_bytes = nullptr;
  decltype(&dsa_prefix_attention) prefix = nullptr;
  decltype(&dsa_prefix_attention_workspace_bytes) prefix_bytes = nullptr;
} lib;

struct NotPlain {};
void require(bool plain) {
  if (!plain) throw NotPlain{};
}

int32_t int32_of(PyObject* o) {
  const long v = PyLong_AsLong(o);
  require(!(v == -1 && PyErr_Occurred()) && v >= std::numeric_limits<int32_t>::min() && v <= std::numeric_limits<int32_t>::max());
  return static_cast<int32_t>(v);
}

double double_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  require(!(v == -1.0 && PyErr_Occurred()));
  return v;
}

int truth_of(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  require(v >= 0);
  return v;
}

// The call's tensors: on the current device, ordinary ones.
struct Call {
  const int device = c10::cuda::current_device();
  void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
  const at::Tensor* optional(PyObject* o, bool contiguous = true) const {
    if (o == Py_None) return nullptr;
    require(THPVariable_Check(o));
    const at::Tensor& t = THPVariable_Unpack(o);
    require(t.is_cuda() && t.get_device() == device && t.layout() == at::kStrided && t.has_storage() &&
            !t.unsafeGetTensorImpl()->is_python_dispatch() && (!contiguous || t.is_contiguous()));
    return &t;
  }
  const at::Tensor& tensor(PyObject* o, bool contiguous = true) const {
    const at::Tensor* t = optional(o, contiguous);
    require(t != nullptr);
    return *t;
  }
  const int32_t* ints(PyObject* o, int64_t n) const {
    const at::Tensor& t = tensor(o);
    require(t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == n);
    return static_cast<const int32_t*>(t.const_data_ptr());
  }
};

// Where a tensor that is only read lies: a lazy clone stays one, where data_ptr() would copy it first.
void* read_only(const at::Tensor& t) { return const_cast<void*>(t.const_data_ptr()); }
void* read_only(const at::Tensor* t) { return t ? read_only(*t) : nullptr; }
void* address(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

dsa_dtype_t float_code(const at::Tensor& t) {
  require(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat);
  return t.scalar_type() == at::kFloat ? DSA_F32 : DSA_BF16;
}

// The tensor that was given, or a new one.
struct Result {
  PyObject* given = nullptr;                             // borrowed
  at::Tensor made;
  void* ptr = nullptr;
  Result(const Call& call, PyObject* o, at::IntArrayRef sizes, at::TensorOptions options) {
    if (o == Py_None) {
      made = at::cuda::empty(sizes, options);
      ptr = made.data_ptr();
      return;
    }
    const at::Tensor& t = call.tensor(o);
    int64_t n = 1;
    for (int64_t s : sizes) n *= s;
    require(t.element_size() == static_cast<int64_t>(options.dtype().itemsize()) && t.numel() == n &&
            (options.dtype() == caffe2::TypeMeta::Make<uint8_t>() || t.dtype() == options.dtype()));
    given = o;
    ptr = t.data_ptr();
  }
  PyObject* object() const { return given ? Py_NewRef(given) : THPVariable_Wrap(made); }
};

dsa_latent_cache_t cache_of(const Call& call, PyObject* latent, PyObject* rope, PyObject* scale, PyObject* page_size, bool written) {
  const at::Tensor& l = call.tensor(latent);
  const at::Tensor* r = call.optional(rope);
  const at::Tensor* s = call.optional(scale);
  const int32_t page = int32_of(page_size);
  require(l.dim() == 2 && page >= 1 && l.size(0) % page == 0 && l.size(0) / page <= std::numeric_limits<int32_t>::max() &&
          l.size(1) <= std::numeric_limits<int32_t>::max());
  const bool fp8 = l.scalar_type() != at::kBFloat16;
  if (fp8)
    require((l.scalar_type() == at::kByte || l.scalar_type() == at::kFloat8_e4m3fn) && s && s->scalar_type() == at::kFloat &&
            s->numel() == l.size(0));
  if (r) require(r->scalar_type() == at::kBFloat16 && r->dim() == 2 && r->size(0) == l.size(0) && r->size(1) <= 4096);
  dsa_latent_cache_t c{};
  c.latent = written ? l.data_ptr() : read_only(l);
  c.scale = fp8 ? static_cast<float*>(written ? s->data_ptr() : read_only(s)) : nullptr;
  c.rope = written ? address(r) : read_only(r);
  c.num_pages = static_cast<int32_t>(l.size(0) / page);
  c.page_size = page;
  c.d_c = static_cast<int32_t>(l.size(1));
  c.d_r = r ? static_cast<int32_t>(r->size(1)) : 0;
  c.dtype = fp8 ? DSA_FP8_E4M3 : DSA_BF16;
  return c;
}

dsa_page_table_t table_of(const Call& call, PyObject* o) {
  const at::Tensor& t = call.tensor(o);
  require(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) <= std::numeric_limits<int32_t>::max() &&
          t.size(1) <= std::numeric_limits<int32_t>::max());
  return dsa_page_table_t{static_cast<const int32_t*>(t.const_data_ptr()), static_cast<int32_t>(t.size(0)), static_cast<int32_t>(t.size(1))};
}

dsa_latent_query_t query_of(const Call& call, PyObject* latent, PyObject* rope, bool rotated) {
  const at::Tensor& l = call.tensor(latent, false);
  require(l.scalar_type() == at::kBFloat16 && l.dim() == 3 && l.size(2) == 512 && l.stride(2) == 1 && l.size(0) >= 1 &&
          l.size(0) <= std::numeric_limits<int32_t>::max() && l.size(1) >= 1 && l.size(1) <= 128);
  dsa_latent_query_t q{};
  q.latent = l.const_data_ptr();
  q.latent_stride_t = l.stride(0);
  q.latent_stride_h = l.stride(1);
  q.T = static_cast<int32_t>(l.size(0));
  q.H = static_cast<int32_t>(l.size(1));
  if (rotated) {
    const at::Tensor& r = call.tensor(rope, false);
    require(r.scalar_type() == at::kBFloat16 && r.dim() == 3 && r.size(0) == l.size(0) && r.size(1) == l.size(1) &&
            r.size(2) == 64 && r.stride(2) == 1);
    q.rope = r.const_data_ptr();
    q.rope_stride_t = r.stride(0);
    q.rope_stride_h = r.stride(1);
  }
  return q;
}

// Another thread may run Python while a launch waits for room in the stream.  The arguments are there before the lock is
// given up (taking a result's address may still copy a lazy clone, which can fail), and it is taken back however f ends.
template <class F, class... Args>
void library_call(F f, Args... args) {
  struct Unlocked {
    PyThreadState* const thread = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(thread); }
  };
  dsa_status_t status;
  {
    const Unlocked unlocked;
    status = f(args...);
  }
  require(status == DSA_OK);
}

// x, weight, eps, residual, group, residual_out, codes, scale, normed
PyObject* rmsnorm(PyObject* const* a) {
  const Call call;
  const at::Tensor &x = call.tensor(a[0], false), &w = call.tensor(a[1]);
  const at::Tensor *residual = call.optional(a[3]), *normed = call.optional(a[8]);
  const int32_t group = int32_of(a[4]);
  require(x.dim() == 2 && x.size(0) >= 1 && x.stride(1) == 1 && x.size(1) <= std::numeric_limits<int32_t>::max() &&
          w.numel() == x.size(1) && (group == 0 || group == 128) && (residual || a[5] == Py_None));
  const int64_t rows = x.size(0), d = x.size(1), groups = group ? (d + 127) / 128 : 1;
  if (residual) require(residual->scalar_type() == x.scalar_type() && residual->numel() == rows * d);
  if (normed) require(normed->scalar_type() == at::kBFloat16 && normed->numel() == rows * d);
  const float eps = static_cast<float>(double_of(a[2]));
  const dsa_dtype_t code = float_code(x), weight_code = float_code(w);
  const Result codes(call, a[6], {rows, d}, x.options().dtype(at::kByte));
  const Result scale(call, a[7], {rows, groups}, x.options().dtype(at::kFloat));
  auto run = [&](void* residual_out) {                   // the residual's address after the result's: they may be one tensor
    library_call(lib.rmsnorm, read_only(x), code, x.stride(0), read_only(residual), residual_out, read_only(w), weight_code, rows,
                 static_cast<int32_t>(d), eps, group, static_cast<uint8_t*>(codes.ptr), static_cast<float*>(scale.ptr),
                 address(normed), call.stream());
  };
  if (!residual) {
    run(nullptr);
    return Py_BuildValue("NNO", codes.object(), scale.object(), Py_None);
  }
  const Result out(call, a[5], residual->sizes(), residual->options());
  run(out.ptr);
  return Py_BuildValue("NNN", codes.object(), scale.object(), out.object());
}

// latent, rope, scale, page_size, page_table, c_new, kr_new, seq_ids, positions, rope_dim, base, interleaved
PyObject* append(PyObject* const* a) {
  const Call call;
  const dsa_latent_cache_t cache = cache_of(call, a[0], a[1], a[2], a[3], true);
  const dsa_page_table_t table = table_of(call, a[4]);
  const at::Tensor& c = call.tensor(a[5], false);
  require(c.dim() == 2 && c.size(0) >= 1 && c.size(0) <= std::numeric_limits<int32_t>::max() && c.size(1) == 512 && c.stride(1) == 1);
  const at::Tensor* kr = nullptr;
  if (cache.rope) {
    kr = &call.tensor(a[6], false);
    require(kr->dim() == 2 && kr->size(0) == c.size(0) && kr->size(1) == 64 && kr->stride(1) == 1 && kr->scalar_type() == c.scalar_type());
  }
  const int32_t *seq = call.ints(a[7], c.size(0)), *pos = call.ints(a[8], c.size(0));
  const dsa_rope_t rope{int32_of(a[9]), truth_of(a[11]), double_of(a[10])};
  const dsa_dtype_t code = float_code(c);
  library_call(lib.append, &cache, &table, read_only(c), c.stride(0), read_only(kr), kr ? kr->stride(0) : 0, code, seq, pos,
               static_cast<int32_t>(c.size(0)), &rope, call.stream());
  return Py_NewRef(Py_True);
}

// What a call of attention returns and works in: out, lse, and a workspace that torch's allocator keeps for a graph.
struct Outputs {
  const Result out, lse;
  at::Tensor made;
  void* workspace = nullptr;
  size_t bytes = 0;
  Outputs(const Call& call, const at::Tensor& like, const dsa_latent_query_t& q, PyObject* o, PyObject* l, PyObject* w, size_t need)
      : out(call, o, {q.T, q.H, 512}, like.options()), lse(call, l, {q.T, q.H}, like.options().dtype(at::kFloat)) {
    if (const at::Tensor* given = call.optional(w)) {
      workspace = given->data_ptr();
      bytes = static_cast<size_t>(given->numel() * given->element_size());
    } else if (need) {
      made = at::cuda::empty({static_cast<int64_t>(need)}, like.options().dtype(at::kByte));
      workspace = made.data_ptr();
      bytes = need;
    }
  }
  PyObject* pair() const { return Py_BuildValue("NN", out.object(), lse.object()); }
};

// q_latent, q_rope, latent, rope, scale, page_size, page_table, seq_ids, idx, sm_scale, out, lse, workspace
PyObject* sparse(PyObject* const* a) {
  const Call call;
  const dsa_latent_cache_t cache = cache_of(call, a[2], a[3], a[4], a[5], false);
  const dsa_latent_query_t q = query_of(call, a[0], a[1], cache.rope != nullptr);
  const dsa_page_table_t table = table_of(call, a[6]);
  const int32_t* seq = call.ints(a[7], q.T);
  const at::Tensor& idx = call.tensor(a[8]);
  require(idx.scalar_type() == at::kInt && idx.dim() == 2 && idx.size(0) == q.T && idx.size(1) <= std::numeric_limits<int32_t>::max());
  const int32_t k = static_cast<int32_t>(idx.size(1));
  const float scale = static_cast<float>(double_of(a[9]));
  const size_t need = a[12] == Py_None ? lib.sparse_bytes(q.T, q.H, k, cache.dtype) : 0;
  const Outputs o(call, THPVariable_Unpack(a[0]), q, a[10], a[11], a[12], need);
  library_call(lib.sparse, &q, &cache, &table, seq, static_cast<const int32_t*>(read_only(idx)), k, scale, o.out.ptr,
               static_cast<float*>(o.lse.ptr), o.workspace, o.bytes, call.stream());
  return o.pair();
}

// q_latent, q_rope, latent, rope, scale, page_size, page_table, seq_ids, key_lens, prefix_len, prefix_seq, max_keys,
// sm_scale, out, lse, workspace
PyObject* prefix(PyObject* const* a) {
  const Call call;
  const dsa_latent_cache_t cache = cache_of(call, a[2], a[3], a[4], a[5], false);
  const dsa_latent_query_t q = query_of(call, a[0], a[1], cache.rope != nullptr);
  const dsa_page_table_t table = table_of(call, a[6]);
  const int32_t *seq = call.ints(a[7], q.T), *lens = call.ints(a[8], q.T);
  const int32_t prefix_len = int32_of(a[9]), prefix_seq = int32_of(a[10]);
  const int64_t most = a[11] == Py_None ? int64_t(table.max_pages) * cache.page_size : int32_of(a[11]);
  require(most <= std::numeric_limits<int32_t>::max());
  const int32_t max_keys = static_cast<int32_t>(most);
  const float scale = static_cast<float>(double_of(a[12]));
  const size_t need = a[15] == Py_None ? lib.prefix_bytes(q.T, q.H, prefix_len, max_keys, cache.dtype) : 0;
  const Outputs o(call, THPVariable_Unpack(a[0]), q, a[13], a[14], a[15], need);
  library_call(lib.prefix, &q, &cache, &table, seq, lens, prefix_len, prefix_seq, max_keys, scale, o.out.ptr,
               static_cast<float*>(o.lse.ptr), o.workspace, o.bytes, call.stream());
  return o.pair();
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n == N && lib.rmsnorm != nullptr) {
    try {
      return F(args);
    } catch (...) {                                      // not plain, or out of memory: the Python form answers
    }
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

// The addresses of the library's functions, in the order of Library.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[6];
  if (n != 6) return PyErr_Format(PyExc_TypeError, "six addresses are wanted");
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  lib.rmsnorm = reinterpret_cast<decltype(lib.rmsnorm)>(p[0]);
  lib.append = reinterpret_cast<decltype(lib.append)>(p[1]);
  lib.sparse = reinterpret_cast<decltype(lib.sparse)>(p[2]);
  lib.sparse_bytes = reinterpret_cast<decltype(lib.sparse_bytes)>(p[3]);
  lib.prefix = reinterpret_cast<decltype(lib.prefix)>(p[4]);
  lib.prefix_bytes = reinterpret_cast<decltype(lib.prefix_bytes)>(p[5]);
  Py_RETURN_NONE;
}

PyCFunction method(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"rmsnorm", method(guarded<rmsnorm, 9>), METH_FASTCALL, nullptr},
    {"append", method(guarded<append, 12>), METH_FASTCALL, nullptr},
    {"sparse", method(guarded<sparse, 13>), METH_FASTCALL, nullptr},
    {"prefix", method(guarded<prefix, 16>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_calls", nullptr, -1, methods};

}  // namespace

// TORCH_BUILT_FOR: the version of torch whose headers these are
extern "C" PyMODINIT_FUNC PyInit__layer_calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
