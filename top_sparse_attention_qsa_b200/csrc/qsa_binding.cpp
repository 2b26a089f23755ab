// qsa_binding.cpp -- CPython binding of the cache appends and of attention
// over a 4-bit cache.
//
// Argument marshalling only, as in _capi.py: tensors are checked and become
// pointers, sizes and strides; every step of the computation runs in
// libqsa.so's kernels.  These calls come once per layer and token, where a
// kernel takes 3 to 10 us and the same checks in Python took 10 to 20: here
// they take about one, and letting go of the interpreter's lock 0.1 to 0.4.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "qsa.h"

namespace {

using at::Tensor;

// ---------------------------------------------------------------- arguments

struct TypeFault : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct ValueFault : std::runtime_error {
  using std::runtime_error::runtime_error;
};

void need(bool ok, const char* what) {
  if (!ok) throw ValueFault(what);
}

// A tensor of type `dt` on CUDA device `dev` (any CUDA device where dev < 0).
const Tensor& tensor(PyObject* o, const char* name, at::ScalarType dt, int dev) {
  if (!THPVariable_Check(o)) throw TypeFault(std::string(name) + " must be a torch.Tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != dt)
    throw TypeFault(std::string(name) + " must be " + c10::toString(dt) + ", got " + c10::toString(t.scalar_type()));
  if (!t.is_cuda() || (dev >= 0 && t.get_device() != dev))
    throw ValueFault(std::string(name) + " must be a CUDA tensor" + (dev >= 0 ? " on cuda:" + std::to_string(dev) : ""));
  return t;
}

bool given(PyObject* o) { return o != Py_None; }

void* ptr(PyObject* o) { return given(o) ? THPVariable_Unpack(o).data_ptr() : nullptr; }

// A contiguous [n] int32 tensor.
const int32_t* per_token(PyObject* o, const char* name, int64_t n, int dev) {
  const Tensor& t = tensor(o, name, at::kInt, dev);
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    throw ValueFault(std::string(name) + " must be a contiguous [T] int32 tensor");
  return static_cast<const int32_t*>(t.data_ptr());
}

int32_t* status_word(PyObject* o, int dev) {
  return given(o) ? static_cast<int32_t*>(tensor(o, "status", at::kInt, dev).data_ptr()) : nullptr;
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}

int64_t integer(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t x = integer(o);
  if (x != static_cast<int32_t>(x)) throw ValueFault(std::string(name) + " is out of range");
  return static_cast<int32_t>(x);
}

// A size as the C ABI's 32 bits.
int32_t size32(int64_t n) {
  need(n <= 0x7fffffff, "a dimension is out of range");
  return static_cast<int32_t>(n);
}

// The stream of a call, current for its time: what the call makes (outputs, a
// workspace that is let go on return with its kernels still to run) then
// belongs to the stream that writes it, and once dropped goes to no work of
// another.
class Launch {
 public:
  Launch(PyObject* o, int dev) {
    const auto d = static_cast<c10::DeviceIndex>(dev);
    if (given(o)) {
      stream_ = PyLong_AsVoidPtr(o);
      if (stream_ == nullptr && PyErr_Occurred()) throw python_error();
      on_stream_.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream_), d));
    } else {
      stream_ = c10::cuda::getCurrentCUDAStream(d).stream();
      if (d != c10::cuda::current_device()) on_device_.set_index(d);
    }
  }
  void* stream() const { return stream_; }

 private:
  void* stream_ = nullptr;
  c10::cuda::OptionalCUDAStreamGuard on_stream_;
  c10::cuda::OptionalCUDAGuard on_device_;
};

// Other Python threads run while a call allocates and launches: an allocation
// may have to free cached memory, a launch may wait for room in its stream's
// queue (which a host function of that stream can hold up).  No Python object
// is touched meanwhile.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// An output on CUDA device `dev`, past the dispatcher: an enqueue with three
// outputs takes 10.5 us instead of 11.6, with one 5.3 instead of 5.7.
Tensor fresh(at::IntArrayRef sizes, at::ScalarType dt, int dev) {
  return at::detail::empty_cuda(sizes, dt, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}

// The status code, or (code 0) the outputs as a tuple.
template <typename... T>
PyObject* result(qsa_status_t rc, const T&... outs) {
  if (rc != QSA_OK) return PyLong_FromLong(rc);
  PyObject* tup = PyTuple_New(sizeof...(outs));
  Py_ssize_t i = 0;
  auto put = [&](const std::optional<Tensor>& t) {
    PyObject* o;
    if (t.has_value()) {
      o = THPVariable_Wrap(*t);
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    PyTuple_SET_ITEM(tup, i++, o);
  };
  (put(outs), ...);
  return tup;
}

template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const TypeFault& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const ValueFault& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

constexpr const char* kInner = "innermost dimensions must be contiguous";

// ---------------------------------------------------------------- append

// kv_append(format, k, v, positions, slots, cos_sin, k_cache, v_cache, k_scale, v_scale, q, q_out, interleaved, k_seen,
// v_seen, want_seen, status, stream) -> status code or (q_out, k_seen, v_seen).  Formats: 0 BF16, 1 E4M3, 2 4-bit (k_cache
// is the buffer, v_cache None).
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 18)) return nullptr;
  return guarded([&]() -> PyObject* {
    const int64_t format = integer(a[0]);
    const auto dt = format == 0 ? at::kBFloat16 : format == 1 ? at::kFloat8_e4m3fn : at::kByte;
    const Tensor& k = tensor(a[1], "k", at::kBFloat16, -1);
    const int dev = k.get_device();
    const Launch on(a[17], dev);
    const Tensor& v = tensor(a[2], "v", at::kBFloat16, dev);
    need(k.dim() == 3 && v.sizes() == k.sizes(), "k and v must be [T, Hkv, 256]");
    const Tensor& kc = tensor(a[6], format == 2 ? "cache" : "k_cache", dt, dev);
    need(kc.dim() == 3 && kc.size(1) == k.size(1) && kc.size(2) == (format == 2 ? 288 : 256),
         format == 2 ? "cache must be [S, Hkv, 288]" : "k_cache must be [S, Hkv, 256]");
    qsa_append_shape_t s = {};
    s.num_tokens = k.size(0);
    s.num_kv_heads = size32(k.size(1));
    s.head_dim = size32(k.size(2));
    s.num_slots = kc.size(0);
    need(k.stride(2) == 1 && v.stride(2) == 1 && kc.stride(2) == 1, kInner);
    if (format != 2) {
      const Tensor& vc = tensor(a[7], "v_cache", dt, dev);
      need(vc.sizes() == kc.sizes() && vc.strides() == kc.strides(), "k_cache and v_cache must have the same shape and strides");
    }
    const int32_t* slots = per_token(a[4], "slots", s.num_tokens, dev);
    const float* table = nullptr;
    const int32_t* positions = nullptr;
    if (given(a[5])) {
      const Tensor& cs = tensor(a[5], "cos_sin", at::kFloat, dev);
      need(cs.dim() == 2 && (cs.size(1) <= 1 || cs.stride(1) == 1), "cos_sin must be [P, R] with contiguous rows");
      need(cs.size(1) <= 256, "cos_sin has more columns than a head has dims");
      s.num_positions = cs.size(0);
      s.rotary_dim = static_cast<int32_t>(cs.size(1));
      s.table_stride = cs.size(0) > 1 ? cs.stride(0) : cs.size(1);
      table = static_cast<const float*>(cs.data_ptr());
      if (s.rotary_dim > 0) positions = per_token(a[3], "positions", s.num_tokens, dev);
    }
    const Tensor* q_in = nullptr;
    std::optional<Tensor> q_out;
    if (given(a[10])) {
      const Tensor& q = *(q_in = &tensor(a[10], "q", at::kBFloat16, dev));
      need(q.dim() == 3 && q.size(0) == s.num_tokens && q.size(2) == s.head_dim && q.stride(2) == 1,
           "q must be [T, Hq, 256] with contiguous rows");
      if (given(a[11])) {
        q_out = tensor(a[11], "q_out", at::kBFloat16, dev);
        need(q_out->sizes() == q.sizes() && q_out->stride(2) == 1, "q_out must have q's shape and contiguous rows");
      }
      s.num_q_heads = size32(q.size(1));
      s.q_stride_tok = q.stride(0);
      s.q_stride_head = q.stride(1);
    } else {
      need(!given(a[11]), "q_out needs q");
    }
    const int yes = PyObject_IsTrue(a[12]), want = PyObject_IsTrue(a[15]);
    if (yes < 0 || want < 0) throw python_error();
    s.interleaved = yes;
    s.k_stride_tok = k.stride(0);
    s.k_stride_head = k.stride(1);
    s.v_stride_tok = v.stride(0);
    s.v_stride_head = v.stride(1);
    s.kv_stride_slot = kc.stride(0);
    s.kv_stride_head = kc.stride(1);
    std::optional<Tensor> seen[2];
    for (int i = 0; i < 2 && format != 0; ++i) {
      const char* name = i ? "v_seen" : "k_seen";
      if (given(a[13 + i])) {
        seen[i] = tensor(a[13 + i], name, at::kBFloat16, dev);
        if (seen[i]->sizes() != k.sizes() || !seen[i]->is_contiguous())
          throw ValueFault(std::string(name) + " must be a contiguous [T, Hkv, 256] tensor");
      }
    }
    int32_t* status = status_word(a[16], dev);
    const float k_scale = static_cast<float>(number(a[8])), v_scale = static_cast<float>(number(a[9]));
    void* v_cache = ptr(a[7]);
    qsa_status_t rc;
    {
      const Unlocked threads;
      if (q_in != nullptr) {
        if (!q_out.has_value()) q_out = fresh(q_in->sizes(), at::kBFloat16, dev);
        s.qo_stride_tok = q_out->stride(0);
        s.qo_stride_head = q_out->stride(1);
      }
      for (auto& x : seen)
        if (format != 0 && want && !x.has_value()) x = fresh(k.sizes(), at::kBFloat16, dev);
      auto data = [](const std::optional<Tensor>& t) { return t.has_value() ? t->data_ptr() : nullptr; };
      void *qi = q_in != nullptr ? q_in->data_ptr() : nullptr, *qo = data(q_out), *ks = data(seen[0]), *vs = data(seen[1]);
      char* c = static_cast<char*>(kc.data_ptr());
      if (format == 0) {
        rc = qsa_kv_append(&s, qi, qo, k.data_ptr(), v.data_ptr(), table, positions, slots, c, v_cache, status,
                           on.stream());
      } else if (format == 1) {
        rc = qsa_kv_append_fp8(&s, qi, qo, k.data_ptr(), v.data_ptr(), table, positions, slots, k_scale, v_scale, c,
                               v_cache, ks, vs, status, on.stream());
      } else {
        s.bscale_stride_slot = s.kv_stride_slot;
        s.bscale_stride_head = s.kv_stride_head;
        rc = qsa_kv_append_fp4(&s, qi, qo, k.data_ptr(), v.data_ptr(), table, positions, slots, k_scale, v_scale, c,
                               c + 256, c + 128, c + 272, ks, vs, status, on.stream());
      }
    }
    return result(rc, q_out, seen[0], seen[1]);
  });
}

// ---------------------------------------------------------------- attention over a 4-bit cache

// sparse_fp4(decode, q, buffer, topk_idx, k_scale, v_scale, n_valid, scale, block_size, last_slot, num_splits, workspace,
// out, lse, status, stream, want_lse) -> status code or (out, lse)
PyObject* sparse_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 17)) return nullptr;
  return guarded([&]() -> PyObject* {
    const bool decode = integer(a[0]) != 0;
    const Tensor& q = tensor(a[1], "q", at::kBFloat16, -1);
    const int dev = q.get_device();
    const Launch on(a[15], dev);
    const Tensor& buf = tensor(a[2], "cache", at::kByte, dev);
    const Tensor& idx = tensor(a[3], "topk_idx", at::kInt, dev);
    need(q.dim() == 3 && idx.dim() == 3 && buf.dim() == 3, "q, the cache and topk_idx must be 3-d");
    need(buf.size(2) == 288, "the cache must be [S, Hkv, 288]");
    qsa_shape_t s = {};
    s.num_tokens = q.size(0);
    s.num_q_heads = size32(q.size(1));
    s.head_dim = size32(q.size(2));
    s.num_slots = buf.size(0);
    s.num_kv_heads = size32(buf.size(1));
    need(idx.size(0) == s.num_tokens && idx.size(1) == s.num_kv_heads, "topk_idx must be [T, Hkv, K]");
    s.topk = size32(idx.size(2));
    const int32_t* n_valid = nullptr;
    if (given(a[6])) {
      const Tensor& nv = tensor(a[6], "n_valid", at::kInt, dev);
      need(nv.dim() == 2 && nv.size(0) == s.num_tokens && nv.size(1) == s.num_kv_heads && nv.is_contiguous(),
           "n_valid must be a contiguous [T, Hkv] tensor");
      n_valid = static_cast<const int32_t*>(nv.data_ptr());
    }
    const int32_t* last = given(a[9]) ? per_token(a[9], "last_slot", s.num_tokens, dev) : nullptr;
    std::optional<Tensor> out;
    if (given(a[12])) {
      out = tensor(a[12], "out", at::kBFloat16, dev);
      need(out->sizes() == q.sizes(), "out must be [T, Hq, D]");
      need(out->stride(2) == 1, kInner);
    }
    need(q.stride(2) == 1 && buf.stride(2) == 1 && (s.topk <= 1 || idx.stride(2) == 1), kInner);
    std::optional<Tensor> lse;
    s.lse_stride_tok = s.num_q_heads;
    const int want = PyObject_IsTrue(a[16]);
    if (want < 0) throw python_error();
    if (given(a[13])) {
      lse = tensor(a[13], "lse", at::kFloat, dev);
      need(lse->dim() == 2 && lse->size(0) == s.num_tokens && lse->size(1) == s.num_q_heads &&
               (s.num_q_heads <= 1 || lse->stride(1) == 1),
           "lse must be [T, Hq] with unit head stride");
      s.lse_stride_tok = lse->stride(0);
    }
    s.q_stride_tok = q.stride(0);
    s.q_stride_head = q.stride(1);
    s.kv_stride_slot = buf.stride(0);
    s.kv_stride_head = buf.stride(1);
    s.idx_stride_tok = idx.stride(0);
    s.idx_stride_head = idx.stride(1);
    int32_t* status = status_word(a[14], dev);
    const float ks = static_cast<float>(number(a[4])), vs = static_cast<float>(number(a[5])),
                scale = static_cast<float>(number(a[7]));
    const int32_t splits = decode ? integer32(a[10], "num_splits") : 0;
    const int32_t block_size = decode ? 1 : integer32(a[8], "block_size");
    Tensor ws;
    size_t bytes = 0;
    const bool own_ws = !decode || !given(a[11]);
    if (!own_ws) {
      if (!THPVariable_Check(a[11])) throw TypeFault("workspace must be a torch.Tensor");
      ws = THPVariable_Unpack(a[11]);
      need(ws.is_cuda() && ws.get_device() == dev && ws.is_contiguous(), "workspace must be a contiguous CUDA tensor");
      bytes = ws.numel() * ws.element_size();
    }
    qsa_status_t rc;
    {
      const Unlocked threads;
      if (!out.has_value()) out = fresh(q.sizes(), at::kBFloat16, dev);
      if (want && !lse.has_value()) lse = fresh({s.num_tokens, s.num_q_heads}, at::kFloat, dev);
      s.o_stride_tok = out->stride(0);
      s.o_stride_head = out->stride(1);
      const char* c = static_cast<const char*>(buf.data_ptr());
      const int32_t* list = static_cast<const int32_t*>(idx.data_ptr());
      float* lp = lse.has_value() ? static_cast<float*>(lse->data_ptr()) : nullptr;
      auto call = [&] {
        if (!decode)
          return qsa_sparse_prefill_fp4_fwd(&s, block_size, last, q.data_ptr(), c, c + 256, c + 128, c + 272,
                                            buf.stride(0), buf.stride(1), list, n_valid, scale, ks, vs,
                                            out->data_ptr(), lp, status, on.stream());
        return qsa_sparse_decode_fp4_fwd(&s, q.data_ptr(), c, c + 256, c + 128, c + 272, buf.stride(0), buf.stride(1),
                                         list, n_valid, scale, ks, vs, out->data_ptr(), lp, status, splits,
                                         ws.defined() ? ws.data_ptr() : nullptr, bytes, on.stream());
      };
      rc = call();
      // refused for want of a workspace, where no cluster serves the call
      if (decode && rc == QSA_ERR_NULL && own_ws && (bytes = qsa_sparse_decode_fp4_workspace_bytes(&s, splits)) > 0) {
        ws = fresh({static_cast<int64_t>(bytes)}, at::kByte, dev);
        rc = call();
      }
    }
    return result(rc, out, lse);
  });
}

PyMethodDef kMethods[] = {
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"sparse_fp4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sparse_fp4)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
