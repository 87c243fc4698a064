// Tensor marshalling of the operators around the loss (embedding, gradient
// clipping, draft verification): the module vocab_wide_logprob_gb300._ops.
//
// It checks the tensors, allocates what the caller did not pass, and calls the
// C ABI of include/grpo.h on the current CUDA stream -- what _native.py does
// through ctypes for the loss calls, in C++ because these calls are short: a
// model's gradients are hundreds of tensors, and a lookup of a few tokens takes
// less time on the GPU than its arguments take in the interpreter.
// _native.py documents the functions and gives them their keywords.
#include <Python.h>

#include <vector>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "grpo.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // GrpoError(status, where)

// Errors of the checks, as Python exceptions.
struct Refused {};
[[noreturn]] void refuse(PyObject* type, const char* format, const char* name) {
  PyErr_Format(type, format, name);
  throw Refused();
}
void check_status(grpo_status s, const char* where) {
  if (s == GRPO_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, where);
  if (e != nullptr) {
    PyErr_SetObject((PyObject*)Py_TYPE(e), e);
    Py_DECREF(e);
  }
  throw Refused();
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}
const Tensor* maybe_tensor(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}
grpo_dtype code(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return GRPO_F32;
  if (t == at::kBFloat16) return GRPO_BF16;
  refuse(PyExc_TypeError, "%s must be float32 or bfloat16", name);
}
// The stream of a call: the given one (anything with a `cuda_stream`), or the
// device's current one.  Until the call returns a given stream is the current one, so
// that what the call allocates comes from that stream's memory: a workspace that
// the caller drops while the kernels still run is handed out to that stream only.
class CallStream {
 public:
  CallStream(PyObject* o, const c10::Device& dev) {
    if (o == Py_None) {
      handle_ = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
      return;
    }
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (h == nullptr) throw Refused();
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Refused();
    handle_ = (cudaStream_t)p;
    PyObject* d = PyObject_GetAttrString(o, "device_index");
    if (d != nullptr) {
      const int64_t index = integer(d);
      Py_DECREF(d);
      if (index != dev.index())
        refuse(PyExc_ValueError, "%s must be of the tensors' device", "stream");
    } else {
      PyErr_Clear();  // (a bare handle)
    }
    guard_.reset_stream(c10::cuda::getStreamFromExternal(handle_, dev.index()));
  }
  operator grpo_stream_t() const { return (grpo_stream_t)handle_; }

 private:
  cudaStream_t handle_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};
void on_device(const Tensor& t, const char* name, const c10::Device& dev) {
  if (!t.is_cuda() || t.device() != dev)
    refuse(PyExc_ValueError, "%s must be a CUDA tensor on the device of the others", name);
}
// The device of a call: its first tensor's, which has to be the current one (the
// library launches there, on that device's streams and with its properties).
c10::Device device_of(const Tensor& t, const char* name) {
  const c10::Device dev = t.device();
  on_device(t, name, dev);
  c10::DeviceIndex current = -1;
  if (c10::cuda::GetDevice(&current) != cudaSuccess) {
    (void)cudaGetLastError();
    current = -1;
  }
  if (dev.index() != current)
    refuse(PyExc_ValueError, "%s must be on the current CUDA device", name);
  return dev;
}
void contiguous(const Tensor& t, const char* name, at::ScalarType dtype, const c10::Device& dev) {
  on_device(t, name, dev);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  if (t.scalar_type() != dtype) refuse(PyExc_TypeError, "%s has the wrong dtype", name);
}
void shaped(const Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) refuse(PyExc_ValueError, "%s has the wrong shape", name);
}
Tensor make(at::IntArrayRef shape, at::ScalarType dtype, const c10::Device& dev) {
  return at::empty(shape, at::TensorOptions().dtype(dtype).device(dev));
}
at::ScalarType dtype_or(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.dtype", "out_dtype");
  return ((THPDtype*)o)->scalar_type;
}
// A workspace of at least `need` bytes: the given one if it is large enough.
Tensor workspace_of(PyObject* o, size_t need, const c10::Device& dev) {
  if (o != Py_None) {
    const Tensor& w = tensor(o, "workspace");
    on_device(w, "workspace", dev);
    if (!w.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", "workspace");
    if ((size_t)w.numel() * w.element_size() >= need) return w;
  }
  return make({(int64_t)need}, at::kByte, dev);
}
// A new workspace of `need` bytes with `count` floats behind them in the same
// memory, as two tensors: one allocation (about 1.3 us each on the host, of the 9
// us of a clipping call on 26 tensors).
Tensor workspace_and(size_t need, int64_t count, const c10::Device& dev, Tensor* floats) {
  const int64_t at = (int64_t)(need + 255) / 256 * 256;
  Tensor w = make({at + 4 * count}, at::kByte, dev);
  w.unsafeGetTensorImpl()->set_sizes_contiguous({(int64_t)need});
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(w.storage()),
                                                   c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                   caffe2::TypeMeta::Make<float>());
  impl->set_storage_offset(at / 4);
  impl->set_sizes_contiguous({count});
  *floats = Tensor(std::move(impl));
  return w;
}
// A tensor of the caller's has new values: autograd refuses a backward pass that
// saved the old ones.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
size_t bytes_of(const Tensor& t) { return (size_t)t.numel() * t.element_size(); }

// Rows of d elements: the pitch of the last-but-one dimension of a tensor of
// `n` rows, either a matrix (possibly part of wider rows) or contiguous.
int64_t row_pitch(const Tensor& t, const char* name, int64_t n, int64_t d) {
  if (t.dim() != 2) {
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must have dense rows", name);
    return d;
  }
  int64_t pitch = t.stride(0);
  if (n <= 1 && pitch < d) pitch = d;
  if ((d > 1 && t.stride(1) != 1) || pitch < d)
    refuse(PyExc_ValueError, "%s must have dense rows", name);
  return pitch;
}
// Whether t is [*ids.shape, d] or [n, d].
bool rows_match(const Tensor& t, const Tensor& ids, int64_t n, int64_t d) {
  if (t.dim() == 2 && t.size(0) == n && t.size(1) == d) return true;
  if (t.dim() != ids.dim() + 1 || t.size(-1) != d) return false;
  for (int64_t k = 0; k < ids.dim(); ++k)
    if (t.size(k) != ids.size(k)) return false;
  return true;
}

template <typename F>
grpo_status launch(F f) {
  grpo_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  return s;
}

// The body of a module function: its result, or NULL with a Python exception
// set; no C++ exception leaves it.
template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

bool count_is(Py_ssize_t have, Py_ssize_t want) {
  if (have == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// embed_fwd(ids, weight, scale, out, out_dtype, stream) -> out
PyObject* embed_fwd(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 6)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& ids = tensor(a[0], "ids");
    const c10::Device dev = device_of(ids, "ids");
    contiguous(ids, "ids", at::kLong, dev);
    const Tensor& weight = tensor(a[1], "weight");
    on_device(weight, "weight", dev);
    const grpo_dtype wcode = code(weight.scalar_type(), "weight");
    if (weight.dim() != 2) refuse(PyExc_ValueError, "%s must have two dimensions", "weight");
    const int64_t n = ids.numel(), V = weight.size(0), d = weight.size(1);
    const int64_t ldw = row_pitch(weight, "weight", V, d);
    const float scale = (float)number(a[2]);
    const at::ScalarType dt = dtype_or(a[4], a[3] == Py_None ? weight.scalar_type()
                                                              : tensor(a[3], "out").scalar_type());
    const CallStream st(a[5], dev);
    Tensor out;
    int64_t ldo = d;
    if (a[3] == Py_None) {
      code(dt, "out");
      c10::SmallVector<int64_t, 5> shape(ids.sizes().begin(), ids.sizes().end());
      shape.push_back(d);
      out = make(shape, dt, dev);
    } else {
      out = tensor(a[3], "out");
      on_device(out, "out", dev);
      if (out.scalar_type() != dt) refuse(PyExc_TypeError, "%s is not of out_dtype", "out");
      if (!rows_match(out, ids, n, d)) refuse(PyExc_ValueError, "%s must be [*ids.shape, d]", "out");
      ldo = row_pitch(out, "out", n, d);
    }
    const grpo_dtype ocode = code(dt, "out");
    check_status(launch([&] {
                   return grpo_embed_fwd((const int64_t*)ids.data_ptr(), n, weight.data_ptr(),
                                         wcode, V, d, ldw, scale, out.data_ptr(), ocode, ldo, st);
                 }),
                 "grpo_embed_fwd");
    if (a[3] == Py_None) return THPVariable_Wrap(out);
    written(out);
    return Py_NewRef(a[3]);
  });
}

PyObject* pair(PyObject* first, PyObject* second) {
  PyObject* t = first != nullptr && second != nullptr ? PyTuple_Pack(2, first, second) : nullptr;
  Py_XDECREF(first);
  Py_XDECREF(second);
  return t;
}
// The caller's own object where it was used, else a new one.
PyObject* wrap(PyObject* given, const Tensor& t) {
  if (given != Py_None && THPVariable_Unpack(given).is_same(t)) return Py_NewRef(given);
  return THPVariable_Wrap(t);
}

// embed_bwd(ids, dout, V, scale, pad_id, dweight, accumulate, out_dtype, workspace, stream)
//   -> (dweight, workspace)
PyObject* embed_bwd(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const bool accumulate = truth(a[6]);
    const Tensor& ids = tensor(a[0], "ids");
    const c10::Device dev = device_of(ids, "ids");
    contiguous(ids, "ids", at::kLong, dev);
    const Tensor& dout = tensor(a[1], "dout");
    on_device(dout, "dout", dev);
    const grpo_dtype dcode = code(dout.scalar_type(), "dout");
    const int64_t n = ids.numel(), V = integer(a[2]);
    if (dout.dim() < 1) refuse(PyExc_ValueError, "%s must be [*ids.shape, d]", "dout");
    const int64_t d = dout.size(-1);
    if (!rows_match(dout, ids, n, d)) refuse(PyExc_ValueError, "%s must be [*ids.shape, d]", "dout");
    const int64_t ldd = row_pitch(dout, "dout", n, d);
    const float scale = (float)number(a[3]);
    const int64_t pad = a[4] == Py_None ? -1 : integer(a[4]);
    const CallStream st(a[9], dev);
    Tensor dw;
    int64_t ldw = d;
    if (a[5] == Py_None) {
      if (accumulate) refuse(PyExc_ValueError, "%s is needed to accumulate", "dweight");
      const at::ScalarType dt = dtype_or(a[7], at::kFloat);
      code(dt, "dweight");
      if (V < 0) refuse(PyExc_ValueError, "%s must not be negative", "V");
      dw = make({V, d}, dt, dev);
    } else {
      dw = tensor(a[5], "dweight");
      on_device(dw, "dweight", dev);
      if (dtype_or(a[7], dw.scalar_type()) != dw.scalar_type())
        refuse(PyExc_TypeError, "%s is not of out_dtype", "dweight");
      shaped(dw, "dweight", {V, d});
      ldw = row_pitch(dw, "dweight", V, d);
    }
    const grpo_dtype wcode = code(dw.scalar_type(), "dweight");
    size_t need = 0;
    check_status(grpo_embed_workspace_size(n, V, d, &need), "grpo_embed_workspace_size");
    const Tensor ws = workspace_of(a[8], need, dev);
    check_status(launch([&] {
                   return grpo_embed_bwd((const int64_t*)ids.data_ptr(), n, dout.data_ptr(), dcode,
                                         V, d, ldd, scale, pad, dw.data_ptr(), wcode, ldw,
                                         accumulate, ws.data_ptr(), bytes_of(ws), st);
                 }),
                 "grpo_embed_bwd");
    if (a[5] != Py_None) written(dw);
    return pair(wrap(a[5], dw), wrap(a[8], ws));
  });
}

// A list or tuple, held for its items.
struct Items {
  PyObject* seq;
  explicit Items(PyObject* o, const char* name) : seq(PySequence_Fast(o, name)) {
    if (seq == nullptr) throw Refused();
  }
  ~Items() { Py_DECREF(seq); }
  Items(const Items&) = delete;
  Items& operator=(const Items&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
  PyObject* at(Py_ssize_t k) const { return PySequence_Fast_GET_ITEM(seq, k); }
};

// clip(grads, max_norm, out, norm_type, eps, stats, workspace, stream, norm_only)
//   -> (stats, workspace)
PyObject* clip(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Items grads(a[0], "grads must be a list of tensors");
    const Py_ssize_t n = grads.size();
    const bool norm_only = truth(a[8]);
    const float max_norm = norm_only ? 0.f : (float)number(a[1]);
    const float eps = norm_only ? 0.f : (float)number(a[4]);
    const grpo_norm_type type = (grpo_norm_type)integer(a[3]);
    const c10::Device dev =
        n > 0 ? device_of(tensor(grads.at(0), "every gradient"), "every gradient")
              : c10::Device(c10::kCUDA, c10::cuda::getCurrentCUDAStream().device_index());
    std::vector<grpo_tensor> table((size_t)n);
    for (Py_ssize_t k = 0; k < n; ++k) {
      const Tensor& t = tensor(grads.at(k), "every gradient");
      on_device(t, "every gradient", dev);
      if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", "every gradient");
      grpo_tensor& g = table[(size_t)k];
      g.data = t.data_ptr();
      g.out = nullptr;
      g.numel = t.numel();
      g.dtype = g.out_dtype = code(t.scalar_type(), "every gradient");
      if (!norm_only && a[2] == Py_None) written(t);
    }
    if (a[2] != Py_None) {
      const Items outs(a[2], "out must be a list of tensors");
      if (outs.size() != n) refuse(PyExc_ValueError, "%s must have one tensor per gradient", "out");
      for (Py_ssize_t k = 0; k < n; ++k) {
        const Tensor& t = tensor(outs.at(k), "every out");
        on_device(t, "every out", dev);
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", "every out");
        grpo_tensor& g = table[(size_t)k];
        if (t.numel() != g.numel)
          refuse(PyExc_ValueError, "%s must have its gradient's size", "every out");
        g.out = t.data_ptr();
        g.out_dtype = code(t.scalar_type(), "every out");
        if (!norm_only) written(t);
      }
    }
    size_t need = 0;
    check_status(grpo_grad_norm_workspace_size(n, &need), "grpo_grad_norm_workspace_size");
    const CallStream st(a[7], dev);
    Tensor stats, ws;
    if (a[5] == Py_None && a[6] == Py_None) {
      ws = workspace_and(need, 2, dev, &stats);
    } else if (a[5] == Py_None) {
      stats = make({2}, at::kFloat, dev);
    } else {
      stats = tensor(a[5], "stats");
      contiguous(stats, "stats", at::kFloat, dev);
      if (stats.numel() < 2) refuse(PyExc_ValueError, "%s must hold two values", "stats");
    }
    if (!ws.defined()) ws = workspace_of(a[6], need, dev);
    float* sp = (float*)stats.data_ptr();
    check_status(launch([&] {
                   return norm_only
                              ? grpo_grad_norm(table.data(), n, type, sp, ws.data_ptr(),
                                               bytes_of(ws), st)
                              : grpo_clip_grad_norm(table.data(), n, type, max_norm, eps, sp,
                                                    ws.data_ptr(), bytes_of(ws), st);
                 }),
                 norm_only ? "grpo_grad_norm" : "grpo_clip_grad_norm");
    if (a[5] != Py_None) written(stats);
    return pair(wrap(a[5], stats), wrap(a[6], ws));
  });
}

// Strides of [N, R, V] logits whose rows are dense and apart.
void logit_strides(const Tensor& t, const char* name, int64_t N, int64_t R, int64_t V,
                   int64_t* seq, int64_t* row) {
  shaped(t, name, {N, R, V});
  *seq = t.stride(0);
  *row = t.stride(1);
  if (R <= 1 && *row < V) *row = V;
  if (N <= 1 && *seq < R * *row) *seq = R * *row;
  if ((V > 1 && t.stride(2) != 1) || *row < V || *seq < (R - 1) * *row + V)
    refuse(PyExc_ValueError, "%s must have dense rows that do not overlap", name);
}

// An entry of the caller's dict of outputs.
const Tensor& entry(PyObject* dict, const char* key) {
  PyObject* o = PyDict_GetItemString(dict, key);
  if (o == nullptr) refuse(PyExc_ValueError, "out has no %s", key);
  return tensor(o, key);
}

// verify(target_logits, draft_tokens, u, noise, draft_logits, draft_lens, temperature, out,
//        workspace, stream) -> out
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (!count_is(n_args, 10)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Tensor& z = tensor(a[0], "target_logits");
    const c10::Device dev = device_of(z, "target_logits");
    if (z.dim() != 3) refuse(PyExc_ValueError, "%s must be [N, K+1, V]", "target_logits");
    const int64_t N = z.size(0), rows = z.size(1), V = z.size(2), K = rows - 1;
    if (K < 0) refuse(PyExc_ValueError, "%s must have a row per sequence", "target_logits");
    const grpo_dtype dt = code(z.scalar_type(), "target_logits");
    int64_t tseq, trow, dseq = 0, drow = 0;
    logit_strides(z, "target_logits", N, rows, V, &tseq, &trow);
    const Tensor* y = maybe_tensor(a[4], "draft_logits");
    if (y != nullptr) {
      on_device(*y, "draft_logits", dev);
      if (y->scalar_type() != z.scalar_type())
        refuse(PyExc_TypeError, "%s must have target_logits' dtype", "draft_logits");
      logit_strides(*y, "draft_logits", N, K, V, &dseq, &drow);
    }
    const Tensor& x = tensor(a[1], "draft_tokens");
    contiguous(x, "draft_tokens", at::kLong, dev);
    shaped(x, "draft_tokens", {N, K});
    const Tensor& u = tensor(a[2], "u");
    contiguous(u, "u", at::kFloat, dev);
    shaped(u, "u", {N, K});
    const Tensor& noise = tensor(a[3], "noise");
    on_device(noise, "noise", dev);
    if (noise.scalar_type() != at::kFloat) refuse(PyExc_TypeError, "%s must be float32", "noise");
    shaped(noise, "noise", {N, V});
    const int64_t nrow = row_pitch(noise, "noise", N, V);
    const Tensor* lens = maybe_tensor(a[5], "draft_lens");
    if (lens != nullptr) {
      contiguous(*lens, "draft_lens", at::kInt, dev);
      shaped(*lens, "draft_lens", {N});
    }
    const Tensor* temp = maybe_tensor(a[6], "temperature");
    if (temp != nullptr) {
      contiguous(*temp, "temperature", at::kFloat, dev);
      shaped(*temp, "temperature", {N});
    }
    const CallStream st(a[9], dev);
    Tensor tokens, accepted, logp;
    PyObject* given_ws = a[8];
    if (a[7] == Py_None) {
      tokens = make({N, rows}, at::kLong, dev);
      accepted = make({N}, at::kInt, dev);
      logp = make({N, rows}, at::kFloat, dev);
    } else {
      if (!PyDict_Check(a[7])) refuse(PyExc_TypeError, "%s must be a dict", "out");
      tokens = entry(a[7], "tokens");
      contiguous(tokens, "tokens", at::kLong, dev);
      shaped(tokens, "tokens", {N, rows});
      accepted = entry(a[7], "n_accepted");
      contiguous(accepted, "n_accepted", at::kInt, dev);
      shaped(accepted, "n_accepted", {N});
      logp = entry(a[7], "logp");
      contiguous(logp, "logp", at::kFloat, dev);
      shaped(logp, "logp", {N, rows});
      if (given_ws == Py_None) {
        PyObject* w = PyDict_GetItemString(a[7], "workspace");
        if (w != nullptr) given_ws = w;
      }
    }
    size_t need = 0;
    check_status(grpo_verify_workspace_size(N, K, &need), "grpo_verify_workspace_size");
    const Tensor ws = workspace_of(given_ws, need, dev);
    check_status(
        launch([&] {
          return grpo_verify_drafts(
              z.data_ptr(), y != nullptr ? y->data_ptr() : nullptr, dt, N, K, V, tseq, trow, dseq,
              drow, (const int64_t*)x.data_ptr(),
              lens != nullptr ? (const int32_t*)lens->data_ptr() : nullptr,
              (const float*)u.data_ptr(), (const float*)noise.data_ptr(), nrow,
              temp != nullptr ? (const float*)temp->data_ptr() : nullptr,
              (int64_t*)tokens.data_ptr(), (int32_t*)accepted.data_ptr(), (float*)logp.data_ptr(),
              ws.data_ptr(), bytes_of(ws), st);
        }),
        "grpo_verify_drafts");
    if (a[7] != Py_None)
      for (const Tensor* t : {&tokens, &accepted, &logp}) written(*t);
    PyObject* out = a[7] == Py_None ? PyDict_New() : Py_NewRef(a[7]);
    if (out == nullptr) return nullptr;
    auto put = [&](const char* key, PyObject* v) {  // takes v
      const bool ok = v != nullptr && PyDict_SetItemString(out, key, v) == 0;
      Py_XDECREF(v);
      return ok;
    };
    bool ok = put("workspace", wrap(given_ws, ws));
    if (a[7] == Py_None)
      ok = ok && put("tokens", THPVariable_Wrap(tokens)) &&
           put("n_accepted", THPVariable_Wrap(accepted)) && put("logp", THPVariable_Wrap(logp));
    if (!ok) {
      Py_DECREF(out);
      return nullptr;
    }
    return out;
  });
}

// set_error(GrpoError): the exception of a status other than GRPO_OK
PyObject* set_error(PyObject*, PyObject* type) {
  Py_XSETREF(g_error, Py_NewRef(type));
  Py_RETURN_NONE;
}

#define FAST(f) (PyCFunction)(void (*)(void))f, METH_FASTCALL
PyMethodDef methods[] = {{"embed_fwd", FAST(embed_fwd), nullptr},
                         {"embed_bwd", FAST(embed_bwd), nullptr},
                         {"clip", FAST(clip), nullptr},
                         {"verify", FAST(verify), nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() {
  PyObject* m = PyModule_Create(&module);
  // what it was compiled against; _native.py compares
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", GRPO_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
