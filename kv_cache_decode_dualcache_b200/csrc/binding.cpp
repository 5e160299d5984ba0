// Python binding of the stream-ordered operators (fdllm_kv8_*, fdllm_sample):
// torch tensors in, torch tensors out, nothing computed here.  These calls
// take a few microseconds on the GPU, which marshalling in Python (attribute
// reads, argument structs, allocations) would more than double: measured 13.5
// us a call for an attention and 17.8 us for an append against 2.5 us for
// each kernel launch in them.  The C entry points come as addresses from the
// library that fdllm.py loaded, so this module links against torch only.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/fdllm.h"

namespace {

decltype(&fdllm_kv8_append) c_append;
decltype(&fdllm_kv8_attention) c_attention;
decltype(&fdllm_kv8_attention_workspace) c_workspace;
decltype(&fdllm_sample) c_sample;

struct Refused {   // becomes a ValueError
  std::string what;
};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::nullopt;
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(name) + " must fit in 32 bits"};
  return (int32_t)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw std::nullopt;
  return v;
}
int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return FDLLM_DTYPE_F32;
    case at::kBFloat16: return FDLLM_DTYPE_BF16;
    case at::kHalf: return FDLLM_DTYPE_F16;
    default: throw Refused{std::string(c10::toString(t)) +
                           " is not a type of this call (float32, bfloat16, float16)"};
  }
}

// Address of a contiguous 1-D tensor of n elements; None gives NULL.
template <typename E> E* vector(PyObject* o, const char* name, int64_t n, at::ScalarType type, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.dim() != 1 || t.numel() != n || !t.is_contiguous())
    throw Refused{std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of " +
                  std::to_string(n) + " elements"};
  if (t.get_device() != dev)
    throw Refused{std::string(name) + " must be on the same CUDA device as the other operands"};
  return static_cast<E*>(t.data_ptr());
}

// [tokens, heads, hd] rows with contiguous vectors; the strides of dims of
// one element do not matter.  heads < 0: any.
void* rows(const at::Tensor& t, const char* name, int64_t tokens, int64_t heads, int64_t hd,
           at::ScalarType type, int dev, int64_t* strides) {
  if (t.dim() != 3 || t.size(2) != hd || (heads >= 0 && t.size(1) != heads) ||
      (t.stride(2) != 1 && t.size(0) > 0))
    throw Refused{std::string(name) + " must be [tokens, " + (heads >= 0 ? std::to_string(heads) : "heads") +
                  ", " + std::to_string(hd) + "] with contiguous vectors"};
  if (t.size(0) != tokens || t.scalar_type() != type)
    throw Refused{"all rows of a call must have the same number of tokens and the same type"};
  if (t.get_device() != dev)
    throw Refused{std::string(name) + " must be on the same CUDA device as the other operands"};
  strides[0] = tokens > 1 ? t.stride(0) : 0;
  strides[1] = t.size(1) > 1 ? t.stride(1) : 0;
  return t.data_ptr();
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
}
// The call's device and stream (None: torch's current one) while it is made.
// Results and workspaces then come from the memory of the stream that writes
// them: none is handed out again before the stream is past the call.
struct OnStream {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard stream;
  void* handle;
  OnStream(PyObject* o, int dev) {
    const c10::DeviceIndex d = (c10::DeviceIndex)dev;
    if (c10::cuda::current_device() != d) device.set_index(d);
    handle = c10::cuda::getCurrentCUDAStream(d).stream();
    if (o == Py_None) return;
    void* given = reinterpret_cast<void*>((uintptr_t)integer(o));
    if (given == handle) return;
    handle = given;
    stream.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(given), d));
  }
};

// fn's result: a tuple, or the status of the C call as an int.
template <typename F> PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F fn) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return fn();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const std::nullopt_t&) {   // a Python error is set
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
PyObject* status_or(int rc, std::initializer_list<const at::Tensor*> out) {
  if (rc != FDLLM_OK) return PyLong_FromLong(rc);
  PyObject* r = PyTuple_New((Py_ssize_t)out.size());
  Py_ssize_t i = 0;
  for (const at::Tensor* t : out) {
    if (t->defined()) {
      PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(*t));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, i++, Py_None);
    }
  }
  return r;
}

// (append, attention, workspace, sample): addresses of the C entry points
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    c_append = reinterpret_cast<decltype(c_append)>((uintptr_t)integer(a[0]));
    c_attention = reinterpret_cast<decltype(c_attention)>((uintptr_t)integer(a[1]));
    c_workspace = reinterpret_cast<decltype(c_workspace)>((uintptr_t)integer(a[2]));
    c_sample = reinterpret_cast<decltype(c_sample)>((uintptr_t)integer(a[3]));
    Py_RETURN_NONE;
  });
}

// (cache struct, device, k, v, starts, lens, pos, rope, q, max_new, stored,
// lens_out, status, stream) -> (q_out, k_out, v_out)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const fdllm_kv8& c = *reinterpret_cast<const fdllm_kv8*>((uintptr_t)integer(a[0]));
    const int dev = (int)integer(a[1]);
    const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    const int64_t T = k.dim() > 0 ? k.size(0) : 0;
    const at::ScalarType type = k.scalar_type();
    fdllm_kv8_append_args p{};
    p.dtype = dtype_code(type);
    p.k = rows(k, "k", T, c.n_kv_heads, c.head_dim, type, dev, p.k_strides);
    p.v = rows(v, "v", T, c.n_kv_heads, c.head_dim, type, dev, p.v_strides);
    if (T > INT32_MAX) throw Refused{"too many tokens"};
    p.n_tokens = (int32_t)T;
    p.max_new = integer32(a[9], "max_new");
    p.starts = vector<int32_t>(a[4], "starts", c.n_seqs + 1, at::kInt, dev);
    p.lens = vector<int32_t>(a[5], "lens", c.n_seqs, at::kInt, dev);
    p.pos = vector<int32_t>(a[6], "pos", c.n_seqs, at::kInt, dev);
    p.lens_out = vector<int32_t>(a[11], "lens_out", c.n_seqs, at::kInt, dev);
    p.status = vector<int32_t>(a[12], "status", 1, at::kInt, dev);
    if (a[7] != Py_None) {
      const at::Tensor& r = tensor(a[7], "rope");
      if (r.scalar_type() != at::kFloat || r.dim() != 3 || r.size(1) != c.head_dim / 2 || r.size(2) != 2 ||
          !r.is_contiguous() || r.get_device() != dev || r.size(0) > INT32_MAX)
        throw Refused{"rope must be contiguous float32 [positions, " + std::to_string(c.head_dim / 2) +
                      ", 2] on the cache's device"};
      p.rope = static_cast<const float*>(r.data_ptr());
      p.rope_len = (int32_t)r.size(0);
    }
    const OnStream on(a[13], dev);
    at::Tensor q_out, k_out, v_out;
    if (a[8] != Py_None) {
      const at::Tensor& q = tensor(a[8], "q");
      p.q = rows(q, "q", T, -1, c.head_dim, type, dev, p.q_strides);
      p.n_heads = (int32_t)q.size(1);
      q_out = empty(q.sizes(), type, dev);
      p.q_out = q_out.data_ptr();
    }
    if (PyObject_IsTrue(a[10])) {
      k_out = empty(k.sizes(), type, dev);
      v_out = empty(k.sizes(), type, dev);
      p.k_out = k_out.data_ptr();
      p.v_out = v_out.data_ptr();
    }
    return status_or(c_append(&c, &p, on.handle), {&q_out, &k_out, &v_out});
  });
}

// (cache struct, device, q, starts, lens, scale, out, max_q, max_len,
// workspace, status, stream) -> (out,)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const fdllm_kv8& c = *reinterpret_cast<const fdllm_kv8*>((uintptr_t)integer(a[0]));
    const int dev = (int)integer(a[1]);
    const at::Tensor& q = tensor(a[2], "q");
    const int64_t T = q.dim() > 0 ? q.size(0) : 0;
    const at::ScalarType type = q.scalar_type();
    fdllm_kv8_attention_args p{};
    p.dtype = dtype_code(type);
    p.q = rows(q, "q", T, -1, c.head_dim, type, dev, p.q_strides);
    if (T > INT32_MAX) throw Refused{"too many tokens"};
    p.n_tokens = (int32_t)T;
    p.n_heads = (int32_t)q.size(1);
    p.max_q = integer32(a[7], "max_q");
    p.max_len = integer32(a[8], "max_len");
    p.scale = a[5] == Py_None ? 1.0f / std::sqrt((float)c.head_dim) : (float)number(a[5]);
    p.starts = vector<int32_t>(a[3], "starts", c.n_seqs + 1, at::kInt, dev);
    p.lens = vector<int32_t>(a[4], "lens", c.n_seqs, at::kInt, dev);
    p.status = vector<int32_t>(a[10], "status", 1, at::kInt, dev);
    const OnStream on(a[11], dev);
    at::Tensor out, space;
    if (a[6] == Py_None) {
      out = empty(q.sizes(), type, dev);
      p.out = out.data_ptr();
      p.out_strides[0] = q.size(1) * q.size(2);
      p.out_strides[1] = q.size(2);
    } else {
      out = tensor(a[6], "out");
      p.out = rows(out, "out", T, q.size(1), c.head_dim, type, dev, p.out_strides);
    }
    if (a[9] == Py_None) {
      const int rc = c_workspace(&c, &p, &p.workspace_bytes);
      if (rc != FDLLM_OK) return PyLong_FromLong(rc);
      if (p.workspace_bytes) {
        space = empty({(int64_t)p.workspace_bytes}, at::kByte, dev);
        p.workspace = space.data_ptr();
      }
    } else {
      const at::Tensor& w = tensor(a[9], "workspace");
      if (w.get_device() != dev || !w.is_contiguous())
        throw Refused{"workspace must be contiguous and on the cache's device"};
      p.workspace = w.data_ptr();
      p.workspace_bytes = (size_t)w.numel() * w.element_size();
    }
    return status_or(c_attention(&c, &p, on.handle), {&out});
  });
}

// (logits, u, temperature, top_k, top_p, min_p, mask_id, tok, prob, stream)
// -> (tok, prob)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "logits");
    if (x.dim() != 2 || (x.stride(1) != 1 && x.size(1) > 1))
      throw Refused{"logits must be [rows, vocab] with contiguous rows"};
    if (!x.is_cuda()) throw Refused{"logits must be on a CUDA device"};
    const int dev = (int)x.get_device();
    const int64_t R = x.size(0), V = x.size(1);
    if (R > INT32_MAX || V > INT32_MAX) throw Refused{"logits are too large"};
    fdllm_sample_args p{};
    p.logits = x.data_ptr();
    p.row_stride = R > 1 ? x.stride(0) : V;
    p.dtype = dtype_code(x.scalar_type());
    p.rows = (int32_t)R;
    p.vocab = (int32_t)V;
    p.mask_id = integer32(a[6], "mask_id");
    if (a[1] == Py_None) throw Refused{"u must be a tensor"};
    p.u = vector<double>(a[1], "u", R, at::kDouble, dev);
    p.temperature = vector<float>(a[2], "temperature", R, at::kFloat, dev);
    p.top_k = vector<int32_t>(a[3], "top_k", R, at::kInt, dev);
    p.top_p = vector<float>(a[4], "top_p", R, at::kFloat, dev);
    p.min_p = vector<float>(a[5], "min_p", R, at::kFloat, dev);
    const OnStream on(a[9], dev);
    at::Tensor tok = a[7] == Py_None ? empty({R}, at::kInt, dev) : tensor(a[7], "tok");
    at::Tensor prob = a[8] == Py_None ? empty({R}, at::kFloat, dev) : tensor(a[8], "prob");
    p.tok = a[7] == Py_None ? static_cast<int32_t*>(tok.data_ptr()) : vector<int32_t>(a[7], "tok", R, at::kInt, dev);
    p.prob = a[8] == Py_None ? static_cast<float*>(prob.data_ptr()) : vector<float>(a[8], "prob", R, at::kFloat, dev);
    return status_or(c_sample(&p, on.handle), {&tok, &prob});
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(bind), nullptr},
                         {"append", FAST(append), nullptr},
                         {"attention", FAST(attention), nullptr},
                         {"sample", FAST(sample), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
