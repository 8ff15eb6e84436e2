// The calls that a decode step makes for every layer, from torch tensors: argument checks, outputs and the C entry
// points of include/gqa_decode.h.  The rest of the binding is ctypes (_binding.py, which wraps these functions
// too); here the host's time for a call counts against a kernel of a few microseconds, and reading a tensor's
// fields through Python takes most of it (one token appended: 15 us a call with the checks in Python).
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/gqa_decode.h"

namespace {

struct Refused {
  std::string what;
};

[[noreturn]] void refuse(const char* name, const std::string& what) {
  throw Refused{std::string(name) + " must be " + what};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, "a tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, "a whole number");
  }
  return v;
}

// an int argument of the C call
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse(name, "a 32-bit number");
  return (int)v;
}

double real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, "a number");
  }
  return v;
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(name, "true or false");
  }
  return v == 1;
}

bool is_half(const at::Tensor& t) { return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16; }

// the CUDA device of the first tensor of a call, which has to be the current one
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(name, "a CUDA tensor");
  const int dev = t.get_device(), now = c10::cuda::current_device();
  if (dev != now)
    throw Refused{"the tensors are on device " + std::to_string(dev) + ", the current device is " + std::to_string(now)};
  return dev;
}

bool has(const at::Tensor& t, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  return t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.sizes() == at::IntArrayRef(shape);
}

// a contiguous tensor of this type and shape on the device: its address
template <typename T>
T* whole(const at::Tensor& t, const char* name, at::ScalarType type, int dev, std::initializer_list<int64_t> shape) {
  if (!has(t, type, dev, shape) || !t.is_contiguous()) {
    std::string s = std::string("a contiguous ") + c10::toString(type) + " tensor of shape (";
    for (int64_t n : shape) s += std::to_string(n) + ", ";
    refuse(name, s + ") on the device of the others");
  }
  return static_cast<T*>(t.data_ptr());
}

// a (tokens, cols) tensor whose rows are dense: its address, and the distance of two rows
uint16_t* rows(const at::Tensor& t, const char* name, at::ScalarType type, int dev, int64_t tokens, int64_t cols,
               int64_t* stride) {
  if (!has(t, type, dev, {tokens, cols}) || (cols > 1 && t.stride(1) != 1))
    refuse(name, std::string("a ") + c10::toString(type) + " tensor of shape (" + std::to_string(tokens) + ", " +
                     std::to_string(cols) + ") with dense rows on the device of the others");
  *stride = tokens > 1 ? t.stride(0) : cols;
  return static_cast<uint16_t*>(t.data_ptr());
}

struct Workspace {
  void* at;
  size_t bytes;
};

Workspace workspace(PyObject* o, int dev) {
  const at::Tensor& t = tensor(o, "workspace_tensor");
  if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    refuse("workspace_tensor", "a contiguous tensor on the device of the others");
  return {t.data_ptr(), (size_t)t.nbytes()};
}

// where a call reports: a workspace, or None, the library's own status word
Workspace status_word(PyObject* o, int dev) {
  if (o != Py_None) return workspace(o, dev);
  return {gqa_device_status(), 256};
}

int32_t as_int(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(name, "smaller");
  return (int32_t)n;
}

// block size of an 8-bit cache of D-element heads (h_kv < 0: any number of heads)
int kv8_block_size(const at::Tensor& cache, int64_t h_kv, int64_t D, int dev) {
  const int64_t row = 2 * D + 2;
  if (cache.scalar_type() != at::kByte || cache.dim() != 3 || !cache.is_cuda() || cache.get_device() != dev ||
      !cache.is_contiguous() || (h_kv >= 0 && cache.size(1) != h_kv) || row < 4 || cache.size(2) % row != 0)
    refuse("an 8-bit cache",
           "a contiguous uint8 tensor (num_blocks, h_kv, block_size * (2 * d_head + 2)) on the device of the others");
  return as_int(cache.size(2) / row, "the blocks of the cache");
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

// append(q|None, k, v, h_q, h_kv, slots, k_cache, v_cache|None, positions|None, cos_sin|None, interleaved, q_weight|None,
//        k_weight|None, eps, q_out|None, workspace|None) -> q_out or None, or a status
PyObject* append(PyObject* const* p) {
  const at::Tensor *q = optional(p[0], "q"), &k = tensor(p[1], "k"), &v = tensor(p[2], "v");
  if (k.dim() != 2 || !is_half(k)) refuse("k", "a float16 or bfloat16 CUDA tensor (tokens, h_kv*d_head)");
  const int dev = device_of(k, "k");
  gqa_append_args a = {};
  a.h_kv = small(p[4], "h_kv");
  const int64_t T = k.size(0), kc = k.size(1);
  if (a.h_kv < 1 || kc % a.h_kv != 0) refuse("k", "a float16 or bfloat16 CUDA tensor (tokens, h_kv*d_head)");
  const int64_t D = kc / a.h_kv;
  const at::ScalarType type = k.scalar_type();
  a.num_tokens = as_int(T, "the number of tokens");
  a.d_head = as_int(D, "d_head");
  a.bf16 = type == at::kBFloat16;
  a.k = rows(k, "k", type, dev, T, kc, &a.k_stride);
  a.v = rows(v, "v", type, dev, T, kc, &a.v_stride);
  at::Tensor made;
  const at::Tensor* q_out = nullptr;
  if (q != nullptr) {
    a.h_q = small(p[3], "h_q");
    const int64_t qc = a.h_q * D;
    a.q = rows(*q, "q", type, dev, T, qc, &a.q_stride);
    q_out = optional(p[14], "q_out");
    if (q_out == nullptr) {
      made = at::empty({T, qc}, k.options());
      q_out = &made;
    }
    a.q_out = rows(*q_out, "q_out", type, dev, T, qc, &a.q_out_stride);
  }
  if (const at::Tensor* cs = optional(p[9], "cos_sin")) {
    const at::Tensor* pos = optional(p[8], "positions");
    if (cs->dim() != 2 || pos == nullptr) refuse("cos_sin", "(max_position, rot_dim), and comes with positions");
    a.max_position = as_int(cs->size(0), "the rows of cos_sin");
    a.rot_dim = as_int(cs->size(1), "rot_dim");
    a.cos_sin = whole<float>(*cs, "cos_sin", at::kFloat, dev, {cs->size(0), cs->size(1)});
    a.positions = whole<int32_t>(*pos, "positions", at::kInt, dev, {T});
    if (T == 0) a.positions = reinterpret_cast<const int32_t*>(a.cos_sin);   // (an empty tensor has no address; none is read)
  }
  a.interleaved = truth(p[10], "interleaved");
  if (const at::Tensor* w = optional(p[11], "q_weight")) a.q_weight = whole<uint16_t>(*w, "q_weight", type, dev, {D});
  if (const at::Tensor* w = optional(p[12], "k_weight")) a.k_weight = whole<uint16_t>(*w, "k_weight", type, dev, {D});
  a.eps = (float)real(p[13], "eps");
  a.slots = whole<int64_t>(tensor(p[5], "slots"), "slots", at::kLong, dev, {T});
  const at::Tensor &kc_t = tensor(p[6], "k_cache"), *vc_t = optional(p[7], "v_cache");
  if (kc_t.scalar_type() == at::kByte) {
    if (vc_t != nullptr) throw Refused{"an 8-bit cache holds K and V: pass no v_cache"};
    a.cache_layout = GQA_CACHE_KV8;
    a.block_size = kv8_block_size(kc_t, a.h_kv, D, dev);
    a.k_cache = kc_t.data_ptr();
  } else {
    if (vc_t == nullptr) throw Refused{"a 16-bit cache needs k_cache and v_cache"};
    const int64_t nb = kc_t.dim() > 0 ? kc_t.size(0) : 0;
    if (kc_t.dim() == 5) {
      const int64_t bs = kc_t.size(3);
      a.cache_layout = GQA_CACHE_VLLM;
      a.block_size = as_int(bs, "block_size");
      a.k_cache = whole<void>(kc_t, "k_cache", type, dev, {nb, a.h_kv, D / 8, bs, 8});
      a.v_cache = whole<void>(*vc_t, "v_cache", type, dev, {nb, a.h_kv, D, bs});
    } else {
      const int64_t bs = kc_t.dim() == 3 ? kc_t.size(1) : 0;
      a.cache_layout = GQA_CACHE_ROWS;
      a.block_size = as_int(bs, "block_size");
      a.k_cache = whole<void>(kc_t, "k_cache", type, dev, {nb, bs, kc});
      a.v_cache = whole<void>(*vc_t, "v_cache", type, dev, {nb, bs, kc});
    }
  }
  a.num_blocks = as_int(kc_t.size(0), "num_blocks");
  const Workspace ws = status_word(p[15], dev);
  void* st = stream_of(dev);
  gqa_status s;
  Py_BEGIN_ALLOW_THREADS
  s = gqa_append(&a, ws.at, ws.bytes, st);
  Py_END_ALLOW_THREADS
  if (s != GQA_OK) return PyLong_FromLong(s);
  if (q_out == nullptr) Py_RETURN_NONE;
  if (q_out != &made) return Py_NewRef(p[14]);
  return THPVariable_Wrap(std::move(made));
}

// decode(q, cache, block_tables, seq_lens, h_q, h_kv, scale|None, causal, out|None, workspace, status|None, timeout_us, stall)
// -> out, or a status
PyObject* decode(PyObject* const* p) {
  const at::Tensor& q = tensor(p[0], "q");
  const int64_t dim = q.dim();
  const int h_q = small(p[4], "h_q"), h_kv = small(p[5], "h_kv");
  if (!is_half(q) || (dim != 2 && dim != 3) || !q.is_contiguous() || h_q < 1 || q.size(dim - 1) % h_q != 0)
    refuse("q", "a contiguous float16 or bfloat16 CUDA tensor (N, h_q*d_head) or (N, T_q, h_q*d_head)");
  const int dev = device_of(q, "q");
  const int64_t N = q.size(0), T_q = dim == 3 ? q.size(1) : 1, D = q.size(dim - 1) / h_q;
  const at::Tensor &cache = tensor(p[1], "cache"), &tables = tensor(p[2], "block_tables");
  const int bs = kv8_block_size(cache, h_kv, D, dev);
  if (tables.dim() != 2) refuse("block_tables", "(N, max_blocks)");
  const int64_t mb = tables.size(1);
  const int32_t* tp = whole<int32_t>(tables, "block_tables", at::kInt, dev, {N, mb});
  const int32_t* lp = whole<int32_t>(tensor(p[3], "seq_lens"), "seq_lens", at::kInt, dev, {N});
  const float scale = p[6] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)real(p[6], "scale");
  const at::Tensor* out = optional(p[8], "out");
  at::Tensor made;
  if (out == nullptr) {
    made = at::empty(q.sizes(), q.options());
    out = &made;
  } else if (out->scalar_type() != q.scalar_type() || !out->is_cuda() || out->get_device() != dev ||
             out->sizes() != q.sizes() || !out->is_contiguous()) {
    refuse("out", "like q");
  }
  gqa_options opt = {};
  const int64_t limit = integer(p[11], "timeout_us");
  if (limit < 0 || limit > UINT32_MAX) refuse("timeout_us", "a number of microseconds in 32 bits");
  opt.timeout_us = (uint32_t)limit;
  opt.test_stall_cta = small(p[12], "test_stall_cta");
  opt.causal = truth(p[7], "causal");
  opt.bf16 = q.scalar_type() == at::kBFloat16;
  const Workspace ws = workspace(p[9], dev), status = status_word(p[10], dev);
  if (status.bytes < 256) return PyLong_FromLong(GQA_ERR_WORKSPACE);
  void* st = stream_of(dev);
  const int n = as_int(N, "N"), t = as_int(T_q, "T_q"), blocks = as_int(mb, "max_blocks"),
            nb = as_int(cache.size(0), "num_blocks"), d = as_int(D, "d_head");
  gqa_status s;
  Py_BEGIN_ALLOW_THREADS
  s = gqa_decode_kv8_status(static_cast<const uint16_t*>(q.data_ptr()), cache.data_ptr(), tp, lp,
                            static_cast<uint16_t*>(out->data_ptr()), n, t, blocks, nb, bs, h_q, h_kv, d, scale, ws.at,
                            ws.bytes, status.at, st, &opt);
  Py_END_ALLOW_THREADS
  if (s != GQA_OK) return PyLong_FromLong(s);
  if (out != &made) return Py_NewRef(p[8]);
  return THPVariable_Wrap(std::move(made));
}

// read(cache, block_tables, seq_lens, d_head, begins|None, k_out|None, v_out|None, workspace|None) -> a status
PyObject* read(PyObject* const* p) {
  const at::Tensor &cache = tensor(p[0], "cache"), &tables = tensor(p[1], "block_tables");
  const int dev = device_of(cache, "cache");
  const int64_t D = integer(p[3], "d_head");
  const int bs = kv8_block_size(cache, -1, D, dev);
  if (tables.dim() != 2) refuse("block_tables", "(N, max_blocks)");
  const int64_t N = tables.size(0), mb = tables.size(1), h_kv = cache.size(1);
  const int32_t* tp = whole<int32_t>(tables, "block_tables", at::kInt, dev, {N, mb});
  const int32_t* lp = whole<int32_t>(tensor(p[2], "seq_lens"), "seq_lens", at::kInt, dev, {N});
  const at::Tensor* begins = optional(p[4], "begins");
  const int32_t* bp = begins != nullptr ? whole<int32_t>(*begins, "begins", at::kInt, dev, {N}) : nullptr;
  const at::Tensor *ko = optional(p[5], "k_out"), *vo = optional(p[6], "v_out"), *one = ko != nullptr ? ko : vo;
  if (one == nullptr || one->dim() != 3 || !is_half(*one))
    refuse("k_out and v_out", "float16 or bfloat16 tensors (N, out_len, h_kv*d_head)");
  const at::ScalarType type = one->scalar_type();
  const int64_t n = one->size(1);
  uint16_t* kp = ko != nullptr ? whole<uint16_t>(*ko, "k_out", type, dev, {N, n, h_kv * D}) : nullptr;
  uint16_t* vp = vo != nullptr ? whole<uint16_t>(*vo, "v_out", type, dev, {N, n, h_kv * D}) : nullptr;
  gqa_options opt = {};
  opt.test_stall_cta = -1;
  opt.bf16 = type == at::kBFloat16;
  const Workspace ws = status_word(p[7], dev);
  void* st = stream_of(dev);
  const int num = as_int(N, "N"), blocks = as_int(mb, "max_blocks"), nb = as_int(cache.size(0), "num_blocks"),
            heads = as_int(h_kv, "h_kv"), d = as_int(D, "d_head");
  gqa_status s;
  Py_BEGIN_ALLOW_THREADS
  s = gqa_kv8_read(cache.data_ptr(), tp, lp, bp, kp, vp, num, n, blocks, nb, bs, heads, d, ws.at, ws.bytes, st, &opt);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

// no C++ exception reaches Python
template <PyObject* (*CALL)(PyObject* const*), Py_ssize_t ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, %zd given", ARGS, n);
    return nullptr;
  }
  try {
    return CALL(args);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

template <PyObject* (*CALL)(PyObject* const*), Py_ssize_t ARGS>
PyCFunction function() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<CALL, ARGS>));
}

PyMethodDef kMethods[] = {{"append", function<append, 16>(), METH_FASTCALL, nullptr},
                          {"decode", function<decode, 13>(), METH_FASTCALL, nullptr},
                          {"read", function<read, 8>(), METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", GQA_TORCH) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
