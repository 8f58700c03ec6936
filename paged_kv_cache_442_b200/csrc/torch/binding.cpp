// Marshalling of the rotary and block-scale entry points for Python (_pa_torch.so): checks of
// torch tensors, then one call of the C entry point in libpa.so. A decode step's launches take
// a few microseconds of GPU time each, less than the same checks cost as Python statements
// (13 - 22 us a call measured through ctypes), so they are made on the tensors directly here.
// Every function takes its arguments by position and returns the entry point's status; what is
// wrong with an argument raises TypeError or ValueError, as the rest of the binding does.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "pa.h"

namespace {

struct Error {
  PyObject* type;
  std::string what;
};
[[noreturn]] void type_error(std::string what) { throw Error{PyExc_TypeError, std::move(what)}; }
[[noreturn]] void value_error(std::string what) { throw Error{PyExc_ValueError, std::move(what)}; }
// a Python error is already set
struct Raised {};

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

// The tensors of one call, all on the current device.
class Call {
 public:
  const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType dtype, const char* dtype_name,
                           int64_t ndim) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda())
      value_error(std::string(name) + " must be a CUDA tensor (the library has no CPU path)");
    if (dtype != at::ScalarType::Undefined && t.scalar_type() != dtype)
      type_error(std::string(name) + " must be " + dtype_name + ", got " + c10::toString(t.scalar_type()));
    if (ndim >= 0 && t.dim() != ndim)
      value_error(std::string(name) + " must have " + std::to_string(ndim) + " dims, got " +
                  std::to_string(t.dim()));
    if (device_ < 0) device_ = c10::cuda::current_device();
    if (t.get_device() != device_)
      value_error(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                  ", the current device is cuda:" + std::to_string(device_));
    return t;
  }
  const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType dtype, const char* dtype_name,
                          int64_t ndim) {
    const at::Tensor& t = tensor(o, name, dtype, dtype_name, ndim);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t;
  }
  const at::Tensor& bf16(PyObject* o, const char* name, int64_t ndim) {
    return dense(o, name, at::kBFloat16, "torch.bfloat16", ndim);
  }
  const at::Tensor& i32(PyObject* o, const char* name, int64_t ndim) {
    return dense(o, name, at::kInt, "torch.int32", ndim);
  }
  const at::Tensor& f32(PyObject* o, const char* name, int64_t ndim) {
    return dense(o, name, at::kFloat, "torch.float32", ndim);
  }
  const at::Tensor& u8(PyObject* o, const char* name, int64_t ndim) {
    return dense(o, name, at::kByte, "torch.uint8", ndim);
  }

  // bf16 [tokens, heads, dim] whose tokens' rows are dense, the tokens any stride apart.
  // Negative expectations are not checked.
  struct Rows {
    void* p = nullptr;
    int64_t stride = 0, tokens = 0, heads = 0, dim = 0;
  };
  Rows rows(PyObject* o, const char* name, int64_t tokens, int64_t heads, int64_t dim) {
    const at::Tensor& t = tensor(o, name, at::kBFloat16, "torch.bfloat16", 3);
    Rows r{t.data_ptr(), 0, t.size(0), t.size(1), t.size(2)};
    if ((tokens >= 0 && r.tokens != tokens) || (heads >= 0 && r.heads != heads) ||
        (dim >= 0 && r.dim != dim)) {
      auto want = [](int64_t n, const char* any) { return n >= 0 ? std::to_string(n) : std::string(any); };
      value_error(std::string(name) + " has shape " + shape_of(t) + ", expected [" +
                  want(tokens, "tokens") + ", " + want(heads, "heads") + ", " + want(dim, "dim") + "]");
    }
    if ((r.dim > 1 && t.stride(2) != 1) || (r.heads > 1 && t.stride(1) != r.dim))
      value_error(std::string(name) + ": each token's heads must be contiguous");
    r.stride = r.tokens > 1 ? t.stride(0) : (r.heads * r.dim + 7) / 8 * 8;
    return r;
  }

  void* stream(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream();
    if (PyLong_Check(o)) return integer_pointer(o);
    PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
    if (!raw) throw Raised{};
    void* p = integer_pointer(raw);
    Py_DECREF(raw);
    return p;
  }

 private:
  static void* integer_pointer(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
  }
  int device_ = -1;
};

int32_t int_of(PyObject* o, const char* name) {
  PyObject* i = PyNumber_Index(o);
  if (!i) throw Raised{};
  const long long v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}

int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(n);
}

float float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}

pa_rope_desc rope_of(Call& c, PyObject* inv_freq, PyObject* interleaved, PyObject* amplitude) {
  const at::Tensor& f = c.f32(inv_freq, "inv_freq", 1);
  const int inter = PyObject_IsTrue(interleaved);
  if (inter < 0) throw Raised{};
  return pa_rope_desc{f.numel() ? static_cast<const float*>(f.data_ptr()) : nullptr,
                      size32(2 * f.numel(), "inv_freq"), inter, float_of(amplitude)};
}

const int32_t* positions_of(Call& c, PyObject* o, int64_t tokens) {
  const at::Tensor& t = c.i32(o, "positions", 1);
  if (t.size(0) != tokens) value_error("positions must be [num_tokens]");
  return static_cast<const int32_t*>(t.data_ptr());
}

// q_out, q (both may be None), k and v of a step.
struct Step {
  Call::Rows q_out, q, k, v;
};
Step step_of(Call& c, PyObject* const* a, int64_t hkv, int64_t d) {
  Step s;
  s.k = c.rows(a[2], "k", -1, hkv, d);
  s.v = c.rows(a[3], "v", s.k.tokens, hkv, d);
  if ((a[0] == Py_None) != (a[1] == Py_None)) value_error("q and q_out come together");
  if (a[1] != Py_None) {
    s.q = c.rows(a[1], "q", s.k.tokens, -1, d);
    s.q_out = c.rows(a[0], "q_out", s.k.tokens, s.q.heads, d);
  }
  return s;
}

struct Pools {
  pa_cache_desc desc;
  void *k, *v;
  float *ks, *vs;
};
pa_cache_desc desc_of(const at::Tensor& pool) {
  return pa_cache_desc{size32(pool.size(0), "num_blocks"), size32(pool.size(1), "block_size"),
                       size32(pool.size(2), "num_kv_heads"), size32(pool.size(3), "head_dim")};
}
Pools pools_of(Call& c, PyObject* const* a) {  // k_codes, v_codes, k_scales, v_scales
  const at::Tensor& k = c.u8(a[0], "k_codes", 4);
  const at::Tensor& v = c.u8(a[1], "v_codes", 4);
  const at::Tensor& ks = c.f32(a[2], "k_scales", 2);
  const at::Tensor& vs = c.f32(a[3], "v_scales", 2);
  if (!k.sizes().equals(v.sizes())) value_error("K and V pools must have the same shapes");
  for (const at::Tensor* s : {&ks, &vs})
    if (s->size(0) != k.size(0) || s->size(1) != k.size(2))
      value_error("scales must be [num_blocks, num_kv_heads] fp32");
  return Pools{desc_of(k), k.data_ptr(), v.data_ptr(), static_cast<float*>(ks.data_ptr()),
               static_cast<float*>(vs.data_ptr())};
}

// Runs `body` (checks, then the entry point without the interpreter's lock held).
template <class Body>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, Body body) {
  try {
    if (nargs != want) type_error("expected " + std::to_string(want) + " arguments");
    return PyLong_FromLong(body());
  } catch (const Raised&) {
  } catch (const Error& e) {
    PyErr_SetString(e.type, e.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

template <class Entry, class... A>
pa_status unlocked(Entry entry, A... args) {
  PyThreadState* state = PyEval_SaveThread();
  const pa_status st = entry(args...);
  PyEval_RestoreThread(state);
  return st;
}

// out, x, positions, inv_freq, interleaved, amplitude, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    Call c;
    const auto x = c.rows(a[1], "x", -1, -1, -1);
    const auto out = c.rows(a[0], "out", x.tokens, x.heads, x.dim);
    const int32_t* pos = positions_of(c, a[2], x.tokens);
    const pa_rope_desc r = rope_of(c, a[3], a[4], a[5]);
    return unlocked(pa_rope, out.p, out.stride, x.p, x.stride, size32(x.tokens, "x"),
                    size32(x.heads, "x"), size32(x.dim, "x"), pos, r, c.stream(a[6]));
  });
}

// q_out, q, k, v, k_cache, v_cache, slot_mapping, positions, inv_freq, interleaved, amplitude,
// stream
PyObject* rope_store_kvcache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    Call c;
    const at::Tensor& kc = c.bf16(a[4], "k_cache", 4);
    const at::Tensor& vc = c.bf16(a[5], "v_cache", 4);
    if (!kc.sizes().equals(vc.sizes())) value_error("k_cache/v_cache shapes must match");
    const Step s = step_of(c, a, kc.size(2), kc.size(3));
    const at::Tensor& slots = c.i32(a[6], "slot_mapping", 1);
    if (slots.size(0) != s.k.tokens) value_error("slot_mapping must be [num_tokens]");
    const int32_t* pos = positions_of(c, a[7], s.k.tokens);
    const pa_rope_desc r = rope_of(c, a[8], a[9], a[10]);
    return unlocked(pa_rope_store_kvcache, s.q_out.p, s.q_out.stride, s.q.p, s.q.stride, s.k.p,
                    s.k.stride, s.v.p, s.v.stride, kc.data_ptr(), vc.data_ptr(), desc_of(kc),
                    static_cast<const int32_t*>(slots.data_ptr()), size32(s.k.tokens, "k"),
                    size32(s.q.heads, "q"), pos, r, c.stream(a[11]));
  });
}

struct Batch {
  const int32_t *tables, *cu, *ctx;
  int32_t width, seqs;
};
Batch batch_of(Call& c, PyObject* const* a) {  // block_tables, cu_seqlens_q, context_lens
  const at::Tensor& bt = c.i32(a[0], "block_tables", 2);
  const at::Tensor& cu = c.i32(a[1], "cu_seqlens_q", 1);
  const at::Tensor& ctx = c.i32(a[2], "context_lens", 1);
  if (cu.size(0) != bt.size(0) + 1 || ctx.size(0) != bt.size(0))
    value_error("cu_seqlens_q/block_tables/context_lens disagree on num_seqs");
  return Batch{static_cast<const int32_t*>(bt.data_ptr()), static_cast<const int32_t*>(cu.data_ptr()),
               static_cast<const int32_t*>(ctx.data_ptr()), size32(bt.size(1), "block_tables"),
               size32(bt.size(0), "block_tables")};
}

// k, v, k_codes, v_codes, k_scales, v_scales, block_tables, cu_seqlens_q, context_lens,
// max_q_len, stream
PyObject* store_blockscale(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    Call c;
    const Pools p = pools_of(c, a + 2);
    PyObject* const rows[4] = {Py_None, Py_None, a[0], a[1]};
    const Step s = step_of(c, rows, p.desc.num_kv_heads, p.desc.head_dim);
    const Batch b = batch_of(c, a + 6);
    return unlocked(pa_store_kvcache_fp8_blockscale, s.k.p, s.k.stride, s.v.p, s.v.stride, p.k, p.v,
                    p.ks, p.vs, p.desc, b.tables, b.width, b.cu, b.ctx, b.seqs,
                    size32(s.k.tokens, "k"), int_of(a[9], "max_q_len"), c.stream(a[10]));
  });
}

// q_out, q, k, v, k_codes, v_codes, k_scales, v_scales, block_tables, cu_seqlens_q,
// context_lens, max_q_len, positions, inv_freq, interleaved, amplitude, stream
PyObject* rope_store_blockscale(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    Call c;
    const Pools p = pools_of(c, a + 4);
    const Step s = step_of(c, a, p.desc.num_kv_heads, p.desc.head_dim);
    const Batch b = batch_of(c, a + 8);
    const int32_t max_q = int_of(a[11], "max_q_len");
    const int32_t* pos = positions_of(c, a[12], s.k.tokens);
    const pa_rope_desc r = rope_of(c, a[13], a[14], a[15]);
    return unlocked(pa_rope_store_kvcache_fp8_blockscale, s.q_out.p, s.q_out.stride, s.q.p, s.q.stride,
                    s.k.p, s.k.stride, s.v.p, s.v.stride, p.k, p.v, p.ks, p.vs, p.desc, b.tables,
                    b.width, b.cu, b.ctx, b.seqs, size32(s.k.tokens, "k"), max_q,
                    size32(s.q.heads, "q"), pos, r, c.stream(a[16]));
  });
}

// out, q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, scale,
// max_context_len, workspace, stream
PyObject* decode_blockscale(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    Call c;
    const at::Tensor& out = c.bf16(a[0], "out", 3);
    const at::Tensor& q = c.bf16(a[1], "q", 3);
    const Pools p = pools_of(c, a + 2);
    const at::Tensor& bt = c.i32(a[6], "block_tables", 2);
    const at::Tensor& ctx = c.i32(a[7], "context_lens", 1);
    if (!out.sizes().equals(q.sizes()) || bt.size(0) != q.size(0) || ctx.size(0) != q.size(0))
      value_error("out/q/block_tables/context_lens disagree on num_seqs");
    if (q.size(2) != p.desc.head_dim) value_error("q and the pools must have the same head dim");
    const at::Tensor& ws = c.dense(a[10], "workspace", at::ScalarType::Undefined, "", -1);
    return unlocked(pa_decode_fp8_blockscale, out.data_ptr(), q.data_ptr(), p.k, p.v, p.ks, p.vs, p.desc,
                    static_cast<const int32_t*>(bt.data_ptr()), size32(bt.size(1), "block_tables"),
                    static_cast<const int32_t*>(ctx.data_ptr()), size32(q.size(0), "q"),
                    size32(q.size(1), "q"), float_of(a[8]), int_of(a[9], "max_context_len"),
                    ws.data_ptr(), ws.nbytes(), c.stream(a[11]));
  });
}

#define PA_FN(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_FN(rope),
                         PA_FN(rope_store_kvcache),
                         PA_FN(store_blockscale),
                         PA_FN(rope_store_blockscale),
                         PA_FN(decode_blockscale),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_torch", "tensor marshalling of libpa.so", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The torch and the Python of this build, for build.py, which finds it in the file.
extern "C" __attribute__((used, visibility("default"))) const char pa_built_for[] = "pa_built_for{" PA_BUILT_FOR "}";

PyMODINIT_FUNC PyInit__pa_torch(void) { return PyModule_Create(&module); }
