// Python binding of the paged-cache calls: checks the tensors, makes the
// outputs that were not given and calls the C ABI on the current stream.
//
// A serving step makes these calls once per layer, and a small one takes 4 to 11 us on
// the GPU; through ctypes the checks and the 20 to 34 converted arguments took
// 15, 18 and 30 us on the host, launches included. Here a call takes 4, 3 and 5.5 with
// its outputs given, 10 (six of them), 5 and 7.5 with outputs made. Module
// functions take positional arguments only (the Python functions of the package
// hold the names, defaults and documentation) and return the result, or the
// gdn_status as an int where the C entry point refused the call.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "gdn.h"

namespace {

decltype(&gdn_page_plan) page_plan_fn = nullptr;
decltype(&gdn_qk_norm_rope) norm_rope_fn = nullptr;
decltype(&gdn_paged_attention_decode) decode_fn = nullptr;
decltype(&gdn_paged_attention_decode_workspace) decode_workspace_fn = nullptr;

struct Refusal {
  PyObject* type;
  std::string text;
};
[[noreturn]] void refuse(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }

std::string text(at::IntArrayRef v) {
  std::ostringstream s;
  s << '(';
  for (size_t i = 0; i < v.size(); ++i) s << (i ? ", " : "") << v[i];
  s << (v.size() == 1 ? ",)" : ")");
  return s.str();
}
std::string text(at::ScalarType t) {
  std::string s = c10::toString(t);
  if (s == "BFloat16") return "torch.bfloat16";
  if (s == "Half") return "torch.float16";
  if (s == "Float") return "torch.float32";
  if (s == "Double") return "torch.float64";
  if (s == "Int") return "torch.int32";
  if (s == "Long") return "torch.int64";
  return s;
}

// arguments ---------------------------------------------------------------
const at::Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o))
    throw Refusal{PyExc_TypeError, std::string(name) + ": a torch.Tensor is needed"};
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor_or_none(o, name);
  if (!t) throw Refusal{PyExc_TypeError, std::string(name) + ": a torch.Tensor is needed"};
  return *t;
}
struct PythonError {};
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
int integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + ": out of range");
  return (int)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
bool dtype_or_none(PyObject* o, at::ScalarType& t) {
  if (o == Py_None) return false;
  if (!THPDtype_Check(o)) throw Refusal{PyExc_TypeError, "a torch.dtype is needed"};
  t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  return true;
}

// checks ------------------------------------------------------------------
gdn_dtype code(at::ScalarType t, const char* name) {
  if (t == at::kBFloat16) return GDN_BF16;
  if (t == at::kHalf) return GDN_F16;
  if (t == at::kFloat) return GDN_F32;
  throw Refusal{PyExc_TypeError, std::string(name) + ": unsupported dtype " + text(t) +
                                     "; use torch.bfloat16, float16 or float32"};
}
bool half_type(at::ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }

void expect(const at::Tensor& t, at::IntArrayRef shape, const char* name, at::ScalarType type) {
  if (t.sizes() != shape)
    refuse(std::string(name) + ": shape " + text(t.sizes()) + ", expected " + text(shape));
  if (t.scalar_type() != type)
    refuse(std::string(name) + ": dtype " + text(t.scalar_type()) + ", expected " + text(type));
}
void dense(const at::Tensor* t, at::IntArrayRef shape, const char* name, at::ScalarType type) {
  if (!t) return;
  expect(*t, shape, name, type);
  if (!t->is_contiguous()) refuse(std::string(name) + " must be contiguous");
}
// row stride of an int32 [N, M] tensor with dense rows
int64_t rows32(const at::Tensor& t, int64_t N, const char* name) {
  if (t.dim() != 2 || t.size(0) != N)
    refuse(std::string(name) + ": shape " + text(t.sizes()) + ", expected (" +
           std::to_string(N) + ", max_pages)");
  if (t.scalar_type() != at::kInt)
    refuse(std::string(name) + ": dtype " + text(t.scalar_type()) + ", expected torch.int32");
  if (t.size(1) > INT32_MAX) refuse(std::string(name) + ": rows too long");
  if (t.stride(1) != 1 && t.size(1) > 1) refuse(std::string(name) + ": rows must be contiguous");
  return N > 1 ? t.stride(0) : t.size(1);              // one row: no stride is used
}
struct CacheStrides { int64_t page, token, head; };
// strides of a [pages, page_size, H_kv, D] cache view
CacheStrides cache(const at::Tensor& t, at::IntArrayRef shape, const char* name,
                   at::ScalarType type) {
  expect(t, shape, name, type);
  if (t.stride(3) != 1)
    refuse(std::string(name) + ": each row of " + std::to_string(shape[3]) +
           " values must be contiguous");
  // the stride of a dimension of one is never used
  auto at = [&](int i) { return shape[i] > 1 ? t.stride(i) : shape[3]; };
  return {at(0), at(1), at(2)};
}
// row stride of [n, H, D] with dense heads
int64_t heads(const at::Tensor& t, at::IntArrayRef shape, const char* name, at::ScalarType type) {
  expect(t, shape, name, type);
  if (t.stride(2) != 1 || (t.stride(1) != shape[2] && shape[1] != 1))
    refuse(std::string(name) + ": trailing dimensions must be contiguous");
  return shape[0] > 1 ? t.stride(0) : shape[1] * shape[2];
}
void three_dims(const at::Tensor& t, const char* name) {
  if (t.dim() != 3)
    refuse(std::string(name) + ": " + std::to_string(t.dim()) + " dimensions, expected [T, H, D]");
}
int narrow(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + ": too large");
  return (int)v;
}

// the CUDA device that all given tensors are on
template <class... T>
c10::Device one_device(const T*... all) {
  const at::Tensor* first = nullptr;
  for (const at::Tensor* t : {static_cast<const at::Tensor*>(all)...}) {
    if (!t) continue;
    if (!t->is_cuda()) refuse("libgdn takes CUDA tensors only (no CPU path)");
    if (!first) first = t;
    if (t->device() != first->device())
      refuse("tensors on " + first->device().str() + " and " + t->device().str() +
             ": one device is needed");
  }
  return first->device();
}
// The address of a tensor's values; null for none. Tensors that only stand for others
// throw here, or have none, which must not pass for an argument that was left out.
void* addr(const at::Tensor* t) {
  if (!t) return nullptr;
  void* p = t->data_ptr();
  if (!p && t->numel() > 0) refuse("a tensor without memory");
  return p;
}
const int32_t* ints(const at::Tensor* t) { return static_cast<const int32_t*>(addr(t)); }

// result, or what Python is to raise
template <class F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed", want);
    return nullptr;
  }
  try {
    return body(args);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const PythonError&) {
  } catch (...) {
    // torch's own, as torch raises them (out of memory among them), and Python's
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}
// the C entry point without the interpreter's lock: a launch can wait for room in the
// queue. The call must not throw: addresses are taken before it.
template <class F>
gdn_status unlocked(F call) {
  gdn_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  return st;
}
PyObject* status(gdn_status st) { return PyLong_FromLong((long)st); }

// entry points -------------------------------------------------------------

// lens, want, block_table, free_pages, free_count, page_size, token_capacity (-1: slot_map's),
// new_lens, cu_new, slot_map, positions, new_count, info
PyObject* page_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 13, [](PyObject* const* v) -> PyObject* {
    const at::Tensor& lens = tensor(v[0], "lens");
    const at::Tensor& want = tensor(v[1], "want");
    const at::Tensor& table = tensor(v[2], "block_table");
    const at::Tensor& free_pages = tensor(v[3], "free_pages");
    const at::Tensor& free_count = tensor(v[4], "free_count");
    const int page = integer32(v[5], "page_size");
    int64_t capacity = integer(v[6]);
    const char* names[] = {"new_lens", "cu_new", "slot_map", "positions", "new_count", "info"};
    const at::Tensor* given[6];
    for (int i = 0; i < 6; ++i) given[i] = tensor_or_none(v[7 + i], names[i]);
    const int64_t N = lens.numel(), P = free_pages.numel();
    if (given[2]) {
      if (capacity >= 0 && capacity != given[2]->numel())
        refuse("token_capacity is not slot_map's length");
      capacity = given[2]->numel();
    }
    if (capacity < 0) refuse("give token_capacity or slot_map");
    // before outputs of that size are made
    if (capacity > (int64_t)1 << 30) return status(GDN_ERR_INVALID_ARG);
    dense(&lens, {N}, "lens", at::kInt);
    dense(&want, {N}, "want", at::kInt);
    const int64_t row = rows32(table, N, "block_table");
    dense(&free_pages, {P}, "free_pages", at::kInt);
    dense(&free_count, {1}, "free_count", at::kInt);
    const int64_t sizes[] = {N, N + 1, capacity, capacity, 1, 4};
    for (int i = 0; i < 6; ++i) dense(given[i], {sizes[i]}, names[i], at::kInt);
    const c10::Device dev = one_device(&lens, &want, &table, &free_pages, &free_count, given[0],
                                       given[1], given[2], given[3], given[4], given[5]);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor out[6];
    int32_t* o[6];
    for (int i = 0; i < 6; ++i) {
      out[i] = given[i] ? *given[i]
                        : at::empty({sizes[i]}, at::TensorOptions().dtype(at::kInt).device(dev));
      o[i] = static_cast<int32_t*>(addr(&out[i]));
    }
    const int n32 = narrow(N, "lens"), p32 = narrow(P, "free_pages");
    const int width = (int)table.size(1);
    const int32_t *lens_p = ints(&lens), *want_p = ints(&want), *count_p = ints(&free_count);
    int32_t *table_p = static_cast<int32_t*>(addr(&table)),
            *free_p = static_cast<int32_t*>(addr(&free_pages));
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    const gdn_status st = unlocked([&] {
      return page_plan_fn(lens_p, want_p, n32, table_p, row, width, free_p, count_p, p32, page,
                          capacity, o[0], o[1], o[2], o[3], o[4], o[5], stream);
    });
    if (st != GDN_OK) return status(st);
    PyObject* r = PyTuple_New(6);
    if (!r) return nullptr;
    for (int i = 0; i < 6; ++i) {
      PyObject* t = given[i] ? Py_NewRef(v[7 + i]) : THPVariable_Wrap(std::move(out[i]));
      if (!t) {
        Py_DECREF(r);
        return nullptr;
      }
      PyTuple_SET_ITEM(r, i, t);
    }
    return r;
  });
}

// q, k, v, k_cache, v_cache, slot_map, q_norm_w, k_norm_w, positions, inv_freq, interleaved,
// rope_scale, eps, q_out, out_dtype
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 15, [](PyObject* const* a) -> PyObject* {
    const at::Tensor* q = tensor_or_none(a[0], "q");
    const at::Tensor* k = tensor_or_none(a[1], "k");
    const at::Tensor* v = tensor_or_none(a[2], "v");
    const at::Tensor* kc = tensor_or_none(a[3], "k_cache");
    const at::Tensor* vc = tensor_or_none(a[4], "v_cache");
    const at::Tensor* slots = tensor_or_none(a[5], "slot_map");
    const at::Tensor* wq = tensor_or_none(a[6], "q_norm_w");
    const at::Tensor* wk = tensor_or_none(a[7], "k_norm_w");
    const at::Tensor* pos = tensor_or_none(a[8], "positions");
    const at::Tensor* inv = tensor_or_none(a[9], "inv_freq");
    const int interleaved = PyObject_IsTrue(a[10]);
    if (interleaved < 0) throw PythonError{};
    const float scale = (float)real(a[11]), eps = (float)real(a[12]);
    const at::Tensor* q_out = tensor_or_none(a[13], "q_out");
    at::ScalarType out_type = at::kHalf;
    const bool out_given = dtype_or_none(a[14], out_type);
    const at::Tensor* x = q ? q : k;
    if (!x || !k != !v || !k != !kc || !k != !vc)
      refuse("give q, or k and v with both caches, or all");
    three_dims(*x, "q, k, v");
    const int64_t T = x->size(0), D = x->size(2);
    const at::ScalarType type = x->scalar_type();
    int64_t Hq = 0, Hkv = 0, P = 0, page = 0, qs = 0, ks = 0, vs = 0;
    CacheStrides kstr{0, 0, 0}, vstr{0, 0, 0};
    if (q) {
      Hq = q->size(1);
      qs = heads(*q, {T, Hq, D}, "q", type);
    } else if (q_out) {
      refuse("q_out without q");
    }
    if (k) {
      three_dims(*k, "k");
      Hkv = k->size(1);
      ks = heads(*k, {T, Hkv, D}, "k", type);
      vs = heads(*v, {T, Hkv, D}, "v", type);
      if (kc->dim() != 4)
        refuse("k_cache: shape " + text(kc->sizes()) +
               ", expected [num_pages, page_size, H_kv, D]");
      P = kc->size(0);
      page = kc->size(1);
      kstr = cache(*kc, {P, page, Hkv, D}, "k_cache", kc->scalar_type());
      vstr = cache(*vc, {P, page, Hkv, D}, "v_cache", kc->scalar_type());
      if (out_given && out_type != kc->scalar_type())
        refuse("out_dtype " + text(out_type) + ": q_out has the caches' dtype");
      out_type = kc->scalar_type();
    } else if (!out_given && q_out) {
      out_type = q_out->scalar_type();
    }
    if (!half_type(out_type))
      refuse("caches and q_out are bf16 or fp16, got " + text(out_type));
    dense(q_out, {T, Hq, D}, "q_out", out_type);
    const at::Tensor* w = wq ? wq : wk;
    if (w) {
      dense(wq, {D}, "q_norm_w", w->scalar_type());
      dense(wk, {D}, "k_norm_w", w->scalar_type());
    }
    dense(slots, {T}, "slot_map", at::kInt);
    int64_t R = 0;
    int axes = 1;
    if (inv) {
      if (!pos) refuse("rotary needs positions");
      R = 2 * inv->numel();
      dense(inv, {R / 2}, "inv_freq", at::kDouble);
      if (pos->dim() == 1) {
        dense(pos, {T}, "positions", at::kInt);
      } else {
        axes = 3;
        dense(pos, {3, T}, "positions", at::kInt);
      }
    } else if (pos) {
      refuse("positions without inv_freq");
    }
    const c10::Device dev = one_device(x, k, v, kc, vc, slots, wq, wk, pos, inv, q_out);
    const gdn_dtype xd = code(type, "q, k, v"),
                    wd = w ? code(w->scalar_type(), "norm weights") : GDN_F32;
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor made;
    if (q && !q_out) {
      made = at::empty({T, Hq, D}, at::TensorOptions().dtype(out_type).device(dev));
      q_out = &made;
    }
    const int hq = narrow(Hq, "H_q"), hkv = narrow(Hkv, "H_kv"), d = narrow(D, "head_dim"),
              r = narrow(R, "rope_dims"), p = narrow(P, "num_pages"), ps = narrow(page, "page_size");
    const gdn_dtype out_code = code(out_type, "q_out");
    const void *q_p = addr(q), *k_p = addr(k), *v_p = addr(v), *wq_p = addr(wq), *wk_p = addr(wk);
    void *out_p = addr(q_out), *kc_p = addr(kc), *vc_p = addr(vc);
    const int32_t *pos_p = ints(pos), *slots_p = ints(slots);
    const double* inv_p = static_cast<const double*>(addr(inv));
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    const gdn_status st = unlocked([&] {
      return norm_rope_fn(q_p, qs, k_p, ks, v_p, vs, xd, wq_p, wk_p, wd, eps, pos_p, axes, inv_p, r,
                          interleaved, scale, slots_p, T, hq, hkv, d, out_p, kc_p, kstr.page,
                          kstr.token, kstr.head, vc_p, vstr.page, vstr.token, vstr.head, p, ps,
                          out_code, stream);
    });
    if (st != GDN_OK) return status(st);
    if (!q) Py_RETURN_NONE;
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[13]);
  });
}

// q, k_cache, v_cache, block_table, kv_lens, gate, scale (None: D ** -0.5), o, o_dtype, lse,
// workspace
PyObject* paged_attention_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 11, [](PyObject* const* a) -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const at::Tensor& kc = tensor(a[1], "k_cache");
    const at::Tensor& vc = tensor(a[2], "v_cache");
    const at::Tensor& table = tensor(a[3], "block_table");
    const at::Tensor& lens = tensor(a[4], "kv_lens");
    const at::Tensor* gate = tensor_or_none(a[5], "gate");
    const at::Tensor* o = tensor_or_none(a[7], "o");
    at::ScalarType o_type = at::kBFloat16;
    const bool o_given = dtype_or_none(a[8], o_type);
    const at::Tensor* lse = tensor_or_none(a[9], "lse");
    const at::Tensor* ws = tensor_or_none(a[10], "workspace");
    if (q.dim() != 3 || kc.dim() != 4)
      refuse("q: shape " + text(q.sizes()) + ", expected [N, H_q, D]; k_cache: shape " +
             text(kc.sizes()) + ", expected [num_pages, page_size, H_kv, D]");
    const at::ScalarType type = kc.scalar_type();
    const int64_t N = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = kc.size(2);
    if (!half_type(type)) refuse("caches are bf16 or fp16, got " + text(type));
    if (kc.size(3) != D)
      refuse("k_cache: head dim " + std::to_string(kc.size(3)) + ", q has " + std::to_string(D));
    const CacheStrides ks = cache(kc, kc.sizes(), "k_cache", type);
    const CacheStrides vs = cache(vc, kc.sizes(), "v_cache", type);
    const int64_t qs = heads(q, q.sizes(), "q", type);
    const int64_t row = rows32(table, N, "block_table");
    dense(&lens, {N}, "kv_lens", at::kInt);
    const int64_t gs = gate ? heads(*gate, q.sizes(), "gate", at::kBFloat16) : 0;
    if (o) {
      if (o_given && o_type != o->scalar_type())
        refuse("o: dtype " + text(o->scalar_type()) + ", expected " + text(o_type));
      o_type = o->scalar_type();
      dense(o, q.sizes(), "o", o_type);
    }
    const gdn_dtype od = code(o_type, "o"), kv_code = code(type, "caches");
    dense(lse, {N, Hq}, "lse", at::kFloat);
    const float scale = a[6] == Py_None ? 1.0f / sqrtf((float)D) : (float)real(a[6]);
    if (ws && !ws->is_contiguous()) refuse("workspace must be contiguous");
    const c10::Device dev = one_device(&q, &kc, &vc, &table, &lens, gate, o, lse, ws);
    const c10::cuda::CUDAGuard guard(dev);
    const int hq = narrow(Hq, "H_q"), hkv = narrow(Hkv, "H_kv"), d = narrow(D, "head_dim"),
              n32 = narrow(N, "N"), p = narrow(kc.size(0), "num_pages"),
              ps = narrow(kc.size(1), "page_size");
    at::Tensor made, made_ws;
    if (!o) {
      made = at::empty(q.sizes(), at::TensorOptions().dtype(o_type).device(dev));
      o = &made;
    }
    if (!ws) {
      const int64_t need = (int64_t)decode_workspace_fn(hq, hkv, d);
      made_ws = at::empty({need > 256 ? need : 256},
                          at::TensorOptions().dtype(at::kByte).device(dev));
      ws = &made_ws;
    }
    const void *q_p = addr(&q), *kc_p = addr(&kc), *vc_p = addr(&vc), *gate_p = addr(gate);
    void *o_p = addr(o), *ws_p = addr(ws);
    const int32_t *table_p = ints(&table), *lens_p = ints(&lens);
    float* lse_p = static_cast<float*>(addr(lse));
    const int width = (int)table.size(1);
    const size_t ws_bytes = ws->nbytes();
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    const gdn_status st = unlocked([&] {
      return decode_fn(q_p, qs, kc_p, ks.page, ks.token, ks.head, vc_p, vs.page, vs.token, vs.head,
                       kv_code, p, ps, table_p, row, width, lens_p, gate_p, gs, n32, hq, hkv, d,
                       scale, o_p, od, lse_p, ws_p, ws_bytes, stream);
    });
    if (st != GDN_OK) return status(st);
    return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[7]);
  });
}

// The addresses of the C entry points, in the order of the pointers above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 4, [](PyObject* const* v) -> PyObject* {
    page_plan_fn = reinterpret_cast<decltype(page_plan_fn)>(integer(v[0]));
    norm_rope_fn = reinterpret_cast<decltype(norm_rope_fn)>(integer(v[1]));
    decode_fn = reinterpret_cast<decltype(decode_fn)>(integer(v[2]));
    decode_workspace_fn = reinterpret_cast<decltype(decode_workspace_fn)>(integer(v[3]));
    Py_RETURN_NONE;
  });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(bind), METH_FASTCALL, nullptr},
    {"page_plan", reinterpret_cast<PyCFunction>(page_plan), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(qk_norm_rope), METH_FASTCALL, nullptr},
    {"paged_attention_decode", reinterpret_cast<PyCFunction>(paged_attention_decode),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged(void) {
  PyObject* m = PyModule_Create(&module);
  // the torch it was compiled against; the package compares it with the one it runs on
  if (m && PyModule_AddStringConstant(m, "built_for", GDN_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
