// fsa_torch.cpp -- the marshalling of the serving calls (fsa.h) for torch tensors, as a
// Python extension module: checks of devices, types, shapes and strides, the current
// stream, and the call into libfsa.  A decode step's kernels run for a few microseconds, so
// the Python side of a call has to cost no more; the same checks in Python took 10 to 20 us.
// Nothing is computed or kept here.
#include <Python.h>
#include <cstdarg>
#include <cstdio>
#include <cuda_runtime.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include "fsa.h"

namespace {

PyObject* g_error = nullptr;      // the package's FsaError(status, what)

// Raised as FsaError; caught at the entry points, with everything that torch throws.
struct Refused {
  int status;
  char what[240];
};
[[noreturn]] void refuse(int status, const char* format, ...) {
  Refused r;
  r.status = status;
  va_list args;
  va_start(args, format);
  std::vsnprintf(r.what, sizeof(r.what), format, args);
  va_end(args);
  throw r;
}
[[noreturn]] void invalid(const char* name, const char* what) { refuse(FSA_ERR_INVALID_ARG, "%s %s", name, what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) invalid(name, "must be a tensor");
  return THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) invalid(name, "must be a CUDA tensor");
  return t.get_device();
}

// A [B, S, heads, D] tensor, rows contiguous; an output's rows lie apart.
fsa_strides strided(const at::Tensor& t, const char* name, int device, bool output, at::ScalarType dtype = at::kBFloat16) {
  if (!t.is_cuda() || t.get_device() != device) invalid(name, "must be a CUDA tensor on the call's device");
  if (t.dim() != 4 || t.scalar_type() != dtype) invalid(name, dtype == at::kFloat ? "must be a 4-dimensional fp32 tensor" : "must be a 4-dimensional bf16 tensor");
  if (t.stride(3) != 1 && t.size(3) > 1) invalid(name, "must be contiguous in its last dimension");
  for (int i = 0; i < 3; ++i)
    if (t.size(i) > 1 && (t.stride(i) % 8 != 0 || (output && t.stride(i) == 0)))
      invalid(name, "strides must be multiples of 8, and an output's rows apart");
  return {t.stride(0), t.stride(1), t.stride(2)};
}

void same_shape(const at::Tensor& t, const at::Tensor& u, const char* what) {
  if (t.sizes() != u.sizes()) refuse(FSA_ERR_INVALID_ARG, "%s shapes", what);
}

// Pointer of a contiguous tensor of the given type and shape (None: null).
template <class T>
T* plain(PyObject* o, const char* name, int device, at::ScalarType dtype, at::IntArrayRef shape) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != dtype || t.sizes() != shape || !t.is_contiguous())
    invalid(name, "must be a contiguous CUDA tensor of the call's device, with the type and shape that the call documents");
  return static_cast<T*>(t.data_ptr());
}

long long number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw 0;
  return v;
}
int small_number(PyObject* o) {
  const long long v = number(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(FSA_ERR_INVALID_ARG, "a number is out of range");
  return (int)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw 0;
  return v;
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw 0;
  return v;
}

// The tensors' device as the current one while the call is made, and its stream.
struct Launch {
  c10::cuda::CUDAGuard guard;
  void* stream;
  Launch(int device, PyObject* given)
      : guard((c10::DeviceIndex)device),
        stream(given == Py_None ? (void*)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream()
                                : (void*)(uintptr_t)PyLong_AsUnsignedLongLong(given)) {
    if (PyErr_Occurred()) throw 0;
  }
};

void done(int status, const char* name) {
  if (status != FSA_OK) refuse(status, "%s", name);
}

// (pages, page_size, Hkv, D, fmt) at args[0..4]
struct CacheArg {
  fsa_cache c;
  int device;
  explicit CacheArg(PyObject* const* a) {
    const at::Tensor& pages = tensor(a[0], "pages");
    device = device_of(pages, "pages");
    c = {pages.data_ptr(), pages.size(0), small_number(a[1]), small_number(a[2]), small_number(a[3]), small_number(a[4])};
    size_t bytes = 0;
    done(fsa_cache_page_bytes(c.page_size, c.Hkv, c.D, c.fmt, &bytes), "fsa_cache_page_bytes");
    if (pages.scalar_type() != at::kByte || pages.dim() != 2 || !pages.is_contiguous() || (size_t)pages.size(1) != bytes)
      invalid("pages", "must be a contiguous uint8 tensor [num_pages, fsa_cache_page_bytes]");
  }
};

struct Table {
  const int32_t* at;
  int width;
  Table(PyObject* o, int B, int device) {
    const at::Tensor& t = tensor(o, "block_table");
    if (t.dim() != 2 || t.size(0) != B || t.size(1) > INT32_MAX) invalid("block_table", "must be [B, max_pages]");
    at = plain<int32_t>(o, "block_table", device, at::kInt, t.sizes());
    width = (int)t.size(1);
  }
};

// norm_rope(q, k, pos, inv_freq, sections, q_weight, k_weight, norm, eps, interleaved, q_out, k_out, stream)
PyObject* norm_rope(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &qo = tensor(a[10], "q_out"), &ko = tensor(a[11], "k_out");
  const int dev = device_of(q, "q");
  fsa_norm_rope r{};
  r.q_strides = strided(q, "q", dev, false);
  r.k_strides = strided(k, "k", dev, false);
  r.q_out_strides = strided(qo, "q_out", dev, true);
  r.k_out_strides = strided(ko, "k_out", dev, true);
  same_shape(qo, q, "q_out, q");
  same_shape(ko, k, "k_out, k");
  if (k.size(0) != q.size(0) || k.size(1) != q.size(1) || k.size(3) != q.size(3)) refuse(FSA_ERR_INVALID_ARG, "q, k shapes");
  const int64_t B = q.size(0), S = q.size(1), D = q.size(3);
  if (B > INT32_MAX || S > INT32_MAX || q.size(2) > INT32_MAX || k.size(2) > INT32_MAX) refuse(FSA_ERR_INVALID_ARG, "q, k shapes");
  int64_t half = 0, axes = 1;
  if (a[3] != Py_None) {
    const at::Tensor& f = tensor(a[3], "inv_freq");
    half = f.numel();
    r.inv_freq = plain<double>(a[3], "inv_freq", dev, at::kDouble, {half});
    if (a[2] == Py_None) refuse(FSA_ERR_INVALID_ARG, "a rotation needs pos");
    const at::Tensor& p = tensor(a[2], "pos");
    if (p.dim() == 3) {
      axes = p.size(2);
      r.pos = plain<int32_t>(a[2], "pos", dev, at::kInt, {B, S, axes});
    } else {
      r.pos = plain<int32_t>(a[2], "pos", dev, at::kInt, {B, S});
    }
  }
  if (half > D / 2) refuse(FSA_ERR_INVALID_ARG, "inv_freq has more than D/2 pairs");
  if (a[4] == Py_None) {
    if (axes != 1) refuse(FSA_ERR_INVALID_ARG, "%lld axes need sections", (long long)axes);
    r.sections[0] = (int)half;
  } else {
    if (!PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != axes || axes > 3)
      refuse(FSA_ERR_INVALID_ARG, "sections must be a tuple of one number for each of %lld axes (1 to 3)", (long long)axes);
    for (int i = 0; i < axes; ++i) r.sections[i] = small_number(PyTuple_GET_ITEM(a[4], i));
  }
  r.q = q.data_ptr(); r.k = k.data_ptr(); r.q_out = qo.data_ptr(); r.k_out = ko.data_ptr();
  r.q_weight = plain<void>(a[5], "q_weight", dev, at::kBFloat16, {D});
  r.k_weight = plain<void>(a[6], "k_weight", dev, at::kBFloat16, {D});
  r.B = (int)B; r.S = (int)S; r.H = (int)q.size(2); r.Hkv = (int)k.size(2); r.D = (int)D;
  r.rotary = (int)(2 * half); r.n_axes = (int)axes;
  r.norm = truth(a[7]); r.eps = (float)real(a[8]); r.interleaved = truth(a[9]);
  const Launch on(dev, a[12]);
  done(fsa_qk_norm_rope(&r, on.stream), "fsa_qk_norm_rope");
  Py_RETURN_NONE;
}

// cache_append(pages, page_size, Hkv, D, fmt, k, v, block_table, lens, new_lens, status, stream)
PyObject* cache_append(PyObject* const* a) {
  const CacheArg c(a);
  const at::Tensor &k = tensor(a[5], "k"), &v = tensor(a[6], "v");
  const fsa_strides ks = strided(k, "k", c.device, false), vs = strided(v, "v", c.device, false);
  same_shape(v, k, "k, v");
  if (k.size(2) != c.c.Hkv || k.size(3) != c.c.D || k.size(0) > INT32_MAX || k.size(1) > INT32_MAX) refuse(FSA_ERR_INVALID_ARG, "k, v shapes");
  const int B = (int)k.size(0), S = (int)k.size(1);
  const Table table(a[7], B, c.device);
  if (a[8] == Py_None) invalid("lens", "must be given");
  const int32_t* lens = plain<int32_t>(a[8], "lens", c.device, at::kInt, {B});
  const int32_t* fresh = plain<int32_t>(a[9], "new_lens", c.device, at::kInt, {B});
  int32_t* status = plain<int32_t>(a[10], "status", c.device, at::kInt, {1});
  const Launch on(c.device, a[11]);
  done(fsa_cache_append(&c.c, k.data_ptr(), v.data_ptr(), &ks, &vs, B, S, table.at, table.width, lens, fresh, status, on.stream),
       "fsa_cache_append");
  Py_RETURN_NONE;
}

// cache_read(pages, page_size, Hkv, D, fmt, k_out, v_out, block_table, lens, start, status, stream)
PyObject* cache_read(PyObject* const* a) {
  const CacheArg c(a);
  const at::Tensor* out[2] = {nullptr, nullptr};
  fsa_strides st[2] = {};
  static const char* const names[2] = {"k_out", "v_out"};
  int64_t B = -1, S = -1;
  for (int i = 0; i < 2; ++i) {
    if (a[5 + i] == Py_None) continue;
    out[i] = &tensor(a[5 + i], names[i]);
    st[i] = strided(*out[i], names[i], c.device, true);
    if (B < 0) { B = out[i]->size(0); S = out[i]->size(1); }
    if (out[i]->size(0) != B || out[i]->size(1) != S || out[i]->size(2) != c.c.Hkv || out[i]->size(3) != c.c.D || B > INT32_MAX || S > INT32_MAX)
      invalid(names[i], "must be [B, S, Hkv, D]");
  }
  if (B < 0) refuse(FSA_ERR_INVALID_ARG, "k_out or v_out must be given");
  const Table table(a[7], (int)B, c.device);
  if (a[8] == Py_None) invalid("lens", "must be given");
  const int32_t* lens = plain<int32_t>(a[8], "lens", c.device, at::kInt, {B});
  const int32_t* start = plain<int32_t>(a[9], "start", c.device, at::kInt, {B});
  int32_t* status = plain<int32_t>(a[10], "status", c.device, at::kInt, {1});
  const Launch on(c.device, a[11]);
  done(fsa_cache_read(&c.c, out[0] ? out[0]->data_ptr() : nullptr, out[1] ? out[1]->data_ptr() : nullptr, &st[0], &st[1],
                      (int)B, (int)S, table.at, table.width, lens, start, status, on.stream), "fsa_cache_read");
  Py_RETURN_NONE;
}

// attention_cache(pages, page_size, Hkv, D, fmt, q, out, lse, block_table, lens, q_lens, causal, scale, workspace,
//                 timeout_ms, status, stream); scale None: D^-1/2; workspace None: one of the call's own
PyObject* attention_cache(PyObject* const* a) {
  const CacheArg c(a);
  const at::Tensor &q = tensor(a[5], "q"), &out = tensor(a[6], "out");
  fsa_cache_attn r{};
  r.q_strides = strided(q, "q", c.device, false);
  if (out.scalar_type() != at::kBFloat16 && out.scalar_type() != at::kFloat) invalid("out", "must be bf16 or fp32");
  r.out_strides = strided(out, "out", c.device, true, out.scalar_type());
  same_shape(out, q, "out, q");
  const int64_t B = q.size(0), Sq = q.size(1), H = q.size(2);
  if (q.size(3) != c.c.D || H % c.c.Hkv != 0 || B > INT32_MAX || Sq > INT32_MAX || H > INT32_MAX)
    refuse(FSA_ERR_INVALID_ARG, "q must have the cache's D and a multiple of its heads");
  const Table table(a[8], (int)B, c.device);
  if (a[9] == Py_None) invalid("lens", "must be given");
  r.q = q.data_ptr();
  r.out = out.data_ptr();
  r.lse = plain<float>(a[7], "lse", c.device, at::kFloat, {B, Sq, H});
  r.cache = &c.c;
  r.block_table = table.at;
  r.lens = plain<int32_t>(a[9], "lens", c.device, at::kInt, {B});
  r.q_lens = plain<int32_t>(a[10], "q_lens", c.device, at::kInt, {B});
  r.status = plain<int32_t>(a[15], "status", c.device, at::kInt, {1});
  r.B = (int)B; r.H = (int)H; r.Sq = (int)Sq; r.max_pages = table.width;
  r.causal = truth(a[11]);
  r.out_dtype = out.scalar_type() == at::kBFloat16 ? FSA_OUT_BF16 : FSA_OUT_F32;
  r.scale = a[12] == Py_None ? (c.c.D == 64 ? 0.125f : 0.08838834764831845f) : (float)real(a[12]);
  const long long limit = number(a[14]);
  if (limit < 0 || limit > UINT32_MAX) invalid("timeout_ms", "is out of range");
  r.timeout_ms = (uint32_t)limit;
  const Launch on(c.device, a[16]);
  at::Tensor own;
  if (a[13] == Py_None) {
    size_t need = 0;
    done(fsa_attention_cache_workspace(&c.c, r.B, r.H, r.Sq, r.max_pages, &need), "fsa_attention_cache_workspace");
    if (need > 0) {
      // made on the call's stream, so that what is freed there is used again only behind it
      c10::cuda::OptionalCUDAStreamGuard guard;
      if (a[16] != Py_None) guard.reset_stream(c10::cuda::getStreamFromExternal((cudaStream_t)on.stream, (c10::DeviceIndex)c.device));
      own = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)c.device));
      r.workspace = own.data_ptr();
      r.workspace_bytes = need;
    }
  } else {
    const at::Tensor& ws = tensor(a[13], "workspace");
    r.workspace = plain<void>(a[13], "workspace", c.device, at::kByte, {ws.numel()});
    r.workspace_bytes = (size_t)ws.numel();
  }
  done(fsa_attention_cache(&r, on.stream), "fsa_attention_cache");
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", r.status, r.what) : nullptr;
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_SetString(PyExc_RuntimeError, r.what);
    }
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

#define FSA_ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FSA_ENTRY(norm_rope, 13), FSA_ENTRY(cache_append, 12), FSA_ENTRY(cache_read, 12),
                         FSA_ENTRY(attention_cache, 17), {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fsa_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fsa_torch(void) { return PyModule_Create(&module); }
