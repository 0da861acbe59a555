// Python entry of the 8-bit cache's calls: argument marshalling only.
//
// These calls take a few microseconds on the GPU, less than checking their
// tensors one attribute at a time in Python takes on the host (a decode step's
// write: 2.1 us on the GPU; 8.9 us a call through ctypes, 3.2 to 3.7 through
// this module).  Every function checks its tensors (type, device, density, shape),
// reads their addresses, and calls the C ABI on the given stream or the current
// one.  It returns the C ABI's code, or kRecheck for arguments that are not what
// the call takes: the Python side then goes through them for its message.
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "pkv.h"

namespace {

constexpr long kRecheck = 1;

// A dense tensor of this type on device `index` (nullptr: it is not).
const at::Tensor *dense(PyObject *o, at::ScalarType type, int index) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor &t = THPVariable_Unpack(o);
  return t.scalar_type() == type && t.get_device() == index && t.is_contiguous() ? &t : nullptr;
}

struct Cache {
  const at::Tensor *k_codes, *v_codes, *k_exps, *v_exps;
  int index;
  int64_t blocks, heads, block_size, dim;
};

// k_codes, v_codes [NB, Hkv, bs, d] e4m3, k_exps, v_exps [NB, Hkv, bs] uint8.
bool read_cache(PyObject *const *a, Cache *c) {
  if (!THPVariable_Check(a[0])) return false;
  c->index = static_cast<int>(THPVariable_Unpack(a[0]).get_device());
  if (c->index < 0) return false;
  c->k_codes = dense(a[0], at::kFloat8_e4m3fn, c->index);
  c->v_codes = dense(a[1], at::kFloat8_e4m3fn, c->index);
  c->k_exps = dense(a[2], at::kByte, c->index);
  c->v_exps = dense(a[3], at::kByte, c->index);
  if (!c->k_codes || !c->v_codes || !c->k_exps || !c->v_exps) return false;
  const auto s = c->k_codes->sizes();
  if (s.size() != 4 || c->v_codes->sizes() != s || c->k_exps->sizes() != s.slice(0, 3) ||
      c->v_exps->sizes() != s.slice(0, 3))
    return false;
  c->blocks = s[0], c->heads = s[1], c->block_size = s[2], c->dim = s[3];
  return true;
}

uint8_t *bytes(const at::Tensor *t) { return static_cast<uint8_t *>(t->data_ptr()); }
pkv_bf16 *bf16(const at::Tensor *t) { return static_cast<pkv_bf16 *>(t->data_ptr()); }

// None, or an int32 tensor on the device.
bool read_status(PyObject *o, int index, int32_t **status) {
  *status = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.scalar_type() != at::kInt || t.get_device() != index) return false;
  *status = static_cast<int32_t *>(t.data_ptr());
  return true;
}

// None (the current stream of the device) or a cudaStream_t's value.
bool read_stream(PyObject *o, int index, void **stream) {
  if (o == Py_None) {
    *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    return true;
  }
  *stream = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// Elements from one token's [heads, dim] rows to the next's, the rows themselves
// dense; -1: they are not.
int64_t token_stride(const at::Tensor &t, int64_t tokens, const Cache &c) {
  if (t.dim() != 3 || t.size(0) != tokens || t.size(1) != c.heads || t.size(2) != c.dim) return -1;
  const int64_t width = c.heads * c.dim;
  if (t.is_contiguous()) return width;
  const auto s = t.strides();
  if ((s[2] != 1 && c.dim > 1) || (s[1] != c.dim && c.heads > 1)) return -1;
  if (tokens <= 1) return width;
  return s[0] >= width && s[0] % 8 == 0 ? s[0] : -1;
}

// f() with the device current and without the interpreter's lock.
template <typename F>
PyObject *call(int index, F &&f) {
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::DeviceType::CUDA, static_cast<c10::DeviceIndex>(index)));
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

PyObject *recheck() { return PyLong_FromLong(kRecheck); }

bool fits_int(int64_t x) { return x >= 0 && x <= INT32_MAX; }

// (k, v, slot_mapping, k_codes, v_codes, k_exps, v_exps, d_status, stream)
PyObject *write_quant(PyObject *, PyObject *const *a, Py_ssize_t n) {
  try {
    Cache c;
    int32_t *status;
    void *stream;
    if (n != 9 || !read_cache(a + 3, &c)) return recheck();
    const at::Tensor *slots = dense(a[2], at::kLong, c.index);
    if (!slots || slots->dim() != 1 || !THPVariable_Check(a[0]) || !THPVariable_Check(a[1])) return recheck();
    const at::Tensor &k = THPVariable_Unpack(a[0]), &v = THPVariable_Unpack(a[1]);
    if (k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16 || k.get_device() != c.index ||
        v.get_device() != c.index)
      return recheck();
    const int64_t T = slots->size(0), ks = token_stride(k, T, c), vs = token_stride(v, T, c);
    if (ks < 0 || vs < 0 || !fits_int(T) || !fits_int(c.blocks) || !read_status(a[7], c.index, &status) ||
        !read_stream(a[8], c.index, &stream))
      return recheck();
    return call(c.index, [&] {
      return pkv_write_quant(bf16(&k), bf16(&v), ks, vs, static_cast<int64_t *>(slots->data_ptr()), static_cast<int>(T),
                             bytes(c.k_codes), bytes(c.v_codes), bytes(c.k_exps), bytes(c.v_exps),
                             static_cast<int>(c.blocks), static_cast<int>(c.block_size), static_cast<int>(c.heads),
                             static_cast<int>(c.dim), status, stream);
    });
  } catch (const std::exception &) {
    return recheck();
  }
}

// (k_codes, v_codes, k_exps, v_exps, slot_mapping, k, v, d_status, stream)
PyObject *read_quant(PyObject *, PyObject *const *a, Py_ssize_t n) {
  try {
    Cache c;
    int32_t *status;
    void *stream;
    if (n != 9 || !read_cache(a, &c)) return recheck();
    const at::Tensor *slots = dense(a[4], at::kLong, c.index);
    const at::Tensor *k = dense(a[5], at::kBFloat16, c.index), *v = dense(a[6], at::kBFloat16, c.index);
    if (!slots || slots->dim() != 1 || !k || !v) return recheck();
    const int64_t T = slots->size(0), shape[3] = {T, c.heads, c.dim};
    if (k->sizes() != at::IntArrayRef(shape, 3) || v->sizes() != k->sizes() || !fits_int(T) || !fits_int(c.blocks) ||
        !read_status(a[7], c.index, &status) || !read_stream(a[8], c.index, &stream))
      return recheck();
    return call(c.index, [&] {
      return pkv_read_quant(bytes(c.k_codes), bytes(c.v_codes), bytes(c.k_exps), bytes(c.v_exps),
                            static_cast<int64_t *>(slots->data_ptr()), static_cast<int>(T), bf16(k), bf16(v),
                            static_cast<int>(c.blocks), static_cast<int>(c.block_size), static_cast<int>(c.heads),
                            static_cast<int>(c.dim), status, stream);
    });
  } catch (const std::exception &) {
    return recheck();
  }
}

// (q, k_codes, v_codes, k_exps, v_exps, block_tables, seq_lens, max_seq_len, scale, out, workspace, d_status, stream)
PyObject *decode_quant(PyObject *, PyObject *const *a, Py_ssize_t n) {
  try {
    Cache c;
    int32_t *status;
    void *stream;
    if (n != 13 || !read_cache(a + 1, &c)) return recheck();
    const at::Tensor *q = dense(a[0], at::kBFloat16, c.index), *out = dense(a[9], at::kBFloat16, c.index);
    const at::Tensor *tables = dense(a[5], at::kInt, c.index), *lens = dense(a[6], at::kInt, c.index);
    if (!q || !out || !tables || !lens) return recheck();
    if (q->dim() != 4 || q->size(1) != 1 || q->size(3) != c.dim || out->sizes() != q->sizes() || tables->dim() != 2 ||
        tables->size(0) != q->size(0) || lens->dim() != 1 || lens->size(0) != q->size(0))
      return recheck();
    const long max_len = PyLong_AsLong(a[7]);
    const double scale = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      return recheck();
    }
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (a[10] != Py_None) {
      if (!THPVariable_Check(a[10])) return recheck();
      const at::Tensor &w = THPVariable_Unpack(a[10]);
      if (w.get_device() != c.index || !w.is_contiguous()) return recheck();
      ws = w.data_ptr();
      ws_bytes = w.nbytes();
    }
    if (max_len < INT32_MIN || max_len > INT32_MAX || !fits_int(q->size(0)) || !fits_int(q->size(2)) || !fits_int(tables->size(1)) ||
        !fits_int(c.blocks) || !read_status(a[11], c.index, &status) || !read_stream(a[12], c.index, &stream))
      return recheck();
    return call(c.index, [&] {
      return paged_attention_decode_quant(
          bf16(q), bytes(c.k_codes), bytes(c.v_codes), bytes(c.k_exps), bytes(c.v_exps),
          static_cast<int32_t *>(tables->data_ptr()), static_cast<int>(tables->size(1)),
          static_cast<int32_t *>(lens->data_ptr()), static_cast<int>(q->size(0)), static_cast<int>(max_len),
          static_cast<int>(q->size(2)), static_cast<int>(c.heads), static_cast<int>(c.dim),
          static_cast<int>(c.block_size), static_cast<int>(c.blocks), static_cast<float>(scale), bf16(out), ws, ws_bytes,
          status, stream);
    });
  } catch (const std::exception &) {
    return recheck();
  }
}

PyMethodDef methods[] = {
    {"write_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write_quant)), METH_FASTCALL, nullptr},
    {"read_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read_quant)), METH_FASTCALL, nullptr},
    {"decode_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_quant)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
