// Python entry of the 8-bit cache's calls, the rotary append and the windowed and
// tree attention: argument marshalling only.
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

// k_cache, v_cache [NB, Hkv, bs, d] bf16 (k_codes, v_codes hold them).
bool read_bf16_cache(PyObject *const *a, Cache *c) {
  if (!THPVariable_Check(a[0])) return false;
  c->index = static_cast<int>(THPVariable_Unpack(a[0]).get_device());
  if (c->index < 0) return false;
  c->k_codes = dense(a[0], at::kBFloat16, c->index);
  c->v_codes = dense(a[1], at::kBFloat16, c->index);
  c->k_exps = c->v_exps = nullptr;
  if (!c->k_codes || !c->v_codes) return false;
  const auto s = c->k_codes->sizes();
  if (s.size() != 4 || c->v_codes->sizes() != s) return false;
  c->blocks = s[0], c->heads = s[1], c->block_size = s[2], c->dim = s[3];
  return true;
}

// None (no bytes), or a dense tensor on the device.
bool read_workspace(PyObject *o, int index, void **ws, size_t *bytes) {
  *ws = nullptr;
  *bytes = 0;
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  const at::Tensor &w = THPVariable_Unpack(o);
  if (w.get_device() != index || !w.is_contiguous()) return false;
  *ws = w.data_ptr();
  *bytes = w.nbytes();
  return true;
}

// An int argument; false where it is not one.
bool read_int(PyObject *o, int *x) {
  const long v = PyLong_AsLong(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *x = static_cast<int>(v);
  return v >= INT32_MIN && v <= INT32_MAX;
}

bool read_float(PyObject *o, float *x) {
  *x = static_cast<float>(PyFloat_AsDouble(o));
  if (!PyErr_Occurred()) return true;
  PyErr_Clear();
  return false;
}

// (q or None, k, v, positions, cos_sin, slot_mapping, q_out or None, interleaved, d_status, stream, cache...)
template <bool QUANT>
PyObject *write_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  try {
    Cache c;
    int32_t *status;
    void *stream;
    int interleaved;
    if (n != (QUANT ? 14 : 12) || !(QUANT ? read_cache(a + 10, &c) : read_bf16_cache(a + 10, &c))) return recheck();
    const at::Tensor *pos = dense(a[3], at::kLong, c.index), *table = dense(a[4], at::kFloat, c.index);
    const at::Tensor *slots = dense(a[5], at::kLong, c.index);
    if (!pos || !table || !slots || pos->dim() != 1 || slots->dim() != 1 || pos->size(0) != slots->size(0) ||
        table->dim() != 2 || !THPVariable_Check(a[1]) || !THPVariable_Check(a[2]))
      return recheck();
    const at::Tensor &k = THPVariable_Unpack(a[1]), &v = THPVariable_Unpack(a[2]);
    auto is_bf16 = [&](const at::Tensor &t) { return t.scalar_type() == at::kBFloat16 && t.get_device() == c.index; };
    if (!is_bf16(k) || !is_bf16(v)) return recheck();
    const int64_t T = slots->size(0), ks = token_stride(k, T, c), vs = token_stride(v, T, c);
    pkv_bf16 *q = nullptr, *q_out = nullptr;
    int64_t qs = 0, qos = 0, hq = 0;
    if (a[0] != Py_None || a[6] != Py_None) {
      if (!THPVariable_Check(a[0]) || !THPVariable_Check(a[6])) return recheck();
      const at::Tensor &tq = THPVariable_Unpack(a[0]), &to = THPVariable_Unpack(a[6]);
      if (!is_bf16(tq) || !is_bf16(to) || tq.dim() != 3) return recheck();
      Cache heads = c;  // a token's query rows are checked as its key rows are, but for their number
      heads.heads = hq = tq.size(1);
      qs = token_stride(tq, T, heads);
      qos = token_stride(to, T, heads);
      if (hq < 1) return recheck();
      q = bf16(&tq);
      q_out = bf16(&to);
    }
    if (ks < 0 || vs < 0 || qs < 0 || qos < 0 || !fits_int(T) || !fits_int(c.blocks) || !fits_int(table->size(0)) ||
        !fits_int(table->size(1)) || !read_int(a[7], &interleaved) || !read_status(a[8], c.index, &status) ||
        !read_stream(a[9], c.index, &stream))
      return recheck();
    const int64_t *p_pos = static_cast<int64_t *>(pos->data_ptr()), *p_slots = static_cast<int64_t *>(slots->data_ptr());
    const float *p_table = static_cast<float *>(table->data_ptr());
    const int tokens = static_cast<int>(T), top = static_cast<int>(table->size(0)), rot = static_cast<int>(table->size(1));
    const int blocks = static_cast<int>(c.blocks), bs = static_cast<int>(c.block_size);
    const int heads = static_cast<int>(c.heads), dim = static_cast<int>(c.dim), nq = static_cast<int>(hq);
    return call(c.index, [&] {
      if constexpr (QUANT)
        return pkv_write_rope_quant(q, bf16(&k), bf16(&v), qs, ks, vs, p_pos, p_table, top, rot, interleaved, p_slots,
                                    tokens, q_out, qos, bytes(c.k_codes), bytes(c.v_codes), bytes(c.k_exps),
                                    bytes(c.v_exps), blocks, bs, nq, heads, dim, status, stream);
      else
        return pkv_write_rope(q, bf16(&k), bf16(&v), qs, ks, vs, p_pos, p_table, top, rot, interleaved, p_slots, tokens,
                              q_out, qos, bf16(c.k_codes), bf16(c.v_codes), blocks, bs, nq, heads, dim, status,
                              stream);
    });
  } catch (const std::exception &) {
    return recheck();
  }
}

// (q, k_cache, v_cache, block_tables, seq_lens, q_start or None, tree_mask or None, first, second, max_seq_len, scale,
//  out, workspace, d_status, stream): first and second are window and sinks, or (with a mask) max_nodes and 0.
PyObject *spans(PyObject *, PyObject *const *a, Py_ssize_t n) {
  try {
    Cache c;
    int32_t *status;
    void *stream, *ws;
    size_t ws_bytes;
    int first, second, max_len;
    float scale;
    if (n != 15 || !read_bf16_cache(a + 1, &c)) return recheck();
    const at::Tensor *q = dense(a[0], at::kBFloat16, c.index), *out = dense(a[11], at::kBFloat16, c.index);
    const at::Tensor *tables = dense(a[3], at::kInt, c.index), *lens = dense(a[4], at::kInt, c.index);
    const bool has_start = a[5] != Py_None, tree = a[6] != Py_None;
    const at::Tensor *start = has_start ? dense(a[5], at::kInt, c.index) : nullptr;
    const at::Tensor *mask = tree ? dense(a[6], at::kLong, c.index) : nullptr;
    if (!q || !out || !tables || !lens || (has_start && !start) || (tree && (!mask || !start))) return recheck();
    if (q->dim() != 3 || q->size(2) != c.dim || out->sizes() != q->sizes() || tables->dim() != 2 || lens->dim() != 1 ||
        tables->size(0) != lens->size(0) ||
        (has_start ? start->dim() != 1 || start->size(0) != lens->size(0) + 1 : q->size(0) != lens->size(0)) ||
        (tree && (mask->dim() != 1 || mask->size(0) != q->size(0))))
      return recheck();
    if (!read_int(a[7], &first) || !read_int(a[8], &second) || !read_int(a[9], &max_len) || !read_float(a[10], &scale) ||
        !read_workspace(a[12], c.index, &ws, &ws_bytes) || !fits_int(q->size(0)) || !fits_int(q->size(1)) ||
        !fits_int(lens->size(0)) || !fits_int(tables->size(1)) || !fits_int(c.blocks) ||
        !read_status(a[13], c.index, &status) || !read_stream(a[14], c.index, &stream))
      return recheck();
    const int32_t *p_start = has_start ? static_cast<int32_t *>(start->data_ptr()) : nullptr;
    const int32_t *p_tables = static_cast<int32_t *>(tables->data_ptr()), *p_lens = static_cast<int32_t *>(lens->data_ptr());
    const int width = static_cast<int>(tables->size(1)), seqs = static_cast<int>(lens->size(0));
    const int rows = static_cast<int>(q->size(0)), hq = static_cast<int>(q->size(1)), hkv = static_cast<int>(c.heads);
    const int dim = static_cast<int>(c.dim), bs = static_cast<int>(c.block_size), blocks = static_cast<int>(c.blocks);
    return call(c.index, [&] {
      if (tree)
        return paged_attention_tree(bf16(q), bf16(c.k_codes), bf16(c.v_codes), p_tables, width, p_lens, p_start,
                                    static_cast<uint64_t *>(mask->data_ptr()), seqs, rows, first, max_len, hq, hkv, dim,
                                    bs, blocks, scale, bf16(out), ws, ws_bytes, status, stream);
      return paged_attention_window(bf16(q), bf16(c.k_codes), bf16(c.v_codes), p_tables, width, p_lens, p_start, seqs,
                                    rows, max_len, first, second, hq, hkv, dim, bs, blocks, scale, bf16(out), ws,
                                    ws_bytes, status, stream);
    });
  } catch (const std::exception &) {
    return recheck();
  }
}

PyMethodDef methods[] = {
    {"write_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write_quant)), METH_FASTCALL, nullptr},
    {"read_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read_quant)), METH_FASTCALL, nullptr},
    {"decode_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_quant)), METH_FASTCALL, nullptr},
    {"write_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write_rope<false>)), METH_FASTCALL, nullptr},
    {"write_rope_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write_rope<true>)), METH_FASTCALL, nullptr},
    {"spans", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(spans)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
