// Marshalling of the window, sink and block-scaled-cache calls: the checks of
// their tensors, their results' allocation, and the C entry.
//
// These calls take 4 to 20 microseconds on the device.  In Python their checks
// and ctypes took 11 (append) to 18 (decode); here they take 3 to 6 with the
// allocations.  The entries are handed over as addresses by the Python module,
// which has loaded the library; its names, signatures and documentation stay
// there.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdarg>

#include "mla.h"

namespace {

struct Entries {
  decltype(&mla_rope_cache_append) append;
  decltype(&mla_gather_cache_scaled) gather;
  decltype(&mla_decode_window_workspace_size) workspace_size;
  decltype(&mla_decode_paged_window) decode_window;
  decltype(&mla_decode_paged_scaled) decode_scaled;
  decltype(&mla_prefill_attn_window) prefill;
} entries;
PyObject *fail = nullptr;   // called with (entry, status): raises the library's error

// Thrown with the interpreter's error set.
struct Refused {};
[[noreturn]] void refuse(PyObject *type, const char *format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Refused();
}
// No C++ exception leaves through the interpreter (an allocation may throw one).
template <typename F>
PyObject *guarded(F &&body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refused &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// The current device, which the first tensor has to be on.
int current_device(const at::Tensor &t, const char *name) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  const int dev = t.get_device();
  if (dev != c10::cuda::current_device())
    refuse(PyExc_ValueError, "%s is on cuda:%d, not on the current device", name, dev);
  return dev;
}

void check(const at::Tensor &t, const char *name, at::ScalarType type, int64_t dims, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(PyExc_ValueError, "%s is not on cuda:%d", name, dev);
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s: dtype %s is not %s", name, c10::toString(t.scalar_type()),
                           c10::toString(type));
  if (t.dim() != dims)
    refuse(PyExc_ValueError, "%s: expected %d dims, got %d", name, static_cast<int>(dims),
                            static_cast<int>(t.dim()));
}
// A contiguous tensor of this dtype, rank and device.
const at::Tensor &dense(PyObject *o, const char *name, at::ScalarType type, int64_t dims, int dev) {
  const at::Tensor &t = tensor(o, name);
  check(t, name, type, dims, dev);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}
// A bf16 tensor whose last dim is contiguous; the others may be strided.
const at::Tensor &rows(PyObject *o, const char *name, int64_t dims, int dev) {
  const at::Tensor &t = tensor(o, name);
  check(t, name, at::kBFloat16, dims, dev);
  if (t.stride(dims - 1) != 1 && t.numel() != 0)
    refuse(PyExc_ValueError, "%s: the last dim must be contiguous", name);
  return t;
}
bool shape(const at::Tensor &t, at::IntArrayRef want) { return t.sizes() == want; }

template <typename T>
T *at_(const at::Tensor &t) { return static_cast<T *>(t.data_ptr()); }

// kv_scales [num_blocks, 64 / scale_block]: returns scale_block.
int scale_block(const at::Tensor &s, int64_t num_blocks) {
  const int64_t per = s.size(1);
  if (s.size(0) != num_blocks || (per != 1 && per != 2 && per != 4))
    refuse(PyExc_ValueError, "kv_scales must be [num_blocks, 64 / scale_block], scale_block 16, 32 or 64");
  return static_cast<int>(64 / per);
}

float real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(v);
}
// An integer; beyond 32 bits refused, or where it bounds something the largest.
int integer(PyObject *o, const char *name, bool bound = false) {
  PyObject *i = PyNumber_Index(o);
  if (!i) throw Refused();
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i, &over);
  Py_DECREF(i);
  if (bound && (over > 0 || v > INT_MAX)) return INT_MAX;
  if (over || v > INT_MAX || v < INT_MIN) refuse(PyExc_ValueError, "%s is beyond 32 bits", name);
  return static_cast<int>(v);
}
int narrow(int64_t v, const char *name) {
  if (v > INT_MAX) refuse(PyExc_ValueError, "%s is beyond 32 bits", name);
  return static_cast<int>(v);
}
void arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse(PyExc_TypeError, "%d arguments, not %d", static_cast<int>(got), static_cast<int>(want));
}
// Calls an entry without the interpreter's lock (a launch may have to wait).
template <typename F>
void call(const char *name, F &&entry) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = entry();
  Py_END_ALLOW_THREADS
  if (status == MLA_OK) return;
  PyObject *r = PyObject_CallFunction(fail, "si", name, status);
  Py_XDECREF(r);
  if (!r) throw Refused();
  refuse(PyExc_ValueError, "%s: status %d", name, status);
}
// The result tensor that the caller gave, or a new one.
at::Tensor result(PyObject *o, const char *name, at::IntArrayRef sizes, at::ScalarType type, int dev) {
  if (o == Py_None)
    return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, dev)));
  const at::Tensor &t = dense(o, name, type, static_cast<int64_t>(sizes.size()), dev);
  if (!shape(t, sizes)) refuse(PyExc_ValueError, "%s has another shape than the result", name);
  return t;
}
PyObject *pair(at::Tensor a, at::Tensor b) {
  PyObject *x = THPVariable_Wrap(std::move(a));
  PyObject *y = x ? THPVariable_Wrap(std::move(b)) : nullptr;
  PyObject *t = y ? PyTuple_New(2) : nullptr;
  if (!t) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    throw Refused();
  }
  PyTuple_SET_ITEM(t, 0, x);
  PyTuple_SET_ITEM(t, 1, y);
  return t;
}

// (q_pe | None, k_pe, kv_c, positions, slot_mapping, kv_cache, kv_scales, rope_base, layout,
//  q_out | None, k_out | None)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    arguments(n, 11);
    const int dev = current_device(tensor(a[1], "k_pe"), "k_pe");
    const at::Tensor &k = rows(a[1], "k_pe", 2, dev), &c = rows(a[2], "kv_c", 2, dev);
    const at::Tensor &pos = dense(a[3], "positions", at::kInt, 1, dev);
    const at::Tensor &slots = dense(a[4], "slot_mapping", at::kInt, 1, dev);
    const at::Tensor &cache = dense(a[5], "kv_cache", at::kFloat8_e4m3fn, 3, dev);
    const at::Tensor &scales = dense(a[6], "kv_scales", at::kFloat, 2, dev);
    const int64_t T = k.size(0);
    int64_t H = 0, qt = 0, qh = 0;
    void *q = nullptr, *qo = nullptr, *ko = nullptr;
    if (a[0] != Py_None) {
      const at::Tensor &t = rows(a[0], "q_pe", 3, dev);
      if (t.size(0) != T || t.size(2) != 64) refuse(PyExc_ValueError, "q_pe must be [T, H, 64]");
      q = t.data_ptr();
      H = t.size(1);
      qt = t.stride(0);
      qh = t.stride(1);
    }
    if (k.size(1) != 64 || !shape(c, {T, 512}) || pos.size(0) != T || slots.size(0) != T ||
        cache.size(1) != 64 || cache.size(2) != 576)
      refuse(PyExc_ValueError, "rope / cache-append shapes");
    const int sb = scale_block(scales, cache.size(0));
    if (a[9] != Py_None) {
      const at::Tensor &t = dense(a[9], "q_out", at::kBFloat16, 3, dev);
      if (a[0] == Py_None || !shape(t, {T, H, 64})) refuse(PyExc_ValueError, "q_out must have q_pe's shape");
      qo = t.data_ptr();
    }
    if (a[10] != Py_None) {
      const at::Tensor &t = dense(a[10], "k_out", at::kBFloat16, 2, dev);
      if (!shape(t, {T, 64})) refuse(PyExc_ValueError, "k_out must have k_pe's shape");
      ko = t.data_ptr();
    }
    const float base = real(a[7]);
    const int layout = integer(a[8], "layout"), tokens = narrow(T, "T"), heads = narrow(H, "H");
    const int blocks = narrow(cache.size(0), "num_blocks");
    const auto stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    call("mla_rope_cache_append", [&] {
      return entries.append(q, qt, qh, k.data_ptr(), k.stride(0), c.data_ptr(), c.stride(0),
                            at_<int32_t>(pos), at_<int32_t>(slots), tokens, heads, base, layout, qo, ko,
                            cache.data_ptr(), at_<float>(scales), sb, blocks, stream);
  });
  Py_RETURN_NONE;
  });
}

// (kv_cache, kv_scales, block_table, seq_lens, cu_out, total_rows, seq_starts | None, out | None)
PyObject *gather(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    arguments(n, 8);
    const int dev = current_device(tensor(a[0], "kv_cache"), "kv_cache");
    const at::Tensor &cache = dense(a[0], "kv_cache", at::kFloat8_e4m3fn, 3, dev);
    const at::Tensor &scales = dense(a[1], "kv_scales", at::kFloat, 2, dev);
    const at::Tensor &table = dense(a[2], "block_table", at::kInt, 2, dev);
    const at::Tensor &lens = dense(a[3], "seq_lens", at::kInt, 1, dev);
    const at::Tensor &cu = dense(a[4], "cu_out", at::kInt, 1, dev);
    const int64_t B = table.size(0);
    if (cache.size(1) != 64 || cache.size(2) != 576 || lens.size(0) != B || cu.size(0) != B + 1)
      refuse(PyExc_ValueError, "gather shapes");
    const int32_t *starts = nullptr;
    if (a[6] != Py_None) {
      const at::Tensor &t = dense(a[6], "seq_starts", at::kInt, 1, dev);
      if (t.size(0) != B) refuse(PyExc_ValueError, "seq_starts must be [B]");
      starts = at_<int32_t>(t);
    }
    const int sb = scale_block(scales, cache.size(0)), total = integer(a[5], "total_rows");
    const int requests = narrow(B, "B"), max_blocks = narrow(table.size(1), "max_blocks");
    const int blocks = narrow(cache.size(0), "num_blocks");
    if (total < 0) refuse(PyExc_ValueError, "total_rows must not be negative");
    at::Tensor out = result(a[7], "out", {total, 576}, at::kBFloat16, dev);
    const auto stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    call("mla_gather_cache_scaled", [&] {
      return entries.gather(cache.data_ptr(), at_<float>(scales), sb, at_<int32_t>(table),
                            at_<int32_t>(lens), starts, at_<int32_t>(cu), requests, max_blocks, blocks,
                            total, out.data_ptr(), stream);
  });
  return THPVariable_Wrap(std::move(out));
  });
}

// (q, kv_cache, kv_scales | None, block_table, seq_lens, sm_scale, q_scale, k_scale, window,
//  sinks, split_tiles, out_dtype, out | None, lse | None, workspace | None): with scales the
//  block-scaled form
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    arguments(n, 15);
    const at::Tensor &q0 = tensor(a[0], "q");
    const int dev = current_device(q0, "q");
    const bool scaled = a[2] != Py_None, fp8 = q0.scalar_type() == at::kFloat8_e4m3fn;
    if (!fp8 && (scaled || q0.scalar_type() != at::kBFloat16))
      refuse(PyExc_TypeError, scaled ? "q: dtype %s is not e4m3" : "q: dtype %s is neither bf16 nor e4m3",
                             c10::toString(q0.scalar_type()));
    const at::Tensor &q = dense(a[0], "q", q0.scalar_type(), 4, dev);
    const at::Tensor &cache = dense(a[1], "kv_cache", q0.scalar_type(), 3, dev);
    const at::Tensor &table = dense(a[3], "block_table", at::kInt, 2, dev);
    const at::Tensor &lens = dense(a[4], "seq_lens", at::kInt, 1, dev);
    const int64_t B = q.size(0);
    if (q.size(3) != 576 || cache.size(1) != 64 || cache.size(2) != 576 || table.size(0) != B ||
        lens.size(0) != B)
      refuse(PyExc_ValueError, "decode shapes");
    const int b = narrow(B, "B"), q_len = narrow(q.size(1), "q_len"), H = narrow(q.size(2), "H");
    const int max_blocks = narrow(table.size(1), "max_blocks"), blocks = narrow(cache.size(0), "num_blocks");
    int sb = 0;
    const float *scales = nullptr;
    if (scaled) {
      const at::Tensor &s = dense(a[2], "kv_scales", at::kFloat, 2, dev);
      sb = scale_block(s, cache.size(0));
      scales = at_<float>(s);
    }
    const float sm = real(a[5]), qs = real(a[6]), ks = real(a[7]);
    const int window = integer(a[8], "window", true), sinks = integer(a[9], "sinks", true);
    const int split = integer(a[10], "split_tiles");
    if (!THPDtype_Check(a[11])) refuse(PyExc_TypeError, "out_dtype must be a dtype");
    const at::ScalarType type = reinterpret_cast<THPDtype *>(a[11])->scalar_type;
    if (type != at::kBFloat16 && type != at::kFloat)
      refuse(PyExc_TypeError, "out_dtype %s is neither bf16 nor fp32", c10::toString(type));
    at::Tensor out = result(a[12], "out", {B, q_len, H, 512}, type, dev);
    at::Tensor lse = result(a[13], "lse", {B, q_len, H}, at::kFloat, dev);
    at::Tensor ws;
    if (a[14] != Py_None) {
      ws = dense(a[14], "workspace", at::kByte, 1, dev);
    } else {
      size_t bytes = 0;
      const int64_t tokens = static_cast<int64_t>(max_blocks) * 64;
      if (tokens <= INT_MAX)   // (more are refused below)
        call("mla_decode_window_workspace_size", [&] {
          return entries.workspace_size(b, q_len, H, static_cast<int>(tokens), window, sinks, split, &bytes);
        });
      if (bytes)
        ws = at::empty({static_cast<int64_t>(bytes)},
                       at::TensorOptions().dtype(at::kByte).device(c10::Device(c10::kCUDA, dev)));
    }
    void *w = ws.defined() ? ws.data_ptr() : nullptr;
    const size_t bytes = ws.defined() ? static_cast<size_t>(ws.numel()) : 0;
    const int code = fp8 ? MLA_E4M3 : MLA_BF16, out_code = type == at::kFloat ? MLA_F32 : MLA_BF16;
    const auto stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    if (scaled)
      call("mla_decode_paged_scaled", [&] {
        return entries.decode_scaled(q.data_ptr(), qs, cache.data_ptr(), scales, sb, at_<int32_t>(table),
                                     at_<int32_t>(lens), b, q_len, H, max_blocks, blocks, sm, window, sinks,
                                     split, out.data_ptr(), out_code, at_<float>(lse), w, bytes, stream);
      });
    else
      call("mla_decode_paged_window", [&] {
        return entries.decode_window(q.data_ptr(), code, qs, cache.data_ptr(), code, ks, at_<int32_t>(table),
                                     at_<int32_t>(lens), b, q_len, H, max_blocks, blocks, sm, window, sinks,
                                     split, out.data_ptr(), out_code, at_<float>(lse), w, bytes, stream);
      });
    return pair(std::move(out), std::move(lse));
  });
}

// (q, k, v, cu_q, cu_k, max_q_len, window, sinks, sm_scale, out | None, lse | None)
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    arguments(n, 11);
    const int dev = current_device(tensor(a[0], "q"), "q");
    const at::Tensor &q = dense(a[0], "q", at::kBFloat16, 3, dev), &k = dense(a[1], "k", at::kBFloat16, 3, dev);
    const at::Tensor &v = dense(a[2], "v", at::kBFloat16, 3, dev);
    const at::Tensor &cu_q = dense(a[3], "cu_q", at::kInt, 1, dev), &cu_k = dense(a[4], "cu_k", at::kInt, 1, dev);
    const int64_t Tq = q.size(0), H = q.size(1), Nk = k.size(0), B = cu_q.size(0) - 1;
    if (q.size(2) != 192 || !shape(k, {Nk, H, 192}) || !shape(v, {Nk, H, 128}) || cu_k.size(0) != B + 1)
      refuse(PyExc_ValueError, "prefill shapes");
    const int b = narrow(B, "B"), tq = narrow(Tq, "Tq"), nk = narrow(Nk, "Nk"), h = narrow(H, "H");
    const int most = integer(a[5], "max_q_len");
    const int window = integer(a[6], "window", true), sinks = integer(a[7], "sinks", true);
    const float sm = real(a[8]);
    at::Tensor out = result(a[9], "out", {Tq, H, 128}, at::kBFloat16, dev);
    at::Tensor lse = result(a[10], "lse", {Tq, H}, at::kFloat, dev);
    const auto stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    call("mla_prefill_attn_window", [&] {
      return entries.prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), at_<int32_t>(cu_q), at_<int32_t>(cu_k),
                             b, tq, nk, h, most, window, sinks, sm, out.data_ptr(), at_<float>(lse), stream);
  });
  return pair(std::move(out), std::move(lse));
  });
}

// (fail, the entries' addresses in the order of Entries)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    arguments(n, 7);
    void *at[6];
    for (int i = 0; i < 6; ++i) {
      at[i] = PyLong_AsVoidPtr(a[i + 1]);
      if (!at[i]) refuse(PyExc_ValueError, "no address");
    }
    Py_INCREF(a[0]);
    Py_XSETREF(fail, a[0]);
    entries = {reinterpret_cast<decltype(entries.append)>(at[0]), reinterpret_cast<decltype(entries.gather)>(at[1]),
               reinterpret_cast<decltype(entries.workspace_size)>(at[2]),
               reinterpret_cast<decltype(entries.decode_window)>(at[3]),
               reinterpret_cast<decltype(entries.decode_scaled)>(at[4]),
               reinterpret_cast<decltype(entries.prefill)>(at[5])};
    Py_RETURN_NONE;
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f))
PyMethodDef methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                         {"append", FAST(append), METH_FASTCALL, nullptr},
                         {"gather", FAST(gather), METH_FASTCALL, nullptr},
                         {"decode", FAST(decode), METH_FASTCALL, nullptr},
                         {"prefill", FAST(prefill), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mla_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_binding() { return PyModule_Create(&module); }
