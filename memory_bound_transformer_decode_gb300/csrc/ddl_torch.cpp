// ddl_torch.cpp -- the per-layer calls of the 8-bit cache for torch tensors, as
// a CPython module: argument checks and the call of the C entry point.
//
// A serving step makes these calls once a layer and their kernels take 3 us
// and more, while the same checks in Python and a ctypes call took 5 to 9 us
// beside the launch itself (one GB300's host: page plan 8.4 us a call, append
// 8.6, attention 11.3).  Only torch's tensor accessors are used; nothing is
// computed here.  Bad arguments raise ValueError, as the other bindings do;
// the entry point's status is returned.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/ddl.h"

namespace {

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + ": a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(std::string(name) + ": an integer");
  }
  return v;
}

int32_t int32(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + ": a 32-bit integer");
  return (int32_t)v;
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(std::string(name) + ": a number");
  }
  return (float)v;
}

// Data of a contiguous tensor of `n` entries (n < 0: any) of a type on CUDA device `dev`.
void* data(const at::Tensor& t, const char* name, at::ScalarType type, int dev, int64_t n) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous() ||
      (n >= 0 && t.numel() != n))
    bad(std::string(name) + ": a contiguous " + (type == at::kInt ? "int32" : "fp32") + " tensor" +
        (n >= 0 ? " of " + std::to_string(n) + " entries" : "") + " on cuda:" + std::to_string(dev));
  return t.data_ptr();
}
int32_t* i32(PyObject* o, const char* name, int dev, int64_t n) {
  return (int32_t*)data(tensor(o, name), name, at::kInt, dev, n);
}
int32_t* i32_or_null(PyObject* o, const char* name, int dev, int64_t n) {
  return o == Py_None ? nullptr : i32(o, name, dev, n);
}
float* f32_or_null(PyObject* o, const char* name, int dev, int64_t n) {
  return o == Py_None ? nullptr : (float*)data(tensor(o, name), name, at::kFloat, dev, n);
}

int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return DDL_T_F32;
    case at::kBFloat16: return DDL_T_BF16;
    case at::kHalf: return DDL_T_F16;
    default: return -1;
  }
}

struct Pool {
  ddl_kv8 kv;
  int32_t H, hd;
  int dev;
};

Pool pool_of(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) bad("pool: a tuple (k, v, k_scale, v_scale)");
  const at::Tensor &k = tensor(PyTuple_GET_ITEM(o, 0), "k"), &v = tensor(PyTuple_GET_ITEM(o, 1), "v");
  const at::Tensor &ks = tensor(PyTuple_GET_ITEM(o, 2), "k_scale"), &vs = tensor(PyTuple_GET_ITEM(o, 3), "v_scale");
  const bool e4m3 = k.scalar_type() == at::kFloat8_e4m3fn;
  if (k.dim() != 4 || !(e4m3 || k.scalar_type() == at::kChar) || v.scalar_type() != k.scalar_type() ||
      v.sizes() != k.sizes())
    bad("pool: k and v [pages, H_kv, page_size, head_dim] of one 8-bit type");
  const int64_t pages = k.size(0), H = k.size(1), P = k.size(2), hd = k.size(3);
  const int64_t want[3] = {pages, H, P / 16};
  if (ks.scalar_type() != at::kFloat || vs.scalar_type() != at::kFloat || ks.sizes() != at::IntArrayRef(want, 3) ||
      vs.sizes() != ks.sizes())
    bad("pool: scales fp32 [pages, H_kv, page_size / 16]");
  if (!k.is_contiguous() || !v.is_contiguous() || !ks.is_contiguous() || !vs.is_contiguous())
    bad("pool: contiguous tensors");
  if (!k.is_cuda() || !v.is_cuda() || !ks.is_cuda() || !vs.is_cuda() || v.get_device() != k.get_device() ||
      ks.get_device() != k.get_device() || vs.get_device() != k.get_device())
    bad("pool: tensors of one CUDA device");
  if (H > INT32_MAX || P > INT32_MAX || hd > INT32_MAX) bad("pool: too large");
  return {{(uint8_t*)k.data_ptr(), (uint8_t*)v.data_ptr(), (float*)ks.data_ptr(), (float*)vs.data_ptr(), pages,
           (int32_t)P, e4m3 ? DDL_KV8_E4M3 : DDL_KV8_INT8},
          (int32_t)H, (int32_t)hd, (int)k.get_device()};
}

// Row stride of rows [T, heads, hd] of `like`'s type whose heads are contiguous.
int64_t rows_of(const at::Tensor& x, const char* name, int dev, int64_t heads, int64_t hd, at::ScalarType type,
                int64_t T) {
  if (x.dim() != 3 || x.size(0) != T || x.size(1) != heads || x.size(2) != hd || x.scalar_type() != type ||
      dtype_of(x) < 0 || !x.is_cuda() || x.get_device() != dev)
    bad(std::string(name) + ": [" + std::to_string(T) + ", " + std::to_string(heads) + ", " + std::to_string(hd) +
        "] fp32, bf16 or fp16 rows of one type on cuda:" + std::to_string(dev));
  if ((hd > 1 && x.stride(2) != 1) || (heads > 1 && x.stride(1) != hd))
    bad(std::string(name) + ": a row's heads are contiguous");
  return T > 1 ? x.stride(0) : heads * hd;
}

// `device` current for the call, and the stream it goes to.
struct On {
  std::optional<c10::cuda::CUDAGuard> guard;
  void* stream;
  On(int dev, PyObject* s) {
    if (c10::cuda::current_device() != dev) guard.emplace((c10::DeviceIndex)dev);
    stream = s == Py_None ? (void*)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()
                          : (void*)(uintptr_t)integer(s, "stream");
  }
};

template <class F>
PyObject* call(F&& f) {
  try {
    return PyLong_FromLong(f());
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (old_len, add_len, free_pages, page_table, page_size, row_off, kv_len, row_pos, slot, used, status, stream)
PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&]() -> int {
    if (n != 12) bad("page_plan: 12 arguments");
    const at::Tensor& table = tensor(a[3], "page_table");
    const int64_t R = tensor(a[0], "old_len").numel(), T = tensor(a[8], "slot").numel();
    const int64_t nfree = tensor(a[2], "free_pages").numel();
    if (!table.is_cuda() || table.dim() != 2 || table.size(0) != R)
      bad("page_table: [R, pages_per_seq] on a CUDA device");
    if (R > INT32_MAX || T > INT32_MAX || nfree > INT32_MAX || table.size(1) > INT32_MAX) bad("page_plan: too large");
    const int dev = (int)table.get_device();
    const int32_t *old = i32(a[0], "old_len", dev, R), *add = i32(a[1], "add_len", dev, R);
    const int32_t* free = i32(a[2], "free_pages", dev, nfree);
    int32_t* tab = i32(a[3], "page_table", dev, -1);
    const int32_t page = int32(a[4], "page_size");
    int32_t *off = i32(a[5], "row_off", dev, R + 1), *len = i32(a[6], "kv_len", dev, R);
    int32_t *pos = i32(a[7], "row_pos", dev, T), *slot = i32(a[8], "slot", dev, T);
    int32_t *used = i32(a[9], "used", dev, 1), *status = i32(a[10], "status", dev, R);
    On on(dev, a[11]);
    return ddl_page_plan(old, add, (int32_t)R, page, free, (int32_t)nfree, tab, (int32_t)table.size(1), off, len, pos,
                         slot, (int32_t)T, used, status, on.stream);
  });
}

// (pool, k_new, v_new, slot, bad, stream)
PyObject* kv8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&]() -> int {
    if (n != 6) bad("kv8_append: 6 arguments");
    const Pool p = pool_of(a[0]);
    const at::Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new");
    const int64_t T = tensor(a[3], "slot").numel();
    if (T > INT32_MAX) bad("slot: too many");
    const int64_t ks = rows_of(k, "k_new", p.dev, p.H, p.hd, k.scalar_type(), T);
    const int64_t vs = rows_of(v, "v_new", p.dev, p.H, p.hd, k.scalar_type(), T);
    const int32_t* slot = i32(a[3], "slot", p.dev, T);
    int32_t* flag = i32_or_null(a[4], "bad", p.dev, 1);
    On on(p.dev, a[5]);
    return ddl_kv8_append(&p.kv, p.H, p.hd, (ddl_dtype)dtype_of(k), k.data_ptr(), ks, v.data_ptr(), vs, slot,
                          (int32_t)T, flag, on.stream);
  });
}

// (pool, q, kv_len, page_table, max_len, q_off, max_rows, scale, softcap, window, slopes, out, lse, workspace, bad,
// stream); scale None: 1 / sqrt(head_dim)
PyObject* kv8_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&]() -> int {
    if (n != 16) bad("kv8_attention: 16 arguments");
    const Pool p = pool_of(a[0]);
    const at::Tensor &q = tensor(a[1], "q"), &out = tensor(a[11], "out"), &table = tensor(a[3], "page_table");
    const at::Tensor& ws = tensor(a[13], "workspace");
    if (q.dim() != 3 || table.dim() != 2) bad("q: [T, H_q, hd]; page_table: [R, pages_per_seq]");
    const int64_t T = q.size(0), Hq = q.size(1), R = tensor(a[2], "kv_len").numel();
    if (T > INT32_MAX || Hq > INT32_MAX || R > INT32_MAX || table.size(1) > INT32_MAX) bad("q: too large");
    const int64_t qs = rows_of(q, "q", p.dev, Hq, p.hd, q.scalar_type(), T);
    const int64_t os = rows_of(out, "out", p.dev, Hq, p.hd, q.scalar_type(), T);
    if (table.size(0) != R) bad("page_table: a row for each entry of kv_len");
    if (!ws.is_cuda() || ws.get_device() != p.dev || !ws.is_contiguous()) bad("workspace: contiguous, on the pool's device");
    ddl_attn_opts o;
    o.scale = a[7] == Py_None ? 1.f / std::sqrt((float)p.hd) : number(a[7], "scale");
    o.softcap = number(a[8], "softcap");
    o.window = int32(a[9], "window");
    o.slopes = f32_or_null(a[10], "slopes", p.dev, Hq);
    const int32_t *len = i32(a[2], "kv_len", p.dev, R), *tab = i32(a[3], "page_table", p.dev, -1);
    const int32_t* off = i32_or_null(a[5], "q_off", p.dev, R + 1);
    float* lse = f32_or_null(a[12], "lse", p.dev, T * Hq);
    int32_t* flag = i32_or_null(a[14], "bad", p.dev, 1);
    const int32_t max_len = int32(a[4], "max_len"), max_rows = int32(a[6], "max_rows");
    On on(p.dev, a[15]);
    return ddl_kv8_attention(&p.kv, (int32_t)Hq, p.H, p.hd, (ddl_dtype)dtype_of(q), &o, (int32_t)R, (int32_t)T, max_rows,
                             max_len, off, len, tab, (int32_t)table.size(1), q.data_ptr(), qs, out.data_ptr(), os, lse,
                             flag, ws.data_ptr(), ws.nbytes(), on.stream);
  });
}

PyMethodDef methods[] = {{"page_plan", (PyCFunction)(void (*)(void))page_plan, METH_FASTCALL, nullptr},
                         {"kv8_append", (PyCFunction)(void (*)(void))kv8_append, METH_FASTCALL, nullptr},
                         {"kv8_attention", (PyCFunction)(void (*)(void))kv8_attention, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_ddl_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__ddl_torch() { return PyModule_Create(&module_def); }
