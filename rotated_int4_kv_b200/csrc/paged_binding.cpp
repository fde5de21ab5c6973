// paged_binding.cpp -- the paged entry points for Python: argument checks, outputs and the
// current stream taken from torch tensors without an interpreter step per attribute. A
// serving step makes these calls once per layer for a few microseconds of GPU work, so their
// host time counts: 17 - 30 us through ctypes with checks in Python, a few us here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <optional>
#include <vector>

#include "../../include/kvq.h"

namespace {

PyObject* g_check = nullptr;  // check(status, where): raises the library's error

// A refused argument: the Python error is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Refused{};
}

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "torch.int32";
    case at::kHalf: return "torch.float16";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// A CUDA tensor of a type, on `device` (-1: any; set to the tensor's own), contiguous unless said otherwise.
const at::Tensor& cuda(PyObject* o, const char* name, at::ScalarType type, int& device, bool contiguous = true) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be a CUDA tensor", name);
  const int d = t.get_device();
  if (device >= 0 && d != device) refuse(PyExc_ValueError, "%s is on cuda:%d, expected cuda:%d", name, d, device);
  device = d;
  if (t.scalar_type() != type)
    refuse(PyExc_ValueError, "%s must be %s, got %s", name, name_of(type), name_of(t.scalar_type()));
  if (contiguous && !t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}

void shape(const at::Tensor& t, const char* name, std::initializer_list<int64_t> want) {
  if (t.sizes() == at::IntArrayRef(want)) return;
  std::string s;
  for (int64_t v : want) s += (s.empty() ? "" : ", ") + std::to_string(v);
  refuse(PyExc_ValueError, "%s must have shape (%s)", name, s.c_str());
}

int64_t integer(PyObject* o, const char* name, int64_t lo = -0x7fffffff - 1ll, int64_t hi = 0x7fffffff) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    PyObject* i = PyNumber_Index(o);  // integers of other libraries
    if (!i) throw Refused{};
    const int64_t x = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (x == -1 && PyErr_Occurred()) throw Refused{};
    if (x < lo || x > hi) refuse(PyExc_ValueError, "%s out of range", name);
    return x;
  }
  if (v < lo || v > hi) refuse(PyExc_ValueError, "%s out of range", name);
  return v;
}

int extent(int64_t v, const char* name) {
  if (v > 0x7fffffff) refuse(PyExc_ValueError, "%s has a dimension of 2^31 or more", name);
  return (int)v;
}

struct PlanView {
  const kvq_plan* handle;
  int64_t D, G, bits;
  int device;
};

PlanView plan(PyObject* o, const char* name) {
  static PyObject* const key = PyUnicode_InternFromString("_desc");
  PyObject* d = PyObject_GetAttr(o, key);
  if (!d) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "%s must be a Plan", name);
  }
  Py_DECREF(d);  // the plan holds it
  if (!PyTuple_Check(d)) refuse(PyExc_ValueError, "%s is closed", name);
  PlanView v;
  v.handle = static_cast<const kvq_plan*>(PyLong_AsVoidPtr(PyTuple_GET_ITEM(d, 0)));
  v.D = PyLong_AsLong(PyTuple_GET_ITEM(d, 1));
  v.G = PyLong_AsLong(PyTuple_GET_ITEM(d, 2));
  v.bits = PyLong_AsLong(PyTuple_GET_ITEM(d, 3));
  v.device = (int)PyLong_AsLong(PyTuple_GET_ITEM(d, 4));
  return v;
}

void on_device(const PlanView& p, int device) {
  if (p.device != device)
    refuse(PyExc_ValueError, "the plan was made on cuda:%d, the tensors are on cuda:%d", p.device, device);
}
void same_dim(const PlanView& p, int64_t D) {
  if (p.D != D) refuse(PyExc_ValueError, "head_dim %lld does not match the plan's %lld", (long long)D, (long long)p.D);
}

struct Pages {
  const at::Tensor *codes, *scales;
  int64_t n, H, P;
};

Pages pages(PyObject* c, PyObject* s, const PlanView& p, const char* cname, const char* sname, int& device) {
  Pages g;
  g.codes = &cuda(c, cname, at::kByte, device);
  g.scales = &cuda(s, sname, at::kHalf, device);
  if (g.codes->dim() != 4) refuse(PyExc_ValueError, "%s must be [num_pages, Hkv, page_size, code bytes]", cname);
  g.n = g.codes->size(0);
  g.H = g.codes->size(1);
  g.P = g.codes->size(2);
  if (g.P != 16 && g.P != 32 && g.P != 64 && g.P != 128)
    refuse(PyExc_ValueError, "page size must be one of (16, 32, 64, 128), got %lld", (long long)g.P);
  shape(*g.codes, cname, {g.n, g.H, g.P, p.D * p.bits / 8});
  shape(*g.scales, sname, {g.n, g.H, g.P, p.D / p.G});
  extent(g.n, cname);
  extent(g.H, cname);
  return g;
}

// [B, max_pages] with contiguous rows; returns the rows' stride.
int64_t block_table(const at::Tensor& t, int64_t B) {
  if (t.dim() != 2 || t.size(0) != B || (t.numel() > 1 && t.size(1) > 1 && t.stride(1) != 1))
    refuse(PyExc_ValueError, "block_table must be [B, max_pages] with contiguous rows");
  extent(t.size(1), "block_table");
  return B > 1 ? t.stride(0) : t.size(1);
}

// The call's device and stream: the current stream of `device`, or the one given.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  std::optional<c10::cuda::CUDAStreamGuard> sguard;
  void* stream;
  On(int device, PyObject* s) {
    if (s == Py_None) {
      guard.set_index((c10::DeviceIndex)device);
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    } else {
      void* raw = PyLong_AsVoidPtr(s);
      if (PyErr_Occurred()) throw Refused{};
      sguard.emplace(c10::cuda::getStreamFromExternal((cudaStream_t)raw, (c10::DeviceIndex)device));
      stream = raw;
    }
  }
};

at::Tensor fresh(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}

template <typename F>
void call(const char* where, F&& f) {
  kvq_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  if (st == KVQ_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)st, where);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  throw Refused{};
}

int32_t* i32(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }
uint16_t* f16(const at::Tensor& t) { return static_cast<uint16_t*>(t.data_ptr()); }
uint8_t* u8(const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

// No C++ exception reaches the interpreter.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
}

// page_plan(kv_lens, q_lens, block_table, free_pages, free_head, page_size, n_tokens, out, free_head_out, stream)
// -> None (out given) or (slots, positions, q_starts, kv_lens, info)
PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded([&]() -> PyObject* {
    expect(na, 10);
    int dev = -1;
    const at::Tensor& kv = cuda(a[0], "kv_lens", at::kInt, dev);
    if (kv.dim() != 1) refuse(PyExc_ValueError, "kv_lens must be a 1-D tensor");
    const int B = extent(kv.size(0), "kv_lens");
    const at::Tensor& q = cuda(a[1], "q_lens", at::kInt, dev);
    shape(q, "q_lens", {B});
    const at::Tensor& table = cuda(a[2], "block_table", at::kInt, dev, false);
    const int64_t stride = block_table(table, B);
    const at::Tensor& free = cuda(a[3], "free_pages", at::kInt, dev);
    const at::Tensor& head = cuda(a[4], "free_head", at::kInt, dev);
    shape(head, "free_head", {1});
    const int P = (int)integer(a[5], "page_size");
    const at::Tensor& head_out = a[8] == Py_None ? head : cuda(a[8], "free_head_out", at::kInt, dev);
    shape(head_out, "free_head_out", {1});
    On on(dev, a[9]);
    std::vector<at::Tensor> made;
    const at::Tensor* out[5];
    static const char* const names[5] = {"out.slots", "out.positions", "out.q_starts", "out.kv_lens", "out.info"};
    int64_t n;
    if (a[7] == Py_None) {
      if (a[6] == Py_None) refuse(PyExc_ValueError, "page_plan needs n_tokens or out");
      n = integer(a[6], "n_tokens", 0);
      const int64_t len[5] = {n, n, B + 1ll, B, 4};
      made.reserve(5);
      for (int i = 0; i < 5; ++i) {
        made.push_back(fresh({len[i]}, at::kInt, dev));
        out[i] = &made[i];
      }
    } else {
      if (!PyTuple_Check(a[7]) || PyTuple_GET_SIZE(a[7]) != 5) refuse(PyExc_TypeError, "out must be a PagePlan");
      for (int i = 0; i < 5; ++i) out[i] = &cuda(PyTuple_GET_ITEM(a[7], i), names[i], at::kInt, dev);
      n = out[0]->numel();
      shape(*out[0], names[0], {n});
      shape(*out[1], names[1], {n});
      shape(*out[2], names[2], {B + 1ll});
      shape(*out[3], names[3], {B});
      shape(*out[4], names[4], {4});
    }
    const int n_free = extent(free.numel(), "free_pages"), n_slots = extent(n, "out.slots");
    call("kvq_page_plan", [&] {
      return kvq_page_plan(i32(kv), i32(q), B, i32(table), (int)table.size(1), stride, i32(free), n_free, i32(head),
                           i32(head_out), P, i32(*out[0]), i32(*out[1]), n_slots, i32(*out[2]), i32(*out[3]),
                           i32(*out[4]), on.stream);
    });
    if (made.empty()) Py_RETURN_NONE;
    PyObject* r = PyTuple_New(5);
    for (int i = 0; r && i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(made[i]));
    return r;
  });
}

// page_release(done, kv_lens, block_table, free_pages, free_head, page_size, stream)
PyObject* page_release(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded([&]() -> PyObject* {
    expect(na, 7);
    int dev = -1;
    const at::Tensor& kv = cuda(a[1], "kv_lens", at::kInt, dev);
    if (kv.dim() != 1) refuse(PyExc_ValueError, "kv_lens must be a 1-D tensor");
    const int B = extent(kv.size(0), "kv_lens");
    const at::Tensor& any = tensor(a[0], "done");
    if (any.scalar_type() != at::kBool && any.scalar_type() != at::kByte)
      refuse(PyExc_ValueError, "done must be a bool or uint8 tensor");
    const at::Tensor& done = cuda(a[0], "done", any.scalar_type(), dev);
    shape(done, "done", {B});
    const at::Tensor& table = cuda(a[2], "block_table", at::kInt, dev, false);
    const int64_t stride = block_table(table, B);
    const at::Tensor& free = cuda(a[3], "free_pages", at::kInt, dev);
    const at::Tensor& head = cuda(a[4], "free_head", at::kInt, dev);
    shape(head, "free_head", {1});
    const int P = (int)integer(a[5], "page_size"), n_free = extent(free.numel(), "free_pages");
    On on(dev, a[6]);
    call("kvq_page_release", [&] {
      return kvq_page_release(u8(done), i32(kv), i32(table), stride, B, (int)table.size(1), P, i32(free), n_free,
                              i32(head), on.stream);
    });
    Py_RETURN_NONE;
  });
}

// encode_paged(jobs, slots, stream)
PyObject* encode_paged(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded([&]() -> PyObject* {
    expect(na, 3);
    PyObject* seq = PySequence_Fast(a[0], "jobs must be a sequence of (plan, x, codes, scales)");
    if (!seq) return nullptr;
    struct Drop {
      PyObject* o;
      ~Drop() { Py_DECREF(o); }
    } drop{seq};
    const Py_ssize_t nj = PySequence_Fast_GET_SIZE(seq);
    if (nj == 0) Py_RETURN_NONE;
    if (nj > 4096) refuse(PyExc_ValueError, "more than 4096 jobs");
    std::vector<kvq_paged_encode_job> jobs((size_t)nj);
    int dev = -1;
    int64_t n = 0, H = 0;
    Pages g0{};
    const at::Tensor* slots = nullptr;
    for (Py_ssize_t i = 0; i < nj; ++i) {
      PyObject* j = PySequence_Fast_GET_ITEM(seq, i);
      if (!PyTuple_Check(j) || PyTuple_GET_SIZE(j) != 4)
        refuse(PyExc_TypeError, "jobs[%zd] must be a tuple (plan, x, codes, scales)", i);
      const PlanView p = plan(PyTuple_GET_ITEM(j, 0), "a job's plan");
      const at::Tensor& x = cuda(PyTuple_GET_ITEM(j, 1), "a job's x", at::kHalf, dev, false);
      if (x.dim() != 3 || (x.size(2) > 1 && x.stride(2) != 1))
        refuse(PyExc_ValueError, "jobs[%zd].x must be [n, Hkv, head_dim] with contiguous rows", i);
      same_dim(p, x.size(2));
      on_device(p, dev);
      const Pages g = pages(PyTuple_GET_ITEM(j, 2), PyTuple_GET_ITEM(j, 3), p, "a job's codes", "a job's scales", dev);
      if (g.H != x.size(1))
        refuse(PyExc_ValueError, "jobs[%zd]: x has %lld heads, the pages %lld", i, (long long)x.size(1), (long long)g.H);
      if (i == 0) {
        n = x.size(0);
        H = x.size(1);
        g0 = g;
        slots = &cuda(a[1], "slots", at::kInt, dev);
        shape(*slots, "slots", {n});
        extent(n, "x");
      } else if (x.size(0) != n || g.H != H || g.P != g0.P || g.n != g0.n) {
        refuse(PyExc_ValueError, "jobs[%zd] has other sizes than jobs[0]", i);
      }
      jobs[(size_t)i] = {p.handle, f16(x), u8(*g.codes), f16(*g.scales), x.stride(0), x.stride(1)};
    }
    if (n == 0 || H == 0) Py_RETURN_NONE;
    On on(dev, a[2]);
    call("kvq_encode_paged", [&] {
      return kvq_encode_paged(jobs.data(), (int)nj, (int)n, (int)H, (int)g0.P, (int)g0.n, i32(*slots), on.stream);
    });
    Py_RETURN_NONE;
  });
}

// decode_paged(plan, codes, scales, slots, out, stream) -> out
PyObject* decode_paged(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded([&]() -> PyObject* {
    expect(na, 6);
    const PlanView p = plan(a[0], "plan");
    int dev = -1;
    const Pages g = pages(a[1], a[2], p, "codes", "scales", dev);
    const at::Tensor& slots = cuda(a[3], "slots", at::kInt, dev);
    if (slots.dim() != 1) refuse(PyExc_ValueError, "slots must be a 1-D tensor");
    on_device(p, dev);
    const int64_t n = extent(slots.size(0), "slots");
    On on(dev, a[5]);
    at::Tensor made;
    const at::Tensor* out = &made;
    if (a[4] == Py_None) {
      made = fresh({n, g.H, p.D}, at::kHalf, dev);
    } else {
      out = &cuda(a[4], "out", at::kHalf, dev);
      shape(*out, "out", {n, g.H, p.D});
    }
    if (n > 0 && g.H > 0)
      call("kvq_decode_paged", [&] {
        return kvq_decode_paged(p.handle, u8(*g.codes), f16(*g.scales), (int)g.n, (int)g.P, (int)g.H, i32(slots),
                                (int)n, f16(*out), on.stream);
      });
    return THPVariable_Wrap(*out);
  });
}

// attend_paged(pk, pv, q, k_codes, k_scales, v_codes, v_scales, block_table, kv_lens, q_starts, max_q_len,
//              max_kv_len, window, softmax_scale, out, workspace, stream) -> out
PyObject* attend_paged(PyObject*, PyObject* const* a, Py_ssize_t na) {
  return guarded([&]() -> PyObject* {
    expect(na, 17);
    int dev = -1;
    const at::Tensor& q = cuda(a[2], "q", at::kHalf, dev, false);
    if (q.dim() != 3 || (q.size(2) > 1 && q.stride(2) != 1))
      refuse(PyExc_ValueError, "q must be [n, Hq, head_dim] with contiguous rows");
    const int n = extent(q.size(0), "q"), Hq = extent(q.size(1), "q");
    const int64_t D = q.size(2);
    const PlanView pk = plan(a[0], "pk"), pv = plan(a[1], "pv");
    same_dim(pk, D);
    same_dim(pv, D);
    on_device(pk, dev);
    on_device(pv, dev);
    const Pages k = pages(a[3], a[4], pk, "k_codes", "k_scales", dev);
    const Pages v = pages(a[5], a[6], pv, "v_codes", "v_scales", dev);
    if (k.n != v.n || k.H != v.H || k.P != v.P) refuse(PyExc_ValueError, "K and V pages differ in size");
    const at::Tensor& lens = cuda(a[8], "kv_lens", at::kInt, dev);
    if (lens.dim() != 1) refuse(PyExc_ValueError, "kv_lens must be 1-D");
    const int B = extent(lens.size(0), "kv_lens");
    const at::Tensor& table = cuda(a[7], "block_table", at::kInt, dev, false);
    const int64_t stride = block_table(table, B);
    const int32_t* starts = nullptr;
    if (a[9] != Py_None) {
      const at::Tensor& s = cuda(a[9], "q_starts", at::kInt, dev);
      shape(s, "q_starts", {B + 1ll});
      starts = i32(s);
    } else if (n != B) {
      refuse(PyExc_ValueError, "without q_starts every request has one query token: q has %d, kv_lens %d", n, B);
    }
    const int64_t max_q = a[10] == Py_None ? (starts ? std::max(1, n) : 1) : integer(a[10], "max_q_len");
    const int64_t cap = std::min<int64_t>(table.size(1) * k.P, 0x7fffffff - 256);
    const int64_t max_kv = a[11] == Py_None ? cap : integer(a[11], "max_kv_len");
    const int64_t window = integer(a[12], "window");
    const double sigma = PyFloat_AsDouble(a[13]);
    if (sigma == -1.0 && PyErr_Occurred()) return nullptr;
    On on(dev, a[16]);
    at::Tensor made, made_ws;
    const at::Tensor* out = &made;
    if (a[14] == Py_None) {
      made = fresh({n, Hq, D}, at::kHalf, dev);
    } else {
      out = &cuda(a[14], "out", at::kHalf, dev);
      shape(*out, "out", {n, Hq, D});
    }
    const at::Tensor* ws = &made_ws;
    if (a[15] == Py_None) {
      const size_t need = kvq_paged_workspace_size(std::max(B, 1), Hq, (int)std::max<int64_t>(k.H, 1), (int)D, n, (int)std::max<int64_t>(max_q, 1));
      made_ws = fresh({(int64_t)std::max<size_t>(need, 16)}, at::kByte, dev);
    } else {
      ws = &cuda(a[15], "workspace", at::kByte, dev);
    }
    call("kvq_attend_paged", [&] {
      return kvq_attend_paged(pk.handle, pv.handle, f16(q), q.stride(0), q.stride(1), u8(*k.codes), f16(*k.scales),
                              u8(*v.codes), f16(*v.scales), (int)k.n, (int)k.P, i32(table), (int)table.size(1), stride,
                              i32(lens), starts, B, n, Hq, (int)k.H, (int)max_q, (int)max_kv, (int)window, (float)sigma,
                              f16(*out), ws->data_ptr(), (size_t)ws->numel(), on.stream);
    });
    return THPVariable_Wrap(*out);
  });
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_check, f);
  Py_RETURN_NONE;
}

#define KVQ_FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KVQ_FAST(page_plan), KVQ_FAST(page_release), KVQ_FAST(encode_paged), KVQ_FAST(decode_paged),
                         KVQ_FAST(attend_paged), {"set_check", set_check, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
