// The Python binding's marshalling for the cache_* calls: checks of tensors
// from their metadata, allocation of outputs, the current stream, and the
// call of the C entry point (include/libtopk.h).  Nothing is computed here.
//
// In C++ because these calls are made once a layer and token: the same checks
// through Python attributes and ctypes took 20 us a call, several times what
// the kernels of a short sequence take.
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>

#include <string>

#include "libtopk.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;       // LibtopkError(status, name)
PyObject* g_raw_stream = nullptr;  // torch's current stream of a device

// A refusal: what is raised.
struct Refusal {
  PyObject* type;
  std::string text;
};
struct PythonError {};  // already set

[[noreturn]] void type_error(const std::string& s) {
  throw Refusal{PyExc_TypeError, s};
}
[[noreturn]] void value_error(const std::string& s) {
  throw Refusal{PyExc_ValueError, s};
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i)
    t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    type_error(std::string(name) + ": expected a torch.Tensor");
  return THPVariable_Unpack(o);
}

void expect_type(const Tensor& x, const char* name, at::ScalarType t) {
  if (x.scalar_type() != t)
    type_error(std::string(name) + ": expected " + c10::toString(t) +
               ", got " + c10::toString(x.scalar_type()));
}

void expect(const Tensor& x, const char* name, at::ScalarType t,
            at::IntArrayRef shape, const at::Device& device,
            bool dense = true) {
  expect_type(x, name, t);
  if (x.device() != device)
    value_error(std::string(name) + ": expected a tensor on " +
                device.str() + ", got " + x.device().str());
  if (x.sizes() != shape)
    value_error(std::string(name) + ": expected shape " + shape_text(shape) +
                ", got " + shape_text(x.sizes()));
  if (dense && !x.is_contiguous())
    value_error(std::string(name) + ": expected a contiguous tensor");
}

void expect_unit(const Tensor& x, const char* name) {
  const int64_t d = x.dim() - 1;
  if (x.size(d) > 1 && x.stride(d) != 1)
    value_error(std::string(name) + ": expected unit stride in the last axis");
}

int64_t step_of(const Tensor& x, int64_t i) {
  return x.size(i) > 1 ? x.stride(i) : 0;
}

void* pointer(const Tensor& x) {
  return x.numel() ? x.data_ptr() : nullptr;
}

int32_t integer(PyObject* o, const char* name, int64_t least) {
  PyObject* n = PyNumber_Index(o);
  if (!n) throw PythonError{};
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(n, &over);
  Py_DECREF(n);
  if (over || v < least || v > INT32_MAX)
    value_error(std::string(name) + ": expected " + std::to_string(least) +
                " .. 2^31 - 1");
  return (int32_t)v;
}

struct Cache {
  libtopk_cache_t c;
  at::Device device{at::kCPU};
  at::ScalarType type{};
};

Cache cache(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo) {
  const Tensor &k = tensor(ko, "k"), &v = tensor(vo, "v");
  Cache r;
  r.device = k.device();
  r.type = k.scalar_type();
  const Tensor* both[2] = {&k, &v};
  const char* names[2] = {"k", "v"};
  for (int i = 0; i < 2; ++i) {
    const Tensor& x = *both[i];
    const at::ScalarType t = x.scalar_type();
    if (t != at::kBFloat16 && t != at::kHalf && t != at::kFloat8_e4m3fn)
      type_error(std::string(names[i]) + ": expected bfloat16, float16 or "
                 "float8_e4m3fn, got " + c10::toString(t));
    if (x.dim() != 4)
      value_error(std::string(names[i]) +
                  ": expected [pages, heads, page, dim]");
    if (x.size(1) < 1 || x.size(2) < 1 || x.size(3) < 1)
      value_error(std::string(names[i]) +
                  ": no axis but the pages may be empty");
    expect_unit(x, names[i]);
  }
  expect(v, "v", r.type, k.sizes(), r.device, false);
  const Tensor& table = tensor(to, "table");
  if (table.dim() != 2)
    value_error("table: expected [batch, pages of a sequence]");
  expect(table, "table", at::kInt, table.sizes(), r.device, false);
  if (table.size(1) < 1) value_error("table: expected at least one column");
  expect_unit(table, "table");
  const Tensor& lens = tensor(lo, "lens");
  expect(lens, "lens", at::kInt, {table.size(0)}, r.device);
  const int64_t bytes = k.size(3) * (int64_t)k.element_size();
  if (k.size(3) > LIBTOPK_MAX_DIM || bytes % 16)
    value_error("rows of " + std::to_string(k.size(3)) + " elements of " +
                c10::toString(r.type) + ": expected at most " +
                std::to_string(LIBTOPK_MAX_DIM) +
                " and a multiple of 16 bytes");
  libtopk_cache_t& c = r.c;
  c.k = pointer(k);
  c.v = pointer(v);
  c.k_page_stride = step_of(k, 0);
  c.k_head_stride = step_of(k, 1);
  c.k_slot_stride = step_of(k, 2);
  c.v_page_stride = step_of(v, 0);
  c.v_head_stride = step_of(v, 1);
  c.v_slot_stride = step_of(v, 2);
  c.pages = k.size(0);
  c.table_stride = step_of(table, 0);
  c.table = (const int32_t*)pointer(table);
  c.lens = (const int32_t*)pointer(lens);
  for (int64_t n : {table.size(0), table.size(1), k.size(1), k.size(2)})
    if (n > INT32_MAX) value_error("an axis of 2^31 or more");
  c.batch = (int32_t)table.size(0);
  c.table_width = (int32_t)table.size(1);
  c.heads = (int32_t)k.size(1);
  c.page = (int32_t)k.size(2);
  c.dim = (int32_t)k.size(3);
  c.dtype = r.type == at::kBFloat16 ? LIBTOPK_BF16
            : r.type == at::kHalf   ? LIBTOPK_F16
                                    : LIBTOPK_E4M3;
  return r;
}

// weights and, where given, positions: [batch, heads, slots].
libtopk_ledger_t ledger(const Cache& r, PyObject* wo, const char* wname,
                        PyObject* po, const char* pname) {
  libtopk_ledger_t l = {};
  int64_t slots = -1;
  for (int i = 0; i < (po ? 2 : 1); ++i) {
    const char* name = i ? pname : wname;
    PyObject* o = i ? po : wo;
    if (o == Py_None) value_error(std::string(name) + ": needed");
    const Tensor& x = tensor(o, name);
    if (x.dim() != 3)
      value_error(std::string(name) + ": expected [batch, heads, slots]");
    if (slots < 0) slots = x.size(2);
    expect(x, name, i ? at::kInt : at::kFloat, {r.c.batch, r.c.heads, slots},
           r.device, false);
    if (slots < 1 || slots > INT32_MAX)
      value_error(std::string(name) + ": expected 1 .. 2^31 - 1 slots");
    expect_unit(x, name);
    (i ? l.positions_batch_stride : l.weights_batch_stride) = step_of(x, 0);
    (i ? l.positions_head_stride : l.weights_head_stride) = step_of(x, 1);
    if (i)
      l.positions = (int32_t*)pointer(x);
    else
      l.weights = (float*)pointer(x);
  }
  l.slots = (int32_t)slots;
  return l;
}

// Torch's current stream on the device, as the C interface takes it.
libtopk_stream_t stream_of(const at::Device& d) {
  if (!d.is_cuda())
    value_error("expected device tensors, got " + d.str());
  PyObject* i = PyLong_FromLong(d.index());
  PyObject* s = i ? PyObject_CallOneArg(g_raw_stream, i) : nullptr;
  Py_XDECREF(i);
  if (!s) throw PythonError{};
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (PyErr_Occurred()) throw PythonError{};
  return (libtopk_stream_t)p;
}

void check(int rc, const char* name) {
  if (rc == LIBTOPK_OK) return;
  if (g_error) {
    PyObject* e = PyObject_CallFunction(g_error, "is", rc, name);
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  } else {
    PyErr_Format(PyExc_RuntimeError, "%s failed (status %d)", name, rc);
  }
  throw PythonError{};
}

// A tensor that a call has changed: gradients that need what it held are
// refused from here on.  (Inference tensors count no changes.)
void changed(const Tensor& x) {
  if (!x.is_inference()) x.unsafeGetTensorImpl()->bump_version();
}

void expect_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("wrong number of arguments");
}

// (q, k, v, table, lens, scale, weights, k_scale, v_scale, out)
PyObject* attend(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 10);
  const Cache r = cache(a[1], a[2], a[3], a[4]);
  const Tensor& q = tensor(a[0], "q");
  const at::ScalarType t = q.scalar_type();
  if (q.dim() != 3) value_error("q: expected [batch, query heads, dim]");
  if (t != at::kBFloat16 && t != at::kHalf)
    type_error(std::string("q: expected bfloat16 or float16, got ") +
               c10::toString(t));
  if (r.c.dtype != LIBTOPK_E4M3 && t != r.type)
    type_error(std::string("q is ") + c10::toString(t) + ", the cache " +
               c10::toString(r.type));
  const int64_t heads = q.size(1);
  expect(q, "q", t, {r.c.batch, heads, r.c.dim}, r.device, false);
  if (heads < 1 || heads > INT32_MAX || heads % r.c.heads)
    value_error("q: " + std::to_string(heads) + " query heads over " +
                std::to_string(r.c.heads) + " heads");
  expect_unit(q, "q");
  double scale = 0;
  if (a[5] == Py_None) {
    scale = 1.0 / std::sqrt((double)r.c.dim);
  } else {
    scale = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) throw PythonError{};
  }
  const float* scales[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i) {
    if (a[7 + i] == Py_None) continue;
    const char* name = i ? "v_scale" : "k_scale";
    const Tensor& x = tensor(a[7 + i], name);
    expect(x, name, at::kFloat, {r.c.heads}, r.device);
    scales[i] = (const float*)pointer(x);
  }
  libtopk_ledger_t l = {};
  const bool weights = a[6] != Py_None;
  if (weights) l = ledger(r, a[6], "weights", nullptr, nullptr);
  const libtopk_stream_t stream = [&] {
    if (a[9] != Py_None && (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 2))
      type_error("out: expected a pair of tensors");
    return stream_of(r.device);
  }();
  Tensor out, lse;
  if (a[9] == Py_None) {
    out = at::empty({r.c.batch, heads, r.c.dim}, q.options());
    lse = at::empty({r.c.batch, heads}, q.options().dtype(at::kFloat));
  } else {
    out = tensor(PyTuple_GET_ITEM(a[9], 0), "out");
    lse = tensor(PyTuple_GET_ITEM(a[9], 1), "lse");
    expect(out, "out", t, {r.c.batch, heads, r.c.dim}, r.device);
    expect(lse, "lse", at::kFloat, {r.c.batch, heads}, r.device);
  }
  const c10::DeviceGuard guard(r.device);
  check(cache_attend(&r.c, pointer(q),
                     t == at::kBFloat16 ? LIBTOPK_BF16 : LIBTOPK_F16,
                     (int32_t)heads, step_of(q, 0), step_of(q, 1), (float)scale,
                     scales[0], scales[1], weights ? &l : nullptr,
                     pointer(out), (float*)pointer(lse), stream),
        "cache_attend");
  if (weights) changed(tensor(a[6], "weights"));
  if (a[9] != Py_None) {
    changed(out);
    changed(lse);
  } else if (at::GradMode::is_enabled()) {
    // There is no backward pass: one that is asked for is an error, and not a
    // gradient of zero.
    torch::autograd::edge_list edges;
    for (int i : {0, 1, 2, 6, 7, 8}) {
      if (a[i] == Py_None) continue;
      const Tensor& x = tensor(a[i], "");
      if (x.requires_grad())
        edges.push_back(torch::autograd::impl::gradient_edge(x));
    }
    if (!edges.empty()) {
      const auto node = std::make_shared<torch::autograd::NotImplemented>(
          "cache_attend", std::move(edges));
      torch::autograd::set_history(out, node);
      torch::autograd::set_history(lse, node);
    }
  }
  PyObject* o = THPVariable_Wrap(std::move(out));
  PyObject* z = THPVariable_Wrap(std::move(lse));
  return Py_BuildValue("(NN)", o, z);
}

// (k_new, v_new, k, v, table, lens, limit, seen, weights, positions, sinks,
// recent)
PyObject* append(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 12);
  const int32_t limit = integer(a[6], "limit", 1);
  const int32_t sinks = integer(a[10], "sinks", 0);
  const int32_t recent = integer(a[11], "recent", 0);
  const Cache r = cache(a[2], a[3], a[4], a[5]);
  const libtopk_ledger_t l = ledger(r, a[8], "weights", a[9], "positions");
  const Tensor &kn = tensor(a[0], "k_new"), &vn = tensor(a[1], "v_new");
  const Tensor* both[2] = {&kn, &vn};
  for (int i = 0; i < 2; ++i) {
    const char* name = i ? "v_new" : "k_new";
    expect(*both[i], name, r.type, {r.c.batch, r.c.heads, r.c.dim}, r.device,
           false);
    expect_unit(*both[i], name);
  }
  for (int i = 0; i < 2; ++i)
    if (step_of(kn, i) != step_of(vn, i))
      value_error("k_new and v_new: expected the same strides");
  const Tensor& seen = tensor(a[7], "seen");
  expect(seen, "seen", at::kInt, {r.c.batch}, r.device);
  const libtopk_stream_t stream = stream_of(r.device);
  Tensor lens = at::empty({r.c.batch}, seen.options());
  Tensor slots = at::empty({r.c.batch, r.c.heads}, seen.options());
  const c10::DeviceGuard guard(r.device);
  check(cache_append(&r.c, pointer(kn), pointer(vn), step_of(kn, 0),
                     step_of(kn, 1), limit, (const int32_t*)pointer(seen), &l,
                     sinks, recent, (int32_t*)pointer(lens),
                     (int32_t*)pointer(slots), stream),
        "cache_append");
  for (int i : {2, 3, 8, 9}) changed(tensor(a[i], ""));
  PyObject* x = THPVariable_Wrap(std::move(lens));
  PyObject* y = THPVariable_Wrap(std::move(slots));
  return Py_BuildValue("(NN)", x, y);
}

// (k, v, table, lens, seen, weights, positions, keep, sinks, recent, out)
PyObject* evict(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 11);
  const int32_t keep = integer(a[7], "keep", 1);
  const int32_t sinks = integer(a[8], "sinks", 0);
  const int32_t recent = integer(a[9], "recent", 0);
  const Cache r = cache(a[0], a[1], a[2], a[3]);
  const libtopk_ledger_t l = ledger(r, a[5], "weights", a[6], "positions");
  const Tensor& seen = tensor(a[4], "seen");
  expect(seen, "seen", at::kInt, {r.c.batch}, r.device);
  libtopk_ledger_t after = {};
  if (a[10] != Py_None) {
    if (!PyTuple_Check(a[10]) || PyTuple_GET_SIZE(a[10]) != 2)
      type_error("out: expected a pair of tensors");
    after = ledger(r, PyTuple_GET_ITEM(a[10], 0), "out[0]",
                   PyTuple_GET_ITEM(a[10], 1), "out[1]");
    if (after.slots != keep)
      value_error("out: expected [batch, heads, " + std::to_string(keep) +
                  "]");
  }
  const libtopk_stream_t stream = stream_of(r.device);
  Tensor w, pos;
  if (a[10] == Py_None) {
    pos = at::empty({r.c.batch, r.c.heads, keep}, seen.options());
    w = at::empty({r.c.batch, r.c.heads, keep},
                  seen.options().dtype(at::kFloat));
    after = {(float*)pointer(w), (int32_t*)pointer(pos), step_of(w, 0),
             step_of(w, 1), step_of(pos, 0), step_of(pos, 1), keep};
  } else {
    w = THPVariable_Unpack(PyTuple_GET_ITEM(a[10], 0));
    pos = THPVariable_Unpack(PyTuple_GET_ITEM(a[10], 1));
  }
  Tensor lens = at::empty({r.c.batch}, seen.options());
  const c10::DeviceGuard guard(r.device);
  check(cache_evict(&r.c, (const int32_t*)pointer(seen), &l, keep, sinks,
                    recent, &after, (int32_t*)pointer(lens), stream),
        "cache_evict");
  for (int i : {0, 1}) changed(tensor(a[i], ""));
  if (a[10] != Py_None) {
    changed(w);
    changed(pos);
  }
  PyObject* x = THPVariable_Wrap(std::move(w));
  PyObject* y = THPVariable_Wrap(std::move(pos));
  PyObject* z = THPVariable_Wrap(std::move(lens));
  return Py_BuildValue("(NNN)", x, y, z);
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define LTK_ENTRY(f) \
  {#f, (PyCFunction)(void (*)(void))entry<f>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LTK_ENTRY(attend),
                         LTK_ENTRY(append),
                         LTK_ENTRY(evict),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject* c = PyImport_ImportModule("torch._C");
  if (!c) return nullptr;
  g_raw_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_DECREF(c);
  if (!g_raw_stream) return nullptr;
  return PyModule_Create(&module);
}
