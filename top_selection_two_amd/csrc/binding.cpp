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

#include <initializer_list>
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

// The scales of 4-bit rows, where the cache has such.
void blocks(const Tensor& x, PyObject* o, const char* name,
            const at::Device& device, void** p, int64_t* page, int64_t* head,
            int64_t* slot) {
  if (x.scalar_type() != at::kFloat4_e2m1fn_x2) {
    if (o != Py_None)
      value_error(std::string(name) + ": only with a float4_e2m1fn_x2 cache");
    return;
  }
  if (o == Py_None)
    value_error(std::string(name) + ": needed with a float4_e2m1fn_x2 cache");
  const Tensor& b = tensor(o, name);
  if (x.size(3) % 16)
    value_error("rows of " + std::to_string(2 * x.size(3)) +
                " elements of 4 bits: expected a multiple of 32");
  expect(b, name, at::kFloat8_e8m0fnu,
         {x.size(0), x.size(1), x.size(2), x.size(3) / 16}, device, false);
  expect_unit(b, name);
  *p = pointer(b);
  *page = step_of(b, 0);
  *head = step_of(b, 1);
  *slot = step_of(b, 2);
}

Cache cache(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo,
            PyObject* kbo = Py_None, PyObject* vbo = Py_None) {
  const Tensor &k = tensor(ko, "k"), &v = tensor(vo, "v");
  Cache r;
  r.device = k.device();
  r.type = k.scalar_type();
  const Tensor* both[2] = {&k, &v};
  const char* names[2] = {"k", "v"};
  for (int i = 0; i < 2; ++i) {
    const Tensor& x = *both[i];
    const at::ScalarType t = x.scalar_type();
    if (t != at::kBFloat16 && t != at::kHalf && t != at::kFloat8_e4m3fn &&
        t != at::kFloat4_e2m1fn_x2)
      type_error(std::string(names[i]) + ": expected bfloat16, float16, "
                 "float8_e4m3fn or float4_e2m1fn_x2, got " + c10::toString(t));
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
  const int64_t dim = k.size(3) * (r.type == at::kFloat4_e2m1fn_x2 ? 2 : 1);
  if (dim > LIBTOPK_MAX_DIM || bytes % 16)
    value_error("rows of " + std::to_string(dim) + " elements of " +
                c10::toString(r.type) + ": expected at most " +
                std::to_string(LIBTOPK_MAX_DIM) +
                " and a multiple of 16 bytes");
  libtopk_cache_t& c = r.c;
  c = {};
  blocks(k, kbo, "k_blocks", r.device, &c.k_blocks, &c.k_block_page_stride,
         &c.k_block_head_stride, &c.k_block_slot_stride);
  blocks(v, vbo, "v_blocks", r.device, &c.v_blocks, &c.v_block_page_stride,
         &c.v_block_head_stride, &c.v_block_slot_stride);
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
  c.dim = (int32_t)dim;
  c.dtype = r.type == at::kBFloat16            ? LIBTOPK_BF16
            : r.type == at::kHalf              ? LIBTOPK_F16
            : r.type == at::kFloat4_e2m1fn_x2 ? LIBTOPK_E2M1
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

// The calls have no derivatives.  Where they make their outputs, one that is
// asked for, by the inputs `in` that outputs depend on smoothly, is an error and
// not zero: a tangent (forward mode) at once, a gradient where it is computed.
void refuse_tangents(const char* name, PyObject* const* a,
                     std::initializer_list<int> in) {
  for (int i : in)
    if (THPVariable_Check(a[i]) &&
        torch::autograd::isFwGradDefined(THPVariable_Unpack(a[i])))
      throw Refusal{PyExc_NotImplementedError,
                    std::string(name) + " has no forward-mode derivative"};
}
void refuse_gradients(const char* name, PyObject* const* a,
                      std::initializer_list<int> in,
                      std::initializer_list<const Tensor*> out) {
  if (!at::GradMode::is_enabled()) return;
  torch::autograd::edge_list edges;
  for (int i : in)
    if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).requires_grad())
      edges.push_back(
          torch::autograd::impl::gradient_edge(THPVariable_Unpack(a[i])));
  if (edges.empty()) return;
  const auto node =
      std::make_shared<torch::autograd::NotImplemented>(name, std::move(edges));
  for (const Tensor* x : out) torch::autograd::set_history(*x, node);
}

void expect_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("wrong number of arguments");
}

// Factors of the heads' rows: float32 [heads], or None.
const float* head_scale(const Cache& r, PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  const Tensor& x = tensor(o, name);
  expect(x, name, at::kFloat, {r.c.heads}, r.device);
  return (const float*)pointer(x);
}

// (q, k, v, table, lens, scale, weights, k_scale, v_scale, out, k_blocks,
// v_blocks)
PyObject* attend(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 12);
  const Cache r = cache(a[1], a[2], a[3], a[4], a[10], a[11]);
  const Tensor& q = tensor(a[0], "q");
  const at::ScalarType t = q.scalar_type();
  if (q.dim() != 3) value_error("q: expected [batch, query heads, dim]");
  if (t != at::kBFloat16 && t != at::kHalf)
    type_error(std::string("q: expected bfloat16 or float16, got ") +
               c10::toString(t));
  if (r.c.dtype != LIBTOPK_E4M3 && r.c.dtype != LIBTOPK_E2M1 && t != r.type)
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
  const float* scales[2] = {head_scale(r, a[7], "k_scale"),
                            head_scale(r, a[8], "v_scale")};
  libtopk_ledger_t l = {};
  const bool weights = a[6] != Py_None;
  const std::initializer_list<int> smooth = {0, 1, 2, 6, 7, 8};
  if (a[9] == Py_None) refuse_tangents("cache_attend", a, smooth);
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
  } else {
    refuse_gradients("cache_attend", a, smooth, {&out, &lse});
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
  const Cache r = cache(a[2], a[3], a[4], a[5]);  // (of no 4-bit type)
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

// (k, v, table, lens, seen, weights, positions, keep, sinks, recent, out,
// k_blocks, v_blocks)
PyObject* evict(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 13);
  const int32_t keep = integer(a[7], "keep", 1);
  const int32_t sinks = integer(a[8], "sinks", 0);
  const int32_t recent = integer(a[9], "recent", 0);
  const Cache r = cache(a[0], a[1], a[2], a[3], a[11], a[12]);
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
  for (int i : {0, 1, 11, 12})
    if (a[i] != Py_None) changed(tensor(a[i], ""));
  if (a[10] != Py_None) {
    changed(w);
    changed(pos);
  }
  PyObject* x = THPVariable_Wrap(std::move(w));
  PyObject* y = THPVariable_Wrap(std::move(pos));
  PyObject* z = THPVariable_Wrap(std::move(lens));
  return Py_BuildValue("(NNN)", x, y, z);
}

// (k_new, v_new, k, v, table, lens, starts, seen, q, freqs, interleaved,
// q_norm, k_norm, eps, k_scale, v_scale, weights, positions, k_blocks,
// v_blocks, out)
PyObject* extend(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 21);
  const Cache r = cache(a[2], a[3], a[4], a[5], a[18], a[19]);
  libtopk_tokens_t t = {};
  const Tensor& kn = tensor(a[0], "k_new");
  const at::ScalarType type = kn.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf)
    type_error(std::string("k_new: expected bfloat16 or float16, got ") +
               c10::toString(type));
  if (r.c.dtype != LIBTOPK_E4M3 && r.c.dtype != LIBTOPK_E2M1 && type != r.type)
    type_error(std::string("k_new is ") + c10::toString(type) +
               ", the cache " + c10::toString(r.type));
  if (kn.dim() != 3) value_error("k_new: expected [tokens, heads, dim]");
  const int64_t tokens = kn.size(0);
  if (tokens > INT32_MAX) value_error("k_new: 2^31 tokens or more");
  struct Rows {
    int arg;
    const char* name;
    const void** p;
    int64_t *token, *head;
  };
  const void* out_p = nullptr;
  const Rows in[3] = {{0, "k_new", &t.k, &t.k_token_stride, &t.k_head_stride},
                      {1, "v_new", &t.v, &t.v_token_stride, &t.v_head_stride},
                      {8, "q", &t.q, &t.q_token_stride, &t.q_head_stride}};
  const bool queries = a[8] != Py_None;
  int64_t q_heads = 0;
  for (int i = 0; i < (queries ? 3 : 2); ++i) {
    const Tensor& x = tensor(a[in[i].arg], in[i].name);
    if (i == 2) {
      if (x.dim() != 3) value_error("q: expected [tokens, query heads, dim]");
      q_heads = x.size(1);
      if (q_heads < 1 || q_heads > INT32_MAX)
        value_error("q: expected at least one head");
    }
    expect(x, in[i].name, type, {tokens, i == 2 ? q_heads : r.c.heads, r.c.dim},
           r.device, false);
    expect_unit(x, in[i].name);
    *in[i].p = pointer(x);
    *in[i].token = step_of(x, 0);
    *in[i].head = step_of(x, 1);
  }
  const Tensor& starts = tensor(a[6], "starts");
  expect(starts, "starts", at::kInt, {(int64_t)r.c.batch + 1}, r.device);
  t.starts = (const int32_t*)pointer(starts);
  if (a[7] != Py_None) {
    const Tensor& seen = tensor(a[7], "seen");
    expect(seen, "seen", at::kInt, {r.c.batch}, r.device);
    t.seen = (const int32_t*)pointer(seen);
  }
  if (a[9] != Py_None) {
    const Tensor& f = tensor(a[9], "freqs");
    if (f.dim() != 1) value_error("freqs: expected [pairs that turn]");
    expect(f, "freqs", at::kFloat, f.sizes(), r.device);
    if (2 * f.size(0) > r.c.dim || f.size(0) % 8)
      value_error("freqs: expected a multiple of 8 and at most " +
                  std::to_string(r.c.dim / 2) + " of them");
    t.freqs = (const float*)pointer(f);
    t.rot = (int32_t)(2 * f.size(0));
  }
  const int turn = PyObject_IsTrue(a[10]);
  if (turn < 0) throw PythonError{};
  t.interleaved = turn;
  t.norm_dtype = type == at::kBFloat16 ? LIBTOPK_BF16 : LIBTOPK_F16;
  t.dtype = t.norm_dtype;
  at::ScalarType norm{};
  for (int i : {0, 1}) {
    if (a[11 + i] == Py_None) continue;
    const char* name = i ? "k_norm" : "q_norm";
    const Tensor& x = tensor(a[11 + i], name);
    if (x.scalar_type() != type && x.scalar_type() != at::kFloat)
      type_error(std::string(name) + ": expected float32 or " +
                 c10::toString(type) + ", got " + c10::toString(x.scalar_type()));
    if (i && a[11] != Py_None && x.scalar_type() != norm)
      type_error("q_norm and k_norm: expected one type");
    norm = x.scalar_type();
    expect(x, name, norm, {r.c.dim}, r.device);
    if (norm == at::kFloat) t.norm_dtype = LIBTOPK_F32;
    (i ? t.k_norm : t.q_norm) = pointer(x);
  }
  const double eps = PyFloat_AsDouble(a[13]);
  if (PyErr_Occurred()) throw PythonError{};
  if (!(eps >= 0)) value_error("eps: expected a number of at least 0");
  t.eps = (float)eps;
  t.k_scale = head_scale(r, a[14], "k_scale");
  t.v_scale = head_scale(r, a[15], "v_scale");
  if ((a[16] == Py_None) != (a[17] == Py_None))
    value_error("weights and positions: expected both or neither");
  libtopk_ledger_t l = {};
  const bool led = a[16] != Py_None;
  if (led) l = ledger(r, a[16], "weights", a[17], "positions");
  const std::initializer_list<int> smooth = {8, 9, 11};
  if (queries && a[20] == Py_None) refuse_tangents("cache_extend", a, smooth);
  const libtopk_stream_t stream = stream_of(r.device);
  Tensor out;
  if (queries) {
    const Tensor& q = tensor(a[8], "q");
    if (a[20] == Py_None) {
      out = at::empty({tokens, q_heads, (int64_t)r.c.dim}, q.options());
      t.rest = 1;  // no row of it is left as memory happens to be
    } else {
      out = tensor(a[20], "out");
      expect(out, "out", type, q.sizes(), r.device, false);
      expect_unit(out, "out");
    }
    out_p = pointer(out);
    t.q_out = const_cast<void*>(out_p);
    t.q_out_token_stride = step_of(out, 0);
    t.q_out_head_stride = step_of(out, 1);
    // An array without elements has no address.
    if (tokens == 0) t.q = nullptr;
  } else if (a[20] != Py_None) {
    value_error("out: only with q");
  }
  t.tokens = (int32_t)tokens;
  t.q_heads = (int32_t)q_heads;
  Tensor lens = at::empty({r.c.batch}, starts.options());
  const c10::DeviceGuard guard(r.device);
  check(cache_extend(&r.c, &t, led ? &l : nullptr, (int32_t*)pointer(lens),
                     stream),
        "cache_extend");
  for (int i : {2, 3, 16, 17, 18, 19})
    if (a[i] != Py_None) changed(tensor(a[i], ""));
  PyObject* x = THPVariable_Wrap(std::move(lens));
  if (!queries) return Py_BuildValue("(NO)", x, Py_None);
  if (a[20] != Py_None) {
    changed(out);
  } else {
    refuse_gradients("cache_extend", a, smooth, {&out});
  }
  return Py_BuildValue("(NN)", x, THPVariable_Wrap(std::move(out)));
}

// (logits, u, temperature, top_k, top_p, min_p, out)
PyObject* sample(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 7);
  const Tensor& x = tensor(a[0], "logits");
  const at::ScalarType t = x.scalar_type();
  if (t != at::kFloat && t != at::kBFloat16 && t != at::kHalf)
    type_error(std::string("logits: expected float32, bfloat16 or float16, "
                           "got ") + c10::toString(t));
  if (x.dim() != 2) value_error("logits: expected [rows, vocabulary]");
  const int64_t rows = x.size(0), cols = x.size(1);
  if (cols < 1) value_error("logits: expected at least one column");
  expect_unit(x, "logits");
  const int64_t ld = rows > 1 ? x.stride(0) : cols;
  if (ld < cols) value_error("logits: expected rows that lie apart");
  const at::Device device = x.device();
  const Tensor& u = tensor(a[1], "u");
  expect(u, "u", at::kFloat, {rows}, device);
  libtopk_sampling_t how = {};
  const char* names[4] = {"temperature", "top_k", "top_p", "min_p"};
  const void* rowwise[4] = {};
  double all[4] = {};
  for (int i = 0; i < 4; ++i) {
    PyObject* o = a[2 + i];
    if (THPVariable_Check(o)) {
      const Tensor& s = THPVariable_Unpack(o);
      expect(s, names[i], i == 1 ? at::kInt : at::kFloat, {rows}, device);
      rowwise[i] = pointer(s);
    } else if (i == 1) {
      how.top_k_all = integer(o, names[i], 0);
    } else {
      all[i] = PyFloat_AsDouble(o);
      if (PyErr_Occurred()) throw PythonError{};
      if (!(all[i] >= 0))
        value_error(std::string(names[i]) + ": expected at least 0");
    }
  }
  how.temperature = (const float*)rowwise[0];
  how.top_k = (const int32_t*)rowwise[1];
  how.top_p = (const float*)rowwise[2];
  how.min_p = (const float*)rowwise[3];
  how.temperature_all = (float)all[0];
  how.top_p_all = (float)all[2];
  how.min_p_all = (float)all[3];
  if (a[6] != Py_None && (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 2))
    type_error("out: expected a pair of tensors");
  // (logprobs depend on u, top_k, top_p and min_p by steps alone)
  const std::initializer_list<int> smooth = {0, 2};
  if (a[6] == Py_None) refuse_tangents("sample_logits", a, smooth);
  const libtopk_stream_t stream = stream_of(device);
  Tensor tokens, logprobs;
  if (a[6] == Py_None) {
    tokens = at::empty({rows}, u.options().dtype(at::kLong));
    logprobs = at::empty({rows}, u.options());
  } else {
    tokens = tensor(PyTuple_GET_ITEM(a[6], 0), "out[0]");
    logprobs = tensor(PyTuple_GET_ITEM(a[6], 1), "out[1]");
    expect(tokens, "out[0]", at::kLong, {rows}, device);
    expect(logprobs, "out[1]", at::kFloat, {rows}, device);
  }
  const c10::DeviceGuard guard(device);
  check(sample_logits(pointer(x),
                      t == at::kFloat      ? LIBTOPK_F32
                      : t == at::kBFloat16 ? LIBTOPK_BF16
                                           : LIBTOPK_F16,
                      rows, cols, ld, &how, (const float*)pointer(u),
                      (int64_t*)pointer(tokens), (float*)pointer(logprobs),
                      stream),
        "sample_logits");
  if (a[6] != Py_None) {
    changed(tokens);
    changed(logprobs);
  } else {
    refuse_gradients("sample_logits", a, smooth, {&logprobs});
  }
  PyObject* y = THPVariable_Wrap(std::move(tokens));
  PyObject* z = THPVariable_Wrap(std::move(logprobs));
  return Py_BuildValue("(NN)", y, z);
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
                         LTK_ENTRY(extend),
                         LTK_ENTRY(sample),
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
