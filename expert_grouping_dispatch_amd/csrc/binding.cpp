// Fast way into the C entry points of the experts' products in floating point
// for torch tensors (module _fast).  A call whose arguments are all as they
// should be -- tensors of the right types, shapes and layout on the current
// device -- goes to the library from here, on the current stream, and returns its
// status.  Any other call returns -1 and does nothing: the Python binding then
// checks the arguments one by one, names what is wrong, or calls with another
// device made current.  The smallest calls take 3 us on the GPU; the same checks
// in Python take 1.9 us of each call's 6.2 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe_experts_float.h"
#include "python_call.h"

#ifndef MOE_MADE_FOR  // the versions of torch and Python that this is compiled for, as the package compares them
#error "MOE_MADE_FOR is not defined"
#endif

namespace {

using moe::guarded;
using moe::kElse;
using moe::status;
using moe::unlocked;

// The tensors of a call: each is checked against the device of the first.
class Call {
 public:
  // The address of `o`, a contiguous tensor of type `t`, or nullptr with ok() false.
  void* at(PyObject* o, c10::ScalarType t, const at::Tensor** out = nullptr) {
    if (!ok_ || !THPVariable_Check(o)) return fail();
    const at::Tensor& v = THPVariable_Unpack(o);
    if (v.scalar_type() != t || v.layout() != c10::kStrided || !v.is_cuda() || !v.is_contiguous()) return fail();
    const int d = v.device().index();
    if (device_ < 0) device_ = d;
    if (d != device_) return fail();
    if (out != nullptr) *out = &v;
    return v.data_ptr();
  }
  void need(bool condition) { ok_ = ok_ && condition; }
  bool ok() const { return ok_; }
  // Whether the call can go from here: its device is the current one.
  bool ready(void** stream) {
    int now = -1;
    if (!ok_ || hipGetDevice(&now) != hipSuccess || now != device_) return false;
    *stream = c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(now)).stream();
    return true;
  }

 private:
  void* fail() {
    ok_ = false;
    return nullptr;
  }
  bool ok_ = true;
  int device_ = -1;
};

int64_t blocks(int64_t n) { return (n + MOE_F8_BLOCK - 1) / MOE_F8_BLOCK; }
bool is(const at::Tensor* t, int64_t a, int64_t b) { return t->dim() == 2 && t->size(0) == a && t->size(1) == b; }
bool is(const at::Tensor* t, int64_t a, int64_t b, int64_t c) {
  return t->dim() == 3 && t->size(0) == a && t->size(1) == b && t->size(2) == c;
}
// Sizes that the C entry points take as 32 bits.
bool fits(int64_t n) { return n >= 0 && n <= INT32_MAX; }

// A whole number that fits 32 bits, not negative.
bool number(PyObject* o, int64_t* out) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  *out = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0 && fits(*out);
}

constexpr auto kBf16 = c10::ScalarType::BFloat16, kF8 = c10::ScalarType::Float8_e4m3fn, kF32 = c10::ScalarType::Float,
               kU32 = c10::ScalarType::UInt32, kI32 = c10::ScalarType::Int, kI64 = c10::ScalarType::Long,
               kU8 = c10::ScalarType::Byte;

// (x, out_q, out_scales, row_count or None)
PyObject* quantize_f8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) return status(kElse);
  Call c;
  const at::Tensor *x = nullptr, *q = nullptr, *s = nullptr, *m = nullptr;
  const auto* px = static_cast<const uint16_t*>(c.at(a[0], kBf16, &x));
  auto* pq = static_cast<uint8_t*>(c.at(a[1], kF8, &q));
  auto* ps = static_cast<float*>(c.at(a[2], kF32, &s));
  const uint32_t* pm = nullptr;
  if (a[3] != Py_None) pm = static_cast<const uint32_t*>(c.at(a[3], kU32, &m));
  if (!c.ok() || x->dim() != 2 || (m != nullptr && m->numel() != 1)) return status(kElse);
  const int64_t rows = x->size(0), h = x->size(1);
  c.need(fits(h) && is(q, rows, h) && is(s, rows, blocks(h)));
  void* stream;
  if (!c.ready(&stream)) return status(kElse);
  return unlocked([&] { return moe_quantize_f8(px, rows, int32_t(h), pm, pq, ps, stream); });
}

// (input_tokens, top_k, restore_token_order, out_q, out_scales)
PyObject* dispatch_f8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int64_t k;
  if (n != 5 || !number(a[1], &k)) return status(kElse);
  Call c;
  const at::Tensor *x = nullptr, *r = nullptr, *q = nullptr, *s = nullptr;
  const auto* px = static_cast<const uint16_t*>(c.at(a[0], kBf16, &x));
  const auto* pr = static_cast<const uint32_t*>(c.at(a[2], kU32, &r));
  auto* pq = static_cast<uint8_t*>(c.at(a[3], kF8, &q));
  auto* ps = static_cast<float*>(c.at(a[4], kF32, &s));
  if (!c.ok() || x->dim() != 2 || q->dim() != 2) return status(kElse);
  const int64_t rows = x->size(0), h = x->size(1), out = q->size(0);
  c.need(fits(h) && fits(rows) && r->numel() == rows * k && is(q, out, h) && is(s, out, blocks(h)));
  void* stream;
  if (!c.ready(&stream)) return status(kElse);
  return unlocked([&] { return moe_dispatch_f8(px, rows, int32_t(h), int32_t(k), pr, pq, ps, out, stream); });
}

// What both grouped products have: the groups, the output and the sizes.
struct Grouped {
  const uint32_t* starts;
  const int32_t* ids;
  uint16_t* out;
  int64_t rows, depth, experts, n_out, halves;
  void* stream;
};
bool grouped(Call& c, const at::Tensor* a, const at::Tensor* w, PyObject* starts, PyObject* ids, PyObject* out,
             int64_t flags, Grouped* g) {
  const at::Tensor *ts = nullptr, *ti = nullptr, *to = nullptr;
  g->starts = static_cast<const uint32_t*>(c.at(starts, kU32, &ts));
  g->ids = static_cast<const int32_t*>(c.at(ids, kI32, &ti));
  g->out = static_cast<uint16_t*>(c.at(out, kBf16, &to));
  if (!c.ok() || a->dim() != 2 || w->dim() != 3) return false;
  g->rows = a->size(0);
  g->depth = a->size(1);
  g->experts = w->size(0);
  g->halves = (flags & MOE_MATMUL_SWIGLU) != 0 ? 2 : 1;
  g->n_out = w->size(1) / g->halves;
  c.need(fits(g->depth) && fits(g->experts) && fits(w->size(1)) && is(w, g->experts, g->halves * g->n_out, g->depth) &&
         is(to, g->rows, g->n_out) && ts->numel() == g->experts + 1 && ti->numel() == g->experts);
  return c.ok();
}

// (a, expert_start_indices, expert_ids, w, out, flags)
PyObject* expert_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int64_t flags;
  if (n != 6 || !number(a[5], &flags)) return status(kElse);
  Call c;
  Grouped g;
  const at::Tensor *ta = nullptr, *tw = nullptr;
  const auto* pa = static_cast<const uint16_t*>(c.at(a[0], kBf16, &ta));
  const auto* pw = static_cast<const uint16_t*>(c.at(a[3], kBf16, &tw));
  if (!c.ok() || !grouped(c, ta, tw, a[1], a[2], a[4], flags, &g) || !c.ready(&g.stream)) return status(kElse);
  return unlocked([&] {
    return moe_expert_matmul(pa, g.rows, g.starts, g.ids, int32_t(g.experts), pw, int32_t(g.n_out), int32_t(g.depth),
                             uint32_t(flags), g.out, g.stream);
  });
}

// (a_q, a_scales, expert_start_indices, expert_ids, w_q, w_scales, out, flags)
PyObject* expert_matmul_f8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int64_t flags;
  if (n != 8 || !number(a[7], &flags)) return status(kElse);
  Call c;
  Grouped g;
  const at::Tensor *ta = nullptr, *sa = nullptr, *tw = nullptr, *sw = nullptr;
  const auto* pa = static_cast<const uint8_t*>(c.at(a[0], kF8, &ta));
  const auto* psa = static_cast<const float*>(c.at(a[1], kF32, &sa));
  const auto* pw = static_cast<const uint8_t*>(c.at(a[4], kF8, &tw));
  const auto* psw = static_cast<const float*>(c.at(a[5], kF32, &sw));
  if (!c.ok() || !grouped(c, ta, tw, a[2], a[3], a[6], flags, &g)) return status(kElse);
  c.need(is(sa, g.rows, blocks(g.depth)) && is(sw, g.experts, g.halves * blocks(g.n_out), blocks(g.depth)));
  if (!c.ready(&g.stream)) return status(kElse);
  return unlocked([&] {
    return moe_expert_matmul_f8(pa, psa, g.rows, g.starts, g.ids, int32_t(g.experts), pw, psw, int32_t(g.n_out),
                                int32_t(g.depth), uint32_t(flags), g.out, g.stream);
  });
}

// (x, topk_ids, router_weights, w_gate_up, w_down, output_tokens, workspace, gate_up_scales, down_scales,
//  real_token_count or None, tp_rank), e4m3 weights
PyObject* layer_few_f8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int64_t rank;
  if (n != 11 || !number(a[10], &rank) || !THPVariable_Check(a[1])) return status(kElse);
  Call c;
  const bool wide = THPVariable_Unpack(a[1]).scalar_type() == kI64;
  const at::Tensor *x = nullptr, *ids = nullptr, *rw = nullptr, *gu = nullptr, *d = nullptr, *out = nullptr,
                   *space = nullptr, *sg = nullptr, *sd = nullptr, *m = nullptr;
  const auto* px = static_cast<const uint16_t*>(c.at(a[0], kBf16, &x));
  const void* pi = c.at(a[1], wide ? kI64 : kI32, &ids);
  const auto* pr = static_cast<const float*>(c.at(a[2], kF32, &rw));
  const auto* pg = static_cast<const uint8_t*>(c.at(a[3], kF8, &gu));
  const auto* pd = static_cast<const uint8_t*>(c.at(a[4], kF8, &d));
  auto* po = static_cast<uint16_t*>(c.at(a[5], kBf16, &out));
  void* ps = c.at(a[6], kU8, &space);
  const auto* psg = static_cast<const float*>(c.at(a[7], kF32, &sg));
  const auto* psd = static_cast<const float*>(c.at(a[8], kF32, &sd));
  const int32_t* pm = nullptr;
  if (a[9] != Py_None) pm = static_cast<const int32_t*>(c.at(a[9], kI32, &m));
  if (!c.ok() || x->dim() != 2 || ids->dim() != 2 || d->dim() != 3 || (m != nullptr && m->numel() != 1))
    return status(kElse);
  const int64_t rows = x->size(0), h = x->size(1), k = ids->size(1), e = d->size(0), i = d->size(2);
  c.need(fits(h) && fits(k) && fits(e) && fits(i) && ids->size(0) == rows && is(rw, rows, k) && is(out, rows, h) &&
         is(d, e, h, i) && is(gu, e, 2 * i, h) && is(sg, e, 2 * blocks(i), blocks(h)) &&
         is(sd, e, blocks(h), blocks(i)));
  void* s;
  if (!c.ready(&s)) return status(kElse);
  const size_t bytes = size_t(space->numel());
  return unlocked([&] {
    return wide ? moe_layer_few_f8_i64(px, rows, int32_t(h), int32_t(k), static_cast<const int64_t*>(pi), pr, pm,
                                       int32_t(rank), int32_t(e), pg, psg, pd, psd, int32_t(i), po, ps, bytes, s)
                : moe_layer_few_f8(px, rows, int32_t(h), int32_t(k), static_cast<const int32_t*>(pi), pr, pm,
                                   int32_t(rank), int32_t(e), pg, psg, pd, psd, int32_t(i), po, ps, bytes, s);
  });
}

#define MOE_METHOD(name) {#name, reinterpret_cast<PyCFunction>(&guarded<name>), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_METHOD(quantize_f8),     MOE_METHOD(dispatch_f8), MOE_METHOD(expert_matmul),
                         MOE_METHOD(expert_matmul_f8), MOE_METHOD(layer_few_f8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() {
  PyObject* const m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "made_for", MOE_MADE_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
