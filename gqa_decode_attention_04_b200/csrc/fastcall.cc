// Marshalling of the 4-bit attention, step, conversion and rotating-append calls without ctypes: the same
// checks as the Python binding's, asked of the tensors directly.  Each function calls the library's
// entry point whose address it is given and returns its status, or None if an argument is not what the
// call takes; the Python binding then goes its own way, which says what is wrong.  An append, of 25
// arguments, costs 13 us of host time through ctypes and 4.9 so, an attention 10 and 3.3; the smallest
// kernels take 2 and 7.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "gqa_int4.h"
#include "gqa_rope.h"

namespace {

// o as a contiguous CUDA tensor of this type on device dev, else nullptr.
const at::Tensor* tensor(PyObject* o, c10::ScalarType type, long dev, int dims, bool contiguous = true) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || t.dim() != dims) return nullptr;
  for (const int64_t n : t.sizes())
    if (n > INT_MAX) return nullptr;
  if (contiguous && !t.is_contiguous()) return nullptr;
  return &t;
}

// The stride between tokens of rows [T, heads, D], else -1.
int64_t row_stride(const at::Tensor& t) {
  const int64_t heads = t.size(1), d = t.size(2);
  if (t.is_contiguous()) return heads * d;
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)) return -1;
  return t.size(0) > 1 ? t.stride(0) : heads * d;
}

void* address(PyObject* o) { return PyLong_AsVoidPtr(o); }

// The entry point at an address, with the type that its header gives it.
#define ENTRY(name, o) reinterpret_cast<decltype(&name)>(address(o))

const int32_t* ints(const at::Tensor* t) { return static_cast<const int32_t*>(t->data_ptr()); }
const float* floats(const at::Tensor* t) { return static_cast<const float*>(t->data_ptr()); }

constexpr auto kBf16 = c10::ScalarType::BFloat16;
constexpr auto kByte = c10::ScalarType::Byte;
constexpr auto kInt = c10::ScalarType::Int;
constexpr auto kFloat = c10::ScalarType::Float;

#define WANT(x) \
  if (!(x)) Py_RETURN_NONE

// attend(fn, device, stream, q, kv_pages, block_table, seq_lens, out, scale, workspace, dims): one query
// token per sequence where q is to have three dimensions, several where it is to have four.
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  WANT(n == 11);
  const long dev = PyLong_AsLong(a[1]);
  void* stream = address(a[2]);
  const int dims = static_cast<int>(PyLong_AsLong(a[10]));
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *q = tensor(a[3], kBf16, dev, dims), *pool = tensor(a[4], kByte, dev, 4), *bt = tensor(a[5], kInt, dev, 2),
                   *sl = tensor(a[6], kInt, dev, 1), *out = tensor(a[7], kBf16, dev, dims), *ws = tensor(a[9], kByte, dev, 1);
  WANT(q && pool && bt && sl && out && ws);
  const int64_t d = q->size(dims - 1), heads = q->size(dims - 2), seqs = q->size(0);
  WANT(pool->size(3) == 18 * d && pool->size(2) <= 256 && bt->size(0) == seqs && sl->size(0) == seqs && out->sizes() == q->sizes());
  const double scale = a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return nullptr;
  const int B = static_cast<int>(seqs), H = static_cast<int>(heads), Hk = static_cast<int>(pool->size(1)), D = static_cast<int>(d),
            ps = static_cast<int>(16 * pool->size(2)), mb = static_cast<int>(bt->size(1)), P = static_cast<int>(pool->size(0));
  const size_t bytes = static_cast<size_t>(ws->numel());
  int status;
  if (dims == 3) {
    status = ENTRY(gqa_paged_decode_attn_int4, a[0])(q->data_ptr(), pool->data_ptr(), ints(bt), ints(sl), out->data_ptr(), B, H, Hk, D,
                                                     ps, static_cast<float>(scale), mb, P, ws->data_ptr(), bytes, stream);
  } else {
    status = ENTRY(gqa_paged_multi_query_attn_int4, a[0])(q->data_ptr(), pool->data_ptr(), ints(bt), ints(sl), out->data_ptr(), B,
                                                          static_cast<int>(q->size(1)), H, Hk, D, ps, static_cast<float>(scale), mb, P,
                                                          ws->data_ptr(), bytes, stream);
  }
  return PyLong_FromLong(status);
}

// convert(fn, device, stream, k_pages, v_pages, kv_pages, back): quantise, or with back != 0 dequantise.
PyObject* convert(PyObject*, PyObject* const* a, Py_ssize_t n) {
  WANT(n == 7);
  const long dev = PyLong_AsLong(a[1]), back = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *k = tensor(a[3], kBf16, dev, 4), *v = tensor(a[4], kBf16, dev, 4), *pool = tensor(a[5], kByte, dev, 4);
  WANT(k && v && pool && v->sizes() == k->sizes());
  const int64_t P = k->size(0), Hk = k->size(1), ps = k->size(2), d = k->size(3);
  WANT(ps % 16 == 0 && d <= 1024 && pool->size(0) == P && pool->size(1) == Hk && pool->size(2) == ps / 16 && pool->size(3) == 18 * d);
  void *x = k->data_ptr(), *y = v->data_ptr(), *z = pool->data_ptr();
  const int p = static_cast<int>(P), h = static_cast<int>(Hk), s = static_cast<int>(ps), dd = static_cast<int>(d);
  return PyLong_FromLong(back ? ENTRY(gqa_kv_dequantize_int4, a[0])(z, x, y, p, h, s, dd, address(a[2]))
                              : ENTRY(gqa_kv_quantize_int4, a[0])(x, y, z, p, h, s, dd, address(a[2])));
}

// rope(fn, device, stream, q, k_new, v_new, cos_sin, q_out, block_table, positions, seq_ids or None,
//      interleaved, pools...): pools are (k, v) in bf16, (k, v, k_scales, v_scales) in e4m3, or (kv,) in 4 bits.
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  WANT(n == 13 || n == 14 || n == 16);
  const long dev = PyLong_AsLong(a[1]);
  void* stream = address(a[2]);
  const int inter = PyObject_IsTrue(a[11]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *q = tensor(a[3], kBf16, dev, 3, false), *k = tensor(a[4], kBf16, dev, 3, false), *v = tensor(a[5], kBf16, dev, 3, false),
                   *cs = tensor(a[6], kFloat, dev, 2), *qo = tensor(a[7], kBf16, dev, 3), *bt = tensor(a[8], kInt, dev, 2),
                   *pos = tensor(a[9], kInt, dev, 1), *ids = nullptr;
  WANT(q && k && v && cs && qo && bt && pos);
  if (a[10] != Py_None) {
    ids = tensor(a[10], kInt, dev, 1);
    WANT(ids);
  }
  const at::Tensor* pool[4] = {};
  const auto type = n == 14 ? kBf16 : kByte;
  for (int i = 0; i < n - 12; ++i) {
    pool[i] = i < 2 ? tensor(a[12 + i], type, dev, 4) : tensor(a[12 + i], kFloat, dev, 1);
    WANT(pool[i]);
  }
  int64_t Hk = pool[0]->size(1), ps = pool[0]->size(2), d = pool[0]->size(3);
  if (n == 13) {
    WANT(d % 18 == 0 && ps <= 256);
    d /= 18;
    ps *= 16;
  } else {
    WANT(pool[1]->sizes() == pool[0]->sizes());
    if (n == 16) WANT(pool[2]->size(0) == Hk && pool[3]->size(0) == Hk);
  }
  const int64_t T = q->size(0), H = q->size(1);
  WANT(q->size(2) == d && k->size(0) == T && k->size(1) == Hk && k->size(2) == d && v->sizes() == k->sizes() &&
       qo->sizes() == q->sizes() && pos->size(0) == T && (ids ? ids->size(0) == T : bt->size(0) == T));
  const int64_t qs = row_stride(*q), ks = row_stride(*k), vs = row_stride(*v);
  WANT(qs >= 0 && ks >= 0 && vs >= 0);
  const int t = static_cast<int>(T), seqs = static_cast<int>(bt->size(0)), h = static_cast<int>(H), hk = static_cast<int>(Hk),
            dd = static_cast<int>(d), r = static_cast<int>(cs->size(1)), mp = static_cast<int>(cs->size(0)),
            page = static_cast<int>(ps), mb = static_cast<int>(bt->size(1)), P = static_cast<int>(pool[0]->size(0));
  const void *qp = q->data_ptr(), *kp = k->data_ptr(), *vp = v->data_ptr();
  const float* cp = floats(cs);
  const int32_t *tp = ints(bt), *pp = ints(pos), *ip = ids ? ints(ids) : nullptr;
  void *op = qo->data_ptr(), *p0 = pool[0]->data_ptr();
  int status;
  if (n == 13) {
    status = ENTRY(gqa_rope_kv_append_int4, a[0])(qp, kp, vp, cp, op, p0, tp, pp, ip, t, seqs, h, hk, dd, r, inter, mp, qs, ks, vs, page,
                                                  mb, P, stream);
  } else if (n == 14) {
    status = ENTRY(gqa_rope_kv_append, a[0])(qp, kp, vp, cp, op, p0, pool[1]->data_ptr(), tp, pp, ip, t, seqs, h, hk, dd, r, inter, mp,
                                             qs, ks, vs, page, mb, P, stream);
  } else {
    status = ENTRY(gqa_rope_kv_append_fp8, a[0])(qp, kp, vp, cp, op, p0, pool[1]->data_ptr(), floats(pool[2]), floats(pool[3]), tp, pp,
                                                 ip, t, seqs, h, hk, dd, r, inter, mp, qs, ks, vs, page, mb, P, stream);
  }
  return PyLong_FromLong(status);
}

// step(fn, device, stream, q, k_new, v_new, kv_pages, block_table, positions, seq_lens, cos_sin or None, interleaved,
//      q_rot (with cos_sin), out, scale, workspace)
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  WANT(n == 16);
  const long dev = PyLong_AsLong(a[1]);
  void* stream = address(a[2]);
  const int inter = PyObject_IsTrue(a[11]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor *q = tensor(a[3], kBf16, dev, 3), *k = tensor(a[4], kBf16, dev, 3), *v = tensor(a[5], kBf16, dev, 3),
                   *pool = tensor(a[6], kByte, dev, 4), *bt = tensor(a[7], kInt, dev, 2), *pos = tensor(a[8], kInt, dev, 1),
                   *sl = tensor(a[9], kInt, dev, 1), *out = tensor(a[13], kBf16, dev, 3), *ws = tensor(a[15], kByte, dev, 1);
  WANT(q && k && v && pool && bt && pos && sl && out && ws);
  const at::Tensor *cs = nullptr, *qr = nullptr;
  if (a[10] != Py_None) {
    cs = tensor(a[10], kFloat, dev, 2);
    qr = tensor(a[12], kBf16, dev, 3);
    WANT(cs && qr && qr->sizes() == q->sizes());
  } else {
    WANT(a[12] == Py_None);
  }
  const int64_t seqs = q->size(0), d = q->size(2), Hk = pool->size(1);
  WANT(pool->size(3) == 18 * d && pool->size(2) <= 256 && k->size(0) == seqs && k->size(1) == Hk && k->size(2) == d &&
       v->sizes() == k->sizes() && bt->size(0) == seqs && pos->size(0) == seqs && sl->size(0) == seqs && out->sizes() == q->sizes());
  const double scale = a[14] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : PyFloat_AsDouble(a[14]);
  if (PyErr_Occurred()) return nullptr;
  const int status = ENTRY(gqa_decode_step_int4, a[0])(
      q->data_ptr(), k->data_ptr(), v->data_ptr(), cs ? floats(cs) : nullptr, qr ? qr->data_ptr() : nullptr, pool->data_ptr(),
      ints(bt), ints(pos), ints(sl), out->data_ptr(), static_cast<int>(seqs), static_cast<int>(q->size(1)),
      static_cast<int>(Hk), static_cast<int>(d), cs ? static_cast<int>(cs->size(1)) : 0, inter, cs ? static_cast<int>(cs->size(0)) : 0,
      static_cast<int>(16 * pool->size(2)), static_cast<float>(scale), static_cast<int>(bt->size(1)),
      static_cast<int>(pool->size(0)), ws->data_ptr(), static_cast<size_t>(ws->numel()), stream);
  return PyLong_FromLong(status);
}

// A tensor without memory, sizes or strides of its own (one that a tracer makes) throws when it is asked
// for them: it is not what the call takes.
template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return f(self, a, n);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef kMethods[] = {
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<attend>)), METH_FASTCALL, nullptr},
    {"convert", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<convert>)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<rope>)), METH_FASTCALL, nullptr},
    {"step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<step>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&kModule); }
