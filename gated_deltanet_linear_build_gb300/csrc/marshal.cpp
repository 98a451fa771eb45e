// Argument marshalling of the attention-side calls for Python: checks dtypes,
// shapes and strides of torch tensors and passes device pointers, sizes and the
// current CUDA stream to the C entry point of the same name. No arithmetic of
// the method happens here. A step of a few tokens is over in 3 to 8 us on the
// GPU, and the same checks written in Python took 8 to 11 us a call (a tensor
// attribute is 0.1 us, a ctypes argument 0.08 us); here they take under one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>

#include <ATen/core/TensorBase.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gdn.h"

namespace {

struct Refused {                       // a failed check: ValueError
  const char* what;
};

int current_device = 0;                // of the call that runs (under the interpreter's lock)

const at::TensorBase& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refused{what};
  const at::TensorBase& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw Refused{what};
  if (t.get_device() != current_device) throw Refused{"a tensor is not on the current device"};
  return t;
}
// A contiguous tensor of `dim` dimensions.
const at::TensorBase& packed(PyObject* o, at::ScalarType type, int64_t dim, const char* what) {
  const at::TensorBase& t = tensor(o, what);
  if (t.scalar_type() != type || t.dim() != dim || !t.is_contiguous()) throw Refused{what};
  return t;
}
template <typename T>
T* ptr(const at::TensorBase& t) { return static_cast<T*>(t.data_ptr()); }

// bfloat16 [T, H, d] with contiguous heads; its token stride in `stride`.
const at::TensorBase& rows(PyObject* o, int64_t* stride, const char* what) {
  const at::TensorBase& t = tensor(o, what);
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3) throw Refused{what};
  const int64_t T = t.size(0), H = t.size(1), d = t.size(2);
  if ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && H > 1)) throw Refused{what};
  *stride = T > 1 ? t.stride(0) : H * d;
  return t;
}
bool same(const at::TensorBase& a, const at::TensorBase& b) { return a.sizes() == b.sizes(); }

int32_t int32(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr};
  if (v != (int32_t)v) throw Refused{"an integer argument exceeds 32 bits"};
  return (int32_t)v;
}
int32_t fits(int64_t v) {
  if (v != (int32_t)v) throw Refused{"a size exceeds 32 bits"};
  return (int32_t)v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr};
  return (float)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{nullptr};
  return v != 0;
}
void* stream(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  void* s = PyLong_AsVoidPtr(o);
  if (!s && PyErr_Occurred()) throw Refused{nullptr};
  return s;
}

struct Cache {
  const at::TensorBase *k, *v, *ks, *vs;
  int32_t blocks, Hk, B, d;
};
Cache cache(PyObject* const* a) {
  Cache c;
  c.k = &tensor(a[0], "k_cache: an 8-bit CUDA tensor expected");
  c.v = &tensor(a[1], "v_cache: an 8-bit CUDA tensor expected");
  // e4m3 codes, or their bytes: another 8-bit type would be read as e4m3 all the same.
  for (const at::TensorBase* t : {c.k, c.v})
    if ((t->scalar_type() != at::kFloat8_e4m3fn && t->scalar_type() != at::kByte) || t->dim() != 4 ||
        !t->is_contiguous() || !same(*t, *c.k))
      throw Refused{"k_cache, v_cache: contiguous float8_e4m3fn or uint8 [num_blocks, Hk, B, d] expected"};
  c.ks = &packed(a[2], at::kFloat, 2, "k_scale: contiguous float32 [num_blocks, Hk] expected");
  c.vs = &packed(a[3], at::kFloat, 2, "v_scale: contiguous float32 [num_blocks, Hk] expected");
  for (const at::TensorBase* s : {c.ks, c.vs})
    if (s->size(0) != c.k->size(0) || s->size(1) != c.k->size(1))
      throw Refused{"k_scale, v_scale: [num_blocks, Hk] of the cache expected"};
  c.blocks = fits(c.k->size(0));
  c.Hk = fits(c.k->size(1));
  c.B = fits(c.k->size(2));
  c.d = fits(c.k->size(3));
  return c;
}

// Row stride of an int32 [N, M] table with contiguous rows.
int64_t table_stride(const at::TensorBase& t) {
  if (t.scalar_type() != at::kInt || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
    throw Refused{"block_table: int32 [N, M] with contiguous rows expected"};
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// Runs `body` (which returns a status) with the argument count checked, and C++
// exceptions turned into Python's.
template <typename F>
PyObject* call(Py_ssize_t n, Py_ssize_t want, F body) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    current_device = c10::cuda::current_device();
    return PyLong_FromLong(body());
  } catch (const Refused& r) {
    if (r.what) PyErr_SetString(PyExc_ValueError, r.what);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// cu_seqlens, context_lens, free_blocks, block_table, kv_lens, positions, slots,
// pieces, counts, block_tokens, device_status, stream
PyObject* build_block_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 12, [&]() -> int {
    const auto& cu = packed(a[0], at::kInt, 1, "cu_seqlens: contiguous int32 [N + 1] expected");
    const auto& ctx = packed(a[1], at::kInt, 1, "context_lens: contiguous int32 [N] expected");
    const auto& fr = packed(a[2], at::kInt, 1, "free_blocks: contiguous int32 [F] expected");
    const auto& table = tensor(a[3], "block_table: int32 [N, M] expected");
    const int64_t stride = table_stride(table), N = table.size(0), M = table.size(1);
    const auto& kv = packed(a[4], at::kInt, 1, "kv_lens: contiguous int32 [N] expected");
    const auto& pos = packed(a[5], at::kInt, 1, "positions: contiguous int32 [T] expected");
    const auto& slots = packed(a[6], at::kLong, 1, "slots: contiguous int64 [T] expected");
    const auto& pieces = packed(a[7], at::kInt, 2, "pieces: contiguous int32 [capacity, 4] expected");
    const auto& counts = packed(a[8], at::kInt, 1, "counts: contiguous int32 [2] expected");
    const int64_t T = pos.size(0);
    if (cu.size(0) != N + 1 || ctx.size(0) != N || kv.size(0) != N || slots.size(0) != T ||
        pieces.size(1) != 4 || counts.size(0) < 2)
      throw Refused{"build_block_tables: sizes do not agree"};
    int32_t* status = nullptr;
    if (a[10] != Py_None)
      status = ptr<int32_t>(packed(a[10], at::kInt, 1, "device_status: contiguous int32 [1] expected"));
    return gdn_build_block_tables(
        ptr<int32_t>(cu), ptr<int32_t>(ctx), ptr<int32_t>(fr), fits(fr.size(0)), fits(N), fits(T),
        int32(a[9]), ptr<int32_t>(table), stride, fits(M), ptr<int32_t>(kv), ptr<int32_t>(pos),
        ptr<int64_t>(slots), ptr<gdn_page_piece_t>(pieces), fits(pieces.size(0)), ptr<int32_t>(counts),
        status, stream(a[11]));
  });
}

// q, k, positions, phases, q_out, k_out, interleaved, inverse, scale, stream
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> int {
    int64_t qs, ks = 0, qos, kos = 0;
    const auto& q = rows(a[0], &qs, "q: bfloat16 [T, Hq, d] with contiguous heads expected");
    const auto& qo = rows(a[4], &qos, "q_out: bfloat16 [T, Hq, d] with contiguous heads expected");
    const auto& pos = packed(a[2], at::kInt, 1, "positions: contiguous int32 [T] expected");
    const auto& ph = packed(a[3], at::kLong, 1, "phases: contiguous int64 [rot_dim / 2] expected");
    const int64_t T = q.size(0), d = q.size(2);
    if (!same(q, qo) || pos.size(0) != T) throw Refused{"rotary: shapes do not agree"};
    void *kp = nullptr, *kop = nullptr;
    int64_t Hk = 0;
    if (a[1] != Py_None) {
      const auto& k = rows(a[1], &ks, "k: bfloat16 [T, Hk, d] with contiguous heads expected");
      const auto& ko = rows(a[5], &kos, "k_out: bfloat16 [T, Hk, d] with contiguous heads expected");
      if (!same(k, ko) || k.size(0) != T || k.size(2) != d) throw Refused{"rotary: shapes do not agree"};
      kp = k.data_ptr();
      kop = ko.data_ptr();
      Hk = k.size(1);
    }
    return gdn_rotary(q.data_ptr(), qs, kp, ks, ptr<int32_t>(pos), ptr<int64_t>(ph), qo.data_ptr(), qos,
                      kop, kos, fits(T), fits(q.size(1)), fits(Hk), fits(d), fits(2 * ph.size(0)),
                      truth(a[6]), truth(a[7]), real(a[8]), stream(a[9]));
  });
}

// q, k, v, positions, phases, pieces, num_pieces, q_out, k_cache, v_cache, k_scale,
// v_scale, interleaved, scale, stream
PyObject* rotary_kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 15, [&]() -> int {
    int64_t qs = 0, ks, vs, qos = 0;
    const auto& k = rows(a[1], &ks, "k: bfloat16 [T, Hk, d] with contiguous heads expected");
    const auto& v = rows(a[2], &vs, "v: bfloat16 [T, Hk, d] with contiguous heads expected");
    const Cache c = cache(a + 8);
    const int64_t T = k.size(0), d = k.size(2);
    if (!same(k, v) || k.size(1) != c.Hk || d != c.d)
      throw Refused{"rotary_kv_append: shapes do not agree"};
    const int32_t* pos = nullptr;
    const int64_t* ph = nullptr;
    int64_t rot = 0;
    if (a[4] != Py_None) {
      const auto& p = packed(a[3], at::kInt, 1, "positions: contiguous int32 [T] expected");
      const auto& f = packed(a[4], at::kLong, 1, "phases: contiguous int64 [rot_dim / 2] expected");
      if (p.size(0) != T) throw Refused{"rotary_kv_append: shapes do not agree"};
      pos = ptr<int32_t>(p);
      ph = ptr<int64_t>(f);
      rot = 2 * f.size(0);
    }
    void *qp = nullptr, *qop = nullptr;
    int64_t Hq = 0;
    if (a[0] != Py_None) {
      const auto& q = rows(a[0], &qs, "q: bfloat16 [T, Hq, d] with contiguous heads expected");
      const auto& qo = rows(a[7], &qos, "q_out: bfloat16 [T, Hq, d] with contiguous heads expected");
      if (!same(q, qo) || q.size(0) != T || q.size(2) != d)
        throw Refused{"rotary_kv_append: shapes do not agree"};
      qp = q.data_ptr();
      qop = qo.data_ptr();
      Hq = q.size(1);
    }
    const auto& pieces = packed(a[5], at::kInt, 2, "pieces: contiguous int32 [capacity, 4] expected");
    const auto& num = packed(a[6], at::kInt, 1, "num_pieces: contiguous int32 [1] expected");
    if (pieces.size(1) != 4 || num.size(0) < 1) throw Refused{"rotary_kv_append: shapes do not agree"};
    return gdn_rotary_kv_append(qp, qs, k.data_ptr(), ks, v.data_ptr(), vs, pos, ph,
                                ptr<gdn_page_piece_t>(pieces), ptr<int32_t>(num), fits(pieces.size(0)),
                                qop, qos, c.k->data_ptr(), c.v->data_ptr(), ptr<float>(*c.ks),
                                ptr<float>(*c.vs), c.blocks, c.B, fits(T), fits(Hq), c.Hk, c.d,
                                fits(rot), truth(a[12]), real(a[13]), stream(a[14]));
  });
}

// q, k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, kv_lens, o,
// workspace, softmax_scale, max_new_tokens, planned, stream
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 14, [&]() -> int {
    int64_t qs;
    const auto& q = rows(a[0], &qs, "q: bfloat16 [T, Hq, d] with contiguous heads expected");
    const Cache c = cache(a + 1);
    const auto& table = tensor(a[5], "block_table: int32 [N, M] expected");
    const int64_t stride = table_stride(table), N = table.size(0), M = table.size(1);
    const auto& cu = packed(a[6], at::kInt, 1, "cu_seqlens: contiguous int32 [N + 1] expected");
    const auto& kv = packed(a[7], at::kInt, 1, "kv_lens: contiguous int32 [N] expected");
    const auto& o = packed(a[8], at::kBFloat16, 3, "o: contiguous bfloat16 [T, Hq, d] expected");
    if (!same(q, o) || q.size(2) != c.d || cu.size(0) != N + 1 || kv.size(0) != N)
      throw Refused{"paged_attention: shapes do not agree"};
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[9] != Py_None) {
      const auto& w = tensor(a[9], "workspace: a CUDA tensor expected");
      if (!w.is_contiguous()) throw Refused{"workspace: a contiguous tensor expected"};
      ws = w.data_ptr();
      bytes = (size_t)w.numel() * w.element_size();
    }
    return gdn_paged_attention(q.data_ptr(), qs, c.k->data_ptr(), c.v->data_ptr(), ptr<float>(*c.ks),
                               ptr<float>(*c.vs), c.blocks, c.B, ptr<int32_t>(table), stride, fits(M),
                               ptr<int32_t>(cu), ptr<int32_t>(kv), fits(N), fits(q.size(0)),
                               int32(a[11]), o.data_ptr(), fits(q.size(1)), c.Hk, c.d, real(a[10]),
                               truth(a[12]) ? GDN_FLAG_PLANNED : 0, ws, bytes, stream(a[13]));
  });
}

#define GDN_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDN_METHOD(build_block_tables), GDN_METHOD(rotary), GDN_METHOD(rotary_kv_append),
                         GDN_METHOD(paged_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
