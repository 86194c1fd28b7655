// Binding of the serving calls (include/sas_serving.h) as a CPython module:
// checks of the tensors, outputs, workspace, and the C call.
//
// A small step (one token a sequence, a few pages) takes the GPU three to six
// microseconds, and the same checks made in Python 11 to 19: this file makes
// them on the C++ tensors. Every function takes its arguments by position, as
// sas.py passes them (None where one is left out), runs on the device of its
// first tensor and launches on that device's current stream; outputs and
// workspace come from the same stream's allocator. No C++ exception leaves it.
#include <torch/csrc/python_headers.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/sas_serving.h"

namespace {

struct PyError {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const std::string& msg) {
  PyErr_SetString(type, msg.c_str());
  throw PyError{};
}

std::string dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kHalf: return "torch.float16";
    case at::kDouble: return "torch.float64";
    default: return c10::toString(t);
  }
}

std::string shape_name(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument; nullptr for None.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = true) {
  if (o == Py_None) {
    if (optional) return nullptr;
    raise(PyExc_TypeError, std::string(name) + " must be a tensor");
  }
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}

int64_t size_of(const at::Tensor& t, const char* name, int64_t dim, int64_t at) {
  if (t.dim() != dim)
    raise(PyExc_ValueError, std::string(name) + " must have " + std::to_string(dim) +
                                " dimensions (got shape " + shape_name(t.sizes()) + ")");
  return t.size(at);
}

int as_int(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is too large");
  return (int)v;
}

int int_arg(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return as_int(v, name);
}
int bool_arg(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError{};
  return v;
}
float float_arg(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return (float)v;
}

sas_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return SAS_BF16;
  if (t.scalar_type() == at::kFloat) return SAS_F32;
  raise(PyExc_TypeError, "unsupported dtype " + dtype_name(t.scalar_type()) + " (bf16 or fp32)");
}

// The call's device (that of its first tensor) and stream.
struct Place {
  int dev;
  c10::cuda::OptionalCUDAGuard guard;
  sas_stream_t stream;

  explicit Place(const at::Tensor& first) {
    if (!first.is_cuda()) raise(PyExc_ValueError, "tensors must all be on one CUDA device");
    dev = first.get_device();
    guard.set_index((c10::DeviceIndex)dev);
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  }

  void check(const at::Tensor& t, const char* name, at::ScalarType dt, at::IntArrayRef shape) const {
    if (!t.is_cuda() || t.get_device() != dev)
      raise(PyExc_ValueError, std::string("tensors must all be on one CUDA device (") + name +
                                  " is on " + t.device().str() + ")");
    if (t.scalar_type() != dt)
      raise(PyExc_TypeError, std::string(name) + " must be " + dtype_name(dt) + " (got " +
                                 dtype_name(t.scalar_type()) + ")");
    if (t.sizes() != shape)
      raise(PyExc_ValueError, std::string(name) + " must have shape " + shape_name(shape) +
                                  " (got " + shape_name(t.sizes()) + ")");
  }

  // Pointer of a contiguous tensor of this type and shape (nullptr passes).
  void* ptr(const at::Tensor* t, const char* name, at::ScalarType dt, at::IntArrayRef shape) const {
    if (!t) return nullptr;
    check(*t, name, dt, shape);
    if (!t->is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    return t->data_ptr();
  }
  int32_t* ints(const at::Tensor* t, const char* name, at::IntArrayRef shape) const {
    return static_cast<int32_t*>(ptr(t, name, at::kInt, shape));
  }

  // Pointer and element strides {batch, head, token} of a tensor whose rows are
  // contiguous.
  void* rows(const at::Tensor* t, const char* name, at::ScalarType dt, at::IntArrayRef shape,
             int64_t (&s)[3]) const {
    if (!t) return nullptr;
    check(*t, name, dt, shape);
    const at::IntArrayRef st = t->strides();
    if (st[3] != 1 && t->size(3) > 1)
      raise(PyExc_ValueError, std::string("the rows of ") + name + " must be contiguous");
    for (int i = 0; i < 3; ++i) s[i] = st[i];
    return t->data_ptr();
  }

  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dt) const {
    return at::detail::empty_cuda(shape, dt, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev),
                                  c10::nullopt);
  }
};

// Outputs of one call. Those below `limit` bytes are carved from one allocation
// (an allocation of its own costs 0.9 us, as much as the call's checks):
// contiguous tensors that share a storage, each from a 16-byte boundary, so that
// one of them that is kept holds less than N limit bytes. Larger ones have
// a storage of their own.
template <int N>
struct Outputs {
  int64_t elems = 0, at[N];
  at::Tensor t[N];

  int64_t padded(at::IntArrayRef s, int64_t per16) const {
    int64_t n = 1;
    for (int64_t d : s) n *= d;
    return (n + per16 - 1) / per16 * per16;
  }
  void make(const Place& pl, at::ScalarType dt, const at::IntArrayRef (&shapes)[N],
            const bool (&wanted)[N], int64_t limit) {
    const int64_t es = (int64_t)c10::elementSize(dt), per16 = 16 / es;
    int count = 0;
    for (int i = 0; i < N; ++i) {
      at[i] = -1;
      if (!wanted[i]) continue;
      const int64_t n = padded(shapes[i], per16);
      if (n * es >= limit) {
        t[i] = pl.empty(shapes[i], dt);
        continue;
      }
      at[i] = elems;
      elems += n;
      ++count;
    }
    if (count == 0) return;
    const at::Tensor base = pl.empty({elems}, dt);
    for (int i = 0; i < N; ++i) {
      if (at[i] < 0) continue;
      t[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(),
                                                      base.dtype());
      t[i].unsafeGetTensorImpl()->set_storage_offset(at[i]);
      t[i].unsafeGetTensorImpl()->set_sizes_contiguous(shapes[i]);
    }
  }
};

// Raises sas.SasError for a status that is not SAS_OK.
void check_status(const char* fn, sas_status st) {
  if (st == SAS_OK) return;
  PyObject* m = PyImport_ImportModule("gated_block_sparse_b200.sas");
  if (m) {
    PyObject* r = PyObject_CallMethod(m, "_raise", "sis", fn, (int)st, sas_last_error_message());
    Py_XDECREF(r);
    Py_DECREF(m);
  }
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
  throw PyError{};
}

// Output: the caller's tensor (a new reference) or a new one.
PyObject* give(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  PyObject* r = THPVariable_Wrap(made);
  if (!r) throw PyError{};
  return r;
}

PyObject* tuple_of(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_DECREF(o);
  }
  if (!t) throw PyError{};
  return t;
}

template <int N, typename F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, F f) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return f(args);
  } catch (const PyError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// rotary(q, inv_freq, k, pos, start, parents, interleaved, amplitude, inverse, qo, ko)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<11>(a, n, [](PyObject* const* a) -> PyObject* {
    const at::Tensor &q = *tensor(a[0], "q", false), &f = *tensor(a[1], "inv_freq", false);
    const at::Tensor *k = tensor(a[2], "k"), *pos = tensor(a[3], "pos"),
                     *start = tensor(a[4], "start"), *parents = tensor(a[5], "parents");
    const at::Tensor *qo = tensor(a[9], "qo"), *ko = tensor(a[10], "ko");
    const Place pl(q);
    const sas_dtype dt = dtype_of(q);
    const at::ScalarType st = q.scalar_type();
    const int64_t B = size_of(q, "q", 4, 0), Hq = q.size(1), N = q.size(2), d = q.size(3);
    const int64_t Hkv = k ? size_of(*k, "k", 4, 1) : 0, half = f.numel();
    const int64_t qshape[4] = {B, Hq, N, d}, kshape[4] = {B, Hkv, N, d};
    Outputs<2> made;
    made.make(pl, st, {qshape, kshape}, {!qo, k && !ko}, 1 << 20);  // used and dropped together
    if (!qo) qo = &made.t[0];
    if (k && !ko) ko = &made.t[1];
    int64_t s[4][3];
    void* pq = pl.rows(&q, "q", st, qshape, s[0]);
    void* pqo = pl.rows(qo, "qo", st, qshape, s[1]);
    void* pk = pl.rows(k, "k", st, kshape, s[2]);
    void* pko = k ? pl.rows(ko, "ko", st, kshape, s[3]) : nullptr;
    check_status("sas_rotary",
                 sas_rotary(pq, s[0], pqo, s[1], as_int(Hq, "Hq"), pk, k ? s[2] : nullptr, pko,
                            k ? s[3] : nullptr, as_int(Hkv, "Hkv"), dt, as_int(B, "B"),
                            as_int(N, "N"), as_int(d, "d"),
                            static_cast<float*>(pl.ptr(&f, "inv_freq", at::kFloat, {half})),
                            as_int(2 * half, "rot"), bool_arg(a[6]), float_arg(a[7]),
                            bool_arg(a[8]), pl.ints(pos, "pos", {B, N}),
                            pl.ints(start, "start", {B}), pl.ints(parents, "parents", {B, N}),
                            pl.stream));
    if (!k) return give(a[9], *qo);
    PyObject* r = give(a[9], *qo);
    return tuple_of({r, give(a[10], *ko)});
  });
}

// page_map(lens, nnew, block_table, free_pages, free_head, T, npages, slots, new_lens, taken, head)
PyObject* page_map(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<11>(a, n, [](PyObject* const* a) -> PyObject* {
    const at::Tensor &lens = *tensor(a[0], "lens", false), &nnew = *tensor(a[1], "nnew", false),
                     &table = *tensor(a[2], "block_table", false),
                     &fr = *tensor(a[3], "free_pages", false),
                     &head = *tensor(a[4], "free_head", false);
    const Place pl(lens);
    const int64_t B = size_of(lens, "lens", 1, 0), width = size_of(table, "block_table", 2, 1),
                  nfree = fr.numel();
    const int T = int_arg(a[5], "T"), npages = int_arg(a[6], "npages");
    if (T < 0) raise(PyExc_ValueError, "T must be >= 0");
    const at::Tensor* out[4] = {tensor(a[7], "slots"), tensor(a[8], "new_lens"),
                                tensor(a[9], "taken"), tensor(a[10], "head")};
    const int64_t s0[2] = {B, T}, s1[1] = {B}, s3[1] = {1};
    Outputs<4> made;
    // a loop keeps lengths and head, not slots
    made.make(pl, at::kInt, {s0, s1, s1, s3}, {!out[0], !out[1], !out[2], !out[3]}, 4096);
    for (int i = 0; i < 4; ++i)
      if (!out[i]) out[i] = &made.t[i];
    check_status("sas_page_map",
                 sas_page_map(pl.ints(&lens, "lens", {B}), pl.ints(&nnew, "nnew", {B}),
                              pl.ints(&table, "block_table", {B, width}),
                              pl.ints(&fr, "free_pages", {nfree}),
                              pl.ints(&head, "free_head", {1}), as_int(B, "B"), T,
                              as_int(width, "width"), npages, as_int(nfree, "nfree"),
                              pl.ints(out[0], "slots", {B, T}),
                              pl.ints(out[1], "new_lens", {B}), pl.ints(out[2], "taken", {B}),
                              pl.ints(out[3], "head", {1}), pl.stream));
    PyObject* r[4];
    for (int i = 0; i < 4; ++i) r[i] = give(a[7 + i], *out[i]);
    return tuple_of({r[0], r[1], r[2], r[3]});
  });
}

// cache_append(k, v, lens, kc, vc, ksum, ntok, rows, slots, inv_freq, interleaved, amplitude, q, out)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<14>(a, n, [](PyObject* const* a) -> PyObject* {
    const at::Tensor &k = *tensor(a[0], "k", false), &v = *tensor(a[1], "v", false),
                     &lens = *tensor(a[2], "lens", false), &kc = *tensor(a[3], "kc", false),
                     &vc = *tensor(a[4], "vc", false);
    const at::Tensor *ksum = tensor(a[5], "ksum"), *ntok = tensor(a[6], "ntok"),
                     *rows = tensor(a[7], "rows"), *slots = tensor(a[8], "slots"),
                     *f = tensor(a[9], "inv_freq"), *q = tensor(a[12], "q"),
                     *out = tensor(a[13], "out");
    const Place pl(k);
    const sas_dtype dt = dtype_of(k);
    const at::ScalarType st = k.scalar_type();
    const int64_t B = size_of(k, "k", 4, 0), Hkv = k.size(1), T = k.size(2), d = k.size(3);
    size_of(kc, "kc", 4, 0);
    const int64_t N = slots ? 0 : kc.size(2), npages = slots ? kc.size(0) : 0;
    const int64_t shape[4] = {B, Hkv, T, d};
    const int64_t cshape[4] = {slots ? npages : B, Hkv, slots ? 64 : N, d};
    const int64_t sshape[4] = {slots ? npages : B, Hkv, slots ? d : N / 64, d};
    const int64_t Hq = q ? size_of(*q, "q", 4, 1) : Hkv, half = f ? f->numel() : 0;
    const int64_t qshape[4] = {B, Hq, T, d};
    if (out && !q) raise(PyExc_ValueError, "out goes with q");
    at::Tensor made;
    if (q && !out) out = &(made = pl.empty(qshape, st));
    int64_t s[3][3];
    void* pq = pl.rows(q, "q", st, qshape, s[0]);
    void* pk = pl.rows(&k, "k", st, shape, s[1]);
    void* pv = pl.rows(&v, "v", st, shape, s[2]);
    void* ps = ksum ? pl.ptr(ksum, "ksum", ksum->scalar_type(),
                             at::IntArrayRef(sshape, slots ? 3 : 4))
                    : nullptr;
    check_status(
        "sas_cache_append",
        sas_cache_append(pq, q ? s[0] : nullptr, pl.ptr(out, "out", st, qshape), pk, s[1], pv, s[2],
                         dt, as_int(B, "B"), as_int(Hq, "Hq"), as_int(Hkv, "Hkv"), as_int(T, "T"),
                         as_int(d, "d"), pl.ints(rows, "rows", {B, T}),
                         pl.ints(&lens, "lens", {B}), pl.ints(ntok, "ntok", {B}),
                         static_cast<float*>(pl.ptr(f, "inv_freq", at::kFloat, {half})),
                         as_int(2 * half, "rot"), bool_arg(a[10]), float_arg(a[11]),
                         pl.ints(slots, "slots", {B, T}), pl.ptr(&kc, "kc", st, cshape),
                         pl.ptr(&vc, "vc", st, cshape), as_int(N, "N"), as_int(npages, "npages"),
                         ps, ksum ? dtype_of(*ksum) : SAS_F32, pl.stream));
    if (!q) Py_RETURN_NONE;
    return give(a[13], *out);
  });
}

// decode_tree(q, kd, vd, kc, vc, lens, ksum, topk, parents, ntok, block_table, gated, scale, out,
//             idx_out, ws)
PyObject* decode_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<16>(a, n, [](PyObject* const* a) -> PyObject* {
    const at::Tensor &q = *tensor(a[0], "q", false), &kd = *tensor(a[1], "kd", false),
                     &vd = *tensor(a[2], "vd", false), &kc = *tensor(a[3], "kc", false),
                     &vc = *tensor(a[4], "vc", false), &lens = *tensor(a[5], "lens", false);
    const at::Tensor *ksum = tensor(a[6], "ksum"), *parents = tensor(a[8], "parents"),
                     *ntok = tensor(a[9], "ntok"), *table = tensor(a[10], "block_table"),
                     *out = tensor(a[13], "out"), *idx = tensor(a[14], "idx_out"),
                     *ws = tensor(a[15], "ws");
    const Place pl(q);
    const sas_dtype dt = dtype_of(q);
    const at::ScalarType st = q.scalar_type();
    const int64_t B = size_of(q, "q", 4, 0), Hq = q.size(1), T = q.size(2), d = q.size(3);
    const int64_t Hkv = size_of(kd, "kd", 4, 1);
    size_of(kc, "kc", 4, 0);
    const int64_t N = table ? 64 * size_of(*table, "block_table", 2, 1) : kc.size(2);
    const int64_t npages = table ? kc.size(0) : 0;
    const int topk = int_arg(a[7], "topk"), gated = int_arg(a[11], "gated");
    const float scale = float_arg(a[12]);
    const int64_t qshape[4] = {B, Hq, T, d}, dshape[4] = {B, Hkv, T, d};
    const int64_t cshape[4] = {table ? npages : B, Hkv, table ? 64 : N, d};
    const int64_t sshape[4] = {table ? npages : B, Hkv, table ? d : N / 64, d};
    const int64_t ishape[4] = {B, Hkv, T, topk};
    at::Tensor made, mws;
    if (!out) out = &(made = pl.empty(qshape, st));
    const int iB = as_int(B, "B"), iHq = as_int(Hq, "Hq"), iHkv = as_int(Hkv, "Hkv"),
              iT = as_int(T, "T"), iN = as_int(N, "N"), id = as_int(d, "d");
    const size_t need = sas_decode_tree_workspace_size(iB, iHq, iHkv, iT, iN, id, topk, dt);
    if (!ws || ws->nbytes() < need)
      ws = &(mws = pl.empty({(int64_t)(need < 16 ? 16 : need)}, at::kByte));
    void* ps = ksum ? pl.ptr(ksum, "ksum", ksum->scalar_type(),
                             at::IntArrayRef(sshape, table ? 3 : 4))
                    : nullptr;
    check_status(
        "sas_decode_tree",
        sas_decode_tree(pl.ptr(&q, "q", st, qshape), pl.ptr(&kd, "kd", st, dshape),
                        pl.ptr(&vd, "vd", st, dshape), pl.ptr(&kc, "kc", st, cshape),
                        pl.ptr(&vc, "vc", st, cshape), dt, iB, iHq, iHkv, iT, iN, id,
                        pl.ints(parents, "parents", {B, T}), pl.ints(ntok, "ntok", {B}),
                        pl.ints(&lens, "lens", {B}), ps, ksum ? dtype_of(*ksum) : SAS_F32,
                        pl.ints(table, "block_table", {B, N / 64}), as_int(npages, "npages"), topk,
                        gated, scale, pl.ptr(out, "out", st, qshape),
                        topk > 0 ? pl.ints(idx, "idx_out", ishape) : nullptr,
                        pl.ptr(ws, "ws", ws->scalar_type(), ws->sizes()), ws->nbytes(),
                        pl.stream));
    return give(a[13], *out);
  });
}

#define METHOD(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(rotary), METHOD(page_map), METHOD(cache_append),
                         METHOD(decode_tree), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
