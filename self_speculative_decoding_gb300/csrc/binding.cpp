// Python binding of the tree-decoding calls (ssd_ops.h): checks the tensors
// (the library sees bare pointers), allocates results and workspaces, and
// calls the library.  Marshalling only, as _abi.py is for the other calls;
// these run several times per layer or token, and through ctypes the checks
// and the allocations cost as much host time as the launches (one small tree
// 22 us a call against 9 us on the device).
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <string>

#include "../../include/ssd_ops.h"

namespace {

// The library's functions, as the Python side loaded them.
struct Library {
  decltype(&ssd_op_tree_attention_workspace) tree_workspace = nullptr;
  decltype(&ssd_op_tree_attention) tree_attention = nullptr;
  decltype(&ssd_op_cache_evict) cache_evict = nullptr;
  decltype(&ssd_op_beam_select_workspace) select_workspace = nullptr;
  decltype(&ssd_op_beam_select) beam_select = nullptr;
  decltype(&ssd_op_beam_reorder) beam_reorder = nullptr;
  decltype(&ssd_ops_last_error) last_error = nullptr;
  PyObject* error = nullptr;  // SSDError
} lib;

constexpr int kMostWidth = 256;  // of a selection (ssd_ops.h)

// Thrown with a Python exception set.
struct Refused {};

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

const at::Tensor* optional(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}

int32_t whole(PyObject* o, const char* name) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (over || v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
    refuse(std::string(name) + ": does not fit 32 bits");
  return (int32_t)v;
}

// The address of a tensor of this type, shape and device.
void* arg(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape,
          int device) {
  if (t.scalar_type() != type || t.sizes() != shape)
    refuse(std::string(name) + ": expected " + c10::toString(type) + " of shape " +
           shape_text(shape) + ", got " + c10::toString(t.scalar_type()) + " of shape " +
           shape_text(t.sizes()));
  if (!t.is_cuda() || t.get_device() != device)
    refuse(std::string(name) + ": expected a tensor on CUDA device " + std::to_string(device) +
           ", got " + t.device().str());
  if (!t.is_contiguous()) refuse(std::string(name) + ": expected a contiguous tensor");
  return t.data_ptr();
}

void check(ssd_status st) {
  if (st == SSD_OK) return;
  PyObject* e = PyObject_CallFunction(lib.error, "is", (int)st, lib.last_error());
  if (e) {
    PyErr_SetObject(lib.error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

void want(Py_ssize_t n, Py_ssize_t got) {
  if (n == got) return;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, got);
  throw Refused();
}

// The device of the call's tensors made current, and its current stream.
struct Place {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Place(const at::Tensor& t)
      : guard(t.device()), stream(c10::cuda::getCurrentCUDAStream(t.get_device()).stream()) {}
};

// Other Python threads run while this one allocates and launches: either may
// wait for the device, whose queue may hold a callback into Python.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + ": expected a CUDA tensor, got " + t.device().str());
  return t.get_device();
}

at::Tensor make(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false));
}

#define SSD_BEGIN \
  HANDLE_TH_ERRORS try {
#define SSD_END              \
  }                          \
  catch (const Refused&) {   \
    return nullptr;          \
  }                          \
  END_HANDLE_TH_ERRORS

// (qkv, parents, k_cache, v_cache, n_ctx, pos0, H, Hkv, dh, theta, weights,
//  weights_out, out) -> out
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  SSD_BEGIN
  want(13, n);
  const at::Tensor &qkv = tensor(a[0], "qkv"), &parents = tensor(a[1], "parents");
  const at::Tensor &k = tensor(a[2], "k_cache"), &v = tensor(a[3], "v_cache");
  const int32_t n_ctx = whole(a[4], "n_ctx"), pos0 = whole(a[5], "pos0"), H = whole(a[6], "H");
  const int32_t Hkv = whole(a[7], "Hkv"), dh = whole(a[8], "dh");
  const double theta = PyFloat_AsDouble(a[9]);
  if (theta == -1.0 && PyErr_Occurred()) throw Refused();
  const at::Tensor *w = optional(a[10], "weights"), *wo = optional(a[11], "weights_out");
  const at::Tensor* given = optional(a[12], "out");
  if (qkv.dim() != 2 || k.dim() != 3)
    refuse("expected qkv [T, (H + 2 Hkv) dh] and k_cache [Hkv, max_seq, dh]");
  const int dev = device_of(qkv, "qkv");
  const int64_t T = qkv.size(0), S = k.size(1);
  if (T > std::numeric_limits<int32_t>::max() || S > std::numeric_limits<int32_t>::max())
    refuse("too many rows");
  const int64_t cache[3] = {Hkv, S, dh}, per_key[2] = {Hkv, S};
  // (unsigned: counts that do not fit wrap, and the library refuses them)
  const int64_t row[2] = {T, (int64_t)(((uint64_t)H + 2 * (uint64_t)Hkv) * (uint64_t)dh)};
  const int64_t res[2] = {T, (int64_t)H * dh};
  void* pq = arg(qkv, "qkv", at::kFloat, row, dev);
  void* pp = arg(parents, "parents", at::kInt, at::IntArrayRef(&T, 1), dev);
  void* pk = arg(k, "k_cache", at::kBFloat16, cache, dev);
  void* pv = arg(v, "v_cache", at::kBFloat16, cache, dev);
  void* pw = w ? arg(*w, "weights", at::kFloat, per_key, dev) : nullptr;
  void* pwo = wo ? arg(*wo, "weights_out", at::kFloat, per_key, dev) : nullptr;
  const Place place(qkv);
  void* po = given ? arg(*given, "out", at::kBFloat16, res, dev) : nullptr;
  at::Tensor out;
  ssd_status st;
  {
    const Unlocked unlocked;
    // (rows that the cache does not have are refused)
    const size_t need = n_ctx <= S - T ? lib.tree_workspace((int32_t)T, n_ctx, H, Hkv, dh) : 0;
    if (!given && need) {                        // (0: refused sizes)
      out = make(qkv, res, at::kBFloat16);
      po = out.data_ptr();
    }
    const at::Tensor ws = make(qkv, {(int64_t)(need ? need : 256)}, at::kByte);
    st = lib.tree_attention((const float*)pq, (const int32_t*)pp, (int32_t)T, n_ctx, pos0, pk, pv,
                            (int32_t)S, H, Hkv, dh, (float)theta, (const float*)pw, (float*)pwo, po,
                            ws.data_ptr(), need, place.stream);
  }
  check(st);
  return THPVariable_Wrap(given ? *given : out);
  SSD_END
}

// (k, v, weights, n, keep, k_out, v_out, weights_out, sinks, recent) -> kept
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  SSD_BEGIN
  want(10, n_args);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &w = tensor(a[2], "weights");
  const int32_t n = whole(a[3], "n"), keep = whole(a[4], "keep");
  const at::Tensor &ko = tensor(a[5], "k_out"), &vo = tensor(a[6], "v_out");
  const at::Tensor* wo = optional(a[7], "weights_out");
  const int32_t sinks = whole(a[8], "sinks"), recent = whole(a[9], "recent");
  const at::ScalarType type = k.scalar_type();
  if ((type != at::kBFloat16 && type != at::kFloat) || k.dim() != 3 || ko.dim() != 3)
    refuse("k, k_out: expected bf16 or fp32 tensors [Hkv, rows, dh]");
  const int dev = device_of(k, "k");
  for (int64_t x : {k.size(0), k.size(1), k.size(2), ko.size(1)})
    if (x > std::numeric_limits<int32_t>::max()) refuse("too many rows");
  const int64_t to[3] = {k.size(0), ko.size(1), k.size(2)};
  void* pk = arg(k, "k", type, k.sizes(), dev);
  void* pv = arg(v, "v", type, k.sizes(), dev);
  void* pw = arg(w, "weights", at::kFloat, k.sizes().slice(0, 2), dev);
  void* pko = arg(ko, "k_out", type, to, dev);
  void* pvo = arg(vo, "v_out", type, to, dev);
  void* pwo = wo ? arg(*wo, "weights_out", at::kFloat, at::IntArrayRef(to, 2), dev) : nullptr;
  const Place place(k);
  at::Tensor kept;
  ssd_status st;
  {
    const Unlocked unlocked;
    const bool fits = keep > 0 && keep <= n && n <= k.size(1) && keep <= ko.size(1);  // (else refused)
    kept = make(k, {k.size(0), fits ? keep : 0}, at::kInt);
    st = lib.cache_evict(pk, pv, (const float*)pw, n, keep, sinks, recent, (int32_t)k.size(1),
                         (int32_t)k.size(0), (int32_t)k.size(2),
                         type == at::kBFloat16 ? SSD_DTYPE_BF16 : SSD_DTYPE_FP32, pko, pvo,
                         (float*)pwo, (int32_t)ko.size(1), (int32_t*)kept.data_ptr(), place.stream);
  }
  check(st);
  return THPVariable_Wrap(kept);
  SSD_END
}

// (logits, scores, width, lse, done, end_id) -> (tokens, parents, scores, done)
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  SSD_BEGIN
  want(6, n);
  const at::Tensor &z = tensor(a[0], "logits"), &scores = tensor(a[1], "scores");
  const int32_t W = whole(a[2], "width");
  const at::Tensor *lse = optional(a[3], "lse"), *done = optional(a[4], "done");
  const int32_t end_id = whole(a[5], "end_id");
  if (z.dim() != 2) refuse("logits: expected [B, V]");
  const int dev = device_of(z, "logits");
  const int64_t B = z.size(0), V = z.size(1);
  if (B > std::numeric_limits<int32_t>::max() || V > std::numeric_limits<int32_t>::max())
    refuse("logits: too many");
  const at::IntArrayRef per_beam(&B, 1);
  void* pz = arg(z, "logits", at::kFloat, z.sizes(), dev);
  void* ps = arg(scores, "scores", at::kFloat, per_beam, dev);
  void* pd = done ? arg(*done, "done", at::kInt, per_beam, dev) : nullptr;
  const float* pl = nullptr;
  int32_t step = 1;
  if (lse && lse->scalar_type() == at::kInt) {
    // ssd_row_stats records
    const int64_t records[2] = {B, (int64_t)(sizeof(ssd_row_stats) / 4)};
    const auto* st = (const ssd_row_stats*)arg(*lse, "lse", at::kInt, records, dev);
    pl = &st->lse;
    step = (int32_t)records[1];
  } else if (lse) {
    if (lse->scalar_type() != at::kFloat || lse->sizes() != per_beam || !lse->is_cuda() ||
        lse->get_device() != dev)
      refuse("lse: expected fp32 [B] on the logits' device, or the LM head's records");
    const int64_t s = B > 1 ? lse->stride(0) : 1;
    if (s < 1 || s > std::numeric_limits<int32_t>::max()) refuse("lse: stride");
    step = (int32_t)s;
    pl = (const float*)lse->data_ptr();
  }
  const Place place(z);
  at::Tensor tok, par, best, end;
  ssd_status st;
  {
    const Unlocked unlocked;
    const size_t need = lib.select_workspace((int32_t)B, (int32_t)V, W);
    const int64_t w = W > 0 && W <= kMostWidth ? W : 0;  // (else refused)
    const at::Tensor ws = need ? make(z, {(int64_t)need}, at::kByte) : at::Tensor();
    tok = make(z, {w}, at::kInt);
    par = make(z, {w}, at::kInt);
    best = make(z, {w}, at::kFloat);
    end = make(z, {w}, at::kInt);
    st = lib.beam_select((const float*)pz, (int32_t)B, (int32_t)V, pl, step, (const float*)ps,
                         (const int32_t*)pd, end_id, W, (int32_t*)tok.data_ptr(),
                         (int32_t*)par.data_ptr(), (float*)best.data_ptr(), (int32_t*)end.data_ptr(),
                         need ? ws.data_ptr() : nullptr, need, place.stream);
  }
  check(st);
  PyObject* r = PyTuple_New(4);
  if (!r) return nullptr;
  int i = 0;
  for (const at::Tensor* t : {&tok, &par, &best, &end}) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(*t));
  return r;
  SSD_END
}

// (k, v, parents, start, stop, k_out, v_out) -> None
PyObject* beam_reorder(PyObject*, PyObject* const* a, Py_ssize_t n) {
  SSD_BEGIN
  want(7, n);
  const at::Tensor& k = tensor(a[0], "k");
  const at::Tensor *v = optional(a[1], "v"), *vo = optional(a[6], "v_out");
  const at::Tensor &parents = tensor(a[2], "parents"), &ko = tensor(a[5], "k_out");
  const int32_t start = whole(a[3], "start"), stop = whole(a[4], "stop");
  if (k.dim() < 3) refuse("k: expected [B, ..., max_seq, dh]");
  if (!v != !vo) refuse("v and v_out go together");
  const int dev = device_of(k, "k");
  const at::ScalarType type = k.scalar_type();
  c10::SmallVector<int64_t, 6> to(k.sizes().begin(), k.sizes().end());
  to[0] = ko.dim() ? ko.size(0) : 0;
  const int64_t W = to[0], rows = k.size(k.dim() - 2), bytes = k.size(k.dim() - 1) * k.element_size();
  int64_t groups = 1;
  for (int64_t i = 1; i + 2 < k.dim(); ++i) groups *= k.size(i);
  for (int64_t x : {k.size(0), W, groups, rows, bytes})
    if (x > std::numeric_limits<int32_t>::max()) refuse("too many rows");
  void* pk = arg(k, "k", type, k.sizes(), dev);
  void* pko = arg(ko, "k_out", type, to, dev);
  void* pv = v ? arg(*v, "v", type, k.sizes(), dev) : nullptr;
  void* pvo = vo ? arg(*vo, "v_out", type, to, dev) : nullptr;
  void* pp = arg(parents, "parents", at::kInt, at::IntArrayRef(&W, 1), dev);
  const Place place(k);
  ssd_status st;
  {
    const Unlocked unlocked;
    st = lib.beam_reorder(pk, pv, (const int32_t*)pp, (int32_t)k.size(0), (int32_t)W,
                          (int32_t)groups, (int32_t)rows, start, stop, (int32_t)bytes, pko, pvo,
                          place.stream);
  }
  check(st);
  Py_RETURN_NONE;
  SSD_END
}

// ({name: address}, SSDError)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  SSD_BEGIN
  want(2, n);
  auto at = [&](const char* name) -> void* {
    PyObject* p = PyDict_GetItemString(a[0], name);
    if (!p) refuse(std::string("no address of ") + name);
    return PyLong_AsVoidPtr(p);
  };
  lib.tree_workspace = (decltype(lib.tree_workspace))at("ssd_op_tree_attention_workspace");
  lib.tree_attention = (decltype(lib.tree_attention))at("ssd_op_tree_attention");
  lib.cache_evict = (decltype(lib.cache_evict))at("ssd_op_cache_evict");
  lib.select_workspace = (decltype(lib.select_workspace))at("ssd_op_beam_select_workspace");
  lib.beam_select = (decltype(lib.beam_select))at("ssd_op_beam_select");
  lib.beam_reorder = (decltype(lib.beam_reorder))at("ssd_op_beam_reorder");
  lib.last_error = (decltype(lib.last_error))at("ssd_ops_last_error");
  if (PyErr_Occurred()) throw Refused();
  Py_INCREF(a[1]);
  Py_XDECREF(lib.error);
  lib.error = a[1];
  Py_RETURN_NONE;
  SSD_END
}

#define SSD_METHOD(f) \
  { #f, (PyCFunction)(void*)f, METH_FASTCALL, "" }
PyMethodDef methods[] = {SSD_METHOD(bind),        SSD_METHOD(tree_attention),
                         SSD_METHOD(cache_evict), SSD_METHOD(beam_select),
                         SSD_METHOD(beam_reorder), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
