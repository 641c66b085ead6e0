// Native side of the Python binding of the calls that a decode loop makes: checks
// the tensors, allocates the outputs and workspaces that were not given and calls the
// C ABI (msa.h) on torch's current stream.  api.py holds the public functions and
// their documentation; a call through plain ctypes spent 10 to 20 us on the same
// checks, more than most of these calls take on the GPU.
//
// No computation happens here.  A wrong argument raises ValueError, a refusal of the
// library raises MSAError, as everywhere in the package.
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <sstream>
#include <string>

#include "../../include/msa.h"

namespace {

using at::Tensor;

struct ValueErr : std::exception {
  std::string msg;
  explicit ValueErr(std::string m) : msg(std::move(m)) {}
  const char* what() const noexcept override { return msg.c_str(); }
};

struct PyErrSet : std::exception {};     // a Python error is set already

constexpr int64_t kD = 128, kTopK = 16, kSlab = 9216;

bool none(PyObject* o) { return o == Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw ValueErr(std::string(name) + " must be a CUDA tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw ValueErr(std::string(name) + " must be a CUDA tensor");
  return t;
}

std::string text(at::IntArrayRef shape) {
  std::ostringstream s;
  s << "(";
  for (size_t i = 0; i < shape.size(); ++i) s << (i ? ", " : "") << shape[i];
  s << (shape.size() == 1 ? ",)" : ")");
  return s.str();
}

// The call's device: the current one, which every tensor has to be on.
struct Call {
  int dev;
  explicit Call(PyObject* first, const char* name) {
    const Tensor& t = tensor(first, name);
    dev = c10::cuda::current_device();
    if (t.get_device() != dev) wrong_device(t, name);
  }
  [[noreturn]] void wrong_device(const Tensor& t, const char* name) const {
    std::ostringstream s;
    s << name << " is on " << t.device() << ", the current device is cuda:" << dev;
    throw ValueErr(s.str());
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
  // straight from the allocator: 0.3 us less per output than by at::empty
  Tensor fresh(at::ScalarType type, at::IntArrayRef shape) const {
    return Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, dev), std::nullopt));
  }
  // Address of a contiguous tensor of this type, shape and device
  void* arg(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (t.scalar_type() != type) {
      std::ostringstream s;
      s << name << " must be " << type << ", got " << t.scalar_type();
      throw ValueErr(s.str());
    }
    if (!t.is_contiguous()) throw ValueErr(std::string(name) + " must be contiguous");
    if (t.sizes() != shape)
      throw ValueErr(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
    if (t.get_device() != dev) wrong_device(t, name);
    return t.data_ptr();
  }
  void* arg(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    return arg(tensor(o, name), name, type, shape);
  }
  template <class T>
  T* opt(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    return none(o) ? nullptr : static_cast<T*>(arg(o, name, type, shape));
  }
  // The given output, or a new one
  Tensor out(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (none(o)) return fresh(type, shape);
    const Tensor& t = tensor(o, name);
    arg(t, name, type, shape);
    return t;
  }
};

struct Workspace {
  Tensor t;
  size_t bytes = 0;
  Workspace(const Call& c, PyObject* o, size_t size) {
    if (none(o)) {
      bytes = size < 256 ? 256 : size;
      t = c.fresh(at::kByte, {static_cast<int64_t>(bytes)});
      return;
    }
    t = tensor(o, "workspace");
    if (!t.is_contiguous()) throw ValueErr("workspace must be contiguous");
    if (t.get_device() != c.dev) c.wrong_device(t, "workspace");
    bytes = t.nbytes();
    if (bytes < size) throw ValueErr("workspace needs " + std::to_string(size) + " bytes");
  }
  void* ptr() const { return t.data_ptr(); }
};

void check(msa_status_t code) {
  if (code == MSA_OK) return;
  PyObject* mod = PyImport_ImportModule("msa_block_sparse_gb300.api");
  PyObject* cls = mod ? PyObject_GetAttrString(mod, "MSAError") : nullptr;
  PyObject* err = cls ? PyObject_CallFunction(cls, "is", static_cast<int>(code), msa_last_error()) : nullptr;
  if (err) PyErr_SetObject(cls, err);
  Py_XDECREF(err);
  Py_XDECREF(cls);
  Py_XDECREF(mod);
  throw PyErrSet();
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyErrSet();
  return v;
}

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyErrSet();
  return v;
}

// A size as the C ABI takes it
int size32(int64_t v, const char* name) {
  if (v > INT32_MAX || v < INT32_MIN) throw ValueErr(std::string(name) + " is too large");
  return static_cast<int>(v);
}

const msa_rope_t* rope_at(PyObject* o) { return static_cast<const msa_rope_t*>(PyLong_AsVoidPtr(o)); }

// cu_seqlens: address and number of sequences
std::pair<const int32_t*, int> sequences(const Call& c, PyObject* o) {
  const Tensor& t = tensor(o, "cu_seqlens");
  if (t.dim() != 1 || t.numel() < 2) throw ValueErr("cu_seqlens must be a tensor of shape (S + 1,)");
  const int64_t n = t.numel();
  return {static_cast<const int32_t*>(c.arg(t, "cu_seqlens", at::kInt, {n})), size32(n - 1, "cu_seqlens")};
}

struct Where {
  const int32_t *positions = nullptr, *cu = nullptr;
  int S = 1;
  Where(const Call& c, PyObject* cu_o, PyObject* pos_o, int64_t T) {
    if (none(cu_o) == none(pos_o)) throw ValueErr("give either cu_seqlens or positions");
    if (!none(pos_o)) {
      positions = static_cast<const int32_t*>(c.arg(pos_o, "positions", at::kInt, {T}));
    } else {
      std::tie(cu, S) = sequences(c, cu_o);
    }
  }
};

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyErrSet();
  PyTuple_SET_ITEM(r, 0, wrap(a));
  PyTuple_SET_ITEM(r, 1, wrap(b));
  return r;
}

// ---------------------------------------------------------------- prologue

// x, w, rope, cu_seqlens, positions, out, eps
PyObject* qk_norm_rope_ex(PyObject* const* a) {
  const Call c(a[0], "x");
  const Tensor& x = tensor(a[0], "x");
  if (x.dim() != 3) throw ValueErr("x must have shape (T, H, D)");
  const auto s = x.sizes();
  const void* xp = c.arg(x, "x", at::kBFloat16, s);
  const void* w = c.opt<void>(a[1], "w", at::kBFloat16, {s[2]});
  const Where at(c, a[3], a[4], s[0]);
  const Tensor y = c.out(a[5], "out", at::kBFloat16, s);
  check(msa_qk_norm_rope_ex(xp, y.data_ptr(), size32(s[0], "T"), size32(s[1], "H"), size32(s[2], "D"), w,
                            at.positions, at.cu, at.S, rope_at(a[2]), number(a[6]), c.stream()));
  return wrap(y);
}

// x, dy, w, rope, cu_seqlens, positions, dx, dw, eps, workspace
PyObject* qk_norm_rope_bwd_ex(PyObject* const* a) {
  const Call c(a[1], "dy");
  const Tensor& dy = tensor(a[1], "dy");
  if (dy.dim() != 3) throw ValueErr("dy must have shape (T, H, D)");
  const auto s = dy.sizes();
  const int T = size32(s[0], "T"), H = size32(s[1], "H"), D = size32(s[2], "D");
  const void* dyp = c.arg(dy, "dy", at::kBFloat16, s);
  const Where at(c, a[4], a[5], s[0]);
  const Tensor dx = c.out(a[6], "dx", at::kBFloat16, s);
  if (none(a[2])) {
    if (!none(a[7])) throw ValueErr("dw needs w");
    check(msa_qk_norm_rope_bwd_ex(nullptr, dyp, dx.data_ptr(), nullptr, T, H, D, nullptr, at.positions,
                                  at.cu, at.S, rope_at(a[3]), number(a[8]), nullptr, 0, c.stream()));
    PyObject* r = PyTuple_New(2);
    if (!r) throw PyErrSet();
    PyTuple_SET_ITEM(r, 0, wrap(dx));
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 1, Py_None);
    return r;
  }
  const void* w = c.arg(a[2], "w", at::kBFloat16, {s[2]});
  const void* x = c.arg(a[0], "x", at::kBFloat16, s);
  const Tensor dw = c.out(a[7], "dw", at::kFloat, {s[2]});
  const Workspace ws(c, a[9], msa_qk_norm_rope_bwd_ex_workspace_size(T, H, D));
  check(msa_qk_norm_rope_bwd_ex(x, dyp, dx.data_ptr(), static_cast<float*>(dw.data_ptr()), T, H, D, w,
                                at.positions, at.cu, at.S, rope_at(a[3]), number(a[8]), ws.ptr(), ws.bytes,
                                c.stream()));
  return pair(dx, dw);
}

// ---------------------------------------------------------------- 4-bit cache

struct Table4 {
  int64_t P = 0, Hkv = 0, maxp = 0;
  const int32_t* table = nullptr;
  Table4(const Call& c, const Tensor& first, PyObject* table_o, int64_t rows) {
    if (first.dim() != 3) throw ValueErr("a 4-bit cache must have shape (num_pages, Hkv, 9216)");
    P = first.size(0);
    Hkv = first.size(1);
    const Tensor& t = tensor(table_o, "block_table");
    if (t.dim() != 2 || t.size(0) != rows)
      throw ValueErr("block_table must have shape (" + std::to_string(rows) + ", max_pages)");
    maxp = t.size(1);
    table = static_cast<const int32_t*>(c.arg(t, "block_table", at::kInt, {rows, maxp}));
  }
  void* cache(const Call& c, PyObject* o, const char* name) const {
    return c.arg(o, name, at::kByte, {P, Hkv, kSlab});
  }
  int pages() const { return size32(P, "num_pages"); }
  int heads() const { return size32(Hkv, "Hkv"); }
  int per_row() const { return size32(maxp, "max_pages"); }
};

const char* const kPack[3] = {"k", "v", "k_idx"};
const char* const kCaches[3] = {"k_cache", "v_cache", "kidx_cache"};

// k, v, k_idx, k_cache, v_cache, kidx_cache, block_table, cu_seqlens, start, gains x 3
PyObject* cache4_store(PyObject* const* a) {
  int n = -1;
  for (int i = 2; i >= 0; --i) {
    if (none(a[i]) != none(a[3 + i]))
      throw ValueErr(std::string(kPack[i]) + " and its cache must be given together");
    if (!none(a[i])) n = i;
  }
  if (n < 0) throw ValueErr("k, v or k_idx must be given, with its cache");
  const Call c(a[n], kPack[n]);
  const Tensor& x = tensor(a[n], kPack[n]);
  if (x.dim() != 3) throw ValueErr(std::string(kPack[n]) + " must have shape (T, Hkv, 128)");
  const int64_t T = x.size(0);
  const auto [cu, S] = sequences(c, a[7]);
  const Table4 t(c, tensor(a[3 + n], kCaches[n]), a[6], S);
  void *xp[3] = {}, *cp[3] = {};
  for (int i = 0; i < 3; ++i)
    if (!none(a[i])) {
      xp[i] = c.arg(a[i], kPack[i], at::kBFloat16, {T, t.Hkv, kD});
      cp[i] = t.cache(c, a[3 + i], kCaches[i]);
    }
  const int32_t* start = c.opt<int32_t>(a[8], "start", at::kInt, {S});
  check(msa_cache4_store(xp[0], xp[1], xp[2], cp[0], cp[1], cp[2], t.table, cu, start, S, size32(T, "T"),
                         t.heads(), t.pages(), t.per_row(), number(a[9]), number(a[10]), number(a[11]),
                         c.stream()));
  Py_RETURN_NONE;
}

// k_cache, v_cache, kidx_cache, block_table, cu_seqlens, T, start, gains x 3, k, v, k_idx
PyObject* cache4_load(PyObject* const* a) {
  int n = -1;
  for (int i = 2; i >= 0; --i) {
    if (none(a[i]) && !none(a[10 + i])) throw ValueErr(std::string(kPack[i]) + " needs its cache");
    if (!none(a[i])) n = i;
  }
  if (n < 0) throw ValueErr("no cache given");
  const Call c(a[n], kCaches[n]);
  const int64_t T = whole(a[5]);
  if (T < 0) throw ValueErr("T must be >= 0");
  const auto [cu, S] = sequences(c, a[4]);
  const Table4 t(c, tensor(a[n], kCaches[n]), a[3], S);
  void *xp[3] = {}, *cp[3] = {};
  Tensor out[3];
  for (int i = 0; i < 3; ++i)
    if (!none(a[i])) {
      cp[i] = t.cache(c, a[i], kCaches[i]);
      out[i] = c.out(a[10 + i], kPack[i], at::kBFloat16, {T, t.Hkv, kD});
      xp[i] = out[i].data_ptr();
    }
  const int32_t* start = c.opt<int32_t>(a[6], "start", at::kInt, {S});
  check(msa_cache4_load(cp[0], cp[1], cp[2], t.table, cu, start, S, size32(T, "T"), t.heads(), t.pages(),
                        t.per_row(), number(a[7]), number(a[8]), number(a[9]), xp[0], xp[1], xp[2],
                        c.stream()));
  PyObject* r = PyTuple_New(3);
  if (!r) throw PyErrSet();
  for (int i = 0; i < 3; ++i) {
    PyObject* o = Py_None;
    if (cp[i]) o = wrap(out[i]);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}

// q and its (B, Hq), checked later
std::pair<int64_t, int64_t> rows_heads(PyObject* o, const char* name) {
  const Tensor& q = tensor(o, name);
  if (q.dim() != 3) throw ValueErr(std::string(name) + " must have shape (B, Hq, 128)");
  return {q.size(0), q.size(1)};
}

// q, q_idx, k, v, k_idx, w_q, w_qi, w_k, w_ki, k_cache, v_cache, kidx_cache, block_table,
// cache_lens, rope, gains x 3, q_out, q_idx_out, eps
PyObject* decode4_append(PyObject* const* a) {
  const Call c(a[0], "q");
  const auto [B, Hq] = rows_heads(a[0], "q");
  const Table4 t(c, tensor(a[9], "k_cache"), a[12], B);
  static const char* const xn[5] = {"q", "q_idx", "k", "v", "k_idx"};
  static const char* const wn[4] = {"w_q", "w_qi", "w_k", "w_ki"};
  const void *x[5], *w[4];
  void* cp[3];
  for (int i = 0; i < 5; ++i) x[i] = c.arg(a[i], xn[i], at::kBFloat16, {B, i ? t.Hkv : Hq, kD});
  for (int i = 0; i < 4; ++i) w[i] = c.arg(a[5 + i], wn[i], at::kBFloat16, {kD});
  for (int i = 0; i < 3; ++i) cp[i] = t.cache(c, a[9 + i], kCaches[i]);
  const auto* lens = static_cast<const int32_t*>(c.arg(a[13], "cache_lens", at::kInt, {B}));
  const Tensor q_out = c.out(a[18], "q_out", at::kBFloat16, {B, Hq, kD});
  const Tensor qi_out = c.out(a[19], "q_idx_out", at::kBFloat16, {B, t.Hkv, kD});
  check(msa_decode4_append(x[0], x[1], x[2], x[3], x[4], w[0], w[1], w[2], w[3], cp[0], cp[1], cp[2],
                           t.table, lens, size32(B, "B"), size32(Hq, "Hq"), t.heads(), t.pages(),
                           t.per_row(), rope_at(a[14]), number(a[15]), number(a[16]), number(a[17]),
                           number(a[20]), q_out.data_ptr(), qi_out.data_ptr(), c.stream()));
  return pair(q_out, qi_out);
}

// q, q_idx, k_cache, v_cache, kidx_cache, block_table, cache_lens, scale, k_gain, v_gain, out,
// sel_out, workspace, n_init
PyObject* decode4_step(PyObject* const* a) {
  const Call c(a[0], "q");
  const auto [B, Hq] = rows_heads(a[0], "q");
  const Table4 t(c, tensor(a[2], "k_cache"), a[5], B);
  const void* q = c.arg(a[0], "q", at::kBFloat16, {B, Hq, kD});
  const void* qi = c.arg(a[1], "q_idx", at::kBFloat16, {B, t.Hkv, kD});
  const void* cp[3];
  for (int i = 0; i < 3; ++i) cp[i] = t.cache(c, a[2 + i], kCaches[i]);
  const auto* lens = static_cast<const int32_t*>(c.arg(a[6], "cache_lens", at::kInt, {B}));
  const Tensor o = c.out(a[10], "out", at::kBFloat16, {B, Hq, kD});
  const Tensor sel = c.out(a[11], "sel_out", at::kInt, {B, t.Hkv, kTopK});
  const int b = size32(B, "B"), hq = size32(Hq, "Hq");
  const Workspace ws(c, a[12], msa_decode4_step_workspace_size(b, hq, t.heads(), t.per_row()));
  check(msa_decode4_step(q, qi, cp[0], cp[1], cp[2], t.table, lens, b, hq, t.heads(), t.pages(),
                         t.per_row(), number(a[7]), number(a[8]), number(a[9]),
                         size32(whole(a[13]), "n_init"), o.data_ptr(), static_cast<int32_t*>(sel.data_ptr()),
                         ws.ptr(), ws.bytes, c.stream()));
  return pair(o, sel);
}

// ---------------------------------------------------------------- pages

struct Tables {
  int32_t *table, *lens, *ref;
  int B, P, maxp;
  Tables(const Call& c, PyObject* table_o, PyObject* lens_o, PyObject* ref_o) {
    const Tensor &t = tensor(table_o, "block_table"), &r = tensor(ref_o, "ref_count");
    if (t.dim() != 2) throw ValueErr("block_table must have shape (B, max_pages)");
    if (r.dim() != 1) throw ValueErr("ref_count must be a tensor of shape (num_pages,)");
    B = size32(t.size(0), "B");
    maxp = size32(t.size(1), "max_pages");
    P = size32(r.size(0), "num_pages");
    table = static_cast<int32_t*>(c.arg(t, "block_table", at::kInt, {B, maxp}));
    lens = static_cast<int32_t*>(c.arg(lens_o, "cache_lens", at::kInt, {B}));
    ref = static_cast<int32_t*>(c.arg(r, "ref_count", at::kInt, {P}));
  }
};

struct Caches {
  void* ptr[8] = {};
  int64_t bytes[8] = {};
  int n = 0;
  Caches(const Call& c, PyObject* list, int64_t P) {
    PyObject* seq = PySequence_Fast(list, "caches must be a sequence of tensors");
    if (!seq) throw PyErrSet();
    try {
      const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
      if (len > 8) throw ValueErr("at most 8 caches, got " + std::to_string(len));
      for (Py_ssize_t i = 0; i < len; ++i) {
        const std::string name = "cache " + std::to_string(i);
        const Tensor& t = tensor(PySequence_Fast_GET_ITEM(seq, i), name.c_str());
        if (!t.is_contiguous()) throw ValueErr(name + " must be contiguous");
        if (t.get_device() != c.dev) c.wrong_device(t, name.c_str());
        if (t.dim() < 1 || t.size(0) != P)
          throw ValueErr(name + " must have " + std::to_string(P) + " pages in its first dimension");
        ptr[i] = t.data_ptr();
        bytes[i] = P > 0 ? static_cast<int64_t>(t.nbytes()) / P : 0;
      }
      n = static_cast<int>(len);
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
    Py_DECREF(seq);
  }
};

int64_t list_len(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  if (t.dim() != 1 || t.numel() < 1)
    throw ValueErr(std::string(name) + " must be a tensor of shape (n,) with n >= 1");
  return t.numel();
}

// src, dst, block_table, cache_lens, ref_count, keep, forked
PyObject* pages_fork(PyObject* const* a) {
  const Call c(a[2], "block_table");
  const Tables t(c, a[2], a[3], a[4]);
  const int64_t n = list_len(a[0], "src");
  const auto* src = static_cast<const int32_t*>(c.arg(a[0], "src", at::kInt, {n}));
  const auto* dst = static_cast<const int32_t*>(c.arg(a[1], "dst", at::kInt, {n}));
  const int32_t* keep = c.opt<int32_t>(a[5], "keep", at::kInt, {n});
  const Tensor forked = c.out(a[6], "forked", at::kInt, {n});
  check(msa_pages_fork(src, dst, keep, size32(n, "n"), t.table, t.lens, t.ref, t.B, t.P, t.maxp,
                       static_cast<int32_t*>(forked.data_ptr()), c.stream()));
  return wrap(forked);
}

// rows, block_table, cache_lens, ref_count, keep, dropped
PyObject* pages_free(PyObject* const* a) {
  const Call c(a[1], "block_table");
  const Tables t(c, a[1], a[2], a[3]);
  const int64_t n = list_len(a[0], "rows");
  const auto* rows = static_cast<const int32_t*>(c.arg(a[0], "rows", at::kInt, {n}));
  const int32_t* keep = c.opt<int32_t>(a[4], "keep", at::kInt, {n});
  const Tensor dropped = c.out(a[5], "dropped", at::kInt, {n});
  check(msa_pages_free(rows, keep, size32(n, "n"), t.table, t.lens, t.ref, t.B, t.P, t.maxp,
                       static_cast<int32_t*>(dropped.data_ptr()), c.stream()));
  return wrap(dropped);
}

// add, block_table, cache_lens, ref_count, caches, done, workspace
PyObject* pages_extend(PyObject* const* a) {
  const Call c(a[1], "block_table");
  const Tables t(c, a[1], a[2], a[3]);
  const auto* add = static_cast<const int32_t*>(c.arg(a[0], "add", at::kInt, {t.B}));
  const Caches k(c, a[4], t.P);
  const Tensor done = c.out(a[5], "done", at::kInt, {t.B});
  const Workspace ws(c, a[6], msa_pages_extend_workspace_size(t.B, t.P));
  check(msa_pages_extend(add, t.table, t.lens, t.ref, t.B, t.P, t.maxp, k.ptr, k.bytes, k.n,
                         static_cast<int32_t*>(done.data_ptr()), ws.ptr(), ws.bytes, c.stream()));
  return wrap(done);
}

// block_table, cache_lens, ref_count, caches, page_map, n_live, workspace
PyObject* pages_compact(PyObject* const* a) {
  const Call c(a[0], "block_table");
  const Tables t(c, a[0], a[1], a[2]);
  const Caches k(c, a[3], t.P);
  const Tensor map = c.out(a[4], "page_map", at::kInt, {t.P}), live = c.out(a[5], "n_live", at::kInt, {1});
  const Workspace ws(c, a[6], msa_pages_compact_workspace_size(t.P));
  check(msa_pages_compact(t.table, t.lens, t.ref, t.B, t.P, t.maxp, k.ptr, k.bytes, k.n,
                          static_cast<int32_t*>(map.data_ptr()), static_cast<int32_t*>(live.data_ptr()),
                          ws.ptr(), ws.bytes, c.stream()));
  return pair(map, live);
}

// parents, block_table, cache_lens, ref_count, kept, workspace
PyObject* pages_reorder(PyObject* const* a) {
  const Call c(a[1], "block_table");
  const Tables t(c, a[1], a[2], a[3]);
  const auto* parents = static_cast<const int32_t*>(c.arg(a[0], "parents", at::kInt, {t.B}));
  const Tensor kept = c.out(a[4], "kept", at::kInt, {t.B});
  const Workspace ws(c, a[5], msa_pages_reorder_workspace_size(t.B, t.maxp));
  check(msa_pages_reorder(parents, t.table, t.lens, t.ref, t.B, t.P, t.maxp,
                          static_cast<int32_t*>(kept.data_ptr()), ws.ptr(), ws.bytes, c.stream()));
  return wrap(kept);
}

// src, dst, caches
PyObject* pages_copy(PyObject* const* a) {
  const Call c(a[0], "src");
  const int64_t n = list_len(a[0], "src");
  const auto* src = static_cast<const int32_t*>(c.arg(a[0], "src", at::kInt, {n}));
  const auto* dst = static_cast<const int32_t*>(c.arg(a[1], "dst", at::kInt, {n}));
  PyObject* first = PySequence_Check(a[2]) && PySequence_Size(a[2]) > 0 ? PySequence_GetItem(a[2], 0) : nullptr;
  if (!first) {
    PyErr_Clear();
    throw ValueErr("no cache given");
  }
  int64_t P = 0;
  try {
    const Tensor& t = tensor(first, "cache 0");
    if (t.dim() < 1) throw ValueErr("cache 0 must have pages in its first dimension");
    P = t.size(0);
  } catch (...) {
    Py_DECREF(first);
    throw;
  }
  Py_DECREF(first);
  const Caches k(c, a[2], P);
  check(msa_pages_copy(src, dst, size32(n, "n"), size32(P, "num_pages"), k.ptr, k.bytes, k.n, c.stream()));
  Py_RETURN_NONE;
}

// ---------------------------------------------------------------- 16-bit cache

struct Table16 {
  int64_t P = 0, Hkv = 0, maxp = 0;
  const int32_t* table = nullptr;
  Table16(const Call& c, PyObject* first_o, const char* name, PyObject* table_o, int64_t rows) {
    const Tensor& first = tensor(first_o, name);
    if (first.dim() != 4) throw ValueErr(std::string(name) + " must have shape (num_pages, Hkv, 128, 128)");
    P = first.size(0);
    Hkv = first.size(1);
    const Tensor& t = tensor(table_o, "block_table");
    if (t.dim() != 2 || t.size(0) != rows)
      throw ValueErr("block_table must have shape (" + std::to_string(rows) + ", max_pages)");
    maxp = t.size(1);
    table = static_cast<const int32_t*>(c.arg(t, "block_table", at::kInt, {rows, maxp}));
  }
  void* cache(const Call& c, PyObject* o, const char* name) const {
    return c.arg(o, name, at::kBFloat16, {P, Hkv, 128, kD});
  }
  int pages() const { return size32(P, "num_pages"); }
  int heads() const { return size32(Hkv, "Hkv"); }
  int per_row() const { return size32(maxp, "max_pages"); }
};

// q, k, v, k_cache, v_cache, block_table, cu_seqlens, cache_lens, rope, w_q, w_k, q_idx, k_idx,
// kidx_cache, w_qi, w_ki, q_out, q_idx_out, eps
PyObject* cache_append(PyObject* const* a) {
  const Call c(a[0], "q");
  const Tensor& q = tensor(a[0], "q");
  if (q.dim() != 3) throw ValueErr("q must have shape (T, Hq, 128)");
  const int64_t T = q.size(0), Hq = q.size(1);
  const auto [cu, S] = sequences(c, a[6]);
  const Table16 t(c, a[3], "k_cache", a[5], S);
  const void* qp = c.arg(q, "q", at::kBFloat16, {T, Hq, kD});
  const void* kp = c.arg(a[1], "k", at::kBFloat16, {T, t.Hkv, kD});
  const void* vp = c.arg(a[2], "v", at::kBFloat16, {T, t.Hkv, kD});
  void *kc = t.cache(c, a[3], "k_cache"), *vc = t.cache(c, a[4], "v_cache");
  const auto* lens = static_cast<const int32_t*>(c.arg(a[7], "cache_lens", at::kInt, {S}));
  const void* wq = c.opt<void>(a[9], "w_q", at::kBFloat16, {kD});
  const void* wk = c.opt<void>(a[10], "w_k", at::kBFloat16, {kD});
  const bool index = !none(a[11]);
  if (index != !none(a[12]) || index != !none(a[13]))
    throw ValueErr("q_idx, k_idx and kidx_cache must be given together");
  const void *qi = nullptr, *ki = nullptr, *wqi = nullptr, *wki = nullptr;
  void* ic = nullptr;
  const Tensor q_out = c.out(a[16], "q_out", at::kBFloat16, {T, Hq, kD});
  Tensor qi_out;
  if (index) {
    qi = c.arg(a[11], "q_idx", at::kBFloat16, {T, t.Hkv, kD});
    ki = c.arg(a[12], "k_idx", at::kBFloat16, {T, t.Hkv, kD});
    ic = t.cache(c, a[13], "kidx_cache");
    wqi = c.opt<void>(a[14], "w_qi", at::kBFloat16, {kD});
    wki = c.opt<void>(a[15], "w_ki", at::kBFloat16, {kD});
    qi_out = c.out(a[17], "q_idx_out", at::kBFloat16, {T, t.Hkv, kD});
  } else if (!none(a[14]) || !none(a[15]) || !none(a[17])) {
    throw ValueErr("w_qi, w_ki and q_idx_out need q_idx, k_idx and kidx_cache");
  }
  check(msa_cache_append(qp, kp, vp, qi, ki, wq, wk, wqi, wki, kc, vc, ic, t.table, cu, lens, S,
                         size32(T, "T"), size32(Hq, "Hq"), t.heads(), t.pages(), t.per_row(), rope_at(a[8]),
                         number(a[18]), q_out.data_ptr(), index ? qi_out.data_ptr() : nullptr, c.stream()));
  if (index) return pair(q_out, qi_out);
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyErrSet();
  PyTuple_SET_ITEM(r, 0, wrap(q_out));
  Py_INCREF(Py_None);
  PyTuple_SET_ITEM(r, 1, Py_None);
  return r;
}

// q, k_cache, v_cache, block_table, cache_lens, scale, out, lse, workspace
PyObject* decode_shared(PyObject* const* a) {
  const Call c(a[0], "q");
  const auto [B, Hq] = rows_heads(a[0], "q");
  const Table16 t(c, a[1], "k_cache", a[3], B);
  const void* q = c.arg(a[0], "q", at::kBFloat16, {B, Hq, kD});
  const void *kc = t.cache(c, a[1], "k_cache"), *vc = t.cache(c, a[2], "v_cache");
  const auto* lens = static_cast<const int32_t*>(c.arg(a[4], "cache_lens", at::kInt, {B}));
  const Tensor o = c.out(a[6], "out", at::kBFloat16, {B, Hq, kD});
  const Tensor lse = c.out(a[7], "lse", at::kFloat, {B, Hq});
  const int b = size32(B, "B"), hq = size32(Hq, "Hq");
  const Workspace ws(c, a[8], msa_decode_shared_workspace_size(b, hq, t.heads(), t.per_row()));
  check(msa_decode_shared(q, kc, vc, t.table, lens, b, hq, t.heads(), t.pages(), t.per_row(), number(a[5]),
                          o.data_ptr(), static_cast<float*>(lse.data_ptr()), ws.ptr(), ws.bytes, c.stream()));
  return pair(o, lse);
}

// ---------------------------------------------------------------- beams

// logits, scores, beams, n_out, finished, pad_token, scores_out, parents, tokens, workspace
PyObject* beam_select(PyObject* const* a) {
  const Call c(a[0], "logits");
  const Tensor& x = tensor(a[0], "logits");
  if (x.dim() != 2) throw ValueErr("logits must have shape (N * beams, V)");
  int dtype = MSA_F32;
  if (x.scalar_type() == at::kBFloat16) {
    dtype = MSA_BF16;
  } else if (x.scalar_type() != at::kFloat) {
    std::ostringstream s;
    s << "logits must be Float or BFloat16, got " << x.scalar_type();
    throw ValueErr(s.str());
  }
  const int64_t R = x.size(0), V = x.size(1), W = whole(a[2]), K = whole(a[3]);
  if ((V > 1 && x.stride(1) != 1) || (R > 1 && x.stride(0) < V))
    throw ValueErr("rows of logits must be contiguous and must not overlap");
  if (W < 1 || R < 1 || R % W != 0) throw ValueErr("logits must have beams rows for every prompt");
  const int64_t N = R / W;
  const void* scores = c.arg(a[1], "scores", at::kFloat, {R});
  const uint8_t* finished = nullptr;
  if (!none(a[4])) {
    const Tensor& f = tensor(a[4], "finished");
    finished = static_cast<const uint8_t*>(
        c.arg(f, "finished", f.scalar_type() == at::kBool ? at::kBool : at::kByte, {R}));
  }
  const int n = size32(N, "N"), w = size32(W, "beams"), v = size32(V, "V"), k = size32(K, "n_out");
  if (k < 1) throw ValueErr("n_out must be >= 1");
  const Tensor so = c.out(a[6], "scores_out", at::kFloat, {N, K});
  const Tensor po = c.out(a[7], "parents", at::kInt, {N, K});
  const Tensor to = c.out(a[8], "tokens", at::kInt, {N, K});
  const Workspace ws(c, a[9], msa_beam_select_workspace_size(n, w, v, k));
  check(msa_beam_select(x.data_ptr(), dtype, R > 1 ? x.stride(0) : V, static_cast<const float*>(scores),
                        finished, n, w, v, k, size32(whole(a[5]), "pad_token"),
                        static_cast<float*>(so.data_ptr()), static_cast<int32_t*>(po.data_ptr()),
                        static_cast<int32_t*>(to.data_ptr()), ws.ptr(), ws.bytes, c.stream()));
  PyObject* r = PyTuple_New(3);
  if (!r) throw PyErrSet();
  PyTuple_SET_ITEM(r, 0, wrap(so));
  PyTuple_SET_ITEM(r, 1, wrap(po));
  PyTuple_SET_ITEM(r, 2, wrap(to));
  return r;
}

// ---------------------------------------------------------------- module

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PyErrSet&) {
  } catch (const ValueErr& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* mod = PyImport_ImportModule("torch");
    PyObject* cls = mod ? PyObject_GetAttrString(mod, "OutOfMemoryError") : nullptr;
    if (cls) PyErr_SetString(cls, e.what());
    Py_XDECREF(cls);
    Py_XDECREF(mod);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define MSA_ENTRY(f, n) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {
    MSA_ENTRY(qk_norm_rope_ex, 7), MSA_ENTRY(qk_norm_rope_bwd_ex, 10), MSA_ENTRY(cache4_store, 12),
    MSA_ENTRY(cache4_load, 13),    MSA_ENTRY(decode4_append, 21),      MSA_ENTRY(decode4_step, 14),
    MSA_ENTRY(pages_fork, 7),      MSA_ENTRY(pages_free, 6),           MSA_ENTRY(pages_extend, 7),
    MSA_ENTRY(pages_compact, 7),   MSA_ENTRY(pages_copy, 3),
    MSA_ENTRY(pages_reorder, 6),   MSA_ENTRY(cache_append, 19),       MSA_ENTRY(decode_shared, 9),
    MSA_ENTRY(beam_select, 10),    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_msa_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__msa_torch() {
  return PyModule_Create(&kModule);
}
