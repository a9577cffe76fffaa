// Python marshalling of the calls over a paged cache and of the logit
// constraints: tensor checks and the C call in compiled code.  These calls
// take a dozen tensors and run for a few microseconds; checked in Python and
// passed through ctypes their arguments took longer than their kernels (13 us a
// call of dspark_pages_reserve whose kernel takes 4).  Each function takes
// (context handle, device index, stream handle, arguments ...) and returns the
// library's return code; what is wrong with an argument is raised as
// TypeError or ValueError before the library is called.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <exception>

#include "dspark.h"

namespace {

struct Raised {};   // a Python error is set

template <typename... A>
[[noreturn]] void raise(PyObject* type, const char* fmt, A... a) {
  PyErr_Format(type, fmt, a...);
  throw Raised();
}

// The arguments of one call, in order.
class Args {
 public:
  Args(PyObject* const* v, Py_ssize_t n, Py_ssize_t want) : v_(v) {
    if (n != want) raise(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    handle = reinterpret_cast<dspark_ctx*>(PyLong_AsVoidPtr(next()));
    device = (int)integer("device", INT32_MIN, INT32_MAX);
    stream = reinterpret_cast<hipStream_t>(PyLong_AsVoidPtr(next()));
    if (PyErr_Occurred()) throw Raised();
  }

  dspark_ctx* handle;
  int device;
  hipStream_t stream;

  int64_t integer(const char* name, int64_t lo, int64_t hi) {
    int over = 0;
    const long long x = PyLong_AsLongLongAndOverflow(next(), &over);
    if (PyErr_Occurred()) throw Raised();
    if (over || x < lo || x > hi) raise(PyExc_ValueError, "%s is out of range", name);
    return x;
  }
  int int32(const char* name) { return (int)integer(name, INT32_MIN, INT32_MAX); }

  double real64(const char*) {
    const double x = PyFloat_AsDouble(next());
    if (PyErr_Occurred()) throw Raised();
    return x;
  }
  float real(const char* name) { return (float)real64(name); }

  bool truth() {
    const int x = PyObject_IsTrue(next());
    if (x < 0) throw Raised();
    return x != 0;
  }

  // The next argument as a tensor on the context's device, or null for None
  // where that is allowed.
  const at::Tensor* tensor(const char* name, bool optional = false) {
    PyObject* o = next();
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device)
      raise(PyExc_ValueError, "%s is on another device than the context (cuda:%d)", name, device);
    return &t;
  }

  // Of one type and rank, contiguous over its last dimension.
  const at::Tensor* rows(const char* name, at::ScalarType type, int dims, bool optional = false) {
    const at::Tensor* t = tensor(name, optional);
    if (!t) return nullptr;
    if (t->scalar_type() != type) raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type),
                                        c10::toString(t->scalar_type()));
    if (t->dim() != dims) raise(PyExc_ValueError, "%s must have %d dims, got %lld", name, dims, (long long)t->dim());
    if (t->size(dims - 1) > 1 && t->stride(dims - 1) != 1)
      raise(PyExc_ValueError, "%s must be contiguous over its last dimension", name);
    return t;
  }

  // A contiguous vector of n entries (n < 0: of at least -n).
  const at::Tensor* vector(const char* name, at::ScalarType type, int64_t n, bool optional = false) {
    const at::Tensor* t = rows(name, type, 1, optional);
    if (!t) return nullptr;
    if (n < 0 ? t->size(0) < -n : t->size(0) != n)
      raise(PyExc_ValueError, "%s must have %s%lld entries, got %lld", name, n < 0 ? "at least " : "",
            (long long)(n < 0 ? -n : n), (long long)t->size(0));
    return t;
  }
  int32_t* ints(const char* name, int64_t n, bool optional = false) {
    return data<int32_t>(vector(name, at::kInt, n, optional));
  }
  float* floats(const char* name, int64_t n, bool optional = false) {
    return data<float>(vector(name, at::kFloat, n, optional));
  }

  template <typename T>
  static T* data(const at::Tensor* t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
  }

 private:
  PyObject* next() { return v_[at_++]; }
  PyObject* const* v_;
  Py_ssize_t at_ = 0;
};

using T = at::Tensor;

int to_int(const char* name, int64_t x) {
  if (x > INT32_MAX) raise(PyExc_ValueError, "%s is too large", name);
  return (int)x;
}

// Step of dimension i; `alone` where the dimension has a single entry (torch leaves its stride arbitrary).
int64_t step(const T& t, int i, int64_t alone = 0) { return t.size(i) > 1 ? t.stride(i) : alone; }

struct Table {
  int32_t* p;
  int64_t stride;
  int cols;
  Table(Args& a, int64_t B) {
    const T* t = a.rows("table", at::kInt, 2);
    if (t->size(0) != B) raise(PyExc_ValueError, "table must have %lld rows, got %lld", (long long)B, (long long)t->size(0));
    p = Args::data<int32_t>(t);
    cols = to_int("table", t->size(1));
    stride = step(*t, 0, cols);
  }
};

struct Cache {
  void *k, *v;
  float *k_scale = nullptr, *v_scale = nullptr;          // e4m3: a scale a head
  uint8_t *k_power = nullptr, *v_power = nullptr;        // mxfp4: powers of two, a byte a block
  int n_pages, page, heads, d;
  int64_t s_page, s_tok, s_head;
  dspark_dtype type;
  explicit Cache(Args& a) {
    const T* kc = a.tensor("kcache");
    const at::ScalarType st = kc->scalar_type();
    if (st == at::kBFloat16) type = DSPARK_BF16;
    else if (st == at::kFloat8_e4m3fn) type = DSPARK_E4M3;
    else if (st == at::kByte || st == at::kFloat4_e2m1fn_x2) type = DSPARK_MXFP4;
    else raise(PyExc_TypeError, "the cache must be bf16, float8_e4m3fn or uint8 (mxfp4), got %s", c10::toString(st));
    const T* vc = a.rows("vcache", st, 4);
    if (kc->dim() != 4) raise(PyExc_ValueError, "kcache must have 4 dims, got %lld", (long long)kc->dim());
    bool alike = kc->sizes() == vc->sizes();
    for (int i = 0; i < 4; ++i) alike = alike && step(*kc, i) == step(*vc, i);
    if (!alike) raise(PyExc_ValueError, "kcache and vcache must have one shape and one set of strides");
    if (kc->stride(3) != 1) raise(PyExc_ValueError, "the cache must be contiguous over a head's values");
    n_pages = to_int("n_pages", kc->size(0));
    page = to_int("page_size", kc->size(1));
    heads = to_int("heads", kc->size(2));
    d = to_int("d", kc->size(3));
    s_tok = kc->stride(1);
    s_head = step(*kc, 2, d);
    s_page = step(*kc, 0, std::max<int64_t>(page * s_tok, heads * s_head));
    k = kc->data_ptr();
    v = vc->data_ptr();
    if (type == DSPARK_MXFP4) {
      d = to_int("d", 2 * kc->size(3));                  // two values a byte
      k_power = power(a, "k_scale");
      v_power = power(a, "v_scale");
    } else {
      k_scale = a.floats("k_scale", heads, true);
      v_scale = a.floats("v_scale", heads, true);
    }
  }

 private:
  uint8_t* power(Args& a, const char* name) {
    const T* t = a.tensor(name);
    if (t->scalar_type() != at::kByte && t->scalar_type() != at::kFloat8_e8m0fnu)
      raise(PyExc_TypeError, "%s must be uint8 or float8_e8m0fnu for an mxfp4 cache, got %s", name,
            c10::toString(t->scalar_type()));
    if (t->dim() != 4 || t->size(0) != n_pages || t->size(1) != heads || t->size(2) != page || t->size(3) != d / 32 ||
        !t->is_contiguous())
      raise(PyExc_ValueError, "%s must be [n_pages][heads][page_size][d / 32] of an mxfp4 cache, contiguous", name);
    return Args::data<uint8_t>(t);
  }
};

// bf16 rows [n_rows][heads][d].
struct Rows {
  void* p = nullptr;
  int64_t row = 0, head = 0;
  explicit Rows(const T* t) {
    if (!t) return;
    p = t->data_ptr();
    // (a row or head that is the only one: as if the others lay behind it)
    head = step(*t, 1, t->size(2));
    row = step(*t, 0, t->size(1) * head);
  }
};

// page_size, n_pages, n_rows, K, length, table, held, held_out, free_list,
// n_free, n_free_out, t_offsets, row_req, row_pos, row_slot
int pages_reserve(Args& a) {
  const int page = a.int32("page_size"), n_pages = a.int32("n_pages"), n_rows = a.int32("n_rows");
  if (n_rows < 0 || n_pages < 0) raise(PyExc_ValueError, "n_rows and n_pages must be >= 0");
  const T* K = a.rows("K", at::kInt, 1);
  const int64_t B = K->size(0);
  if (!K->is_contiguous()) raise(PyExc_ValueError, "K must be contiguous");
  const int32_t* length = a.ints("length", B);
  const Table table(a, B);
  const int32_t* held = a.ints("held", B);
  int32_t* held_out = a.ints("held_out", B);
  const int32_t* free_list = a.ints("free_list", n_pages);
  const int32_t* n_free = a.ints("n_free", 1);
  int32_t* n_free_out = a.ints("n_free_out", 1);
  int32_t* offs = a.ints("t_offsets", B + 1);
  int32_t* req = a.ints("row_req", n_rows);
  int32_t* pos = a.ints("row_pos", n_rows);
  int32_t* slot = a.ints("row_slot", n_rows);
  return dspark_pages_reserve(a.handle, a.stream, to_int("B", B), page, n_pages, Args::data<int32_t>(K), length,
                              table.p, table.stride, table.cols, held, held_out, free_list, n_free, n_free_out,
                              n_rows, offs, req, pos, slot);
}

// page_size, n_pages, length, len_out, accept_len, finished, table, held,
// held_out, free_list, n_free, n_free_out
int pages_commit(Args& a) {
  const int page = a.int32("page_size"), n_pages = a.int32("n_pages");
  if (n_pages < 0) raise(PyExc_ValueError, "n_pages must be >= 0");
  const T* length = a.rows("length", at::kInt, 1);
  const int64_t B = length->size(0);
  if (!length->is_contiguous()) raise(PyExc_ValueError, "length must be contiguous");
  int32_t* len_out = a.ints("len_out", B);
  const int32_t* accept = a.ints("accept_len", B);
  const int32_t* finished = a.ints("finished", B, true);
  const Table table(a, B);
  const int32_t* held = a.ints("held", B);
  int32_t* held_out = a.ints("held_out", B);
  int32_t* free_list = a.ints("free_list", n_pages);
  const int32_t* n_free = a.ints("n_free", 1);
  int32_t* n_free_out = a.ints("n_free_out", 1);
  return dspark_pages_commit(a.handle, a.stream, to_int("B", B), page, n_pages, Args::data<int32_t>(length), len_out,
                             accept, finished, table.p, table.stride, table.cols, held, held_out, free_list, n_free,
                             n_free_out);
}

// kcache, vcache, k_scale, v_scale, k, v, row_slot
int cache_write(Args& a) {
  const Cache c(a);
  const T* k = a.rows("k", at::kBFloat16, 3);
  const T* v = a.rows("v", at::kBFloat16, 3);
  if (k->size(1) != c.heads || k->size(2) != c.d || v->sizes() != k->sizes())
    raise(PyExc_ValueError, "k and v must be [n_rows][heads][d] of the cache");
  const int32_t* slot = a.ints("row_slot", k->size(0));
  if (c.type == DSPARK_MXFP4)
    return dspark_cache_write_mxfp4(a.handle, a.stream, to_int("n_rows", k->size(0)), c.heads, c.d, c.page, c.n_pages,
                                    k->data_ptr(), step(*k, 0), step(*k, 1), v->data_ptr(), step(*v, 0), step(*v, 1),
                                    slot, c.k, c.v, c.s_page, c.s_tok, c.s_head, c.k_power, c.v_power);
  return dspark_cache_write(a.handle, a.stream, to_int("n_rows", k->size(0)), c.heads, c.d, c.page, c.n_pages,
                            k->data_ptr(), step(*k, 0), step(*k, 1), v->data_ptr(), step(*v, 0), step(*v, 1), slot,
                            c.k, c.v, c.s_page, c.s_tok, c.s_head, c.type, c.k_scale, c.v_scale);
}

// kcache, vcache, k_scale, v_scale, row_slot, k, v
int cache_read(Args& a) {
  const Cache c(a);
  const T* slot = a.rows("row_slot", at::kInt, 1);
  const int64_t n = slot->size(0);
  const T* out[2];
  for (int i = 0; i < 2; ++i) {
    out[i] = a.rows(i ? "v" : "k", at::kBFloat16, 3);
    if (out[i]->size(0) != n || out[i]->size(1) != c.heads || out[i]->size(2) != c.d)
      raise(PyExc_ValueError, "k and v must be [n_rows][heads][d] of the cache");
  }
  const Rows k(out[0]), v(out[1]);
  return dspark_cache_read(a.handle, a.stream, to_int("n_rows", n), c.heads, c.d, c.page, c.n_pages,
                           Args::data<int32_t>(slot), c.k, c.v, c.s_page, c.s_tok, c.s_head, c.type, c.k_scale,
                           c.v_scale, c.k_power, c.v_power, k.p, k.row, k.head, v.p, v.row, v.head);
}

// freq, factor: the turned values of a head, its pairs' frequencies and the factor.
struct Turn {
  const double* freq;
  int rot;
  double factor;
  bool interleaved;
  explicit Turn(Args& a) {
    const T* f = a.vector("freq", at::kDouble, -1);
    rot = to_int("freq", 2 * f->size(0));
    freq = Args::data<double>(f);
    interleaved = a.truth();
    factor = a.real64("factor");
  }
};

// freq, interleaved, factor, row_pos, k, k_out, q, q_out
int rope(Args& a) {
  const Turn turn(a);
  const T* pos = a.rows("row_pos", at::kInt, 1);
  const int64_t n = pos->size(0);
  const T* k = a.rows("k", at::kBFloat16, 3, true);
  const T* ko = a.rows("k_out", at::kBFloat16, 3, !k);
  if (k && (k->size(0) != n || ko->sizes() != k->sizes()))
    raise(PyExc_ValueError, "k and k_out must be [n_rows][heads][d]");
  const T* q = a.rows("q", at::kBFloat16, 3, k != nullptr);
  const T* qo = a.rows("q_out", at::kBFloat16, 3, !q);
  if (q && (q->size(0) != n || (k && q->size(2) != k->size(2)) || qo->sizes() != q->sizes()))
    raise(PyExc_ValueError, "q and q_out must be [n_rows][heads_q][d]");
  const Rows rq(q), rk(k), rqo(qo), rko(ko);
  return dspark_rope(a.handle, a.stream, to_int("n_rows", n), q ? to_int("heads_q", q->size(1)) : 0,
                     k ? to_int("heads", k->size(1)) : 0, to_int("d", (k ? k : q)->size(2)), turn.rot, turn.interleaved,
                     Args::data<int32_t>(pos), turn.freq, turn.factor, rq.p, rq.row, rq.head, rk.p, rk.row, rk.head,
                     rqo.p, rqo.row, rqo.head, rko.p, rko.row, rko.head);
}

// kcache, vcache, k_scale, v_scale, freq, interleaved, factor, row_pos,
// row_slot, k, v, q, q_out
int rope_write(Args& a) {
  const Cache c(a);
  const Turn turn(a);
  const T* pos = a.rows("row_pos", at::kInt, 1);
  const int64_t n = pos->size(0);
  const int32_t* slot = a.ints("row_slot", n);
  const T* k = a.rows("k", at::kBFloat16, 3);
  const T* v = a.rows("v", at::kBFloat16, 3);
  if (k->size(0) != n || k->size(1) != c.heads || k->size(2) != c.d || v->sizes() != k->sizes())
    raise(PyExc_ValueError, "k and v must be [n_rows][heads][d] of the cache");
  const T* q = a.rows("q", at::kBFloat16, 3, true);
  const T* qo = a.rows("q_out", at::kBFloat16, 3, !q);
  if (q && (q->size(0) != n || q->size(2) != c.d || qo->sizes() != q->sizes()))
    raise(PyExc_ValueError, "q and q_out must be [n_rows][heads_q][d]");
  const Rows rq(q), rqo(qo), rk(k), rv(v);
  return dspark_rope_write(a.handle, a.stream, to_int("n_rows", n), q ? to_int("heads_q", q->size(1)) : 0, c.heads, c.d,
                           turn.rot, turn.interleaved, c.page, c.n_pages, Args::data<int32_t>(pos), slot, turn.freq,
                           turn.factor, rq.p, rq.row, rq.head, rqo.p, rqo.row, rqo.head, rk.p, rk.row, rk.head, rv.p,
                           rv.row, rv.head, c.k, c.v, c.s_page, c.s_tok, c.s_head, c.type, c.k_scale, c.v_scale,
                           c.k_power, c.v_power);
}

// kcache, vcache, k_scale, v_scale, q, length, table, gamma, K, t_offsets,
// causal, scale, out, lse
int attend(Args& a) {
  const Cache c(a);
  const T* q = a.rows("q", at::kBFloat16, 3);
  if (q->size(2) != c.d) raise(PyExc_ValueError, "q must be [n_rows][heads_q][d] with the cache's d");
  const T* length = a.rows("length", at::kInt, 1);
  const int64_t B = length->size(0);
  if (!length->is_contiguous()) raise(PyExc_ValueError, "length must be contiguous");
  const Table table(a, B);
  const int gamma = a.int32("gamma");
  const int32_t* K = a.ints("K", B, true);
  const int32_t* offs = a.ints("t_offsets", -B, true);
  const bool causal = a.truth();
  const float scale = a.real("scale");
  const T* out = a.rows("out", at::kBFloat16, 3);
  if (out->sizes() != q->sizes()) raise(PyExc_ValueError, "out must have the shape of q");
  const T* lse = a.rows("lse", at::kFloat, 2, true);
  if (lse && (!lse->is_contiguous() || lse->size(0) != q->size(0) || lse->size(1) != q->size(1)))
    raise(PyExc_ValueError, "lse must be [n_rows][heads_q], contiguous");
  if (c.type == DSPARK_MXFP4)
    return dspark_attend_mxfp4(a.handle, a.stream, to_int("B", B), to_int("n_rows", q->size(0)), gamma,
                               to_int("heads_q", q->size(1)), c.heads, c.d, q->data_ptr(), step(*q, 0), step(*q, 1),
                               c.k, c.v, c.s_page, c.s_tok, c.s_head, c.k_power, c.v_power, c.page, c.n_pages, table.p,
                               table.stride, table.cols, Args::data<int32_t>(length), K, offs, causal ? 1 : 0, scale,
                               out->data_ptr(), step(*out, 0), step(*out, 1), Args::data<float>(lse));
  return dspark_attend(a.handle, a.stream, to_int("B", B), to_int("n_rows", q->size(0)), gamma,
                       to_int("heads_q", q->size(1)), c.heads, c.d, q->data_ptr(), step(*q, 0), step(*q, 1), c.k, c.v,
                       c.s_page, c.s_tok, c.s_head, c.type, c.k_scale, c.v_scale, c.page, c.n_pages, table.p,
                       table.stride, table.cols, Args::data<int32_t>(length), K, offs, causal ? 1 : 0, scale,
                       out->data_ptr(), step(*out, 0), step(*out, 1), Args::data<float>(lse));
}

// logits, out, n_pos, K, t_offsets, hist, n_hist, n_prompt, tokens, rep, freq,
// pres, bias ids, bias values, bias counts, mask
int constrain(Args& a) {
  const T* x = a.tensor("logits");
  const at::ScalarType st = x->scalar_type();
  if (st != at::kBFloat16 && st != at::kFloat)
    raise(PyExc_TypeError, "logits must be bf16 or float32, got %s", c10::toString(st));
  const int dims = (int)x->dim();
  if (dims != 2 && dims != 3) raise(PyExc_ValueError, "logits must have 2 (packed) or 3 dims, got %d", dims);
  const int64_t V = x->size(dims - 1);
  if (V > 1 && x->stride(dims - 1) != 1) raise(PyExc_ValueError, "logits must be contiguous over their last dimension");
  const T* out = a.rows("out", at::kFloat, dims);
  if (out->sizes() != x->sizes()) raise(PyExc_ValueError, "out must have the shape of logits");
  const int n_pos = a.int32("n_pos");
  const bool packed = dims == 2;
  const T* K = a.rows("K", at::kInt, 1, true);
  const T* offs = a.rows("t_offsets", at::kInt, 1, true);
  if (packed != (offs != nullptr))
    raise(PyExc_ValueError, "logits must be [n_rows][V] with t_offsets, [B][n_pos][V] without");
  const int64_t B = packed ? (K ? K->size(0) : offs->size(0)) : x->size(0);
  if (K && (K->size(0) != B || !K->is_contiguous())) raise(PyExc_ValueError, "K must have %lld entries", (long long)B);
  if (offs && (offs->size(0) < B || !offs->is_contiguous()))
    raise(PyExc_ValueError, "t_offsets must have at least %lld entries", (long long)B);
  if (!packed && x->size(1) < n_pos)
    raise(PyExc_ValueError, "logits have %lld positions, n_pos is %d", (long long)x->size(1), n_pos);
  // per-request arrays [B][n]: stride of a request
  auto table = [&](const T* t, const char* name, int64_t at_least) -> int64_t {
    if (!t) return 0;
    if (t->size(0) != B || t->size(1) < at_least)
      raise(PyExc_ValueError, "%s must be [%lld][>= %lld]", name, (long long)B, (long long)at_least);
    return step(*t, 0, t->size(1));
  };
  const T* hist = a.rows("hist", at::kInt, 2, true);
  const int64_t s_hist = table(hist, "hist", 0);
  const int32_t* n_hist = a.ints("n_hist", B, !hist);
  const int32_t* n_prompt = a.ints("n_prompt", B, true);
  const T* tokens = a.rows("tokens", at::kInt, 2, true);
  const int64_t s_tok = table(tokens, "tokens", n_pos - 1);
  const float* rep = a.floats("rep", B, true);
  const float* freq = a.floats("freq", B, true);
  const float* pres = a.floats("pres", B, true);
  const T* ids = a.rows("bias ids", at::kInt, 2, true);
  const int64_t s_bias = table(ids, "bias ids", 0);
  const T* values = a.rows("bias values", at::kFloat, 2, !ids);
  if (ids && (values->sizes() != ids->sizes() || step(*values, 0, ids->size(1)) != s_bias))
    raise(PyExc_ValueError, "bias ids and values must have one shape and one set of strides");
  const int32_t* n_bias = a.ints("bias counts", B, true);
  const T* mask = a.rows("mask", at::kInt, dims, true);
  // strides of a request and of a row; a row that is the only one takes its width
  const int64_t wide = (V + 7) / 8 * 8;
  struct Steps {
    int64_t b, k;
  };
  auto steps = [&](const T& t, int64_t width) {
    return packed ? Steps{0, step(t, 0, width)} : Steps{step(t, 0), step(t, 1, width)};
  };
  Steps m{0, 0};
  if (mask) {
    bool fits = mask->size(dims - 1) >= (V + 31) / 32;
    for (int i = 0; i < dims - 1; ++i) fits = fits && mask->size(i) == x->size(i);
    if (!fits) raise(PyExc_ValueError, "mask must have the rows of logits and %lld words in each", (long long)((V + 31) / 32));
    m = steps(*mask, mask->size(dims - 1));
  }
  const Steps l = steps(*x, wide), o = steps(*out, wide);
  return dspark_constrain(a.handle, a.stream, to_int("B", B), n_pos, to_int("V", V), x->data_ptr(),
                          st == at::kBFloat16 ? DSPARK_BF16 : DSPARK_F32, l.b, l.k, Args::data<int32_t>(offs),
                          Args::data<int32_t>(K), packed ? to_int("n_rows", x->size(0)) : 0,
                          Args::data<int32_t>(hist), s_hist, hist ? to_int("hist", hist->size(1)) : 0, n_hist,
                          n_prompt, Args::data<int32_t>(tokens), s_tok, rep, freq, pres, Args::data<int32_t>(ids),
                          Args::data<float>(values), s_bias, ids ? to_int("bias", ids->size(1)) : 0, n_bias,
                          Args::data<int32_t>(mask), m.b, m.k, static_cast<float*>(out->data_ptr()), o.b, o.k);
}

template <int (*F)(Args&), int N>
PyObject* entry(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    Args a(v, n, N + 3);
    return PyLong_FromLong(F(a));
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <int (*F)(Args&), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<pages_reserve, 15>("pages_reserve"), method<pages_commit, 12>("pages_commit"),
    method<cache_write, 7>("cache_write"),      method<attend, 14>("attend"),
    method<constrain, 16>("constrain"),         method<cache_read, 7>("cache_read"),
    method<rope, 8>("rope"),                    method<rope_write, 13>("rope_write"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
