// Python entry of the operators around the paged cache: argument checks and the call of the C ABI
// (include/nld.h).  A decode step makes these calls with a handful of rows, where the call itself is the
// latency; through ctypes and Python-level checks it took 14 to 20 us, from here 3 to 6 us.
//
// Every function takes its arguments by position (the Python functions of the package give names and
// defaults), raises ValueError for a tensor of the wrong type, shape, layout or device and returns the
// library's status.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdio>
#include <initializer_list>
#include <string>

#include "nld.h"

namespace {

struct Raised {};   // a Python error is set

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Raised();
}

std::string text(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

int as_int(const char* name, int64_t v) {
  if (v < INT_MIN || v > INT_MAX) refuse(std::string(name) + " is too large");
  return static_cast<int>(v);
}

// The arguments of one call, in order.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : args_(args) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments expected, not %zd", want, n);
      throw Raised();
    }
    device_ = c10::cuda::current_device();
  }
  const at::Tensor& tensor(const char* name) {
    PyObject* o = *args_++;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device_)
      refuse(std::string(name) + " must be on the current CUDA device (" + std::to_string(device_) + ")");
    return t;
  }
  const at::Tensor* optional(const char* name) {
    if (*args_ != Py_None) return &tensor(name);
    ++args_;
    return nullptr;
  }
  int integer(const char* name) {
    PyObject* o = PyNumber_Index(*args_++);
    if (!o) throw Raised();
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    Py_DECREF(o);
    return as_int(name, over ? LLONG_MAX : v);
  }
  float number() {
    const double v = PyFloat_AsDouble(*args_++);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return static_cast<float>(v);
  }
  // The caller's stream, else torch's current one on the current device.
  void* stream() {
    PyObject* o = *args_++;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised();
    return p;
  }

 private:
  PyObject* const* args_;
  int device_;
};

void dims(const at::Tensor& t, int n, const char* what) {
  if (t.dim() != n) refuse(std::string(what) + " expected");
}
void check(const char* name, const at::Tensor& t, at::ScalarType type) {
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + toString(type) + ", not " + toString(t.scalar_type()));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}
void check(const char* name, const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) refuse(std::string(name) + " must be " + text(want) + ", not " + text(t.sizes()));
  check(name, t, type);
}
template <typename T = void>
T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T = void>
T* ptr(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
template <typename T = void>
T* ptr(const char* name, const at::Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape) {
  if (!t) return nullptr;
  check(name, *t, type, shape);
  return static_cast<T*>(t->data_ptr());
}
int32_t* error_word(const at::Tensor* t) {
  if (!t) return nullptr;
  check("err", *t, at::kInt);
  if (t->numel() < 1) refuse("err must hold one element");
  return static_cast<int32_t*>(t->data_ptr());
}

// Elements between the token rows of t [batch, m, heads, hd]: heads contiguous, one distance between all tokens.
int64_t token_rows(const char* name, const at::Tensor& t, int64_t batch, int64_t m, int64_t heads, int64_t hd,
                   at::ScalarType type) {
  const int64_t want[4] = {batch, m, heads, hd};
  if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(want, 4))
    refuse(std::string(name) + " must be a " + toString(type) + " tensor " + text(at::IntArrayRef(want, 4)));
  const at::IntArrayRef s = t.strides();
  if ((hd > 1 && s[3] != 1) || (heads > 1 && s[2] != hd) || (m > 1 && batch > 1 && s[0] != m * s[1]))
    refuse(std::string(name) + ": the heads of a token must be contiguous and the tokens evenly spaced");
  return m > 1 ? s[1] : batch > 1 ? s[0] : heads * hd;
}

template <nld_status (*kCall)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return PyLong_FromLong(kCall(args, n));
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

nld_status qk_norm_rope(PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 17);
  const at::Tensor &q = a.tensor("q"), &k = a.tensor("k"), &v = a.tensor("v");
  const at::Tensor *q_gain = a.optional("q_gain"), *k_gain = a.optional("k_gain");
  const float eps = a.number();
  const at::Tensor &rope = a.tensor("rope"), &lens = a.tensor("lens"), &q_out = a.tensor("q_out"), &pool = a.tensor("kv_pool"),
                   &table = a.tensor("page_table");
  const int offset = a.integer("position_offset");
  const at::Tensor *rows = a.optional("rows"), *k_scale = a.optional("k_scale"), *v_scale = a.optional("v_scale"),
                   *err = a.optional("err");
  dims(q, 4, "q [B, m, Hq, hd]");
  dims(k, 4, "k [B, m, Hkv, hd]");
  dims(rope, 3, "rope [positions, hd/2, 2]");
  dims(pool, 5, "kv_pool [n_pages, 2, Hkv, 64, hd]");
  dims(table, 2, "page_table [B, pps]");
  const int64_t B = q.size(0), m = q.size(1), Hq = q.size(2), hd = q.size(3), Hkv = k.size(2);
  const at::ScalarType dt = q.scalar_type(), kv = pool.scalar_type();
  if (dt != at::kBFloat16 && dt != at::kFloat) refuse("q must be bfloat16 or float32");
  if (kv != at::kFloat && kv != at::kBFloat16 && kv != at::kFloat8_e4m3fn) refuse("kv_pool must be float32, bfloat16 or float8_e4m3fn");
  const int64_t q_ld = token_rows("q", q, B, m, Hq, hd, dt), k_ld = token_rows("k", k, B, m, Hkv, hd, dt),
                v_ld = token_rows("v", v, B, m, Hkv, hd, dt);
  check("rope", rope, at::kFloat, {rope.size(0), hd / 2, 2});
  check("lens", lens, at::kInt, {B});
  check("q_out", q_out, dt, {B, m, Hq, hd});
  check("kv_pool", pool, kv, {pool.size(0), 2, Hkv, 64, hd});
  check("page_table", table, at::kInt, {B, table.size(1)});
  return nld_qk_norm_rope(
      ptr(q), q_ld, ptr(k), k_ld, ptr(v), v_ld, dt == at::kFloat ? NLD_F32 : NLD_BF16, ptr("q_gain", q_gain, dt, {hd}),
      ptr("k_gain", k_gain, dt, {hd}), eps, ptr<float>(rope), as_int("rope", rope.size(0)), offset, ptr<int32_t>(lens),
      ptr<int32_t>("rows", rows, at::kInt, {B}), as_int("batch", B), as_int("m", m), as_int("query heads", Hq),
      as_int("kv heads", Hkv), as_int("head_dim", hd), ptr(q_out), ptr(pool),
      kv == at::kFloat ? NLD_F32 : kv == at::kBFloat16 ? NLD_BF16 : NLD_E4M3, ptr<float>("k_scale", k_scale, at::kFloat, {Hkv}),
      ptr<float>("v_scale", v_scale, at::kFloat, {Hkv}), ptr<int32_t>(table), as_int("page_table", table.size(1)),
      as_int("pages", pool.size(0)), error_word(err), a.stream());
}

// What the two attentions have in common: q, the pool, the page table, lens and out.
struct Attention {
  int B, m, Hq, hd, n_pages, Hkv, pps;
  Attention(const at::Tensor& q, const at::Tensor& pool, at::ScalarType kv, const at::Tensor& table, const at::Tensor& lens,
            const at::Tensor& out) {
    dims(q, 4, "q [B, m, Hq, hd]");
    dims(pool, 5, "kv_pool [n_pages, 2, Hkv, 64, hd]");
    dims(table, 2, "page_table [B, pps]");
    B = as_int("batch", q.size(0));
    m = as_int("m", q.size(1));
    Hq = as_int("query heads", q.size(2));
    hd = as_int("head_dim", q.size(3));
    n_pages = as_int("pages", pool.size(0));
    Hkv = as_int("kv heads", pool.size(2));
    pps = as_int("page_table", table.size(1));
    check("q", q, at::kBFloat16);
    check("kv_pool", pool, kv, {n_pages, 2, Hkv, 64, hd});
    check("page_table", table, at::kInt, {B, pps});
    check("lens", lens, at::kInt, {B});
    check("out", out, at::kBFloat16, {B, m, Hq, hd});
  }
};

nld_status attention_q8(PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 11);
  const at::Tensor &q = a.tensor("q"), &pool = a.tensor("kv_pool"), &k_scale = a.tensor("k_scale"),
                   &v_scale = a.tensor("v_scale"), &table = a.tensor("page_table"), &lens = a.tensor("lens");
  const int block = a.integer("block_size"), max_len = a.integer("max_len");
  const at::Tensor& out = a.tensor("out");
  const at::Tensor* err = a.optional("err");
  const Attention t(q, pool, at::kFloat8_e4m3fn, table, lens, out);
  check("k_scale", k_scale, at::kFloat, {t.Hkv});
  check("v_scale", v_scale, at::kFloat, {t.Hkv});
  return nld_attention_q8(ptr(q), ptr(pool), ptr<float>(k_scale), ptr<float>(v_scale), ptr<int32_t>(table), t.pps, t.n_pages,
                          ptr<int32_t>(lens), t.B, t.m, t.Hq, t.Hkv, t.hd, block, max_len, ptr(out), error_word(err),
                          a.stream());
}

nld_status attention_shared(PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 12);
  const at::Tensor &q = a.tensor("q"), &pool = a.tensor("kv_pool");
  const at::Tensor* pages = a.optional("shared_pages");
  const int shared_len = a.integer("shared_len");
  const at::Tensor &table = a.tensor("page_table"), &lens = a.tensor("lens");
  const int block = a.integer("block_size"), max_len = a.integer("max_len");
  const at::Tensor& out = a.tensor("out");
  const at::Tensor *workspace = a.optional("workspace"), *err = a.optional("err");
  const Attention t(q, pool, at::kBFloat16, table, lens, out);
  if (pages) check("shared_pages", *pages, at::kInt, {pages->numel()});
  if (workspace) check("workspace", *workspace, at::kByte);
  return nld_attention_shared(ptr(q), ptr(pool), ptr<int32_t>(pages), pages ? as_int("shared_pages", pages->numel()) : 0,
                              shared_len, ptr<int32_t>(table), t.pps, t.n_pages, ptr<int32_t>(lens), t.B, t.m, t.Hq, t.Hkv, t.hd,
                              block, max_len, ptr(out), ptr(workspace), workspace ? workspace->numel() : 0, error_word(err),
                              a.stream());
}

nld_status sample(PyObject* const* args, Py_ssize_t n) {
  Args a(args, n, 9);
  const at::Tensor &logits = a.tensor("logits"), &u = a.tensor("u"), &tokens = a.tensor("tokens_out");
  const at::Tensor *prob = a.optional("prob_out"), *temperature = a.optional("temperature"), *top_k = a.optional("top_k"),
                   *top_p = a.optional("top_p"), *min_p = a.optional("min_p");
  const at::ScalarType dt = logits.scalar_type();
  if (logits.dim() != 2 || (dt != at::kFloat && dt != at::kBFloat16)) refuse("logits must be [rows, vocab], float32 or bfloat16");
  const int64_t rows = logits.size(0), vocab = logits.size(1);
  if (vocab > 1 && logits.stride(1) != 1) refuse("each row of logits must be contiguous");
  check("u", u, at::kFloat, {rows});
  check("tokens_out", tokens, at::kInt, {rows});
  return nld_sample(ptr(logits), dt == at::kFloat ? NLD_F32 : NLD_BF16, rows > 1 ? logits.stride(0) : vocab,
                    as_int("rows", rows), as_int("vocab", vocab), ptr<float>(u),
                    ptr<float>("temperature", temperature, at::kFloat, {rows}), ptr<int32_t>("top_k", top_k, at::kInt, {rows}),
                    ptr<float>("top_p", top_p, at::kFloat, {rows}), ptr<float>("min_p", min_p, at::kFloat, {rows}),
                    ptr<int32_t>(tokens), ptr<float>("prob_out", prob, at::kFloat, {rows}), a.stream());
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(qk_norm_rope), ENTRY(attention_q8), ENTRY(attention_shared), ENTRY(sample), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operators", NLD_BUILT_FOR, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operators() { return PyModule_Create(&module); }
