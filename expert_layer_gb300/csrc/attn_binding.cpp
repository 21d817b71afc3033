// The Python functions of the attention entry points (attention.py): argument
// checks and marshalling on tensors directly.  A decode step calls them once a
// layer; done through Python attributes and ctypes the checks cost 8 us a call,
// several times the kernels of a small batch (here about 1 us).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <optional>
#include <string>
#include <vector>

#include "moe.h"

namespace {

struct Library {
  decltype(&moe_attn_workspace_size) workspace_size;
  decltype(&moe_rope_append_axes) rope_append;
  decltype(&moe_attn_prefill) prefill;
  decltype(&moe_attn_prefill_paged) prefill_paged;
  decltype(&moe_attn_decode) decode;
  decltype(&moe_rope_append_fp8) rope_append_fp8;
  decltype(&moe_attn_prefill_paged_fp8) prefill_paged_fp8;
  decltype(&moe_attn_decode_fp8) decode_fp8;
  decltype(&moe_attn_key_weights) key_weights;
  decltype(&moe_kv_evict) evict;
  decltype(&moe_error_string) error_string;
} lib = {};
constexpr int kAddresses = sizeof(Library) / sizeof(void*);
PyObject* error_type = nullptr;       // MoEError

struct Refusal {
  std::string text;
};
struct PythonError {};                // the Python error is set already

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i)
    t += (i ? ", " : "") + (s[i] < 0 ? std::string("any") : std::to_string(s[i]));
  return t + (s.size() == 1 ? ",)" : ")");
}
const char* type_text(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return at::toString(t);
  }
}

const at::Tensor& as_tensor(PyObject* o, const char* name) {
  if (!o || !THPVariable_Check(o)) throw Refusal{std::string(name) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

// A CUDA tensor of this type, device and shape (-1: any size)
const at::Tensor& checked(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int device) {
  const at::Tensor& t = as_tensor(o, name);
  const std::string n = name;
  if (!t.is_cuda()) throw Refusal{n + " must be a CUDA tensor"};
  if (t.get_device() != device)
    throw Refusal{n + " must be on cuda:" + std::to_string(device) + ", got cuda:" + std::to_string(t.get_device())};
  if (t.scalar_type() != type) throw Refusal{n + " must be " + type_text(type) + ", got " + type_text(t.scalar_type())};
  if (t.dim() != (int64_t)shape.size())
    throw Refusal{n + " must have " + std::to_string(shape.size()) + " dimensions, got " + std::to_string(t.dim())};
  for (size_t i = 0; i < shape.size(); ++i)
    if (shape[i] >= 0 && shape[i] != t.size(i))
      throw Refusal{n + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes())};
  return t;
}
const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int device) {
  const at::Tensor& t = checked(o, name, type, shape, device);
  if (!t.is_contiguous()) throw Refusal{std::string(name) + " must be contiguous"};
  return t;
}
template <typename T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
bool given(PyObject* o) { return o && o != Py_None; }

// A [tokens, heads, D] view: any token and head stride, dense D
moe_heads heads(const at::Tensor& t, const char* name) {
  if (t.stride(2) != 1 && t.size(2) > 1 && t.numel() > 0)
    throw Refusal{std::string(name) + " must be contiguous in its last dimension"};
  return moe_heads{t.data_ptr(), t.stride(0), t.stride(1)};
}

int whole(int64_t v, const char* name) {
  if (v > INT32_MAX || v < INT32_MIN) throw Refusal{std::string(name) + " is out of range"};
  return (int)v;
}

struct Query {
  moe_heads view;
  at::ScalarType type;
  int T, Hq, D, code, device;
};
Query query(PyObject* o) {
  if (!o || !THPVariable_Check(o)) throw Refusal{"q must be a bfloat16 or float16 torch.Tensor"};
  const at::Tensor& t = THPVariable_Unpack(o);
  Query q;
  q.type = t.scalar_type();
  if (q.type != at::kBFloat16 && q.type != at::kHalf) throw Refusal{"q must be a bfloat16 or float16 torch.Tensor"};
  if (!t.is_cuda()) throw Refusal{"q must be a CUDA tensor"};
  q.device = c10::cuda::current_device();
  checked(o, "q", q.type, {-1, -1, -1}, q.device);
  q.view = heads(t, "q");
  q.T = whole(t.size(0), "q");
  q.Hq = whole(t.size(1), "q");
  q.D = whole(t.size(2), "q");
  q.code = q.type == at::kBFloat16 ? MOE_BF16 : MOE_F16;
  return q;
}

struct Cache {
  moe_kv_cache c;
  int Hkv;
};
Cache cache(PyObject* k, PyObject* v, const Query& q) {
  const at::Tensor& kt = dense(k, "k_cache", q.type, {-1, -1, -1, q.D}, q.device);
  const at::Tensor& vt = dense(v, "v_cache", q.type, kt.sizes(), q.device);
  return Cache{moe_kv_cache{kt.data_ptr(), vt.data_ptr(), whole(kt.size(0), "k_cache"), whole(kt.size(2), "k_cache")},
               whole(kt.size(1), "k_cache")};
}

struct CacheFp8 {
  moe_kv_cache_fp8 c;
  int Hkv;
};
CacheFp8 cache_fp8(PyObject* k, PyObject* v, PyObject* scales, const Query& q) {
  const at::Tensor& kt = dense(k, "k_cache", at::kFloat8_e4m3fn, {-1, -1, -1, q.D}, q.device);
  const at::Tensor& vt = dense(v, "v_cache", at::kFloat8_e4m3fn, kt.sizes(), q.device);
  const at::Tensor& st = dense(scales, "scales", at::kFloat, {kt.size(0), kt.size(1), kt.size(2) / 16, 2}, q.device);
  return CacheFp8{moe_kv_cache_fp8{kt.data_ptr(), vt.data_ptr(), ptr<float>(st), whole(kt.size(0), "k_cache"),
                                   whole(kt.size(2), "k_cache")},
                  whole(kt.size(1), "k_cache")};
}

// Where a call runs.  What it allocates comes from that stream's memory: a
// block of the caller's stream that was just freed may still be in use by work
// queued there, for which another stream does not wait.
struct Run {
  int device;
  void* stream;
  c10::cuda::CUDAStream callers;
  std::optional<c10::cuda::CUDAStreamGuard> guard;        // of a launch stream that is not the caller's
  std::vector<at::Tensor> made;

  Run(PyObject* given_stream, int dev) : device(dev), callers(c10::cuda::getCurrentCUDAStream(dev)) {
    stream = callers.stream();
    if (!given(given_stream)) return;
    PyObject* attr = PyObject_GetAttrString(given_stream, "cuda_stream");
    if (!attr) throw PythonError{};
    stream = PyLong_AsVoidPtr(attr);
    Py_DECREF(attr);
    if (PyErr_Occurred()) throw PythonError{};
    if (stream != callers.stream())
      guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), dev));
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) {
    made.push_back(at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, device))));
    return made.back();
  }
  // a tensor that the caller gets: freed, it is kept until the caller's stream is past it
  at::Tensor returned(const at::Tensor& t) {
    if (guard) t.record_stream(callers.unwrap());
    return t;
  }
};

struct Space {
  void* data;
  size_t bytes;
};
Space workspace(PyObject* o, int T, int n_seq, int Hq, int Hkv, int D, Run& run) {
  if (given(o)) {
    const at::Tensor& t = dense(o, "workspace", at::kByte, {-1}, run.device);
    return Space{t.data_ptr(), (size_t)t.numel()};
  }
  const size_t n = lib.workspace_size(T > 0 ? T : 1, n_seq, Hq, Hkv, D);
  if (n == 0) throw Refusal{"unsupported shape"};
  return Space{run.make({(int64_t)n}, at::kByte).data_ptr(), n};
}

// An output of this shape: the caller's, or a new one (then `wrapped` owns it)
struct Output {
  PyObject* object;
  void* data;
};
Output output(PyObject* o, const char* name, const Query& q, Run& run) {
  if (given(o)) {
    void* data = dense(o, name, q.type, {q.T, q.Hq, q.D}, q.device).data_ptr();
    Py_INCREF(o);
    return Output{o, data};
  }
  at::Tensor t = run.returned(run.make({q.T, q.Hq, q.D}, q.type));
  return Output{THPVariable_Wrap(t), t.data_ptr()};
}
struct Owned {      // gives the reference back unless it is returned
  PyObject* o;
  ~Owned() { Py_XDECREF(o); }
  PyObject* release() {
    PyObject* r = o;
    o = nullptr;
    return r;
  }
};

void check(int rc, const char* what) {
  if (rc != MOE_OK)
    throw Refusal{std::string(what) + " failed: " + lib.error_string(rc) + " (" + std::to_string(rc) + ")"};
}

// ------------------------------------------------------------- arguments
// A function's parameters, defaults and documentation are those of its Python
// definition (attention.py), handed over by bind(); the functions below take
// them in that order.
constexpr int kMost = 19;
struct Spec {
  const char* function;
  int total;
  int required;
  PyObject* names[kMost];         // interned
  PyObject* defaults[kMost];      // null where required
  std::string doc;
};
struct Args {
  PyObject* v[kMost] = {};
};
Args parse(const Spec& s, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
  Args a;
  if (!lib.rope_append) throw Refusal{"the attention functions are not bound to the library"};
  const std::string f = std::string(s.function) + "() ";
  if (n > s.total) {
    PyErr_SetString(PyExc_TypeError, (f + "takes " + std::to_string(s.total) + " arguments at most").c_str());
    throw PythonError{};
  }
  for (Py_ssize_t i = 0; i < n; ++i) a.v[i] = args[i];
  const Py_ssize_t kw = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t i = 0; i < kw; ++i) {
    PyObject* name = PyTuple_GET_ITEM(kwnames, i);
    int at = -1;
    for (int j = 0; j < s.total && at < 0; ++j)
      if (s.names[j] == name) at = j;
    for (int j = 0; j < s.total && at < 0; ++j)
      if (PyUnicode_Compare(s.names[j], name) == 0) at = j;
    if (at < 0 || a.v[at]) {
      PyErr_Format(PyExc_TypeError, "%s() got an unexpected or repeated argument '%U'", s.function, name);
      throw PythonError{};
    }
    a.v[at] = args[n + i];
  }
  for (int j = 0; j < s.total; ++j)
    if (!a.v[j] && !(a.v[j] = s.defaults[j])) {
      PyErr_Format(PyExc_TypeError, "%s() misses the argument '%U'", s.function, s.names[j]);
      throw PythonError{};
    }
  return a;
}
double number(PyObject* o, double otherwise) {
  if (!given(o)) return otherwise;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
long integer(PyObject* o, long otherwise, const char* name) {
  if (!given(o)) return otherwise;
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return whole(v, name);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}
float scale_of(PyObject* o, int D) { return (float)number(o, D > 0 ? 1.0 / std::sqrt((double)D) : 0.0); }

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const PythonError&) {
  } catch (const Refusal& r) {
    PyErr_SetString(error_type ? error_type : PyExc_RuntimeError, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(error_type ? error_type : PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ------------------------------------------------------------- functions
// Positions [T], or with axes (uint8 [rot / 2]) [n_axes, T]
struct Turn {
  const int32_t* positions;
  const uint8_t* axes;
  int n_axes;
};
Turn turn(PyObject* positions, PyObject* axes, const at::Tensor& table, const Query& q) {
  if (!given(axes)) return Turn{ptr<int32_t>(dense(positions, "positions", at::kInt, {q.T}, q.device)), nullptr, 0};
  const at::Tensor& a = dense(axes, "axes", at::kByte, {table.size(1) / 2}, q.device);
  const at::Tensor& p = dense(positions, "positions", at::kInt, {-1, q.T}, q.device);
  // (no pair is turned: no axes, and a pointer that may be null)
  return Turn{ptr<int32_t>(p), a.numel() ? ptr<uint8_t>(a) : nullptr, whole(p.size(0), "positions")};
}

Spec rope_spec = {"rope_append", 16};
PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(rope_spec, args, n, kw);
    const Query q = query(a.v[0]);
    const Cache c = cache(a.v[6], a.v[7], q);
    const moe_heads k = heads(checked(a.v[1], "k", q.type, {q.T, c.Hkv, q.D}, q.device), "k");
    const moe_heads v = heads(checked(a.v[2], "v", q.type, {q.T, c.Hkv, q.D}, q.device), "v");
    const at::Tensor& table = dense(a.v[3], "table", at::kFloat, {-1, -1}, q.device);
    const Turn by = turn(a.v[4], a.v[15], table, q);
    const int32_t* slots = ptr<int32_t>(dense(a.v[5], "slots", at::kInt, {q.T}, q.device));
    const float* qn = given(a.v[8]) ? ptr<float>(dense(a.v[8], "q_norm", at::kFloat, {q.D}, q.device)) : nullptr;
    const float* kn = given(a.v[9]) ? ptr<float>(dense(a.v[9], "k_norm", at::kFloat, {q.D}, q.device)) : nullptr;
    const float eps = (float)number(a.v[10], 1e-6);
    const bool interleaved = truth(a.v[11]);
    Run run(a.v[14], q.device);
    const Output out = output(a.v[12], "q_out", q, run);
    Owned owned{out.object};
    const Space ws = workspace(a.v[13], q.T, 0, q.Hq, c.Hkv, q.D, run);
    check(lib.rope_append(&q.view, &k, &v, qn, kn, eps, ptr<float>(table), whole(table.size(0), "table"),
                          whole(table.size(1), "table"), interleaved, by.positions, by.axes, by.n_axes, slots, q.T,
                          q.Hq, c.Hkv, q.D, q.code, out.data, &c.c, ws.data, ws.bytes, run.stream),
          "moe_rope_append");
    return owned.release();
  });
}

// The page table, starts and lengths of a ragged call
struct Ragged {
  const int32_t* table;
  const int32_t* q_starts;
  const int32_t* lens;
  int pages, seqs;
};
Ragged ragged(PyObject* page_table, PyObject* q_starts, PyObject* kv_lens, int device) {
  Ragged r;
  const at::Tensor& lens = dense(kv_lens, "kv_lens", at::kInt, {-1}, device);
  r.seqs = whole(lens.size(0), "kv_lens");
  r.lens = ptr<int32_t>(lens);
  r.q_starts = ptr<int32_t>(dense(q_starts, "q_starts", at::kInt, {r.seqs + 1}, device));
  const at::Tensor& table = dense(page_table, "page_table", at::kInt, {r.seqs, -1}, device);
  r.table = ptr<int32_t>(table);
  r.pages = whole(table.size(1), "page_table");
  return r;
}

Spec rope_fp8_spec = {"rope_append_fp8", 19};
PyObject* rope_append_fp8(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(rope_fp8_spec, args, n, kw);
    const Query q = query(a.v[0]);
    const CacheFp8 c = cache_fp8(a.v[8], a.v[9], a.v[10], q);
    const moe_heads k = heads(checked(a.v[1], "k", q.type, {q.T, c.Hkv, q.D}, q.device), "k");
    const moe_heads v = heads(checked(a.v[2], "v", q.type, {q.T, c.Hkv, q.D}, q.device), "v");
    const at::Tensor& table = dense(a.v[3], "table", at::kFloat, {-1, -1}, q.device);
    const Turn by = turn(a.v[4], a.v[15], table, q);
    const Ragged r = ragged(a.v[5], a.v[6], a.v[7], q.device);
    const float* qn = given(a.v[11]) ? ptr<float>(dense(a.v[11], "q_norm", at::kFloat, {q.D}, q.device)) : nullptr;
    const float* kn = given(a.v[12]) ? ptr<float>(dense(a.v[12], "k_norm", at::kFloat, {q.D}, q.device)) : nullptr;
    const float eps = (float)number(a.v[13], 1e-6);
    const bool interleaved = truth(a.v[14]);
    Run run(a.v[18], q.device);
    const Output out = output(a.v[16], "q_out", q, run);
    Owned owned{out.object};
    const Space ws = workspace(a.v[17], q.T, r.seqs, q.Hq, c.Hkv, q.D, run);
    check(lib.rope_append_fp8(&q.view, &k, &v, qn, kn, eps, ptr<float>(table), whole(table.size(0), "table"),
                              whole(table.size(1), "table"), interleaved, by.positions, by.axes, by.n_axes, r.table,
                              r.pages, r.q_starts, r.lens, r.seqs, q.T, q.Hq, c.Hkv, q.D, q.code, out.data, &c.c,
                              ws.data, ws.bytes, run.stream),
          "moe_rope_append_fp8");
    return owned.release();
  });
}

float* lse_of(PyObject* o, const Query& q) {
  return given(o) ? ptr<float>(dense(o, "lse", at::kFloat, {q.T, q.Hq}, q.device)) : nullptr;
}

Spec prefill_spec = {"attn_prefill", 11};
PyObject* attn_prefill(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(prefill_spec, args, n, kw);
    const Query q = query(a.v[0]);
    const at::Tensor& kt = checked(a.v[1], "k", q.type, {-1, -1, q.D}, q.device);
    const moe_heads k = heads(kt, "k"), v = heads(checked(a.v[2], "v", q.type, kt.sizes(), q.device), "v");
    const at::Tensor& qs = dense(a.v[3], "q_starts", at::kInt, {-1}, q.device);
    const int seqs = whole(qs.size(0), "q_starts") - 1;
    if (seqs < 0) throw Refusal{"q_starts must have n_seq + 1 entries"};
    const at::Tensor& ks = dense(a.v[4], "kv_starts", at::kInt, {seqs + 1}, q.device);
    const int Tk = whole(kt.size(0), "k"), Hkv = whole(kt.size(1), "k");
    Run run(a.v[10], q.device);
    const Output out = output(a.v[7], "out", q, run);
    Owned owned{out.object};
    float* lse = lse_of(a.v[8], q);
    const Space ws = workspace(a.v[9], q.T, seqs, q.Hq, Hkv, q.D, run);
    check(lib.prefill(&q.view, &k, &v, ptr<int32_t>(qs), ptr<int32_t>(ks), seqs, q.T, Tk, q.Hq, Hkv, q.D, q.code,
                      truth(a.v[5]), scale_of(a.v[6], q.D), out.data, lse, ws.data, ws.bytes, run.stream),
          "moe_attn_prefill");
    return owned.release();
  });
}

Spec paged_spec = {"attn_prefill_paged", 12};
PyObject* attn_prefill_paged(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(paged_spec, args, n, kw);
    const Query q = query(a.v[0]);
    const Cache c = cache(a.v[1], a.v[2], q);
    const Ragged r = ragged(a.v[3], a.v[4], a.v[5], q.device);
    Run run(a.v[11], q.device);
    const Output out = output(a.v[8], "out", q, run);
    Owned owned{out.object};
    float* lse = lse_of(a.v[9], q);
    const Space ws = workspace(a.v[10], q.T, r.seqs, q.Hq, c.Hkv, q.D, run);
    check(lib.prefill_paged(&q.view, &c.c, r.table, r.pages, r.q_starts, r.lens, r.seqs, q.T, q.Hq, c.Hkv, q.D, q.code,
                            truth(a.v[6]), scale_of(a.v[7], q.D), out.data, lse, ws.data, ws.bytes, run.stream),
          "moe_attn_prefill_paged");
    return owned.release();
  });
}

// The pages of a shared prefix (null without one)
const int32_t* prefix_of(PyObject* table, int prefix_len, int page_size, int device) {
  if (prefix_len <= 0) return nullptr;
  if (!given(table)) throw Refusal{"prefix_len > 0 needs a prefix_table"};
  const at::Tensor& pt = dense(table, "prefix_table", at::kInt, {-1}, device);
  if (pt.size(0) * page_size < prefix_len)
    throw Refusal{"prefix_table holds " + std::to_string(pt.size(0)) + " pages, too few for " +
                  std::to_string(prefix_len) + " tokens"};
  return ptr<int32_t>(pt);
}

Spec decode_spec = {"attn_decode", 12};
PyObject* attn_decode(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(decode_spec, args, n, kw);
    const Query q = query(a.v[0]);
    const Cache c = cache(a.v[1], a.v[2], q);
    const at::Tensor& lens = dense(a.v[4], "kv_lens", at::kInt, {q.T}, q.device);
    const at::Tensor& table = dense(a.v[3], "page_table", at::kInt, {q.T, -1}, q.device);
    const int prefix_len = (int)integer(a.v[6], 0, "prefix_len");
    const int32_t* prefix = prefix_of(a.v[5], prefix_len, c.c.page_size, q.device);
    Run run(a.v[11], q.device);
    const Output out = output(a.v[8], "out", q, run);
    Owned owned{out.object};
    float* lse = lse_of(a.v[9], q);
    const Space ws = workspace(a.v[10], q.T, q.T, q.Hq, c.Hkv, q.D, run);
    check(lib.decode(&q.view, &c.c, ptr<int32_t>(table), whole(table.size(1), "page_table"), ptr<int32_t>(lens), prefix,
                     prefix_len, q.T, q.Hq, c.Hkv, q.D, q.code, scale_of(a.v[7], q.D), out.data, lse, ws.data, ws.bytes,
                     run.stream),
          "moe_attn_decode");
    return owned.release();
  });
}

Spec paged_fp8_spec = {"attn_prefill_paged_fp8", 13};
PyObject* attn_prefill_paged_fp8(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(paged_fp8_spec, args, n, kw);
    const Query q = query(a.v[0]);
    const CacheFp8 c = cache_fp8(a.v[1], a.v[2], a.v[3], q);
    const Ragged r = ragged(a.v[4], a.v[5], a.v[6], q.device);
    Run run(a.v[12], q.device);
    const Output out = output(a.v[9], "out", q, run);
    Owned owned{out.object};
    float* lse = lse_of(a.v[10], q);
    const Space ws = workspace(a.v[11], q.T, r.seqs, q.Hq, c.Hkv, q.D, run);
    check(lib.prefill_paged_fp8(&q.view, &c.c, r.table, r.pages, r.q_starts, r.lens, r.seqs, q.T, q.Hq, c.Hkv, q.D,
                                q.code, truth(a.v[7]), scale_of(a.v[8], q.D), out.data, lse, ws.data, ws.bytes,
                                run.stream),
          "moe_attn_prefill_paged_fp8");
    return owned.release();
  });
}

Spec decode_fp8_spec = {"attn_decode_fp8", 13};
PyObject* attn_decode_fp8(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(decode_fp8_spec, args, n, kw);
    const Query q = query(a.v[0]);
    const CacheFp8 c = cache_fp8(a.v[1], a.v[2], a.v[3], q);
    const at::Tensor& lens = dense(a.v[5], "kv_lens", at::kInt, {q.T}, q.device);
    const at::Tensor& table = dense(a.v[4], "page_table", at::kInt, {q.T, -1}, q.device);
    const int prefix_len = (int)integer(a.v[7], 0, "prefix_len");
    const int32_t* prefix = prefix_of(a.v[6], prefix_len, c.c.page_size, q.device);
    Run run(a.v[12], q.device);
    const Output out = output(a.v[9], "out", q, run);
    Owned owned{out.object};
    float* lse = lse_of(a.v[10], q);
    const Space ws = workspace(a.v[11], q.T, q.T, q.Hq, c.Hkv, q.D, run);
    check(lib.decode_fp8(&q.view, &c.c, ptr<int32_t>(table), whole(table.size(1), "page_table"), ptr<int32_t>(lens),
                         prefix, prefix_len, q.T, q.Hq, c.Hkv, q.D, q.code, scale_of(a.v[8], q.D), out.data, lse,
                         ws.data, ws.bytes, run.stream),
          "moe_attn_decode_fp8");
    return owned.release();
  });
}

Spec weights_spec = {"attn_key_weights", 11};
PyObject* attn_key_weights(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(weights_spec, args, n, kw);
    const Query q = query(a.v[0]);
    const at::Tensor& kt = dense(a.v[1], "k_cache", q.type, {-1, -1, -1, q.D}, q.device);
    const int Hkv = whole(kt.size(1), "k_cache");
    const Ragged r = ragged(a.v[2], a.v[3], a.v[4], q.device);
    const float* lse = ptr<float>(dense(a.v[5], "lse", at::kFloat, {q.T, q.Hq}, q.device));
    const at::Tensor& wt = dense(a.v[6], "weights", at::kFloat, {r.seqs, Hkv, -1}, q.device);
    Run run(a.v[10], q.device);
    const Space ws = workspace(a.v[9], q.T, r.seqs, q.Hq, Hkv, q.D, run);
    check(lib.key_weights(&q.view, kt.data_ptr(), whole(kt.size(0), "k_cache"), whole(kt.size(2), "k_cache"), r.table,
                          r.pages, r.q_starts, r.lens, r.seqs, q.T, q.Hq, Hkv, q.D, q.code, truth(a.v[7]),
                          scale_of(a.v[8], q.D), lse, ptr<float>(wt), whole(wt.size(2), "weights"), ws.data, ws.bytes,
                          run.stream),
          "moe_attn_key_weights");
    Py_INCREF(a.v[6]);
    return a.v[6];
  });
}

// The caller's tensor, or a new one
Owned made(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, Run& run, void** data) {
  if (given(o)) {
    *data = dense(o, name, type, shape, run.device).data_ptr();
    Py_INCREF(o);
    return Owned{o};
  }
  const at::Tensor t = run.returned(run.make(shape, type));
  *data = t.data_ptr();
  return Owned{THPVariable_Wrap(t)};
}

Spec evict_spec = {"kv_evict", 14};
PyObject* kv_evict(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    const Args a = parse(evict_spec, args, n, kw);
    const at::Tensor& kt = as_tensor(a.v[0], "k_cache");
    const at::ScalarType type = kt.scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf) throw Refusal{"k_cache must be a bfloat16 or float16 torch.Tensor"};
    if (!kt.is_cuda()) throw Refusal{"k_cache must be a CUDA tensor"};
    const int device = c10::cuda::current_device();
    dense(a.v[0], "k_cache", type, {-1, -1, -1, -1}, device);
    const at::Tensor& vt = dense(a.v[1], "v_cache", type, kt.sizes(), device);
    const moe_kv_cache c{kt.data_ptr(), vt.data_ptr(), whole(kt.size(0), "k_cache"), whole(kt.size(2), "k_cache")};
    const int Hkv = whole(kt.size(1), "k_cache"), D = whole(kt.size(3), "k_cache");
    const at::Tensor& lens = dense(a.v[3], "kv_lens", at::kInt, {-1}, device);
    const int seqs = whole(lens.size(0), "kv_lens");
    const at::Tensor& table = dense(a.v[2], "page_table", at::kInt, {seqs, -1}, device);
    const at::Tensor& wt = dense(a.v[4], "weights", at::kFloat, {seqs, Hkv, -1}, device);
    const at::Tensor& to = dense(a.v[5], "out_table", at::kInt, {seqs, -1}, device);
    const int budget = (int)integer(a.v[6], 0, "budget"), first = (int)integer(a.v[7], 0, "keep_first"),
              last = (int)integer(a.v[8], 0, "keep_last");
    if (budget <= 0) throw Refusal{"budget must be positive"};
    Run run(a.v[13], device);
    void *new_lens, *new_weights, *kept;
    Owned o0 = made(a.v[9], "new_lens", at::kInt, {seqs}, run, &new_lens);
    Owned o1 = made(a.v[10], "new_weights", at::kFloat, {seqs, Hkv, budget}, run, &new_weights);
    Owned o2 = made(a.v[11], "kept", at::kInt, {seqs, Hkv, budget}, run, &kept);
    const Space ws = workspace(a.v[12], 0, seqs, Hkv, Hkv, D, run);
    check(lib.evict(&c, ptr<int32_t>(table), whole(table.size(1), "page_table"), ptr<int32_t>(lens), ptr<float>(wt),
                    whole(wt.size(2), "weights"), ptr<int32_t>(to), whole(to.size(1), "out_table"), budget, first, last,
                    seqs, Hkv, D, static_cast<int32_t*>(new_lens), static_cast<float*>(new_weights),
                    static_cast<int32_t*>(kept), ws.data, ws.bytes, run.stream),
          "moe_kv_evict");
    return PyTuple_Pack(3, o0.o, o1.o, o2.o);
  });
}

PyObject* bind(PyObject*, PyObject* args);

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS
PyMethodDef methods[] = {
    {"rope_append", FAST(rope_append), nullptr},
    {"attn_prefill", FAST(attn_prefill), nullptr},
    {"attn_prefill_paged", FAST(attn_prefill_paged), nullptr},
    {"attn_decode", FAST(attn_decode), nullptr},
    {"rope_append_fp8", FAST(rope_append_fp8), nullptr},
    {"attn_prefill_paged_fp8", FAST(attn_prefill_paged_fp8), nullptr},
    {"attn_decode_fp8", FAST(attn_decode_fp8), nullptr},
    {"attn_key_weights", FAST(attn_key_weights), nullptr},
    {"kv_evict", FAST(kv_evict), nullptr},
    {"bind", bind, METH_VARARGS, "Connect the functions to a loaded library and to their Python definitions."},
    {nullptr, nullptr, 0, nullptr}};

Spec* const specs[] = {&rope_spec,     &prefill_spec,   &paged_spec,      &decode_spec, &rope_fp8_spec,
                       &paged_fp8_spec, &decode_fp8_spec, &weights_spec, &evict_spec};
constexpr int kFunctions = sizeof(specs) / sizeof(specs[0]);
static_assert(sizeof(methods) / sizeof(methods[0]) == kFunctions + 2, "a method per function, bind and the end");

// bind(error type, addresses of the library's functions in the order of
// Library, then for each of the functions above (parameter names, defaults of
// the last of them, documentation))
PyObject* bind(PyObject*, PyObject* args) {
  if (PyTuple_GET_SIZE(args) != 1 + kAddresses + kFunctions) {
    PyErr_Format(PyExc_TypeError, "bind: %d arguments expected", 1 + kAddresses + kFunctions);
    return nullptr;
  }
  void* address[kAddresses];
  for (int i = 0; i < kAddresses; ++i) {
    address[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, 1 + i));
    if (PyErr_Occurred()) return nullptr;
  }
  for (int f = 0; f < kFunctions; ++f) {
    Spec& s = *specs[f];
    PyObject *names, *defaults;
    const char* doc;
    PyObject* given_spec = PyTuple_GET_ITEM(args, 1 + kAddresses + f);
    if (!PyTuple_Check(given_spec)) {
      PyErr_SetString(PyExc_TypeError, "bind: a tuple per function expected");
      return nullptr;
    }
    if (!PyArg_ParseTuple(given_spec, "O!O!s", &PyTuple_Type, &names, &PyTuple_Type, &defaults, &doc)) return nullptr;
    if (PyTuple_GET_SIZE(names) != s.total || PyTuple_GET_SIZE(defaults) > s.total) {
      PyErr_Format(PyExc_TypeError, "%s: %d parameters expected", s.function, s.total);
      return nullptr;
    }
    s.required = s.total - (int)PyTuple_GET_SIZE(defaults);
    for (int i = 0; i < s.total; ++i) {
      PyObject* name = PyTuple_GET_ITEM(names, i);
      if (!PyUnicode_Check(name)) {
        PyErr_SetString(PyExc_TypeError, "parameter names must be strings");
        return nullptr;
      }
      Py_INCREF(name);
      PyUnicode_InternInPlace(&name);
      Py_XSETREF(s.names[i], name);
      PyObject* value = i < s.required ? nullptr : PyTuple_GET_ITEM(defaults, i - s.required);
      Py_XINCREF(value);
      Py_XSETREF(s.defaults[i], value);
    }
    s.doc = doc;
    methods[f].ml_doc = s.doc.c_str();
  }
  PyObject* err = PyTuple_GET_ITEM(args, 0);
  Py_INCREF(err);
  Py_XSETREF(error_type, err);
  std::memcpy(&lib, address, sizeof(lib));
  Py_RETURN_NONE;
}

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding() { return PyModule_Create(&module); }
