// Python wrappers of the decode-step entry points (include/gbfuse_decode.h).
//
// A decode-step call runs for a few microseconds, about what ctypes and a dozen
// Python-level operand checks take, so these wrappers are compiled: the same
// checks as the package's other wrappers (every operand a dense torch tensor of
// the element type and extent the call reads or writes, on the current CUDA
// device), then the C call on the current torch stream.  Nothing is computed or
// kept here.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>

#include "gbfuse_decode.h"

namespace {

PyObject* g_error = nullptr;       // GbfError

// Thrown once a Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw Raised();
}

// ------------------------------------------------------------- call arguments

template <int N>
struct Args {
  PyObject* at[N];

  // Positional arguments, then those by name; the first `required` must be there.
  Args(const char* fn, const char* const (&names)[N], int required, PyObject* const* args, Py_ssize_t nargs,
       PyObject* kwnames) {
    if (nargs > N) raise(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", fn, N, nargs);
    for (int i = 0; i < N; ++i) at[i] = i < nargs ? args[i] : nullptr;
    const Py_ssize_t named = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
    for (Py_ssize_t j = 0; j < named; ++j) {
      PyObject* key = PyTuple_GET_ITEM(kwnames, j);
      int i = 0;
      while (i < N && PyUnicode_CompareWithASCIIString(key, names[i]) != 0) ++i;
      if (i == N) raise(PyExc_TypeError, "%s() got an unexpected keyword argument '%U'", fn, key);
      if (at[i]) raise(PyExc_TypeError, "%s() got multiple values for argument '%s'", fn, names[i]);
      at[i] = args[nargs + j];
    }
    for (int i = 0; i < N; ++i)
      if (!at[i]) {
        if (i < required) raise(PyExc_TypeError, "%s() missing required argument '%s'", fn, names[i]);
        at[i] = Py_None;
      }
  }
};

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    raise(PyExc_TypeError, "%s: expected an int that fits 64 bits, got %R", name, o);
  }
  return v;
}

int narrow(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v != static_cast<int>(v)) raise(PyExc_ValueError, "%s: %lld does not fit 32 bits", name, static_cast<long long>(v));
  return static_cast<int>(v);
}

double real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    raise(PyExc_TypeError, "%s: expected a number, got %R", name, o);
  }
  return v;
}

// ------------------------------------------------------------------- operands

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a torch.Tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// The current CUDA device, or -1 when the call's first operand is on none: the
// other operands' extents are checked all the same, and the call ends in stream().
int device_of(const at::Tensor& first) { return first.is_cuda() ? c10::cuda::current_device() : -1; }

void check_type(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s: expected torch.%s, got torch.%s", name,
          type == at::kInt ? "int32" : type == at::kFloat ? "float32" : type == at::kByte ? "uint8" : "bfloat16",
          c10::toString(t.scalar_type()));
}

void check_device(const at::Tensor& t, const char* name, int device) {
  if (device < 0 || t.get_device() == device) return;
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s: must be on a CUDA device", name);
  raise(PyExc_ValueError, "%s: is on cuda:%d, the current device is cuda:%d", name, static_cast<int>(t.get_device()), device);
}

// Data pointer of a dense operand of n elements; None is an absent optional one.
void* operand(PyObject* o, int64_t n, at::ScalarType type, const char* name, int device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.numel() != n)
    raise(PyExc_ValueError, "%s: holds %lld elements, the call needs %lld", name, static_cast<long long>(t.numel()),
          static_cast<long long>(n));
  check_type(t, type, name);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: must be contiguous", name);
  check_device(t, name, device);
  return t.data_ptr();
}

// A [batch, width] operand whose rows may be apart (a column range of a wider one).
struct Rows {
  void* at;
  int64_t batch, width, apart;
};
Rows rows(const at::Tensor& t, int64_t batch, at::ScalarType type, const char* name, int device) {
  if (t.dim() != 2 || (batch >= 0 && t.size(0) != batch))
    raise(PyExc_ValueError, "%s: expected [batch, n] with one row per request", name);
  Rows r{nullptr, t.size(0), t.size(1), t.stride(0)};
  if (r.width > 1 && t.stride(1) != 1) raise(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
  if (r.batch <= 1) r.apart = r.width;
  else if (r.apart < r.width) raise(PyExc_ValueError, "%s: rows may not overlap", name);
  check_type(t, type, name);
  check_device(t, name, device);
  r.at = t.data_ptr();
  return r;
}

// cudaStream_t of `o`, by default of the current torch stream; the last check.
void* stream(PyObject* o, int device) {
  if (device < 0) raise(PyExc_ValueError, "the operands must be on a CUDA device");
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (!raw) throw Raised();
  void* s = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  if (!s && PyErr_Occurred()) throw Raised();
  return s;
}

PyObject* finish(int status) {
  if (status == GBF_OK) return PyLong_FromLong(0);
  PyObject* e = PyObject_CallFunction(g_error, "is", status, gbf_last_error());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

template <typename Call>
PyObject* guarded(Call call) {
  try {
    return finish(call());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// -------------------------------------------------------------------- the calls

PyObject* paged_slots(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&] {
    static const char* const names[12] = {"ctx_lens", "new_lens", "block_table", "free_ring", "ring", "block_size",
                                          "seq_lens", "ring_out", "slots", "pos", "start", "stream"};
    const Args<12> v("paged_slots", names, 10, args, nargs, kwnames);
    const at::Tensor& ctx = tensor(v.at[0], names[0]);
    const int d = device_of(ctx);
    const int64_t batch = ctx.numel(), blocks = tensor(v.at[3], names[3]).numel(), tokens = tensor(v.at[8], names[8]).numel();
    auto i32 = [&](int i, int64_t n) { return static_cast<int32_t*>(operand(v.at[i], n, at::kInt, names[i], d)); };
    const int32_t *c = i32(0, batch), *n = i32(1, batch), *ring = i32(4, 2);
    const Rows table = rows(tensor(v.at[2], names[2]), batch, at::kInt, names[2], d);
    int32_t *free_ring = i32(3, blocks), *seq = i32(6, batch), *ring_out = i32(7, 2), *slots = i32(8, tokens),
            *pos = i32(9, tokens), *start = i32(10, batch + 1);
    const int block = narrow(v.at[5], names[5]);
    void* s = stream(v.at[11], d);
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = gbfd_paged_slots(c, n, batch, static_cast<int32_t*>(table.at), table.apart, table.width, block, free_ring,
                              ring, blocks, seq, ring_out, slots, pos, tokens, start, s);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

PyObject* paged_attention(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&] {
    static const char* const names[13] = {"q", "k_cache", "v_cache", "block_table", "seq_lens", "block_size", "out",
                                          "workspace", "scale", "window", "lse", "out_scale", "stream"};
    const Args<13> v("paged_attention", names, 8, args, nargs, kwnames);
    const at::Tensor &q = tensor(v.at[0], names[0]), &k = tensor(v.at[1], names[1]);
    const int d = device_of(q);
    if (q.dim() != 3) raise(PyExc_ValueError, "q: expected [batch, n_q_heads, head_dim]");
    if (k.dim() != 3 || k.size(2) != q.size(2))
      raise(PyExc_ValueError, "k_cache: expected [cache_rows, n_kv_heads, %lld]", static_cast<long long>(q.size(2)));
    const int64_t batch = q.size(0), hq = q.size(1), dim = q.size(2), cache_rows = k.size(0), hkv = k.size(1);
    if (hq > 0x7fffffff || hkv > 0x7fffffff || dim > 0x7fffffff) raise(PyExc_ValueError, "q: a dimension does not fit 32 bits");
    const bool codes = v.at[11] != Py_None;
    const double out_scale = codes ? real(v.at[11], names[11]) : 0.0;
    // in float32, as the call reads it: there 0 means bf16 output, twice the bytes of the codes
    if (codes && !(static_cast<float>(out_scale) > 0.0f)) raise(PyExc_ValueError, "out_scale: must be > 0, got %R", v.at[11]);
    const double scale = v.at[8] != Py_None ? real(v.at[8], names[8]) : 1.0 / std::sqrt(static_cast<double>(dim));
    const int64_t window = v.at[9] != Py_None ? integer(v.at[9], names[9]) : 0;
    const void *qp = operand(v.at[0], q.numel(), at::kBFloat16, names[0], d),
               *kp = operand(v.at[1], k.numel(), at::kBFloat16, names[1], d),
               *vp = operand(v.at[2], k.numel(), at::kBFloat16, names[2], d);
    const Rows table = rows(tensor(v.at[3], names[3]), batch, at::kInt, names[3], d);
    const void* lens = operand(v.at[4], batch, at::kInt, names[4], d);
    void* out = operand(v.at[6], q.numel(), codes ? at::kByte : at::kBFloat16, names[6], d);
    void* lse = operand(v.at[10], batch * hq, at::kFloat, names[10], d);
    const at::Tensor& w = tensor(v.at[7], names[7]);
    void* ws = operand(v.at[7], w.numel(), w.scalar_type(), names[7], d);
    const int64_t room = w.numel() * static_cast<int64_t>(w.element_size());
    const int block = narrow(v.at[5], names[5]);
    void* s = stream(v.at[12], d);
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = gbfd_paged_attention(qp, kp, vp, cache_rows, static_cast<const int32_t*>(table.at), table.apart, table.width,
                                  block, static_cast<const int32_t*>(lens), batch, static_cast<int>(hq),
                                  static_cast<int>(hkv), static_cast<int>(dim), static_cast<float>(scale), window, out,
                                  static_cast<float>(out_scale), static_cast<float*>(lse), ws, room, s);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

PyObject* sample_tokens(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  return guarded([&] {
    static const char* const names[9] = {"logits", "uniform", "tokens", "temperature", "top_k",
                                         "top_p", "min_p", "logprob", "stream"};
    const Args<9> v("sample_tokens", names, 3, args, nargs, kwnames);
    const at::Tensor& logits = tensor(v.at[0], names[0]);
    const int d = device_of(logits);
    const at::ScalarType kind = logits.scalar_type();
    if (kind != at::kBFloat16 && kind != at::kFloat)
      raise(PyExc_TypeError, "logits: expected torch.bfloat16 or torch.float32, got torch.%s", c10::toString(kind));
    const Rows l = rows(logits, -1, kind, names[0], d);
    auto f32 = [&](int i) { return static_cast<float*>(operand(v.at[i], l.batch, at::kFloat, names[i], d)); };
    auto i32 = [&](int i) { return static_cast<int32_t*>(operand(v.at[i], l.batch, at::kInt, names[i], d)); };
    const float *u = f32(1), *t = f32(3), *p = f32(5), *mp = f32(6);
    const int32_t* k = i32(4);
    int32_t* tokens = i32(2);
    float* logprob = f32(7);
    void* s = stream(v.at[8], d);
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = gbfd_sample_tokens(l.at, kind == at::kFloat ? 1 : 0, l.batch, l.width, l.apart, u, t, k, p, mp, tokens,
                                logprob, s);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

// The exception class that a status other than GBF_OK raises: (status, message).
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

#define GBF_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS

PyMethodDef methods[] = {
    {"paged_slots", GBF_FAST(paged_slots),
     "paged_slots(ctx_lens, new_lens, block_table, free_ring, ring, block_size, seq_lens, ring_out, slots, pos, "
     "start=None, stream=None)\n--\n\n"
     "gbfd_paged_slots: block tables, slot maps and positions of one step from the\n"
     "requests' lengths.  ctx_lens, new_lens, seq_lens [batch]; block_table [batch,\n"
     "max_blocks] (rows may be apart); free_ring [num_blocks]; ring, ring_out [2];\n"
     "slots, pos [tokens]; start [batch + 1] or None; all int32."},
    {"paged_attention", GBF_FAST(paged_attention),
     "paged_attention(q, k_cache, v_cache, block_table, seq_lens, block_size, out, workspace, scale=None, window=0, "
     "lse=None, out_scale=None, stream=None)\n--\n\n"
     "gbfd_paged_attention: out[b] = attention of q[b] over the seq_lens[b] cached\n"
     "positions of request b.  q [batch, n_q_heads, head_dim]; k_cache, v_cache\n"
     "[cache_rows, n_kv_heads, head_dim]; block_table [batch, max_blocks] (rows may be\n"
     "apart); out as q in bf16, or uint8 E4M3 codes with out_scale; lse float32 [batch,\n"
     "n_q_heads] or None; workspace: any dense tensor of at least\n"
     "paged_attention_workspace() bytes; scale defaults to head_dim ** -0.5."},
    {"sample_tokens", GBF_FAST(sample_tokens),
     "sample_tokens(logits, uniform, tokens, temperature=None, top_k=None, top_p=None, min_p=None, logprob=None, "
     "stream=None)\n--\n\n"
     "gbfd_sample_tokens: tokens[b] drawn from logits[b] (bf16 or float32 [batch,\n"
     "vocab], rows may be apart) with the given uniform[b] and, where the tensors are\n"
     "given, temperature, top_k (int32), top_p and min_p of each row."},
    {"set_error", set_error, METH_O, "set_error(type): the exception class of a failed call"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "decode_binding", "Decode-step entry points of libgbfuse.so.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_decode_binding() {
  PyObject* m = PyModule_Create(&module);
  // torch's C++ interfaces change from version to version: the package looks at this before it uses anything here
  if (m && PyModule_AddStringConstant(m, "built_for_torch", GBF_BUILT_FOR_TORCH) != 0) Py_CLEAR(m);
  return m;
}
