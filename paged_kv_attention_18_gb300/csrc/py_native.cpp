// The Python side of the calls that a decode loop makes for every layer and token: argument
// checks and the C ABI call, compiled, so that a small call costs the host a few
// microseconds. (The same checks in Python over ctypes: 11 to 27 us a call, most of it
// attribute reads of a dozen tensors; here 3 to 6 us.) Only marshalling: every function
// checks that its tensors are CUDA tensors on the current device with the types, ranks and
// shapes the entry point of include/pagedserve.h expects, and passes their addresses on.
// Errors are raised as binding.PagedServeError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <stdexcept>
#include <string>

#include "pagedserve.h"

namespace {

PyObject* g_error = nullptr;  // binding.PagedServeError

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};  // a Python exception is set already

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

int to_int(int64_t x, const char* name) {
  if (x > INT_MAX || x < INT_MIN) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(x);
}

int arg_int(PyObject* o, const char* name) {
  int overflow = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (overflow) refuse(std::string(name) + " does not fit 32 bits");
  if (x == -1 && PyErr_Occurred()) throw PythonError();
  return to_int(x, name);
}

float arg_float(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError();
  return static_cast<float>(x);
}

bool arg_bool(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw PythonError();
  return x != 0;
}

const at::Tensor& arg_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return t;
}

// Tensors of one call, all on the device of the first, which is the current one.
struct Call {
  int dev = -1;

  const at::Tensor& first(PyObject* o, const char* name) {
    const at::Tensor& t = arg_tensor(o, name);
    dev = t.get_device();
    if (dev != c10::cuda::current_device())
      refuse(std::string(name) + " is on device " + std::to_string(dev) +
             ", not on the current CUDA device");
    return t;
  }

  const at::Tensor& any(PyObject* o, const char* name, at::ScalarType type, int64_t ndim) const {
    const at::Tensor& t = arg_tensor(o, name);
    if (t.get_device() != dev)
      refuse(std::string(name) + " is on device " + std::to_string(t.get_device()) +
             ", the other tensors on device " + std::to_string(dev));
    if (t.scalar_type() != type)
      refuse(std::string(name) + " has dtype " + at::toString(t.scalar_type()) + ", expected " +
             at::toString(type));
    if (t.dim() != ndim)
      refuse(std::string(name) + " must have " + std::to_string(ndim) + " dimensions, has " +
             std::to_string(t.dim()));
    return t;
  }

  // a contiguous tensor
  const at::Tensor& on(PyObject* o, const char* name, at::ScalarType type, int64_t ndim) const {
    const at::Tensor& t = any(o, name, type, ndim);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    return t;
  }

  // [T, heads, D] whose tokens are dense rows, at any distance from one another
  const at::Tensor& tokens(PyObject* o, const char* name, at::ScalarType type,
                           int64_t* stride) const {
    const at::Tensor& t = any(o, name, type, 3);
    const int64_t H = t.size(1), D = t.size(2);
    if ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D))
      refuse(std::string(name) + ": a token's heads must lie together");
    *stride = t.size(0) > 1 ? t.stride(0) : H * D;
    return t;
  }
};

int dtype16(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kHalf) return PS_F16;
  if (t.scalar_type() == at::kBFloat16) return PS_BF16;
  refuse(std::string(name) + " must be a float16 or bfloat16 tensor");
}

void* arg_stream(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
  PyObject* a = PyObject_GetAttrString(o, "cuda_stream");
  if (!a) throw PythonError();
  void* s = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  if (!s && PyErr_Occurred()) throw PythonError();
  return s;
}

void check(int rc, const char* what) {
  if (rc == PS_OK) return;
  std::string msg = std::string(what) + " failed: " + ps_status_string(rc);
  if (rc == PS_ERR_CUDA) msg += std::string(" [") + ps_last_error_message() + "]";
  refuse(msg + " (" + std::to_string(rc) + ")");
}

const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.const_data_ptr()); }

PyObject* give(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// New tensors on device `dev`, past the dispatcher (a selection of one prompt with its three
// results: 7.8 -> 6.9 us with a workspace given, 8.9 -> 7.8 without).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, int dev) {
  return at::Tensor(
      at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, dev), std::nullopt));
}

// q, k, v, positions, slots, k_pool, v_pool, inv_freq, interleaved, magnitude, q_out | None,
// stream | None; with several axes (kAxes) the frequencies' axes behind inv_freq
template <bool kAxes>
PyObject* rotary(PyObject* const* a) {
  constexpr int x = kAxes ? 1 : 0;
  Call c;
  const at::Tensor& q = c.first(a[0], "q");
  const int dt = dtype16(q, "q");
  const at::ScalarType st = q.scalar_type();
  int64_t qs, ks, vs, os;
  c.tokens(a[0], "q", st, &qs);
  const at::Tensor& k = c.tokens(a[1], "k", st, &ks);
  const at::Tensor& v = c.tokens(a[2], "v", st, &vs);
  PyObject* out_obj = a[10 + x] == Py_None ? a[0] : a[10 + x];
  const at::Tensor& out = c.tokens(out_obj, "q_out", st, &os);
  const at::Tensor& pos = c.on(a[3], "positions", at::kInt, 1 + x);
  const at::Tensor& slots = c.on(a[4], "slot_mapping", at::kInt, 1);
  const at::Tensor& kp = c.on(a[5], "k_pool", st, 4);
  const at::Tensor& vp = c.on(a[6], "v_pool", st, 4);
  const at::Tensor& freq = c.on(a[7], "inv_freq", at::kDouble, 1);
  const int64_t T = q.size(0), D = q.size(2);
  if (!k.sizes().equals(v.sizes()) || k.size(0) != T || k.size(2) != D ||
      !out.sizes().equals(q.sizes()) || !kp.sizes().equals(vp.sizes()) ||
      kp.size(1) != PS_BLOCK_SIZE || kp.size(2) != k.size(1) || kp.size(3) != D ||
      pos.size(x) != T || slots.size(0) != T)
    refuse(kAxes ? "rotary_axes_reshape_and_cache: inconsistent shapes"
                 : "rotary_reshape_and_cache: inconsistent shapes");
  const int32_t* axes = nullptr;
  int num_axes = 1;
  if constexpr (kAxes) {
    const at::Tensor& t = c.on(a[8], "axes", at::kInt, 1);
    if (t.size(0) != freq.size(0)) refuse("axes: one per frequency");
    axes = ints(t);
    num_axes = to_int(pos.size(0), "axes");
  }
  const bool inter = arg_bool(a[8 + x]);
  const float mag = arg_float(a[9 + x]);
  void* s = arg_stream(a[11 + x], c.dev);
  const int H_q = to_int(q.size(1), "H_q"), H_kv = to_int(k.size(1), "H_kv");
  const int n = to_int(T, "T"), nb = to_int(kp.size(0), "num_blocks");
  const int rot = to_int(2 * freq.size(0), "rotary_dim"), d = to_int(D, "D");
  const double* f = static_cast<const double*>(freq.const_data_ptr());
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  if constexpr (kAxes)
    rc = ps_rotary_axes_reshape_and_cache(
        q.const_data_ptr(), qs, k.const_data_ptr(), ks, v.const_data_ptr(), vs, ints(pos), axes,
        num_axes, ints(slots), kp.mutable_data_ptr(), vp.mutable_data_ptr(), f, rot,
        inter ? 1 : 0, mag, out.mutable_data_ptr(), os, n, H_q, H_kv, d, nb, dt, s);
  else
    rc = ps_rotary_reshape_and_cache(
        q.const_data_ptr(), qs, k.const_data_ptr(), ks, v.const_data_ptr(), vs, ints(pos),
        ints(slots), kp.mutable_data_ptr(), vp.mutable_data_ptr(), f, rot, inter ? 1 : 0, mag,
        out.mutable_data_ptr(), os, n, H_q, H_kv, d, nb, dt, s);
  Py_END_ALLOW_THREADS;
  check(rc, kAxes ? "ps_rotary_axes_reshape_and_cache" : "ps_rotary_reshape_and_cache");
  return give(out_obj);
}

// What the paged attentions' first arguments hold: q, k_pool, v_pool, block_tables, seq_lens,
// query_start_loc.
struct Paged {
  const at::Tensor &q, &kp, &vp, &bt, &sl, &qsl;
  at::ScalarType st;
  int dt, T, H_q, D, B, width, nb, H_kv;

  Paged(Call& c, PyObject* const* a, const char* what)
      : q(c.first(a[0], "q")),
        kp(c.on(a[1], "k_pool", q.scalar_type(), 4)),
        vp(c.on(a[2], "v_pool", q.scalar_type(), 4)),
        bt(c.on(a[3], "block_tables", at::kInt, 2)),
        sl(c.on(a[4], "seq_lens", at::kInt, 1)),
        qsl(c.on(a[5], "query_start_loc", at::kInt, 1)),
        st(q.scalar_type()) {
    dt = dtype16(q, "q");
    c.on(a[0], "q", st, 3);
    T = to_int(q.size(0), "T");
    H_q = to_int(q.size(1), "H_q");
    D = to_int(q.size(2), "D");
    B = to_int(bt.size(0), "B");
    width = to_int(bt.size(1), "max_blocks");
    if (sl.size(0) != B || qsl.size(0) != static_cast<int64_t>(B) + 1)
      refuse("block_tables / query_start_loc do not match seq_lens");
    if (kp.size(1) != PS_BLOCK_SIZE || kp.size(3) != D || !vp.sizes().equals(kp.sizes()))
      refuse(std::string(what) + ": inconsistent pool shape");
    nb = to_int(kp.size(0), "num_blocks");
    H_kv = to_int(kp.size(2), "H_kv");
  }

  at::Tensor out(const Call& c, PyObject* o) const {
    at::Tensor t = o == Py_None ? fresh(q.sizes(), st, c.dev) : c.on(o, "out", st, 3);
    if (!t.sizes().equals(q.sizes())) refuse("out must have q's shape");
    return t;
  }

  at::Tensor workspace(const Call& c, PyObject* o, PyObject* max_seq_len) const {
    if (o != Py_None) return c.on(o, "workspace", at::kByte, 1);
    const int64_t len = max_seq_len == Py_None ? static_cast<int64_t>(width) * PS_BLOCK_SIZE
                                               : arg_int(max_seq_len, "max_seq_len");
    const size_t n =
        ps_paged_attention_workspace_size(T, B, H_q, H_kv, D, to_int(len, "max_seq_len"));
    return fresh({static_cast<int64_t>(n > 256 ? n : 256)}, at::kByte, c.dev);
  }
};

// q, k_pool, v_pool, block_tables, seq_lens, query_start_loc, scale, softcap, slopes | None,
// window, prefix | None, starts | None, out | None, workspace | None, max_seq_len | None,
// stream | None
PyObject* attend(PyObject* const* a) {
  Call c;
  const Paged x(c, a, "masked_paged_attention");
  const float* slopes = nullptr;
  const int32_t *prefix = nullptr, *starts = nullptr;
  if (a[8] != Py_None) {
    const at::Tensor& t = c.on(a[8], "distance_slopes", at::kFloat, 1);
    if (t.size(0) != x.H_q) refuse("distance_slopes: one per query head");
    slopes = static_cast<const float*>(t.const_data_ptr());
  }
  if (a[10] != Py_None) {
    const at::Tensor& t = c.on(a[10], "prefix_lens", at::kInt, 1);
    if (t.size(0) != x.B) refuse("prefix_lens: one per sequence");
    prefix = ints(t);
  }
  if (a[11] != Py_None) {
    const at::Tensor& t = c.on(a[11], "key_starts", at::kInt, 1);
    if (t.size(0) != x.T) refuse("key_starts: one per packed token");
    starts = ints(t);
  }
  const float scale = arg_float(a[6]), cap = arg_float(a[7]);
  const int window = arg_int(a[9], "window");
  void* s = arg_stream(a[15], c.dev);
  const at::Tensor out = x.out(c, a[12]), ws = x.workspace(c, a[13], a[14]);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ps_paged_attention_masked(x.q.const_data_ptr(), x.kp.const_data_ptr(),
                                 x.vp.const_data_ptr(), ints(x.bt), x.width, ints(x.sl),
                                 ints(x.qsl), x.B, x.T, x.H_q, x.H_kv, x.D, x.nb, scale, cap,
                                 slopes, window, prefix, starts, out.mutable_data_ptr(),
                                 ws.mutable_data_ptr(), static_cast<size_t>(ws.numel()), x.dt, s);
  Py_END_ALLOW_THREADS;
  check(rc, "ps_paged_attention_masked");
  return a[12] == Py_None ? THPVariable_Wrap(out) : give(a[12]);
}

// q, k_pool, v_pool, block_tables, seq_lens, query_start_loc, scale, window, sinks, softcap,
// out | None, workspace | None, max_seq_len | None, stream | None
PyObject* stream_attend(PyObject* const* a) {
  Call c;
  const Paged x(c, a, "streaming_paged_attention");
  const float scale = arg_float(a[6]), cap = arg_float(a[9]);
  const int window = arg_int(a[7], "window"), sinks = arg_int(a[8], "sinks");
  void* s = arg_stream(a[13], c.dev);
  const at::Tensor out = x.out(c, a[10]), ws = x.workspace(c, a[11], a[12]);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ps_paged_attention_streaming(x.q.const_data_ptr(), x.kp.const_data_ptr(),
                                    x.vp.const_data_ptr(), ints(x.bt), x.width, ints(x.sl),
                                    ints(x.qsl), x.B, x.T, x.H_q, x.H_kv, x.D, x.nb, scale, cap,
                                    window, sinks, out.mutable_data_ptr(), ws.mutable_data_ptr(),
                                    static_cast<size_t>(ws.numel()), x.dt, s);
  Py_END_ALLOW_THREADS;
  check(rc, "ps_paged_attention_streaming");
  return a[10] == Py_None ? THPVariable_Wrap(out) : give(a[10]);
}

int logits_type(const at::Tensor& x) {
  switch (x.scalar_type()) {
    case at::kHalf: return PS_F16;
    case at::kBFloat16: return PS_BF16;
    case at::kFloat: return PS_F32;
    default: refuse("logits must be a float16, bfloat16 or float32 tensor");
  }
}

// logits, random_bits, temperature | None, top_k | None, top_p | None, min_p | None,
// tokens | None, logprobs | None (both or neither), stream | None
PyObject* sample(PyObject* const* a) {
  Call c;
  const at::Tensor& x = c.first(a[0], "logits");
  const int dt = logits_type(x);
  if (x.dim() != 2) refuse("logits must have 2 dimensions");
  const int64_t B = x.size(0), V = x.size(1), ld = B > 1 ? x.stride(0) : V;
  if (V > 1 && x.stride(1) != 1) refuse("logits: rows must be dense");
  auto row = [&](PyObject* o, const char* name, at::ScalarType type) -> const void* {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = c.on(o, name, type, 1);
    if (t.size(0) != B) refuse(std::string(name) + ": one per row");
    return t.const_data_ptr();
  };
  if (a[1] == Py_None) refuse("random_bits must be a CUDA tensor");
  const void* bits = row(a[1], "random_bits", at::kInt);
  const void* temp = row(a[2], "temperature", at::kFloat);
  const void* k = row(a[3], "top_k", at::kInt);
  const void* tp = row(a[4], "top_p", at::kFloat);
  const void* mp = row(a[5], "min_p", at::kFloat);
  void* s = arg_stream(a[8], c.dev);
  const int b = to_int(B, "B"), v = to_int(V, "V");
  const bool own = a[6] == Py_None;
  at::Tensor tok, lp;
  if (own) {
    tok = fresh({B}, at::kInt, c.dev);
    lp = fresh({B}, at::kFloat, c.dev);
  } else {
    tok = c.on(a[6], "tokens", at::kInt, 1);
    lp = c.on(a[7], "logprobs", at::kFloat, 1);
    if (tok.size(0) != B || lp.size(0) != B) refuse("sample: one result per row");
  }
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ps_sample(x.const_data_ptr(), ld, static_cast<const float*>(temp),
                 static_cast<const int32_t*>(k), static_cast<const float*>(tp),
                 static_cast<const float*>(mp), static_cast<const uint32_t*>(bits), b, v, dt,
                 static_cast<int32_t*>(tok.mutable_data_ptr()),
                 static_cast<float*>(lp.mutable_data_ptr()), s);
  Py_END_ALLOW_THREADS;
  check(rc, "ps_sample");
  if (!own) return PyTuple_Pack(2, a[6], a[7]);
  PyObject* res = PyTuple_New(2);
  if (!res) throw PythonError();
  PyTuple_SET_ITEM(res, 0, THPVariable_Wrap(tok));
  PyTuple_SET_ITEM(res, 1, THPVariable_Wrap(lp));
  return res;
}

// block_tables, seq_lens, new_lens, free_blocks, free_count, num_blocks, query_start_loc,
// slot_mapping, positions, window, sinks, out_seq_lens | None, out_free_count | None,
// held_pages | None, stream | None
PyObject* extend(PyObject* const* a) {
  Call c;
  const at::Tensor& bt = c.first(a[0], "block_tables");
  c.on(a[0], "block_tables", at::kInt, 2);
  const at::Tensor& sl = c.on(a[1], "seq_lens", at::kInt, 1);
  const at::Tensor& nl = c.on(a[2], "new_lens", at::kInt, 1);
  const at::Tensor& fb = c.on(a[3], "free_blocks", at::kInt, 1);
  const at::Tensor& fc = c.on(a[4], "free_count", at::kInt, 1);
  const int nb = arg_int(a[5], "num_blocks");
  const at::Tensor& qsl = c.on(a[6], "query_start_loc", at::kInt, 1);
  const at::Tensor& slots = c.on(a[7], "slot_mapping", at::kInt, 1);
  const at::Tensor& pos = c.on(a[8], "positions", at::kInt, 1);
  const int window = arg_int(a[9], "window"), sinks = arg_int(a[10], "sinks");
  const at::Tensor& ol = c.on(a[11] == Py_None ? a[1] : a[11], "out_seq_lens", at::kInt, 1);
  const at::Tensor& oc = c.on(a[12] == Py_None ? a[4] : a[12], "out_free_count", at::kInt, 1);
  const at::Tensor* held =
      a[13] == Py_None ? nullptr : &c.on(a[13], "held_pages", at::kInt, 1);
  const int64_t B = bt.size(0);
  if (held && held->size(0) != B) refuse("held_pages: one per sequence");
  if (sl.size(0) != B || nl.size(0) != B || ol.size(0) != B || qsl.size(0) != B + 1 ||
      pos.size(0) != slots.size(0) || fc.size(0) != 1 || oc.size(0) != 1)
    refuse("extend_sequences: inconsistent shapes");
  void* s = arg_stream(a[14], c.dev);
  const int b = to_int(B, "B"), w = to_int(bt.size(1), "max_blocks");
  const int T = to_int(slots.size(0), "T"), cap = to_int(fb.size(0), "free_capacity");
  auto out = [](const at::Tensor& t) { return static_cast<int32_t*>(t.mutable_data_ptr()); };
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  if (held)
    rc = ps_extend_held_sequences(out(bt), w, ints(sl), ints(nl), out(*held), out(fb), cap,
                                  ints(fc), b, T, nb, window, sinks, out(qsl), out(slots),
                                  out(pos), out(ol), out(oc), s);
  else
    rc = ps_extend_sequences(out(bt), w, ints(sl), ints(nl), out(fb), cap, ints(fc), b, T, nb,
                             window, sinks, out(qsl), out(slots), out(pos), out(ol), out(oc), s);
  Py_END_ALLOW_THREADS;
  check(rc, held ? "ps_extend_held_sequences" : "ps_extend_sequences");
  return give(Py_None);
}

// logits, scores, n_select, finished | None, pad_token, workspace | None, parents | None,
// tokens | None, best | None (all three or none), stream | None
PyObject* select(PyObject* const* a) {
  Call c;
  const at::Tensor& x = c.first(a[0], "logits");
  const int dt = logits_type(x);
  if (x.dim() != 3) refuse("logits must have 3 dimensions");
  const int64_t B = x.size(0), W = x.size(1), V = x.size(2);
  const int64_t ld = W > 1 ? x.stride(1) : B > 1 ? x.stride(0) : V;
  if ((V > 1 && x.stride(2) != 1) || (B > 1 && W > 1 && x.stride(0) != W * x.stride(1)))
    refuse("logits: rows must be dense and equally far apart");
  const at::Tensor& scores = c.on(a[1], "scores", at::kFloat, 2);
  const int n = arg_int(a[2], "n_select");
  if (n < 1 || n > 32) refuse("beam_select: n_select must be 1 to 32");
  const uint8_t* fin = nullptr;
  if (a[3] != Py_None) {
    const at::Tensor& t = arg_tensor(a[3], "finished");
    c.on(a[3], "finished", t.scalar_type() == at::kBool ? at::kBool : at::kByte, 2);
    if (t.size(0) != B || t.size(1) != W) refuse("beam_select: inconsistent shapes");
    fin = static_cast<const uint8_t*>(t.const_data_ptr());
  }
  if (scores.size(0) != B || scores.size(1) != W) refuse("beam_select: inconsistent shapes");
  const int pad = arg_int(a[4], "pad_token");
  void* s = arg_stream(a[9], c.dev);
  const int b = to_int(B, "B"), w = to_int(W, "W"), v = to_int(V, "V");
  at::Tensor ws;
  if (a[5] == Py_None) {
    const size_t need = ps_beam_select_workspace_size(b, w, v, n);
    ws = fresh({static_cast<int64_t>(need > 256 ? need : 256)}, at::kByte, c.dev);
  } else {
    ws = c.on(a[5], "workspace", at::kByte, 1);
  }
  const bool own = a[6] == Py_None;
  at::Tensor par, tok, best;
  if (own) {
    par = fresh({B, n}, at::kInt, c.dev);
    tok = fresh({B, n}, at::kInt, c.dev);
    best = fresh({B, n}, at::kFloat, c.dev);
  } else {
    par = c.on(a[6], "parents", at::kInt, 2);
    tok = c.on(a[7], "tokens", at::kInt, 2);
    best = c.on(a[8], "best", at::kFloat, 2);
  }
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ps_beam_select(x.const_data_ptr(), ld, static_cast<const float*>(scores.const_data_ptr()),
                      fin, pad, b, w, v, n, dt, static_cast<int32_t*>(par.mutable_data_ptr()),
                      static_cast<int32_t*>(tok.mutable_data_ptr()),
                      static_cast<float*>(best.mutable_data_ptr()), ws.mutable_data_ptr(),
                      static_cast<size_t>(ws.numel()), s);
  Py_END_ALLOW_THREADS;
  check(rc, "ps_beam_select");
  if (!own) return PyTuple_Pack(3, a[6], a[7], a[8]);
  PyObject* res = PyTuple_New(3);
  if (!res) throw PythonError();
  PyTuple_SET_ITEM(res, 0, THPVariable_Wrap(par));
  PyTuple_SET_ITEM(res, 1, THPVariable_Wrap(tok));
  PyTuple_SET_ITEM(res, 2, THPVariable_Wrap(best));
  return res;
}

// block_tables, seq_lens, parents, tail_blocks, k_pool, v_pool, out_block_tables,
// out_seq_lens, stream | None
PyObject* fork(PyObject* const* a) {
  Call c;
  const at::Tensor& kp = c.first(a[4], "k_pool");
  const int dt = dtype16(kp, "k_pool");
  const int64_t nd = kp.dim();
  if (nd != 4 && nd != 5) refuse("k_pool must have 4 or 5 dimensions");
  c.on(a[4], "k_pool", kp.scalar_type(), nd);
  const at::Tensor& vp = c.on(a[5], "v_pool", kp.scalar_type(), nd);
  const at::Tensor& bt = c.on(a[0], "block_tables", at::kInt, 2);
  const at::Tensor& sl = c.on(a[1], "seq_lens", at::kInt, 1);
  const at::Tensor& par = c.on(a[2], "parents", at::kInt, 2);
  const at::Tensor& tails = c.on(a[3], "tail_blocks", at::kInt, 2);
  const at::Tensor& obt = c.on(a[6], "out_block_tables", at::kInt, 2);
  const at::Tensor& ol = c.on(a[7], "out_seq_lens", at::kInt, 1);
  const int64_t groups = par.size(0), n_out = par.size(1), n = bt.size(0), width = bt.size(1);
  if (!vp.sizes().equals(kp.sizes()) || kp.size(-3) != PS_BLOCK_SIZE || sl.size(0) != n ||
      !tails.sizes().equals(par.sizes()) || obt.size(0) != groups * n_out ||
      obt.size(1) != width || ol.size(0) != groups * n_out || (groups > 0 && n % groups != 0))
    refuse("fork_sequences: inconsistent shapes");
  if (groups == 0) return give(Py_None);
  void* s = arg_stream(a[8], c.dev);
  const int w = to_int(width, "max_blocks"), g = to_int(groups, "groups");
  const int n_in = to_int(n / groups, "n_in"), no = to_int(n_out, "n_out");
  const int layers = nd == 5 ? to_int(kp.size(0), "layers") : 1;
  const int nb = to_int(kp.size(-4), "num_blocks"), H = to_int(kp.size(-2), "H_kv");
  const int D = to_int(kp.size(-1), "D");
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ps_fork_sequences(ints(bt), w, ints(sl), ints(par), ints(tails), g, n_in, no,
                         kp.mutable_data_ptr(), vp.mutable_data_ptr(), layers, nb, H, D, dt,
                         static_cast<int32_t*>(obt.mutable_data_ptr()),
                         static_cast<int32_t*>(ol.mutable_data_ptr()), s);
  Py_END_ALLOW_THREADS;
  check(rc, "ps_fork_sequences");
  return give(Py_None);
}

// Calls f with exactly kArgs arguments; no C++ exception leaves.
template <PyObject* (*f)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return f(args);
  } catch (const PythonError&) {
  } catch (const Refused& e) {
    PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, kArgs>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<rotary<false>, 12>("rotary"),
                           method<rotary<true>, 13>("rotary_axes"),
                           method<stream_attend, 14>("stream_attend"),
                           method<sample, 9>("sample"),
                           method<extend, 15>("extend"),
                           method<attend, 16>("attend"),
                           method<select, 10>("select"),
                           method<fork, 9>("fork"),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
