// Python binding of the block-sparse and scored steps' calls for torch tensors.
//
// Argument marshalling only, as in ops.py, but compiled: these calls take 3
// to 15 us on the device for a decode batch, and checking a dozen tensors
// and handing their addresses over by ctypes took 6 to 11 us of host time a
// call.  Each function checks the sizes that the C ABI cannot see through
// its pointers (ValueError), makes the tensors' device current, takes that
// device's current stream unless one is given, and returns the C entry's
// status.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "pa.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

std::string text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

bool is(at::IntArrayRef s, std::initializer_list<int64_t> want) {
  return s.equals(at::IntArrayRef(want));
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

int32_t to_int32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " does not fit 32 bits");
  return (int32_t)v;
}

int32_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be an integer");
  }
  return to_int32(v, name);
}

int32_t flag(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be true or false");
  }
  return v;
}

// A device, and the tensors that have to be on it.
class OnDevice {
 public:
  explicit OnDevice(const at::Tensor& first, const char* name) {
    if (!first.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
    device_ = first.device().index();
  }
  void check(const at::Tensor& t, const char* name, at::ScalarType type) const {
    if (!t.is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor");
    if (t.device().index() != device_)
      throw Refused(std::string(name) + " is on " + t.device().str() + ", other tensors are on cuda:" +
                    std::to_string(device_));
    if (t.scalar_type() != type)
      throw Refused(std::string(name) + " must have dtype " + c10::toString(type) + ", got " +
                    c10::toString(t.scalar_type()));
  }
  // What a call reads.
  template <typename T = void>
  const T* in(const at::Tensor& t, const char* name, at::ScalarType type) const {
    whole(t, name, type);
    return static_cast<const T*>(t.const_data_ptr());
  }
  template <typename T = void>
  const T* optional(PyObject* o, const char* name, at::ScalarType type) const {
    return o == Py_None ? nullptr : in<T>(tensor(o, name), name, type);
  }
  // What a call writes: a lazy clone gets memory of its own here, so these
  // are taken before the addresses of inputs, which may be views of them.
  template <typename T = void>
  T* out(const at::Tensor& t, const char* name, at::ScalarType type) const {
    whole(t, name, type);
    return static_cast<T*>(t.mutable_data_ptr());
  }
  // Rows [heads, d] of a [tokens, heads, d] tensor whose tokens may lie apart.
  const void* rows(const at::Tensor& t, const char* name, int64_t* stride) const {
    check(t, name, at::kBFloat16);
    const auto s = t.sizes(), st = t.strides();
    if ((st[2] != 1 && s[2] > 1) || (st[1] != s[2] && s[1] > 1))
      throw Refused(std::string(name) + ": a token's heads and channels must be contiguous");
    *stride = s[0] > 1 ? st[0] : s[1] * s[2];
    return t.const_data_ptr();
  }
  // Runs call(stream) with the device current.
  template <typename F>
  PyObject* run(PyObject* stream, F&& call) const {
    pa_stream_t raw;
    if (stream == Py_None) {
      raw = reinterpret_cast<pa_stream_t>(c10::cuda::getCurrentCUDAStream(device_).stream());
    } else {
      PyObject* handle = PyLong_Check(stream) ? Py_NewRef(stream)
                                              : PyObject_GetAttrString(stream, "cuda_stream");
      raw = handle ? static_cast<pa_stream_t>(PyLong_AsVoidPtr(handle)) : nullptr;
      Py_XDECREF(handle);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused("stream must be a CUDA stream or its handle");
      }
    }
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != device_) guard.set_index(device_);
    pa_status status;
    Py_BEGIN_ALLOW_THREADS;  // a C call: nothing throws in here
    status = call(raw);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
  }

 private:
  void whole(const at::Tensor& t, const char* name, at::ScalarType type) const {
    check(t, name, type);
    if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
  }
  c10::DeviceIndex device_;
};

// Descriptor of a [num_blocks, block_size, num_kv_heads, head_dim] cache.
pa_cache_desc describe(const at::Tensor& cache) {
  const auto s = cache.sizes();
  if (s.size() != 4)
    throw Refused("cache must be [num_blocks, block_size, num_kv_heads, head_dim]");
  pa_cache_desc d;
  if (cache.scalar_type() == at::kBFloat16)
    d.dtype = PA_KV_BF16;
  else if (cache.scalar_type() == at::kFloat8_e4m3fn || cache.scalar_type() == at::kByte)
    d.dtype = PA_KV_FP8_E4M3;
  else
    throw Refused(std::string("cache dtype must be bfloat16 or float8_e4m3fn/uint8, got ") +
                  c10::toString(cache.scalar_type()));
  d.num_blocks = to_int32(s[0], "num_blocks");
  d.block_size = to_int32(s[1], "block_size");
  d.num_kv_heads = to_int32(s[2], "num_kv_heads");
  d.head_dim = to_int32(s[3], "head_dim");
  return d;
}

pa_cache_desc describe(const at::Tensor& k, const at::Tensor& v, PyObject* ks, PyObject* vs) {
  if (!k.sizes().equals(v.sizes()) || k.scalar_type() != v.scalar_type())
    throw Refused("k_cache and v_cache must have the same shape and dtype");
  const pa_cache_desc d = describe(k);
  if (d.dtype == PA_KV_BF16 && (ks != Py_None || vs != Py_None))
    throw Refused("k_scale/v_scale are only for fp8 caches");
  if (d.dtype != PA_KV_BF16 && (ks == Py_None || vs == Py_None))
    throw Refused("fp8 caches need k_scale and v_scale (device float32 scalars)");
  return d;
}

// The same of a cache that may hold 8-bit rows; their units.
pa_cache_desc describe_any(const at::Tensor& k, const at::Tensor& v, PyObject* ks, PyObject* vs) {
  if (k.scalar_type() != at::kChar) {
    const pa_cache_desc d = describe(k, v, ks, vs);
    for (PyObject* s : {ks, vs})
      if (s != Py_None && tensor(s, "k_scale and v_scale").numel() != 1)
        throw Refused("k_scale and v_scale of an fp8 cache must have one element");
    return d;
  }
  const auto s = k.sizes();
  if (s.size() != 4)
    throw Refused("cache must be [num_blocks, block_size, num_kv_heads, head_dim]");
  if (!v.sizes().equals(s) || v.scalar_type() != at::kChar)
    throw Refused("k_cache and v_cache must have the same shape and dtype");
  for (PyObject* u : {ks, vs}) {
    if (u == Py_None) throw Refused("int8 caches need k_scale and v_scale (their units)");
    const auto got = tensor(u, "k_scale and v_scale").sizes();
    if (!got.equals(s.slice(0, 3)))
      throw Refused("k_scale and v_scale of an int8 cache must be " + text(s.slice(0, 3)) +
                    ", got " + text(got));
  }
  return {to_int32(s[0], "num_blocks"), to_int32(s[1], "block_size"),
          to_int32(s[2], "num_kv_heads"), to_int32(s[3], "head_dim"), PA_KV_INT8};
}

float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be a number");
  }
  return (float)v;
}

void check_ranges(const pa_cache_desc& d, const at::Tensor& codes, const at::Tensor& scales) {
  const int64_t want[] = {d.num_blocks, d.num_kv_heads, 2, d.head_dim};
  if (!codes.sizes().equals(want))
    throw Refused("codes must be [num_blocks, num_kv_heads, 2, head_dim] = " + text(want) +
                  ", got " + text(codes.sizes()));
  if (!scales.sizes().equals(at::IntArrayRef(want, 2)))
    throw Refused("scales must be [num_blocks, num_kv_heads] = " + text({want, 2}) + ", got " +
                  text(scales.sizes()));
}

// Sizes shared by the calls over query rows.
struct Rows {
  int32_t rows, heads, seqs, max_blocks, top;
};
Rows check_rows(const at::Tensor& q, const at::Tensor& tables, const at::Tensor& lens,
                PyObject* row_seqs, const at::Tensor& selected, const pa_cache_desc& d) {
  const auto qs = q.sizes(), ts = tables.sizes(), ss = selected.sizes();
  if (qs.size() != 3) throw Refused("q must be [num_rows, num_heads, head_dim]");
  const std::string n = std::to_string(qs[0]);
  if (ts.size() != 2 || (row_seqs == Py_None && ts[0] != qs[0]))
    throw Refused("block_tables must be [" + (row_seqs == Py_None ? n : std::string("num_seqs")) +
                  ", max_blocks_per_seq], got " + text(ts));
  if (lens.numel() != qs[0])
    throw Refused("context_lens needs " + n + " entries, got " + std::to_string(lens.numel()));
  if (row_seqs != Py_None) {
    const int64_t m = tensor(row_seqs, "row_seqs").numel();
    if (m != qs[0]) throw Refused("row_seqs needs " + n + " entries, got " + std::to_string(m));
  }
  if (ss.size() != 3 || ss[0] != qs[0] || ss[1] != d.num_kv_heads)
    throw Refused("selected must be [" + n + ", " + std::to_string(d.num_kv_heads) +
                  ", top], got " + text(ss));
  if (qs[2] != d.head_dim)
    throw Refused("q's head_dim " + std::to_string(qs[2]) + " differs from the cache's " +
                  std::to_string(d.head_dim));
  return {to_int32(qs[0], "num_rows"), to_int32(qs[1], "num_heads"), to_int32(ts[0], "num_seqs"),
          to_int32(ts[1], "max_blocks_per_seq"), to_int32(ss[2], "top")};
}

// Every entry: the expected number of positional arguments, and C++
// exceptions turned into Python's.
template <Py_ssize_t N, typename F>
PyObject* entry(const char* name, Py_ssize_t nargs, F&& body) {
  if (nargs != N)
    return PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, N, nargs);
  try {
    return body();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The position axes and their sections.
pa_rope_desc rope_of(at::IntArrayRef ps, at::IntArrayRef ts, PyObject* sections, PyObject* in_turn,
                     PyObject* adjacent) {
  pa_rope_desc rope = {};
  rope.max_position = to_int32(ts[0], "max_position");
  rope.rot_dim = to_int32(ts[1], "rot_dim");
  const int64_t axes = ps.size() == 1 ? 1 : ps[0];
  if (axes > 4) throw Refused("at most 4 position axes");
  rope.num_axes = (int32_t)axes;
  if (sections == Py_None && axes == 1) {
    rope.sections[0] = rope.rot_dim / 2;
  } else {
    PyObject* list = sections == Py_None ? nullptr : PySequence_Fast(sections, "sections");
    PyErr_Clear();
    const bool ok = list && PySequence_Fast_GET_SIZE(list) == axes;
    try {
      for (int64_t i = 0; ok && i < axes; ++i)
        rope.sections[i] = integer(PySequence_Fast_GET_ITEM(list, i), "sections");
    } catch (...) {
      Py_DECREF(list);
      throw;
    }
    Py_XDECREF(list);
    if (!ok)
      throw Refused("sections must have one entry for each of the " + std::to_string(axes) +
                    " position axes");
  }
  rope.sections_in_turn = flag(in_turn, "sections_in_turn");
  rope.adjacent_pairs = flag(adjacent, "adjacent_pairs");
  return rope;
}

// Sizes shared by the rotating writes: one row per slot; positions and table
// (where there are any).  Returns the number of tokens.
int64_t check_write(const at::Tensor& q_out, const at::Tensor& query, const at::Tensor& key,
                    const at::Tensor& value, const at::Tensor& slots, const at::Tensor* pos,
                    const at::Tensor* table, const pa_cache_desc& d) {
  const int64_t n = slots.numel();
  if (!is(key.sizes(), {n, d.num_kv_heads, d.head_dim}) || !value.sizes().equals(key.sizes())) {
    const int64_t want[] = {n, d.num_kv_heads, d.head_dim};
    throw Refused("key and value must be " + text(want) + " (one row per slot), got " +
                  text(key.sizes()) + " and " + text(value.sizes()));
  }
  const auto qs = query.sizes();
  if (qs.size() != 3 || qs[0] != n || qs[2] != d.head_dim || !q_out.sizes().equals(qs))
    throw Refused("query and q_out must be [" + std::to_string(n) + ", num_heads, " +
                  std::to_string(d.head_dim) + "], got " + text(qs) + " and " +
                  text(q_out.sizes()));
  if (!pos) return n;
  const auto ps = pos->sizes();
  if ((ps.size() != 1 && ps.size() != 2) || ps.back() != n)
    throw Refused("positions must be [" + std::to_string(n) + "] or [axes, " + std::to_string(n) +
                  "], got " + text(ps));
  if (table->sizes().size() != 2) throw Refused("cos_sin must be [max_position, rot_dim]");
  return n;
}

// q_out, query, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin,
// k_scale, v_scale, sections, sections_in_turn, adjacent_pairs, stream
PyObject* rope_and_cache(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return entry<15>("rope_and_cache", nargs, [&] {
    const at::Tensor &q_out = tensor(a[0], "q_out"), &query = tensor(a[1], "query"),
                     &key = tensor(a[2], "key"), &value = tensor(a[3], "value"),
                     &kc = tensor(a[4], "k_cache"), &vc = tensor(a[5], "v_cache"),
                     &slots = tensor(a[6], "slot_mapping"), &pos = tensor(a[7], "positions"),
                     &table = tensor(a[8], "cos_sin");
    const pa_cache_desc d = describe(kc, vc, a[9], a[10]);
    const int64_t n = check_write(q_out, query, key, value, slots, &pos, &table, d);
    const pa_rope_desc rope = rope_of(pos.sizes(), table.sizes(), a[11], a[12], a[13]);
    const OnDevice on(kc, "k_cache");
    void* o = on.out(q_out, "q_out", at::kBFloat16);
    void *kp = on.out(kc, "k_cache", kc.scalar_type()), *vp = on.out(vc, "v_cache", kc.scalar_type());
    int64_t q_stride, k_stride, v_stride;
    const void *q = on.rows(query, "query", &q_stride), *k = on.rows(key, "key", &k_stride),
               *v = on.rows(value, "value", &v_stride);
    const auto* sp = on.in<int32_t>(slots, "slot_mapping", at::kInt);
    const auto* pp = on.in<int32_t>(pos, "positions", at::kInt);
    const auto* cs = on.in<float>(table, "cos_sin", at::kFloat);
    const auto* ks = on.optional<float>(a[9], "k_scale", at::kFloat);
    const auto* vs = on.optional<float>(a[10], "v_scale", at::kFloat);
    const int32_t heads = to_int32(query.sizes()[1], "num_heads"), tokens = to_int32(n, "num_tokens");
    return on.run(a[14], [&](pa_stream_t stream) {
      return pa_rope_and_cache(o, q, q_stride, heads, k, k_stride, v, v_stride, kp, vp, d, sp, pp,
                               cs, rope, tokens, ks, vs, stream);
    });
  });
}

// k_cache, slot_mapping, codes, scales, stream
PyObject* summarize_blocks(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return entry<5>("summarize_blocks", nargs, [&] {
    const at::Tensor &kc = tensor(a[0], "k_cache"), &slots = tensor(a[1], "slot_mapping"),
                     &codes = tensor(a[2], "codes"), &scales = tensor(a[3], "scales");
    const pa_cache_desc d = describe(kc);
    check_ranges(d, codes, scales);
    const OnDevice on(kc, "k_cache");
    auto* cp = on.out<int8_t>(codes, "codes", at::kChar);
    auto* up = on.out<float>(scales, "scales", at::kFloat);
    const void* kp = on.in(kc, "k_cache", kc.scalar_type());
    const auto* sp = on.in<int32_t>(slots, "slot_mapping", at::kInt);
    const int32_t tokens = to_int32(slots.numel(), "num_tokens");
    return on.run(a[4], [&](pa_stream_t stream) {
      return pa_summarize_blocks(kp, d, sp, tokens, cp, up, stream);
    });
  });
}

// selected, q, codes, scales, block_tables, context_lens, block_size, sink,
// recent, row_seqs, stream
PyObject* select_blocks(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return entry<11>("select_blocks", nargs, [&] {
    const at::Tensor &selected = tensor(a[0], "selected"), &q = tensor(a[1], "q"),
                     &codes = tensor(a[2], "codes"), &scales = tensor(a[3], "scales"),
                     &tables = tensor(a[4], "block_tables"), &lens = tensor(a[5], "context_lens");
    const auto cs = codes.sizes();
    if (cs.size() != 4 || cs[2] != 2)
      throw Refused("codes must be [num_blocks, num_kv_heads, 2, head_dim]");
    const pa_cache_desc d = {to_int32(cs[0], "num_blocks"), integer(a[6], "block_size"),
                             to_int32(cs[1], "num_kv_heads"), to_int32(cs[3], "head_dim"),
                             PA_KV_BF16};
    check_ranges(d, codes, scales);
    const Rows r = check_rows(q, tables, lens, a[9], selected, d);
    const int32_t sink = integer(a[7], "sink"), recent = integer(a[8], "recent");
    const OnDevice on(codes, "codes");
    auto* out = on.out<int32_t>(selected, "selected", at::kInt);
    const void* qp = on.in(q, "q", at::kBFloat16);
    const auto* cp = on.in<int8_t>(codes, "codes", at::kChar);
    const auto* up = on.in<float>(scales, "scales", at::kFloat);
    const auto* tp = on.in<int32_t>(tables, "block_tables", at::kInt);
    const auto* lp = on.in<int32_t>(lens, "context_lens", at::kInt);
    const auto* rp = on.optional<int32_t>(a[9], "row_seqs", at::kInt);
    return on.run(a[10], [&](pa_stream_t stream) {
      return pa_select_blocks(out, qp, cp, up, d, tp, r.max_blocks, lp, rp, r.rows, r.seqs,
                              r.heads, r.top, sink, recent, stream);
    });
  });
}

// out, q, k_cache, v_cache, block_tables, context_lens, selected, scale,
// k_scale, v_scale, row_seqs, stream
PyObject* decode_selected(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return entry<12>("decode_selected", nargs, [&] {
    const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "q"),
                     &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache"),
                     &tables = tensor(a[4], "block_tables"), &lens = tensor(a[5], "context_lens"),
                     &selected = tensor(a[6], "selected");
    const pa_cache_desc d = describe(kc, vc, a[8], a[9]);
    if (!out.sizes().equals(q.sizes()))
      throw Refused("q and out must both be [num_rows, num_heads, head_dim]");
    const Rows r = check_rows(q, tables, lens, a[10], selected, d);
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused("scale must be a number");
    }
    const OnDevice on(kc, "k_cache");
    void* op = on.out(out, "out", at::kBFloat16);
    const void* qp = on.in(q, "q", at::kBFloat16);
    const void *kp = on.in(kc, "k_cache", kc.scalar_type()),
               *vp = on.in(vc, "v_cache", kc.scalar_type());
    const auto* tp = on.in<int32_t>(tables, "block_tables", at::kInt);
    const auto* lp = on.in<int32_t>(lens, "context_lens", at::kInt);
    const auto* sp = on.in<int32_t>(selected, "selected", at::kInt);
    const auto* ks = on.optional<float>(a[8], "k_scale", at::kFloat);
    const auto* vs = on.optional<float>(a[9], "v_scale", at::kFloat);
    const auto* rp = on.optional<int32_t>(a[10], "row_seqs", at::kInt);
    return on.run(a[11], [&](pa_stream_t stream) {
      return pa_decode_selected(op, qp, kp, vp, d, tp, r.max_blocks, lp, rp, sp, r.rows, r.seqs,
                                r.heads, r.top, (float)scale, ks, vs, stream);
    });
  });
}

// q_out, query, key, value, k_cache, v_cache, slot_mapping, positions, cos_sin,
// q_weight, k_weight, eps, k_scale, v_scale, sections, sections_in_turn,
// adjacent_pairs, stream
PyObject* norm_rope_and_cache(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return entry<18>("norm_rope_and_cache", nargs, [&] {
    const at::Tensor &q_out = tensor(a[0], "q_out"), &query = tensor(a[1], "query"),
                     &key = tensor(a[2], "key"), &value = tensor(a[3], "value"),
                     &kc = tensor(a[4], "k_cache"), &vc = tensor(a[5], "v_cache"),
                     &slots = tensor(a[6], "slot_mapping");
    const pa_cache_desc d = describe_any(kc, vc, a[12], a[13]);
    if ((a[7] == Py_None) != (a[8] == Py_None))
      throw Refused("positions and cos_sin are given together or not at all");
    const bool rotates = a[7] != Py_None;
    const at::Tensor *pos = rotates ? &tensor(a[7], "positions") : nullptr,
                     *table = rotates ? &tensor(a[8], "cos_sin") : nullptr;
    const int64_t n = check_write(q_out, query, key, value, slots, pos, table, d);
    pa_rope_desc rope = {};
    if (rotates) {
      rope = rope_of(pos->sizes(), table->sizes(), a[14], a[15], a[16]);
      if (rope.rot_dim == 0) throw Refused("cos_sin must have columns");
    }
    for (int i : {9, 10}) {
      if (a[i] != Py_None && !is(tensor(a[i], "q_weight and k_weight").sizes(), {d.head_dim}))
        throw Refused("q_weight and k_weight must be [" + std::to_string(d.head_dim) + "]");
    }
    const float eps = number(a[11], "eps");
    const OnDevice on(kc, "k_cache");
    void* o = on.out(q_out, "q_out", at::kBFloat16);
    void *kp = on.out(kc, "k_cache", kc.scalar_type()), *vp = on.out(vc, "v_cache", kc.scalar_type());
    const bool units = d.dtype == PA_KV_INT8;
    auto scale = [&](PyObject* s, const char* name) {
      return units ? on.out<float>(tensor(s, name), name, at::kFloat)
                   : const_cast<float*>(on.optional<float>(s, name, at::kFloat));
    };
    float *ks = scale(a[12], "k_scale"), *vs = scale(a[13], "v_scale");
    int64_t q_stride, k_stride, v_stride;
    const void *q = on.rows(query, "query", &q_stride), *k = on.rows(key, "key", &k_stride),
               *v = on.rows(value, "value", &v_stride);
    const auto* sp = on.in<int32_t>(slots, "slot_mapping", at::kInt);
    const auto* pp = on.optional<int32_t>(a[7], "positions", at::kInt);
    const auto* cs = on.optional<float>(a[8], "cos_sin", at::kFloat);
    const auto* qw = on.optional<float>(a[9], "q_weight", at::kFloat);
    const auto* kw = on.optional<float>(a[10], "k_weight", at::kFloat);
    const int32_t heads = to_int32(query.sizes()[1], "num_heads"), tokens = to_int32(n, "num_tokens");
    return on.run(a[17], [&](pa_stream_t stream) {
      return pa_norm_rope_and_cache(o, q, q_stride, heads, k, k_stride, v, v_stride, kp, vp, d, sp,
                                    pp, cs, rope, qw, kw, eps, tokens, ks, vs, stream);
    });
  });
}

// k_out, v_out, k_cache, v_cache, block_tables, context_lens, out_start_loc,
// first_tokens, k_scale, v_scale, stream
PyObject* gather_cache(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return entry<11>("gather_cache", nargs, [&] {
    const at::Tensor &ko = tensor(a[0], "k_out"), &vo = tensor(a[1], "v_out"),
                     &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache"),
                     &tables = tensor(a[4], "block_tables"), &lens = tensor(a[5], "context_lens"),
                     &starts = tensor(a[6], "out_start_loc");
    const pa_cache_desc d = describe_any(kc, vc, a[8], a[9]);
    const auto os = ko.sizes(), ts = tables.sizes();
    if (os.size() != 3 || os[1] != d.num_kv_heads || os[2] != d.head_dim || !vo.sizes().equals(os))
      throw Refused("k_out and v_out must be [num_rows, " + std::to_string(d.num_kv_heads) + ", " +
                    std::to_string(d.head_dim) + "], got " + text(os) + " and " + text(vo.sizes()));
    if (ts.size() != 2) throw Refused("block_tables must be [num_seqs, max_blocks_per_seq]");
    const std::string n = std::to_string(ts[0]);
    if (lens.numel() != ts[0])
      throw Refused("context_lens needs " + n + " entries, got " + std::to_string(lens.numel()));
    if (starts.numel() != ts[0] + 1)
      throw Refused("out_start_loc needs num_seqs + 1 = " + std::to_string(ts[0] + 1) +
                    " entries, got " + std::to_string(starts.numel()));
    if (a[7] != Py_None && tensor(a[7], "first_tokens").numel() != ts[0])
      throw Refused("first_tokens needs " + n + " entries, got " +
                    std::to_string(tensor(a[7], "first_tokens").numel()));
    const OnDevice on(kc, "k_cache");
    void *kop = on.out(ko, "k_out", at::kBFloat16), *vop = on.out(vo, "v_out", at::kBFloat16);
    const void *kp = on.in(kc, "k_cache", kc.scalar_type()),
               *vp = on.in(vc, "v_cache", kc.scalar_type());
    const auto* tp = on.in<int32_t>(tables, "block_tables", at::kInt);
    const auto* lp = on.in<int32_t>(lens, "context_lens", at::kInt);
    const auto* sp = on.in<int32_t>(starts, "out_start_loc", at::kInt);
    const auto* fp = on.optional<int32_t>(a[7], "first_tokens", at::kInt);
    const auto* ks = on.optional<float>(a[8], "k_scale", at::kFloat);
    const auto* vs = on.optional<float>(a[9], "v_scale", at::kFloat);
    const int32_t max_blocks = to_int32(ts[1], "max_blocks_per_seq"),
                  seqs = to_int32(ts[0], "num_seqs"), rows = to_int32(os[0], "num_rows");
    return on.run(a[10], [&](pa_stream_t stream) {
      return pa_gather_cache(kop, vop, kp, vp, d, tp, max_blocks, lp, fp, sp, seqs, rows, ks, vs,
                             stream);
    });
  });
}

// What decode_scored and varlen_scored share: a holds out, q, k_cache,
// v_cache, block_tables, lens; then (varlen) query_start_loc; then, from
// a[at] on, scale, cap, window, slopes, (varlen) prefix_lens, k_scale,
// v_scale, workspace, stream.
template <bool kVarlen>
PyObject* scored(PyObject* const* a) {
  constexpr int at = kVarlen ? 7 : 6, rest = kVarlen ? at + 5 : at + 4;
  const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "q"), &kc = tensor(a[2], "k_cache"),
                   &vc = tensor(a[3], "v_cache"), &tables = tensor(a[4], "block_tables"),
                   &lens = tensor(a[5], kVarlen ? "seq_lens" : "context_lens"),
                   &ws = tensor(a[rest + 2], "workspace");
  const pa_cache_desc d = describe_any(kc, vc, a[rest], a[rest + 1]);
  const auto qs = q.sizes(), ts = tables.sizes();
  if (qs.size() != 3 || !out.sizes().equals(qs))
    throw Refused("q and out must both be [num_rows, num_heads, head_dim]");
  if (qs[2] != d.head_dim)
    throw Refused("q's head_dim " + std::to_string(qs[2]) + " differs from the cache's " +
                  std::to_string(d.head_dim));
  const int64_t n = kVarlen ? lens.numel() : qs[0];
  if (ts.size() != 2 || ts[0] != n)
    throw Refused("block_tables must be [" + std::to_string(n) + ", max_blocks_per_seq], got " +
                  text(ts));
  if (lens.numel() != n)
    throw Refused("context_lens needs " + std::to_string(n) + " entries, got " +
                  std::to_string(lens.numel()));
  if (kVarlen && tensor(a[6], "query_start_loc").numel() != n + 1)
    throw Refused("query_start_loc needs num_seqs + 1 = " + std::to_string(n + 1) + " entries");
  if (a[at + 3] != Py_None && !is(tensor(a[at + 3], "slopes").sizes(), {qs[1]}))
    throw Refused("slopes must be [" + std::to_string(qs[1]) + "]");
  if (kVarlen && a[at + 4] != Py_None && tensor(a[at + 4], "prefix_lens").numel() != n)
    throw Refused("prefix_lens needs " + std::to_string(n) + " entries");
  const float scale = number(a[at], "scale");
  pa_score_desc score = {number(a[at + 1], "cap"), integer(a[at + 2], "window"), nullptr};
  const OnDevice on(kc, "k_cache");
  void* op = on.out(out, "out", at::kBFloat16);
  void* wp = on.out(ws, "workspace", at::kByte);
  score.slopes = on.optional<float>(a[at + 3], "slopes", at::kFloat);
  const void* qp = on.in(q, "q", at::kBFloat16);
  const void *kp = on.in(kc, "k_cache", kc.scalar_type()),
             *vp = on.in(vc, "v_cache", kc.scalar_type());
  const auto* tp = on.in<int32_t>(tables, "block_tables", at::kInt);
  const auto* lp = on.in<int32_t>(lens, "context_lens", at::kInt);
  const auto* ks = on.optional<float>(a[rest], "k_scale", at::kFloat);
  const auto* vs = on.optional<float>(a[rest + 1], "v_scale", at::kFloat);
  const int32_t rows = to_int32(qs[0], "num_rows"), heads = to_int32(qs[1], "num_heads"),
                seqs = to_int32(n, "num_seqs"), max_blocks = to_int32(ts[1], "max_blocks_per_seq");
  const size_t bytes = ws.numel();
  if constexpr (kVarlen) {
    const auto* sp = on.in<int32_t>(tensor(a[6], "query_start_loc"), "query_start_loc", at::kInt);
    const auto* pp = on.optional<int32_t>(a[at + 4], "prefix_lens", at::kInt);
    return on.run(a[rest + 3], [&](pa_stream_t stream) {
      return pa_varlen_scored(op, qp, kp, vp, d, tp, max_blocks, lp, sp, seqs, rows, heads, scale,
                              score, pp, ks, vs, wp, bytes, stream);
    });
  } else {
    return on.run(a[rest + 3], [&](pa_stream_t stream) {
      return pa_decode_scored(op, qp, kp, vp, d, tp, max_blocks, lp, seqs, heads, scale, score, ks,
                              vs, wp, bytes, stream);
    });
  }
}

// out, q, k_cache, v_cache, block_tables, context_lens, scale, cap, window,
// slopes, k_scale, v_scale, workspace, stream
PyObject* decode_scored(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return entry<14>("decode_scored", nargs, [&] { return scored<false>(a); });
}

// out, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale,
// cap, window, slopes, prefix_lens, k_scale, v_scale, workspace, stream
PyObject* varlen_scored(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return entry<16>("varlen_scored", nargs, [&] { return scored<true>(a); });
}

PyMethodDef kMethods[] = {
    {"rope_and_cache", (PyCFunction)(void (*)(void))rope_and_cache, METH_FASTCALL, nullptr},
    {"summarize_blocks", (PyCFunction)(void (*)(void))summarize_blocks, METH_FASTCALL, nullptr},
    {"select_blocks", (PyCFunction)(void (*)(void))select_blocks, METH_FASTCALL, nullptr},
    {"decode_selected", (PyCFunction)(void (*)(void))decode_selected, METH_FASTCALL, nullptr},
    {"norm_rope_and_cache", (PyCFunction)(void (*)(void))norm_rope_and_cache, METH_FASTCALL,
     nullptr},
    {"gather_cache", (PyCFunction)(void (*)(void))gather_cache, METH_FASTCALL, nullptr},
    {"decode_scored", (PyCFunction)(void (*)(void))decode_scored, METH_FASTCALL, nullptr},
    {"varlen_scored", (PyCFunction)(void (*)(void))varlen_scored, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
