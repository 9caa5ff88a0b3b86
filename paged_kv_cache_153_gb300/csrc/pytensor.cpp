// Module _tensor: the rotary append, the block index, the sparse, the shared-prefix
// and the window decode, and the drafted tokens' calls, straight from torch tensors.  Each reads
// shapes, strides and addresses, refuses what does not fit, and calls the
// library's entry point; the same steps in Python take 2 to 6 us of a call
// whose kernels run for 2 to 8 (rope: 8.3 us a call in Python, 2.9 here; sparse
// decode 9.8 against 4.9).
#include "pycall.h"

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

namespace pkv_py {
namespace {

struct Refused {};   // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const char* what) {
  PyErr_SetString(type, what);
  throw Refused{};
}

const at::Tensor& need(PyObject* o, int dims, const char* what) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "expected a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (dims >= 0 && t.dim() != dims) refuse(PyExc_ValueError, what);
  return t;
}

thread_local int call_device;   // the current device, asked once per call (-1: not yet)

// t's address, on the device that the call will launch on
void* ptr(const at::Tensor& t) {
  if (t.is_cuda() && call_device < 0) call_device = c10::cuda::current_device();
  if (!t.is_cuda() || t.get_device() != call_device)
    refuse(PyExc_ValueError, "tensors must be on the current CUDA device");
  return t.data_ptr();
}

void* address(PyObject* o) { return o == Py_None ? nullptr : ptr(need(o, -1, "")); }

template <typename T>
T number(PyObject* o) {
  T v;
  if (!convert(o, v)) throw Refused{};
  return v;
}

void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  if (PyLong_Check(o)) return number<void*>(o);
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (h == nullptr) throw Refused{};
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (s == nullptr && PyErr_Occurred()) throw Refused{};
  return s;
}

// The 16-bit type of a call: PKV_F16 / PKV_BF16 by t, or as given.  Where it is
// given, tensors of any two-byte type hold its bits; else all have t's own type.
struct Type16 {
  pkv_dtype code;
  bool given;
  at::ScalarType own;
  Type16(const at::Tensor& t, PyObject* tag) : code(PKV_F16), given(tag != Py_None), own(t.scalar_type()) {
    if (given) {
      code = number<pkv_dtype>(tag);
      check(t);
    } else if (own == at::kBFloat16) {
      code = PKV_BF16;
    } else if (own != at::kHalf) {
      refuse(PyExc_TypeError, "cannot infer the 16-bit kind; pass dtype=PKV_F16/PKV_BF16");
    }
  }
  void check(const at::Tensor& t) const {
    if (given ? t.element_size() != 2 : t.scalar_type() != own)
      refuse(PyExc_TypeError, "the 16-bit tensors of a call must have one type, or two-byte elements and dtype given");
  }
};

// Index tensors are contiguous int32: another type would be read as garbage indices.
void index_check(const at::Tensor& t) {
  if (t.scalar_type() != at::kInt || !t.is_contiguous())
    refuse(PyExc_TypeError, "tables, lengths, positions and lists must be contiguous int32 tensors");
}

void contiguous(const at::Tensor& t) {
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "q, out, caches, bounds, scores and slots must be contiguous");
}

// a cache of the element size that the call reads and writes
void cache_check(const at::Tensor& t, int64_t itemsize) {
  if (static_cast<int64_t>(t.element_size()) != itemsize)
    refuse(PyExc_ValueError, "caches must have the call's element type");
  contiguous(t);
}

void caches_check(const at::Tensor& k, const at::Tensor& v, int64_t itemsize) {
  if (k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
    refuse(PyExc_ValueError, "caches must have one shape and type");
  cache_check(k, itemsize);
  contiguous(v);
}

// What a cache holds, its element size being right: kind 0 the call's 16-bit
// type; 1 (E4M3) and 2 (E5M2) codes of any one-byte type but the other format's.
void cache_type(const at::Tensor& t, int kind, const Type16& type) {
  if (kind == 0)
    type.check(t);
  else if (t.scalar_type() == (kind == 1 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn))
    refuse(PyExc_TypeError, "the cache holds the other FP8 format's codes");
}

// scales per KV head (None: none given)
void scales_check(PyObject* o, int64_t heads) {
  if (o == Py_None) return;
  const at::Tensor& t = need(o, -1, "");
  if (t.scalar_type() != at::kFloat || !t.is_contiguous()) refuse(PyExc_TypeError, "scales must be contiguous fp32");
  if (t.numel() != heads) refuse(PyExc_ValueError, "scales must have one entry per KV head");
}

// the device error word (None: none given)
void flag_check(PyObject* o) {
  if (o == Py_None) return;
  const at::Tensor& t = need(o, -1, "");
  if (t.scalar_type() != at::kInt || t.numel() < 1) refuse(PyExc_TypeError, "err_flag must be int32, one entry");
}

void per_sequence(int64_t b, const at::Tensor& tables, const at::Tensor& lens) {
  if (tables.size(0) != b || lens.numel() != b)
    refuse(PyExc_ValueError, "block_tables and context_lens must have a row per sequence");
}

int to_int(int64_t v) {
  if (v > INT32_MAX) refuse(PyExc_OverflowError, "a size does not fit its C type");
  return static_cast<int>(v);
}

constexpr const char* kTableDims = "block_tables must be [batch, max_blocks]";
constexpr const char* kCacheDims = "caches must be [num_blocks, num_kv_heads, 16, head_dim]";

template <typename F>
PyObject* status(F&& call) {
  pkv_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

// Runs f; what it refuses, or what torch throws, becomes a Python exception.
template <Py_ssize_t N, PyObject* (*F)(PyObject* const*)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  call_device = -1;
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// elements between the tokens of t [T, heads, d], whose heads are contiguous
int64_t token_stride(const at::Tensor& t, const char* what) {
  const int64_t heads = t.size(1), d = t.size(2);
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)) refuse(PyExc_ValueError, what);
  return t.size(0) > 1 ? t.stride(0) : heads * d;
}

// kind (0: 16-bit cache, 1: E4M3, 2: E5M2), q, k_new, v_new, positions,
// slot_mapping, turns, q_out, k_cache, v_cache, k_scale, v_scale, layout,
// amplitude, dtype, err_flag, stream
PyObject* rope_append(PyObject* const* a) {
  const int kind = number<int>(a[0]);
  const bool has_q = a[1] != Py_None, has_k = a[2] != Py_None;
  pkv_rope_layout layout;
  if (PyUnicode_Check(a[12])) {
    if (PyUnicode_CompareWithASCIIString(a[12], "half") == 0)
      layout = PKV_ROPE_HALF;
    else if (PyUnicode_CompareWithASCIIString(a[12], "interleaved") == 0)
      layout = PKV_ROPE_INTERLEAVED;
    else
      refuse(PyExc_ValueError, "unknown layout");
  } else {
    layout = number<pkv_rope_layout>(a[12]);
  }
  const at::Tensor &pos = need(a[4], -1, ""), &turns = need(a[6], 1, "turns must be [rot_dim / 2]");
  index_check(pos);
  if ((turns.scalar_type() != at::kLong && turns.scalar_type() != at::kUInt64) || !turns.is_contiguous())
    refuse(PyExc_TypeError, "turns must be the int64 tensor of pkv_rope_plan");
  if (!has_q && !has_k) refuse(PyExc_ValueError, "q, or k_new and v_new, must be given");
  const Type16 type(need(has_q ? a[1] : a[2], -1, ""), a[14]);
  flag_check(a[15]);
  const int64_t n = pos.numel();
  void *q = nullptr, *q_out = nullptr, *k = nullptr, *v = nullptr, *kc = nullptr, *vc = nullptr;
  int64_t q_stride = 0, o_stride = 0, k_stride = 0, v_stride = 0, nb = 0;
  int hq = 0, hkv = 0, d = 0, bs = 16;
  if (has_q) {
    const at::Tensor &tq = need(a[1], 3, "q must be [T, num_q_heads, head_dim]"), &to = need(a[7], -1, "");
    if (tq.size(0) != n || to.sizes() != tq.sizes())
      refuse(PyExc_ValueError, "q, q_out and positions differ in shape");
    type.check(to);
    hq = to_int(tq.size(1)), d = to_int(tq.size(2));
    q_stride = token_stride(tq, "q: a token's heads must be contiguous");
    o_stride = token_stride(to, "q_out: a token's heads must be contiguous");
  }
  if (has_k) {
    const at::Tensor &tk = need(a[2], 3, "k_new must be [T, num_kv_heads, head_dim]"), &tv = need(a[3], -1, ""),
                     &ck = need(a[8], 4, kCacheDims), &cv = need(a[9], -1, ""), &ts = need(a[5], -1, "");
    nb = ck.size(0), hkv = to_int(ck.size(1)), bs = to_int(ck.size(2));
    if (tk.size(0) != n || tk.size(1) != hkv || tk.size(2) != ck.size(3) || tv.sizes() != tk.sizes() ||
        (has_q && ck.size(3) != d))
      refuse(PyExc_ValueError, "k_new and v_new must be [T, num_kv_heads, head_dim] of the cache");
    if (ts.numel() != n || ts.scalar_type() != at::kLong || !ts.is_contiguous())
      refuse(PyExc_ValueError, "slot_mapping must be contiguous int64, one slot per position");
    caches_check(ck, cv, kind == 0 ? 2 : 1);
    type.check(tk);
    type.check(tv);
    cache_type(ck, kind, type);
    d = to_int(ck.size(3));
    scales_check(a[10], hkv);
    scales_check(a[11], hkv);
    k_stride = token_stride(tk, "k_new: a token's heads must be contiguous");
    v_stride = token_stride(tv, "v_new: a token's heads must be contiguous");
    k = ptr(tk), v = ptr(tv), kc = ptr(ck), vc = ptr(cv);
  }
  if (has_q) q = address(a[1]), q_out = address(a[7]);
  const auto* pos_p = static_cast<const int32_t*>(ptr(pos));
  const auto* slots = static_cast<const int64_t*>(address(a[5]));
  const auto* turns_p = static_cast<const uint64_t*>(ptr(turns));
  const auto* ks = static_cast<const float*>(address(a[10]));
  const auto* vs = static_cast<const float*>(address(a[11]));
  const int rot = to_int(2 * turns.numel());
  const float amplitude = number<float>(a[13]);
  const pkv_dtype dt = type.code;
  auto* err = static_cast<int32_t*>(address(a[15]));
  void* s = stream_of(a[16]);
  if (kind == 0)
    return status([&] {
      return pkv_rope_append(q, q_stride, k, k_stride, v, v_stride, pos_p, slots, n, turns_p, rot, layout, amplitude,
                             q_out, o_stride, kc, vc, nb, hq, hkv, d, bs, dt, err, s);
    });
  const auto fn = kind == 1 ? pkv_rope_append_fp8 : pkv_rope_append_e5m2;
  return status([&] {
    return fn(q, q_stride, k, k_stride, v, v_stride, pos_p, slots, n, turns_p, rot, layout, amplitude, q_out, o_stride,
              static_cast<uint8_t*>(kc), static_cast<uint8_t*>(vc), nb, ks, vs, hq, hkv, d, bs, dt, err, s);
  });
}

// kind, k_cache, block_tables, context_lens, bounds, new_lens, max_new_len,
// dtype, err_flag, stream
PyObject* block_bounds(PyObject* const* a) {
  const int kind = number<int>(a[0]);
  const at::Tensor &kc = need(a[1], 4, kCacheDims), &tab = need(a[2], 2, kTableDims), &len = need(a[3], -1, ""),
                   &out = need(a[4], 4, "bounds must be [num_blocks, num_kv_heads, 2, head_dim]");
  if (out.size(0) != kc.size(0) || out.size(1) != kc.size(1) || out.size(2) != 2 || out.size(3) != kc.size(3))
    refuse(PyExc_ValueError, "bounds must be [num_blocks, num_kv_heads, 2, head_dim] of the cache");
  index_check(tab);
  index_check(len);
  if (a[5] != Py_None) {
    const at::Tensor& t = need(a[5], -1, "");
    index_check(t);
    if (t.numel() != len.numel()) refuse(PyExc_ValueError, "new_lens and context_lens differ in length");
  }
  cache_check(kc, kind == 0 ? 2 : 1);
  contiguous(out);
  per_sequence(len.numel(), tab, len);
  const Type16 type(out, a[7]);
  cache_type(kc, kind, type);
  flag_check(a[8]);
  const auto* fresh = static_cast<const int32_t*>(address(a[5]));
  const auto* tp = static_cast<const int32_t*>(ptr(tab));
  const auto* lp = static_cast<const int32_t*>(ptr(len));
  const int max_new = number<int>(a[6]), b = to_int(len.numel()), hkv = to_int(kc.size(1)), d = to_int(kc.size(3)),
            bs = to_int(kc.size(2)), width = to_int(tab.size(1));
  const int64_t nb = kc.size(0);
  const pkv_dtype dt = type.code;
  auto* err = static_cast<int32_t*>(address(a[8]));
  void *s = stream_of(a[9]), *k = ptr(kc), *o = ptr(out);
  if (kind == 0)
    return status([&] {
      return pkv_kv_block_bounds(k, tp, lp, fresh, max_new, b, hkv, d, bs, width, nb, o, dt, err, s);
    });
  const auto fn = kind == 1 ? pkv_kv_block_bounds_fp8 : pkv_kv_block_bounds_e5m2;
  return status([&] {
    return fn(static_cast<const uint8_t*>(k), tp, lp, fresh, max_new, b, hkv, d, bs, width, nb, o, dt, err, s);
  });
}

// q, bounds, block_tables, context_lens, scores, scale, max_context_len,
// k_scale, dtype, err_flag, stream
PyObject* block_scores(PyObject* const* a) {
  const at::Tensor &q = need(a[0], 3, "q must be [batch, num_q_heads, head_dim]"),
                   &lo_hi = need(a[1], 4, "bounds must be [num_blocks, num_kv_heads, 2, head_dim]"),
                   &tab = need(a[2], 2, kTableDims), &len = need(a[3], -1, ""),
                   &out = need(a[4], 3, "scores must be [batch, num_kv_heads, max_blocks]");
  const int64_t b = q.size(0), hkv = lo_hi.size(1), d = q.size(2), width = tab.size(1);
  if (out.size(0) != b || out.size(1) != hkv || out.size(2) != width || lo_hi.size(2) != 2 || lo_hi.size(3) != d)
    refuse(PyExc_ValueError,
           "scores must be [batch, num_kv_heads, max_blocks], bounds [num_blocks, num_kv_heads, 2, head_dim]");
  if (lo_hi.scalar_type() != q.scalar_type()) refuse(PyExc_TypeError, "bounds and q differ in dtype");
  if (out.scalar_type() != at::kFloat) refuse(PyExc_TypeError, "scores must be fp32");
  index_check(tab);
  index_check(len);
  contiguous(q);
  contiguous(lo_hi);
  contiguous(out);
  per_sequence(b, tab, len);
  const Type16 type(q, a[8]);
  scales_check(a[7], hkv);
  flag_check(a[9]);
  const int bi = to_int(b), hq = to_int(q.size(1)), h = to_int(hkv), di = to_int(d), w = to_int(width),
            max_ctx = number<int>(a[6]);
  const int64_t nb = lo_hi.size(0);
  const float scale = number<float>(a[5]);
  const auto* ks = static_cast<const float*>(address(a[7]));
  const pkv_dtype dt = type.code;
  auto* err = static_cast<int32_t*>(address(a[9]));
  void *s = stream_of(a[10]), *qp = ptr(q), *lp = ptr(lo_hi);
  const auto* tp = static_cast<const int32_t*>(ptr(tab));
  const auto* np = static_cast<const int32_t*>(ptr(len));
  auto* op = static_cast<float*>(ptr(out));
  return status([&] {
    return pkv_block_scores(qp, lp, tp, np, ks, bi, hq, h, di, 16, w, nb, max_ctx, scale, op, dt, err, s);
  });
}

// scores, context_lens, selected, num_first, num_last, err_flag, stream
PyObject* select_blocks(PyObject* const* a) {
  const at::Tensor &sc = need(a[0], 3, "scores must be [batch, num_kv_heads, max_blocks]"), &len = need(a[1], -1, ""),
                   &sel = need(a[2], 3, "selected must be [batch, num_kv_heads, budget]");
  if (sel.size(0) != sc.size(0) || sel.size(1) != sc.size(1))
    refuse(PyExc_ValueError, "selected must be [batch, num_kv_heads, budget]");
  index_check(len);
  index_check(sel);
  contiguous(sc);
  if (sc.scalar_type() != at::kFloat || len.numel() != sc.size(0))
    refuse(PyExc_ValueError, "scores must be fp32, with a context length per sequence");
  flag_check(a[5]);
  const auto* sp = static_cast<const float*>(ptr(sc));
  const auto* lp = static_cast<const int32_t*>(ptr(len));
  auto* op = static_cast<int32_t*>(ptr(sel));
  const int b = to_int(sc.size(0)), h = to_int(sc.size(1)), w = to_int(sc.size(2)), budget = to_int(sel.size(2)),
            first = number<int>(a[3]), last = number<int>(a[4]);
  auto* err = static_cast<int32_t*>(address(a[5]));
  void* s = stream_of(a[6]);
  return status([&] { return pkv_select_blocks(sp, lp, b, h, 16, w, first, last, budget, op, err, s); });
}

// what the two attention calls have in common
struct Attention {
  void *q, *k, *v, *out, *ws;
  const int32_t *tab, *len;
  int b, hq, hkv, d, bs, width;
  int64_t nb;
  size_t ws_bytes;
  pkv_dtype dtype;
  // kind as in cache_type; the scales and the flag are only checked here
  Attention(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* tab_, PyObject* len_, PyObject* out_, PyObject* ws_,
            int kind, PyObject* dtype_, PyObject* k_scale, PyObject* v_scale, PyObject* flag) {
    const at::Tensor &tq = need(q_, 3, "q must be [batch, num_q_heads, head_dim]"), &kc = need(k_, 4, kCacheDims),
                     &vc = need(v_, -1, ""), &t = need(tab_, 2, kTableDims), &l = need(len_, -1, ""),
                     &o = need(out_, -1, ""), &w = need(ws_, -1, "");
    index_check(t);
    index_check(l);
    contiguous(tq);
    contiguous(o);
    caches_check(kc, vc, kind == 0 ? 2 : 1);
    per_sequence(tq.size(0), t, l);
    if (o.sizes() != tq.sizes()) refuse(PyExc_ValueError, "q and out differ in shape");
    if (kc.size(3) != tq.size(2)) refuse(PyExc_ValueError, "q and the caches differ in head_dim");
    const Type16 type(tq, dtype_);
    type.check(o);
    cache_type(kc, kind, type);
    dtype = type.code;
    scales_check(k_scale, kc.size(1));
    scales_check(v_scale, kc.size(1));
    flag_check(flag);
    if (!w.is_contiguous()) refuse(PyExc_ValueError, "the workspace must be contiguous");
    q = ptr(tq), k = ptr(kc), v = ptr(vc), out = ptr(o), ws = ptr(w);
    tab = static_cast<const int32_t*>(ptr(t)), len = static_cast<const int32_t*>(ptr(l));
    b = to_int(tq.size(0)), hq = to_int(tq.size(1)), d = to_int(tq.size(2)), width = to_int(t.size(1));
    nb = kc.size(0), hkv = to_int(kc.size(1)), bs = to_int(kc.size(2));
    ws_bytes = w.nbytes();
  }
};

// kind, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
// selected, out, scale, workspace, dtype, err_flag, stream
PyObject* sparse_decode(PyObject* const* a) {
  const int kind = number<int>(a[0]);
  const at::Tensor& sel = need(a[8], 3, "selected must be [batch, num_kv_heads, budget]");
  index_check(sel);
  const Attention x(a[1], a[2], a[3], a[6], a[7], a[9], a[11], kind, a[12], a[4], a[5], a[13]);
  if (sel.size(0) != x.b || sel.size(1) != x.hkv)
    refuse(PyExc_ValueError, "selected must be [batch, num_kv_heads, budget]");
  const auto* lists = static_cast<const int32_t*>(ptr(sel));
  const int budget = to_int(sel.size(2));
  const float scale = number<float>(a[10]);
  const pkv_dtype dt = x.dtype;
  const auto* ks = static_cast<const float*>(address(a[4]));
  const auto* vs = static_cast<const float*>(address(a[5]));
  auto* err = static_cast<int32_t*>(address(a[13]));
  void* s = stream_of(a[14]);
  if (kind == 0)
    return status([&] {
      return pkv_paged_decode_attention_sparse(x.q, x.k, x.v, x.tab, x.len, lists, budget, x.b, x.hq, x.hkv, x.d, x.bs,
                                               x.width, x.nb, scale, x.out, dt, x.ws, x.ws_bytes, err, s);
    });
  const auto fn = kind == 1 ? pkv_paged_decode_attention_sparse_fp8 : pkv_paged_decode_attention_sparse_e5m2;
  return status([&] {
    return fn(x.q, static_cast<const uint8_t*>(x.k), static_cast<const uint8_t*>(x.v), ks, vs, x.tab, x.len, lists,
              budget, x.b, x.hq, x.hkv, x.d, x.bs, x.width, x.nb, scale, x.out, dt, x.ws, x.ws_bytes, err, s);
  });
}

// kind, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, out,
// scale, window, num_sinks, workspace, dtype, err_flag, stream
PyObject* window_decode(PyObject* const* a) {
  const int kind = number<int>(a[0]);
  const Attention x(a[1], a[2], a[3], a[6], a[7], a[8], a[12], kind, a[13], a[4], a[5], a[14]);
  const float scale = number<float>(a[9]);
  const int window = number<int>(a[10]), sinks = number<int>(a[11]);
  const pkv_dtype dt = x.dtype;
  const auto* ks = static_cast<const float*>(address(a[4]));
  const auto* vs = static_cast<const float*>(address(a[5]));
  auto* err = static_cast<int32_t*>(address(a[14]));
  void* s = stream_of(a[15]);
  if (kind == 0)
    return status([&] {
      return pkv_paged_decode_attention_window(x.q, x.k, x.v, x.tab, x.len, x.b, x.hq, x.hkv, x.d, x.bs, x.width, x.nb,
                                               window, sinks, scale, x.out, dt, x.ws, x.ws_bytes, err, s);
    });
  const auto fn = kind == 1 ? pkv_paged_decode_attention_window_fp8 : pkv_paged_decode_attention_window_e5m2;
  return status([&] {
    return fn(x.q, static_cast<const uint8_t*>(x.k), static_cast<const uint8_t*>(x.v), ks, vs, x.tab, x.len, x.b, x.hq,
              x.hkv, x.d, x.bs, x.width, x.nb, window, sinks, scale, x.out, dt, x.ws, x.ws_bytes, err, s);
  });
}

// q, k_cache, v_cache, block_tables, context_lens, group_starts, prefix_lens,
// out, scale, max_context_len, max_prefix_len, workspace, dtype, err_flag, stream
PyObject* prefix_decode(PyObject* const* a) {
  const at::Tensor &starts = need(a[5], -1, ""), &pre = need(a[6], -1, "");
  if (starts.numel() != pre.numel() + 1)
    refuse(PyExc_ValueError, "group_starts must have one entry more than prefix_lens");
  index_check(starts);
  index_check(pre);
  const Attention x(a[0], a[1], a[2], a[3], a[4], a[7], a[11], 0, a[12], Py_None, Py_None, a[13]);
  const auto* sp = static_cast<const int32_t*>(ptr(starts));
  const auto* pp = static_cast<const int32_t*>(ptr(pre));
  const int groups = to_int(pre.numel()), max_ctx = number<int>(a[9]), max_pre = number<int>(a[10]);
  const float scale = number<float>(a[8]);
  const pkv_dtype dt = x.dtype;
  auto* err = static_cast<int32_t*>(address(a[13]));
  void* s = stream_of(a[14]);
  return status([&] {
    return pkv_paged_decode_attention_prefix(x.q, x.k, x.v, x.tab, x.len, sp, pp, groups, x.b, x.hq, x.hkv, x.d, x.bs,
                                             x.width, x.nb, max_ctx, max_pre, scale, x.out, dt, x.ws, x.ws_bytes, err,
                                             s);
  });
}

// a step's drafted tokens: offsets [batch + 1], one context length per sequence
int drafted_batch(const at::Tensor& cu, const at::Tensor& len) {
  index_check(cu);
  index_check(len);
  if (cu.numel() != len.numel() + 1)
    refuse(PyExc_ValueError, "cu_nodes must have one entry more than context_lens");
  return to_int(len.numel());
}

void mask_check(const at::Tensor& t, int64_t tokens) {
  if ((t.scalar_type() != at::kLong && t.scalar_type() != at::kUInt64) || !t.is_contiguous())
    refuse(PyExc_TypeError, "tree_mask must be contiguous int64");
  if (t.size(0) != tokens) refuse(PyExc_ValueError, "tree_mask must have a row per token");
}
constexpr const char* kMaskDims = "tree_mask must be [num_tokens, words]";

// parents, cu_nodes, block_tables, context_lens, tree_mask, positions,
// slot_mapping, num_blocks, err_flag, stream
PyObject* tree_plan(PyObject* const* a) {
  const at::Tensor &par = need(a[0], -1, ""), &cu = need(a[1], -1, ""), &len = need(a[3], -1, ""),
                   &mask = need(a[4], 2, kMaskDims);
  index_check(par);
  const int b = drafted_batch(cu, len), words = to_int(mask.size(1));
  const int64_t tokens = par.numel(), nb = number<int64_t>(a[7]);
  mask_check(mask, tokens);
  int width = 0;
  if (a[6] != Py_None) {
    const at::Tensor &t = need(a[2], 2, kTableDims), &s = need(a[6], -1, "");
    index_check(t);
    per_sequence(b, t, len);
    if (s.numel() != tokens || s.scalar_type() != at::kLong || !s.is_contiguous())
      refuse(PyExc_ValueError, "slot_mapping must be contiguous int64, one slot per token");
    width = to_int(t.size(1));
  }
  if (a[5] != Py_None) {
    const at::Tensor& t = need(a[5], -1, "");
    index_check(t);
    if (t.numel() != tokens) refuse(PyExc_ValueError, "positions must have an entry per token");
  }
  flag_check(a[8]);
  const auto* tab = static_cast<const int32_t*>(a[6] != Py_None ? address(a[2]) : nullptr);
  auto* mp = static_cast<uint64_t*>(ptr(mask));
  const auto* pp = static_cast<const int32_t*>(ptr(par));
  const auto* cp = static_cast<const int32_t*>(ptr(cu));
  const auto* lp = static_cast<const int32_t*>(ptr(len));
  auto* pos = static_cast<int32_t*>(address(a[5]));
  auto* slots = static_cast<int64_t*>(address(a[6]));
  auto* err = static_cast<int32_t*>(address(a[8]));
  void* s = stream_of(a[9]);
  return status([&] {
    return pkv_tree_plan(pp, cp, tab, lp, b, tokens, words, 16, width, nb, mp, pos, slots, err, s);
  });
}

// kind, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
// cu_nodes, tree_mask, out, scale, max_context_len, max_nodes, workspace, dtype,
// err_flag, stream
PyObject* tree_attention(PyObject* const* a) {
  const int kind = number<int>(a[0]);
  const at::Tensor &q = need(a[1], 3, "q must be [num_tokens, num_q_heads, head_dim]"), &kc = need(a[2], 4, kCacheDims),
                   &vc = need(a[3], -1, ""), &tab = need(a[6], 2, kTableDims), &len = need(a[7], -1, ""),
                   &cu = need(a[8], -1, ""), &mask = need(a[9], 2, kMaskDims), &out = need(a[10], -1, ""),
                   &ws = need(a[14], -1, "");
  const int b = drafted_batch(cu, len), words = to_int(mask.size(1));
  index_check(tab);
  per_sequence(b, tab, len);
  contiguous(q);
  contiguous(out);
  caches_check(kc, vc, kind == 0 ? 2 : 1);
  if (out.sizes() != q.sizes()) refuse(PyExc_ValueError, "q and out differ in shape");
  if (kc.size(3) != q.size(2)) refuse(PyExc_ValueError, "q and the caches differ in head_dim");
  const Type16 type(q, a[15]);
  type.check(out);
  cache_type(kc, kind, type);
  scales_check(a[4], kc.size(1));
  scales_check(a[5], kc.size(1));
  flag_check(a[16]);
  if (!ws.is_contiguous()) refuse(PyExc_ValueError, "the workspace must be contiguous");
  const int64_t tokens = q.size(0), nb = kc.size(0);
  mask_check(mask, tokens);
  const auto* mp = static_cast<const uint64_t*>(ptr(mask));
  const int hq = to_int(q.size(1)), hkv = to_int(kc.size(1)), d = to_int(q.size(2)), bs = to_int(kc.size(2)),
            width = to_int(tab.size(1)), max_ctx = number<int>(a[12]), max_nodes = number<int>(a[13]);
  const float scale = number<float>(a[11]);
  const pkv_dtype dt = type.code;
  void *qp = ptr(q), *kp = ptr(kc), *vp = ptr(vc), *op = ptr(out), *wp = ptr(ws);
  const size_t bytes = ws.nbytes();
  const auto* tp = static_cast<const int32_t*>(ptr(tab));
  const auto* lp = static_cast<const int32_t*>(ptr(len));
  const auto* cp = static_cast<const int32_t*>(ptr(cu));
  const auto* ks = static_cast<const float*>(address(a[4]));
  const auto* vs = static_cast<const float*>(address(a[5]));
  auto* err = static_cast<int32_t*>(address(a[16]));
  void* s = stream_of(a[17]);
  if (kind == 0)
    return status([&] {
      return pkv_paged_tree_attention(qp, kp, vp, tp, lp, cp, mp, words, max_nodes, tokens, b, hq, hkv, d, bs, width,
                                      nb, max_ctx, scale, op, dt, wp, bytes, err, s);
    });
  const auto fn = kind == 1 ? pkv_paged_tree_attention_fp8 : pkv_paged_tree_attention_e5m2;
  return status([&] {
    return fn(qp, static_cast<const uint8_t*>(kp), static_cast<const uint8_t*>(vp), ks, vs, tp, lp, cp, mp, words,
              max_nodes, tokens, b, hq, hkv, d, bs, width, nb, max_ctx, scale, op, dt, wp, bytes, err, s);
  });
}

// q, k_cache, v_cache, block_tables, context_lens, cu_seqlens, out, scale,
// max_query_len, window, num_sinks, dtype, err_flag, stream
PyObject* window_prefill(PyObject* const* a) {
  const at::Tensor &q = need(a[0], 3, "q must be [num_tokens, num_q_heads, head_dim]"), &kc = need(a[1], 4, kCacheDims),
                   &vc = need(a[2], -1, ""), &tab = need(a[3], 2, kTableDims), &len = need(a[4], -1, ""),
                   &cu = need(a[5], -1, ""), &out = need(a[6], -1, "");
  index_check(len);
  index_check(cu);
  index_check(tab);
  if (cu.numel() != len.numel() + 1)
    refuse(PyExc_ValueError, "cu_seqlens must have one entry more than context_lens");
  per_sequence(len.numel(), tab, len);
  contiguous(q);
  contiguous(out);
  caches_check(kc, vc, 2);
  if (out.sizes() != q.sizes()) refuse(PyExc_ValueError, "q and out differ in shape");
  if (kc.size(3) != q.size(2)) refuse(PyExc_ValueError, "q and the caches differ in head_dim");
  const Type16 type(q, a[11]);
  type.check(out);
  cache_type(kc, 0, type);
  flag_check(a[12]);
  const int64_t tokens = q.size(0), nb = kc.size(0);
  const int b = to_int(len.numel()), hq = to_int(q.size(1)), hkv = to_int(kc.size(1)), d = to_int(q.size(2)),
            bs = to_int(kc.size(2)), width = to_int(tab.size(1)), longest = number<int>(a[8]),
            window = number<int>(a[9]), sinks = number<int>(a[10]);
  const float scale = number<float>(a[7]);
  const pkv_dtype dt = type.code;
  void *qp = ptr(q), *kp = ptr(kc), *vp = ptr(vc), *op = ptr(out);
  const auto* tp = static_cast<const int32_t*>(ptr(tab));
  const auto* lp = static_cast<const int32_t*>(ptr(len));
  const auto* cp = static_cast<const int32_t*>(ptr(cu));
  auto* err = static_cast<int32_t*>(address(a[12]));
  void* s = stream_of(a[13]);
  return status([&] {
    return pkv_paged_prefill_attention_window(qp, kp, vp, tp, lp, cp, tokens, b, hq, hkv, d, bs, width, nb, longest,
                                              window, sinks, scale, op, dt, err, s);
  });
}

// k_cache, v_cache, block_tables, context_lens, cu_nodes, accepted, new_lens,
// err_flag, stream
PyObject* tree_commit(PyObject* const* a) {
  const at::Tensor &kc = need(a[0], -1, ""), &vc = need(a[1], -1, ""), &tab = need(a[2], 2, kTableDims),
                   &len = need(a[3], -1, ""), &cu = need(a[4], -1, ""),
                   &acc = need(a[5], 2, "accepted must be [batch, max_accept]");
  if (kc.dim() != 4 && kc.dim() != 5)
    refuse(PyExc_ValueError, "caches must be [num_blocks, num_kv_heads, 16, head_dim], or with num_layers second");
  const int b = drafted_batch(cu, len), n = static_cast<int>(kc.dim());
  index_check(tab);
  index_check(acc);
  per_sequence(b, tab, len);
  if (acc.size(0) != b) refuse(PyExc_ValueError, "accepted must have a row per sequence");
  if (kc.element_size() != 1 && kc.element_size() != 2)
    refuse(PyExc_TypeError, "caches must have elements of one or two bytes");
  caches_check(kc, vc, static_cast<int64_t>(kc.element_size()));
  if (a[6] != Py_None) {
    const at::Tensor& t = need(a[6], -1, "");
    index_check(t);
    if (t.numel() != b) refuse(PyExc_ValueError, "new_lens and context_lens differ in length");
  }
  flag_check(a[7]);
  const int64_t nb = kc.size(0);
  const int heads = to_int(n == 5 ? kc.size(1) * kc.size(2) : kc.size(1)), bs = to_int(kc.size(n - 2)),
            d = to_int(kc.size(n - 1)), elt = static_cast<int>(kc.element_size()), width = to_int(tab.size(1)),
            most = to_int(acc.size(1));
  void *kp = ptr(kc), *vp = ptr(vc);
  const auto* tp = static_cast<const int32_t*>(ptr(tab));
  const auto* lp = static_cast<const int32_t*>(ptr(len));
  const auto* cp = static_cast<const int32_t*>(ptr(cu));
  const auto* ap = static_cast<const int32_t*>(ptr(acc));
  auto* np = static_cast<int32_t*>(address(a[6]));
  auto* err = static_cast<int32_t*>(address(a[7]));
  void* s = stream_of(a[8]);
  return status([&] {
    return pkv_tree_commit(kp, vp, tp, lp, cp, ap, most, b, heads, d, bs, width, nb, elt, np, err, s);
  });
}

#define PKV_TENSOR_CALL(f, n) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<n, &f>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    PKV_TENSOR_CALL(rope_append, 17),
    PKV_TENSOR_CALL(block_bounds, 10),
    PKV_TENSOR_CALL(block_scores, 11),
    PKV_TENSOR_CALL(select_blocks, 7),
    PKV_TENSOR_CALL(sparse_decode, 15),
    PKV_TENSOR_CALL(prefix_decode, 15),
    PKV_TENSOR_CALL(window_decode, 16),
    PKV_TENSOR_CALL(window_prefill, 14),
    PKV_TENSOR_CALL(tree_plan, 10),
    PKV_TENSOR_CALL(tree_attention, 18),
    PKV_TENSOR_CALL(tree_commit, 9),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_tensor", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace
}  // namespace pkv_py

PyMODINIT_FUNC PyInit__tensor(void) { return PyModule_Create(&pkv_py::module_def); }
