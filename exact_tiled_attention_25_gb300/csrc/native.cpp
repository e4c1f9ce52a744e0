// Argument marshalling of the short calls, compiled: the functions of
// exact_tiled_attention_25_gb300 for cross attention, rotary positions, block tables
// and cache appends check tensor metadata, allocate outputs and call the C ABI
// here.  Their kernels take 3 to 10 us in a decode step; the same marshalling in
// Python with ctypes took 20 to 22 us a call on a Grace core, this 5 to 12.
//
// Each function takes its Python namesake's arguments, all positional, None for
// those left out, and leaves the computation to libattn_gb300.so.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/attn_gb300.h"

namespace {

struct Api {
#define ATTN_FN(name) decltype(&::name) name = nullptr
  ATTN_FN(attn_cross_workspace_size);
  ATTN_FN(attn_cross_fwd);
  ATTN_FN(attn_cross_bwd_workspace_size);
  ATTN_FN(attn_cross_bwd);
  ATTN_FN(attn_rope_table);
  ATTN_FN(attn_rope);
  ATTN_FN(attn_block_tables);
  ATTN_FN(attn_cache_append);
  ATTN_FN(attn_cache_append_fp8);
#undef ATTN_FN
} api;
PyObject* on_error = nullptr;      // called with (code, name); raises
PyObject* out_of_memory = nullptr; // torch.OutOfMemoryError

// A refused argument: becomes a ValueError.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
// A Python exception is already set.
struct Raised {};

void require(bool ok, const char* text) {
  if (!ok) throw Refused(text);
}

// An optional tensor argument.
struct Arg {
  const char* name;
  at::Tensor t;      // undefined: None
  Arg(const char* n, PyObject* o) : name(n) {
    if (o == Py_None) return;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s must be a tensor", n);
      throw Raised{};
    }
    t = THPVariable_Unpack(o);
  }
  explicit operator bool() const { return t.defined(); }
  void* ptr() const { return t.defined() ? t.data_ptr() : nullptr; }
  template <typename T>
  T* as() const { return static_cast<T*>(ptr()); }
  int64_t size(int i) const { return t.size(i); }
};

const Arg& given(const Arg& a) {
  if (!a) throw Refused(std::string(a.name) + " is missing");
  return a;
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

void like(const Arg& a, at::IntArrayRef shape, at::ScalarType type) {
  given(a);
  if (a.t.scalar_type() != type || a.t.sizes() != shape || !a.t.is_contiguous())
    throw Refused(std::string(a.name) + " must be contiguous " + c10::toString(type) + " " + shape_text(shape));
}

// The current CUDA device, where every tensor of a call has to be, and the call's
// stream.  Outputs and scratch are allocated as that stream's: freed scratch is not
// handed to another stream while the kernel that uses it may still run.
struct Device {
  c10::DeviceIndex index = -1;
  cudaStream_t stream = nullptr;
  bool other = false;      // not the current stream
  void check(const Arg& a) {
    if (!a) return;
    if (a.t.is_cuda() && index < 0) index = c10::cuda::current_device();
    if (!a.t.is_cuda() || a.t.get_device() != index)
      throw Refused(std::string(a.name) + " must be on the current CUDA device");
  }
  template <typename... A>
  explicit Device(PyObject* stream_arg, const A&... args) {
    (check(args), ...);
    if (index < 0) index = c10::cuda::current_device();
    stream = c10::cuda::getCurrentCUDAStream(index).stream();
    if (stream_arg == Py_None) return;
    PyObject* h = PyObject_GetAttrString(stream_arg, "cuda_stream");
    if (!h) throw Raised{};
    void* p = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (!p && PyErr_Occurred()) throw Raised{};
    other = static_cast<cudaStream_t>(p) != stream;
    stream = static_cast<cudaStream_t>(p);
  }
  // (straight from the allocator: the dispatcher takes half a microsecond a tensor)
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    const c10::Device on(c10::kCUDA, index);
    if (!other) return at::detail::empty_cuda(shape, type, on, std::nullopt);
    const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(stream, index));
    return at::detail::empty_cuda(shape, type, on, std::nullopt);
  }
  // Several small outputs, those not given as parts of one allocation (an allocation and
  // its release take most of a microsecond each).
  struct Wanted {
    Arg* a;
    std::vector<int64_t> shape;
    at::ScalarType type;
    size_t at = 0;
  };
  void outputs(std::vector<Wanted> all) const {
    size_t bytes = 0;
    for (Wanted& w : all) {
      if (*w.a) {
        like(*w.a, w.shape, w.type);
        continue;
      }
      w.at = bytes;
      bytes += (c10::multiply_integers(w.shape) * c10::elementSize(w.type) + 255) / 256 * 256;
    }
    at::Tensor whole;
    for (Wanted& w : all) {
      if (*w.a) continue;
      if (!whole.defined()) whole = empty({static_cast<int64_t>(bytes)}, at::kByte);
      w.a->t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                        c10::scalarTypeToTypeMeta(w.type));
      c10::TensorImpl* t = w.a->t.unsafeGetTensorImpl();
      t->set_sizes_contiguous(w.shape);
      t->set_storage_offset(static_cast<int64_t>(w.at / c10::elementSize(w.type)));
    }
  }
  // a given output of that shape and type, or a new one
  void output(Arg& a, at::IntArrayRef shape, at::ScalarType type) const {
    if (a) like(a, shape, type);
    else a.t = empty(shape, type);
  }
  void workspace(Arg& a, size_t bytes) const {
    if (!a && bytes > 0) a.t = empty({static_cast<int64_t>(bytes)}, at::kByte);
  }
};

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int small(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < -2147483648LL || v > 2147483647LL) throw Refused(std::string(name) + " out of range");
  return static_cast<int>(v);
}
int extent(int64_t n) {
  require(n <= 2147483647LL, "a dimension exceeds 2^31 - 1");
  return static_cast<int>(n);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}
float scale_of(PyObject* o, int d) {
  return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : static_cast<float>(number(o));
}

attn_dtype_t dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kHalf ? ATTN_FP16 : ATTN_BF16; }
bool is16(const at::Tensor& t) { return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16; }

// Run a C entry point without the interpreter's lock; a status other than 0 raises.  The
// lock is held again before an exception of f (a dimension out of range) leaves.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F>
void call(const char* name, F f) {
  attn_status_t s;
  {
    const Unlocked unlocked;
    s = f();
  }
  if (s == ATTN_OK) return;
  PyObject* r = PyObject_CallFunction(on_error, "is", static_cast<int>(s), name);
  Py_XDECREF(r);
  if (r) PyErr_Format(PyExc_RuntimeError, "%s failed with status %d", name, static_cast<int>(s));
  throw Raised{};
}

PyObject* tuple(std::initializer_list<const Arg*> out) {
  PyObject* r = PyTuple_New(out.size());
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const Arg* a : out) {
    PyObject* o = *a ? THPVariable_Wrap(a->t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

template <PyObject* (*Body)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return Body(a);
  } catch (const Raised&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(out_of_memory, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// ------------------------------------------------------------------ cross attention ----
struct CrossShape {
  int B, H, H_kv, N_q, N_k, d;
};
CrossShape cross_shape(const Arg& q, const Arg& k, const Arg& v, const Arg& lens) {
  for (const Arg* a : {&q, &k, &v}) {
    if (given(*a).t.dim() != 4) throw Refused(std::string(a->name) + " must be [B, H, N, d]");
    if (!a->t.is_contiguous()) throw Refused(std::string(a->name) + " must be contiguous");
  }
  require(k.size(0) == q.size(0) && k.size(3) == q.size(3) && v.t.sizes() == k.t.sizes(),
          "k and v must be [B, H_kv, N_k, d] with q's B and d");
  require(is16(q.t) && k.t.scalar_type() == q.t.scalar_type() && v.t.scalar_type() == q.t.scalar_type(),
          "q, k, v must all be bfloat16 or all float16");
  if (lens) like(lens, {q.size(0)}, at::kInt);
  return {extent(q.size(0)), extent(q.size(1)), extent(k.size(1)), extent(q.size(2)), extent(k.size(2)),
          extent(q.size(3))};
}

PyObject* cross_fwd(PyObject* const* a) {
  Arg q("q", a[0]), k("k", a[1]), v("v", a[2]), lens("kv_lens", a[3]), o("o", a[5]), lse("lse", a[6]), ws("workspace", a[7]);
  const CrossShape s = cross_shape(q, k, v, lens);
  const float scale = scale_of(a[4], s.d);
  const Device dev(a[8], q, k, v, lens, o, lse, ws);
  dev.output(o, q.t.sizes(), q.t.scalar_type());
  dev.output(lse, {s.B, s.H, s.N_q}, at::kFloat);
  dev.workspace(ws, api.attn_cross_workspace_size(s.B, s.H, s.H_kv, s.N_q, s.N_k, s.d));
  call("attn_cross_fwd", [&] {
    return api.attn_cross_fwd(q.ptr(), k.ptr(), v.ptr(), lens.as<int>(), o.ptr(), lse.as<float>(), ws.ptr(),
                              ws ? ws.t.nbytes() : 0, s.B, s.H, s.H_kv, s.N_q, s.N_k, s.d, scale, dtype_of(q.t), dev.stream);
  });
  return tuple({&o, &lse});
}

PyObject* cross_bwd(PyObject* const* a) {
  Arg q("q", a[0]), k("k", a[1]), v("v", a[2]), o("o", a[3]), dout("dout", a[4]), lse("lse", a[5]), lens("kv_lens", a[6]),
      dq("dq", a[8]), dk("dk", a[9]), dv("dv", a[10]), ws("workspace", a[11]);
  const CrossShape s = cross_shape(q, k, v, lens);
  like(o, q.t.sizes(), q.t.scalar_type());
  like(dout, q.t.sizes(), q.t.scalar_type());
  like(lse, {s.B, s.H, s.N_q}, at::kFloat);
  const float scale = scale_of(a[7], s.d);
  const Device dev(a[12], q, k, v, o, dout, lse, lens, dq, dk, dv, ws);
  dev.output(dq, q.t.sizes(), q.t.scalar_type());
  dev.output(dk, k.t.sizes(), q.t.scalar_type());
  dev.output(dv, k.t.sizes(), q.t.scalar_type());
  dev.workspace(ws, api.attn_cross_bwd_workspace_size(s.B, s.H, s.N_q, s.N_k, s.d));
  call("attn_cross_bwd", [&] {
    return api.attn_cross_bwd(q.ptr(), k.ptr(), v.ptr(), o.ptr(), dout.ptr(), lse.as<float>(), lens.as<int>(), dq.ptr(),
                              dk.ptr(), dv.ptr(), ws.ptr(), ws ? ws.t.nbytes() : 0, s.B, s.H, s.H_kv, s.N_q, s.N_k, s.d,
                              scale, dtype_of(q.t), dev.stream);
  });
  return tuple({&dq, &dk, &dv});
}

// ------------------------------------------------------------------- rotary ----
// (max_pos, rot_dim) of a pair of tables, {0, 0} without.
struct Tables {
  int max_pos = 0, rot = 0;
  Tables(const Arg& cos, const Arg& sin) {
    if (!cos && !sin) return;
    require(cos && sin, "give both rope_cos and rope_sin, or neither");
    require(cos.t.dim() == 2, "rope_cos must be [positions, rot_dim / 2]");
    like(cos, cos.t.sizes(), at::kFloat);
    like(sin, cos.t.sizes(), at::kFloat);
    max_pos = extent(cos.size(0));
    rot = extent(2 * cos.size(1));
  }
};

// Stride of dimension i of a tensor of contiguous rows; a dimension of extent 1 may
// have any, and is given a row's length.
long long row_stride(const Arg& a, int i) { return a.size(i) > 1 ? a.t.stride(i) : a.size(a.t.dim() - 1); }
void rows_contiguous(const Arg& a) {
  if (a.t.stride(-1) != 1) throw Refused(std::string(a.name) + "'s rows must be contiguous");
}
struct Strides3 {
  long long s[3];      // batch, head, token
  Strides3(const Arg& a, bool packed) {
    rows_contiguous(a);
    if (packed) {
      s[0] = a.size(2);
      s[1] = row_stride(a, 1);
      s[2] = row_stride(a, 0);
    } else {
      for (int i = 0; i < 3; ++i) s[i] = row_stride(a, i);
    }
  }
};

PyObject* rope_table(PyObject* const* a) {
  const long long n = integer(a[0]);
  const int rot = small(a[1], "rot_dim");
  require(n >= 1 && rot >= 2, "n and rot_dim must be positive");
  const double base = number(a[2]), factor = number(a[3]), low = number(a[5]), high = number(a[6]), attn = number(a[7]);
  const long long orig = integer(a[4]), first = integer(a[8]);
  Arg cos("rope_cos", a[9]), sin("rope_sin", a[10]);
  if (cos) like(cos, {n, rot / 2}, at::kFloat);
  if (sin) like(sin, {n, rot / 2}, at::kFloat);
  const Device dev(a[11], cos, sin);
  dev.output(cos, {n, rot / 2}, at::kFloat);
  dev.output(sin, {n, rot / 2}, at::kFloat);
  call("attn_rope_table", [&] {
    return api.attn_rope_table(cos.as<float>(), sin.as<float>(), n, rot, base, factor, orig, low, high, attn, first, dev.stream);
  });
  return tuple({&cos, &sin});
}

PyObject* rope(PyObject* const* a) {
  Arg q("q", a[0]), k("k", a[1]), cos("rope_cos", a[2]), sin("rope_sin", a[3]), pos("positions", a[4]), qo("q_out", a[7]),
      ko("k_out", a[8]);
  given(cos);
  const Tables tab(cos, sin);
  given(q);
  const bool packed = q.t.dim() == 3;
  require(packed || q.t.dim() == 4, "q must be [B, H, N, d] or packed [total, H, d]");
  require(is16(q.t), "q and k must be bfloat16 or float16");
  require(q.t.numel() > 0, "q is empty");
  const int64_t B = packed ? 1 : q.size(0), H = q.size(1), N = packed ? q.size(0) : q.size(2), d = q.size(-1);
  int64_t H_kv = 0;
  if (k) {
    require(k.t.dim() == q.t.dim(), "k must match q in dtype and shape, up to its heads");
    H_kv = k.size(1);
    const bool same = packed ? k.t.sizes() == at::IntArrayRef({N, H_kv, d}) : k.t.sizes() == at::IntArrayRef({B, H_kv, N, d});
    require(same && k.t.scalar_type() == q.t.scalar_type(), "k must match q in dtype and shape, up to its heads");
  }
  require(k || !ko, "k_out without k");
  if (pos) {
    if (packed) like(pos, {N}, at::kInt);
    else like(pos, {B, N}, at::kInt);
  }
  for (auto* x : {&qo, &ko}) {
    const Arg& in = x == &qo ? q : k;
    if (*x && (x->t.sizes() != in.t.sizes() || x->t.scalar_type() != in.t.scalar_type()))
      throw Refused(std::string(x->name) + " must match its input in shape and dtype");
  }
  const Device dev(a[9], q, k, cos, sin, pos, qo, ko);
  if (!qo) qo.t = dev.empty(q.t.sizes(), q.t.scalar_type());
  if (k && !ko) ko.t = dev.empty(k.t.sizes(), q.t.scalar_type());
  const Strides3 sq(q, packed), sqo(qo, packed), sk(k ? k : q, packed), sko(k ? ko : qo, packed);
  const int inter = truth(a[5]), inv = truth(a[6]);
  call("attn_rope", [&] {
    return api.attn_rope(q.ptr(), qo.ptr(), k.ptr(), ko.ptr(), cos.as<float>(), sin.as<float>(), pos.as<int>(),
                         extent(B), extent(N), extent(H), extent(H_kv), extent(d), tab.rot, tab.max_pos, sq.s, sqo.s, sk.s,
                         sko.s, inter, inv, dtype_of(q.t), dev.stream);
  });
  return tuple({&qo, &ko});
}

// -------------------------------------------------------------------- cache ----
PyObject* block_tables(PyObject* const* a) {
  Arg bt("block_table", a[0]), old("old_lens", a[1]), add("new_lens", a[2]), free_("free_pages", a[3]), lens("seq_lens", a[6]),
      cu("cu_seqlens", a[7]), slots("slots", a[8]), pos("positions", a[9]), used("used", a[10]);
  const int page = small(a[4], "page_size"), cap = small(a[5], "capacity");
  require(given(bt).t.dim() == 2 && given(free_).t.dim() == 1, "block_table must be [B, max_pages] and free_pages a vector");
  require(cap >= 0, "capacity must be >= 0");
  const int B = extent(bt.size(0)), max_pages = extent(bt.size(1));
  like(bt, bt.t.sizes(), at::kInt);
  like(old, {B}, at::kInt);
  like(add, {B}, at::kInt);
  like(free_, free_.t.sizes(), at::kInt);
  const Device dev(a[11], bt, old, add, free_, lens, cu, slots, pos, used);
  dev.outputs({{&lens, {B}, at::kInt},
               {&cu, {B + 1}, at::kInt},
               {&slots, {cap}, at::kLong},
               {&pos, {cap}, at::kInt},
               {&used, {1}, at::kInt}});
  call("attn_block_tables", [&] {
    return api.attn_block_tables(bt.as<int>(), old.as<int>(), add.as<int>(), free_.as<int>(), lens.as<int>(), cu.as<int>(),
                                 slots.as<long long>(), pos.as<int>(), used.as<int>(), B, max_pages, extent(free_.size(0)),
                                 page, cap, dev.stream);
  });
  return tuple({&lens, &cu, &slots, &pos, &used});
}

// Sizes and {token, head} strides of an append: k, v [total, H_kv, d], q [total, H, d].
struct Rows {
  int total, H = 0, H_kv, d;
  long long qs[2] = {0, 0}, ks[2], vs[2];
  Rows(const Arg& k, const Arg& v, const Arg& q, const Arg& qo, const Arg& cache) {
    require(given(k).t.dim() == 3 && given(v).t.sizes() == k.t.sizes() && is16(k.t) && v.t.scalar_type() == k.t.scalar_type(),
            "k and v must be bfloat16 or float16 [total, H_kv, d]");
    total = extent(k.size(0)), H_kv = extent(k.size(1)), d = extent(k.size(2));
    require(given(cache).t.dim() == 4 && cache.size(2) == H_kv && cache.size(3) == d,
            "the caches must be [num_pages, page_size, H_kv, d]");
    strides(k, ks);
    strides(v, vs);
    require(q || !qo, "q_out without q");
    if (q) {
      require(q.t.dim() == 3 && q.size(0) == total && q.size(2) == d && q.t.scalar_type() == k.t.scalar_type(),
              "q must be [total, H, d] in k's dtype");
      H = extent(q.size(1));
      strides(q, qs);
    }
  }
  static void strides(const Arg& a, long long* s) {
    rows_contiguous(a);
    s[0] = row_stride(a, 0);
    s[1] = row_stride(a, 1);
  }
};

PyObject* cache_append(PyObject* const* a) {
  Arg k("k", a[0]), v("v", a[1]), kc("k_cache", a[2]), vc("v_cache", a[3]), slots("slots", a[4]), cos("rope_cos", a[5]),
      sin("rope_sin", a[6]), pos("positions", a[7]), q("q", a[8]), qo("q_out", a[10]);
  const Rows r(k, v, q, qo, kc);
  like(kc, kc.t.sizes(), k.t.scalar_type());
  like(vc, kc.t.sizes(), k.t.scalar_type());
  like(slots, {r.total}, at::kLong);
  const Tables tab(cos, sin);
  if (cos) {
    require(static_cast<bool>(pos), "rotation needs positions");
    like(pos, {r.total}, at::kInt);
  }
  const Device dev(a[11], k, v, kc, vc, slots, cos, sin, pos, q, qo);
  if (q) dev.output(qo, {r.total, r.H, r.d}, k.t.scalar_type());
  const int inter = truth(a[9]);
  call("attn_cache_append", [&] {
    return api.attn_cache_append(q.ptr(), qo.ptr(), k.ptr(), v.ptr(), kc.ptr(), vc.ptr(), slots.as<long long>(),
                                 cos.as<float>(), sin.as<float>(), pos.as<int>(), r.total, r.H, r.H_kv, r.d, tab.rot,
                                 tab.max_pos, extent(kc.size(0)), extent(kc.size(1)), r.qs, r.ks, r.vs, inter,
                                 dtype_of(k.t), dev.stream);
  });
  return qo ? THPVariable_Wrap(qo.t) : Py_NewRef(Py_None);
}

PyObject* cache_append_fp8(PyObject* const* a) {
  Arg k("k", a[0]), v("v", a[1]), kc("k_cache", a[2]), vc("v_cache", a[3]), kd("k_descale", a[4]), vd("v_descale", a[5]),
      bt("block_table", a[6]), lens("seq_lens", a[7]), cu("cu_seqlens", a[8]), cos("rope_cos", a[9]), sin("rope_sin", a[10]),
      signs("hadamard_signs", a[11]), q("q", a[12]), qo("q_out", a[14]);
  const Rows r(k, v, q, qo, kc);
  like(kc, kc.t.sizes(), at::kByte);
  like(vc, kc.t.sizes(), at::kByte);
  like(kd, {kc.size(0), r.H_kv}, at::kFloat);
  like(vd, {kc.size(0), r.H_kv}, at::kFloat);
  require(given(bt).t.dim() == 2, "block_table must be [B, max_pages]");
  const int B = extent(bt.size(0));
  like(bt, bt.t.sizes(), at::kInt);
  like(lens, {B}, at::kInt);
  like(cu, {B + 1}, at::kInt);
  if (signs) like(signs, {r.d}, at::kFloat);
  const Tables tab(cos, sin);
  const Device dev(a[15], k, v, kc, vc, kd, vd, bt, lens, cu, cos, sin, signs, q, qo);
  if (q) dev.output(qo, {r.total, r.H, r.d}, k.t.scalar_type());
  const int inter = truth(a[13]);
  call("attn_cache_append_fp8", [&] {
    return api.attn_cache_append_fp8(q.ptr(), qo.ptr(), k.ptr(), v.ptr(), kc.as<uint8_t>(), vc.as<uint8_t>(),
                                     kd.as<float>(), vd.as<float>(), bt.as<int>(), lens.as<int>(), cu.as<int>(),
                                     cos.as<float>(), sin.as<float>(), signs.as<float>(), B, r.total, r.H, r.H_kv, r.d,
                                     tab.rot, tab.max_pos, extent(kc.size(0)), extent(kc.size(1)), extent(bt.size(1)),
                                     r.qs, r.ks, r.vs, inter, dtype_of(k.t), dev.stream);
  });
  return qo ? THPVariable_Wrap(qo.t) : Py_NewRef(Py_None);
}

// bind(path of libattn_gb300.so, on_error): before any other call.
PyObject* bind(PyObject* const* a) {
  const char* path = PyUnicode_AsUTF8(a[0]);
  if (!path) throw Raised{};
  void* lib = dlopen(path, RTLD_NOW);
  if (!lib) throw std::runtime_error(dlerror());
#define ATTN_FN(name)                                                       \
  api.name = reinterpret_cast<decltype(&::name)>(dlsym(lib, #name));        \
  if (!api.name) throw std::runtime_error("libattn_gb300.so lacks " #name)
  ATTN_FN(attn_cross_workspace_size);
  ATTN_FN(attn_cross_fwd);
  ATTN_FN(attn_cross_bwd_workspace_size);
  ATTN_FN(attn_cross_bwd);
  ATTN_FN(attn_rope_table);
  ATTN_FN(attn_rope);
  ATTN_FN(attn_block_tables);
  ATTN_FN(attn_cache_append);
  ATTN_FN(attn_cache_append_fp8);
#undef ATTN_FN
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
  Py_XDECREF(torch);
  if (!type) throw Raised{};
  Py_XSETREF(out_of_memory, type);
  Py_XSETREF(on_error, Py_NewRef(a[1]));
  return Py_NewRef(Py_None);
}

#define ATTN_METHOD(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<&name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    ATTN_METHOD(bind, 2),        ATTN_METHOD(cross_fwd, 9),     ATTN_METHOD(cross_bwd, 13),
    ATTN_METHOD(rope_table, 12), ATTN_METHOD(rope, 10),         ATTN_METHOD(block_tables, 12),
    ATTN_METHOD(cache_append, 12), ATTN_METHOD(cache_append_fp8, 16), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
