// Argument marshalling of the cache, latent and long-cache calls as a CPython extension: checks of
// tensors against one another, outputs and workspaces that the caller left out, and the C
// ABI call.  A decode step's kernels take a few microseconds and so does a Python
// function that looks at nine tensors (5 to 11 us here, against 0.5 us); nothing is
// computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/decode_attn.h"

namespace {

using at::Tensor;
constexpr int64_t kLatentRope = 64;

template <typename... I>
std::array<int64_t, sizeof...(I)> dims(I... n) {
  return {(int64_t)n...};
}

// Becomes a ValueError.
struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};
// Becomes the binding's DecodeAttnError (entry point, status).
struct Failed {
  const char* fn;
  int status;
};

struct Library {
  void* handle = nullptr;
  decltype(&::rope_apply) rope_apply = nullptr;
  decltype(&::kv_write_contig) kv_write_contig = nullptr;
  decltype(&::kv_write_paged) kv_write_paged = nullptr;
  decltype(&::kv_write_int8_contig) kv_write_int8_contig = nullptr;
  decltype(&::kv_write_int8_paged) kv_write_int8_paged = nullptr;
  decltype(&::kv_read_paged) kv_read_paged = nullptr;
  decltype(&::kv_read_int8_contig) kv_read_int8_contig = nullptr;
  decltype(&::kv_read_int8_paged) kv_read_int8_paged = nullptr;
  decltype(&::kv_read_paged_filled) kv_read_paged_filled = nullptr;
  decltype(&::kv_read_int8_contig_filled) kv_read_int8_contig_filled = nullptr;
  decltype(&::kv_read_int8_paged_filled) kv_read_int8_paged_filled = nullptr;
  decltype(&::latent_attn_contig) latent_attn_contig = nullptr;
  decltype(&::latent_attn_paged) latent_attn_paged = nullptr;
  decltype(&::latent_workspace_bytes) latent_workspace_bytes = nullptr;
  decltype(&::latent_prefill_contig) latent_prefill_contig = nullptr;
  decltype(&::latent_prefill_workspace_bytes) latent_prefill_workspace_bytes = nullptr;
  decltype(&::prefix_attn_contig) prefix_attn_contig = nullptr;
  decltype(&::prefix_attn_paged) prefix_attn_paged = nullptr;
  decltype(&::prefix_attn_workspace_bytes) prefix_attn_workspace_bytes = nullptr;
  decltype(&::block_means_contig) block_means_contig = nullptr;
  decltype(&::block_means_paged) block_means_paged = nullptr;
  decltype(&::block_select) block_select = nullptr;
  decltype(&::sparse_attn_contig) sparse_attn_contig = nullptr;
  decltype(&::sparse_attn_paged) sparse_attn_paged = nullptr;
  decltype(&::kv_weights_contig) kv_weights_contig = nullptr;
  decltype(&::kv_weights_paged) kv_weights_paged = nullptr;
  decltype(&::kv_weights_int8_contig) kv_weights_int8_contig = nullptr;
  decltype(&::kv_weights_int8_paged) kv_weights_int8_paged = nullptr;
  decltype(&::kv_weights_workspace_bytes) kv_weights_workspace_bytes = nullptr;
  decltype(&::kv_evict_contig) kv_evict_contig = nullptr;
  decltype(&::kv_evict_paged) kv_evict_paged = nullptr;
  decltype(&::kv_evict_int8_contig) kv_evict_int8_contig = nullptr;
  decltype(&::kv_evict_int8_paged) kv_evict_int8_paged = nullptr;
};
Library g_lib;
PyObject* g_error = nullptr;  // DecodeAttnError

// ---------------------------------------------------------------- arguments

const Tensor* opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Bad(std::string(name) + ": expected a tensor or None");
  return &THPVariable_Unpack(o);
}

const Tensor& ten(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Bad(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// An int argument of the C ABI.
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Bad(std::string(name) + ": does not fit 32 bits");
  return (int)v;
}
int small(int64_t v, const char* name) {
  if (v > INT32_MAX) throw Bad(std::string(name) + ": a size does not fit 32 bits");
  return (int)v;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}

int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}

[[noreturn]] void mismatch(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int64_t dev,
                           const char* how) {
  std::ostringstream s;
  s << name << ": expected a " << how << type << " tensor of shape " << shape << " on cuda:" << dev << ", got "
    << t.scalar_type() << " " << t.sizes() << ", strides " << t.strides() << ", on " << t.device();
  throw Bad(s.str());
}

int64_t cuda_index(const Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

// t must be a contiguous tensor of this type and shape on device dev.
void plain(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int64_t dev) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || cuda_index(t) != dev)
    mismatch(t, name, type, shape, dev, "contiguous ");
}

// The library launches on the current device: the tensors' device must be that one.
void on_current(int64_t dev) {
  if (dev < 0) throw Bad("expected tensors on the current CUDA device, got them on the CPU");
  if (dev != c10::cuda::current_device())
    throw Bad("expected tensors on the current CUDA device, got them on cuda:" + std::to_string(dev));
}

// The stream of a call; what the call allocates belongs to that stream.
struct Stream {
  cudaStream_t raw;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  Stream(PyObject* o, int64_t dev) {
    if (o == Py_None) {
      raw = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    } else {
      PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
      if (!h) throw python_error();
      raw = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
      Py_DECREF(h);
      if (PyErr_Occurred()) throw python_error();
      guard.emplace(c10::cuda::getStreamFromExternal(raw, (c10::DeviceIndex)dev));
    }
  }
};

template <typename T = void>
T* ptr(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
template <typename T = void>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// Elements from one token to the next of t [.., H, D] (lead leading dims that are one run of
// tokens), a head's elements consecutive.
int64_t token_stride(const Tensor& t, const char* name, int lead) {
  const auto sz = t.sizes();
  const auto st = t.strides();
  const int64_t D = sz[lead + 1];
  bool ok = D <= 1 || st[lead + 1] == 1;
  int64_t step = st[lead - 1];
  if (lead == 2 && sz[0] > 1 && sz[1] > 0) {
    if (sz[1] > 1)
      ok = ok && st[0] == sz[1] * st[1];
    else
      step = st[0];
  }
  if (!ok) {
    std::ostringstream s;
    s << name << ": tokens must be equally far apart and a head's elements consecutive, got strides " << st
      << " of shape " << sz;
    throw Bad(s.str());
  }
  return step;
}

// The C ABI call, without the GIL: f neither throws nor touches Python.
template <typename F>
void call(const char* fn, F f) {
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  if (st != DA_OK) throw Failed{fn, st};
}

// The call has written t (null: nothing): autograd notices where it had saved it.
void written(const Tensor* t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// Autograd records none of these calls, so what it tracks cannot be written by one.
void not_tracked(const Tensor* t, const char* name) {
  if (t && t->requires_grad() && at::GradMode::is_enabled())
    throw Bad(std::string(name) + ": it requires a gradient, and autograd does not record this call; write into a "
              "detached tensor or under torch.no_grad()");
}

void need_library() {
  if (!g_lib.handle) throw std::runtime_error("the library is not open");
}

// Runs a method's body: its exceptions become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  HANDLE_TH_ERRORS
  try {
    if (got != want) throw std::runtime_error("wrong number of arguments");
    need_library();
    return body();
  } catch (const Bad& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Failed& e) {
    PyObject* x = PyObject_CallFunction(g_error, "si", e.fn, e.status);
    if (x) {
      PyErr_SetObject(g_error, x);
      Py_DECREF(x);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// ---------------------------------------------------------------- rope_apply

// (x, positions, inv_freq, offset, interleaved, magnitude, backward, out, stream)
PyObject* rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Tensor &x = ten(a[0], "x"), &positions = ten(a[1], "positions"), &w = ten(a[2], "inv_freq");
    const auto type = x.scalar_type();
    const int dtype = type == at::kBFloat16 ? DA_BF16 : type == at::kHalf ? DA_F16 : type == at::kFloat ? DA_F32 : -1;
    const int lead = (int)x.dim() - 2;
    if (dtype < 0 || (lead != 1 && lead != 2)) {
      std::ostringstream s;
      s << "x: expected bf16, fp16 or fp32 [T, H, D] or [B, T, H, D], got " << type << " " << x.sizes();
      throw Bad(s.str());
    }
    const auto shape = x.sizes();
    const int64_t dev = cuda_index(x), H = shape[lead], D = shape[lead + 1];
    plain(positions, "positions", at::kInt, shape.slice(0, lead), dev);
    const int64_t rot = w.dim() == 1 ? w.size(0) : -1;
    plain(w, "inv_freq", at::kDouble, dims(std::max<int64_t>(rot, 0)), dev);
    const Tensor* given = opt(a[7], "out");
    if (given && (given->scalar_type() != type || given->sizes() != shape || cuda_index(*given) != dev))
      mismatch(*given, "out", type, shape, dev, "");
    not_tracked(given, "out");
    const int64_t xt = token_stride(x, "x", lead), ot = given ? token_stride(*given, "out", lead) : H * D;
    on_current(dev);
    Stream st(a[8], dev);
    const Tensor out = given ? *given : at::empty(shape, x.options());
    const int64_t oh = given ? out.strides()[lead] : D, xh = x.strides()[lead];
    const int off = small(a[3], "offset"), il = truth(a[4]), back = truth(a[6]);
    const int Hi = small(H, "x"), Di = small(D, "x"), roti = small(2 * rot, "inv_freq");
    const float mag = real(a[5]);
    call("rope_apply", [&] {
      return g_lib.rope_apply(ptr(x), ptr(out), ptr<int>(positions), ptr<double>(w), positions.numel(), Hi, Di, off,
                              roti, il, mag, back, dtype, xt, xh, ot, oh, st.raw);
    });
    written(given);
    return given ? same(a[7]) : THPVariable_Wrap(out);
  });
}

// ---------------------------------------------------------------- caches

struct Cache {
  int64_t slabs, slab, cols;
  bool paged, int8;
};

// Checks a cache of batch B and its lengths against the call's heads.
Cache check_cache(const Tensor& k, const Tensor* v, const Tensor* ks, const Tensor* vs, const Tensor* table,
                  const Tensor* lens, int64_t B, int64_t H, int64_t D, int64_t dev) {
  if (k.dim() != 4) throw Bad("k: expected 4 dims");
  Cache c{table ? k.size(0) : B, k.size(1), 0, table != nullptr, ks != nullptr};
  if (table) {
    c.cols = table->dim() == 2 ? table->size(1) : 0;
    plain(*table, "page_table", at::kInt, dims(B, c.cols), dev);
    if (!lens) throw Bad("seq_lens: a paged cache needs them");
  }
  if (lens) plain(*lens, "seq_lens", at::kInt, dims(B), dev);
  const auto type = c.int8 ? at::kChar : at::kBFloat16;
  plain(k, "k", type, dims(c.slabs, c.slab, H, D), dev);
  if (v) plain(*v, "v", type, dims(c.slabs, c.slab, H, D), dev);
  if (c.int8) {
    plain(*ks, "k_scale", at::kFloat, dims(c.slabs, H, c.slab), dev);
    if (v) {
      if (!vs) throw Bad("v: an int8 cache needs its scales");
      plain(*vs, "v_scale", at::kFloat, dims(c.slabs, H, c.slab), dev);
    }
  }
  return c;
}

// The token stride of new tokens [B, q_len, H, D], a token's heads consecutive.
int64_t new_tokens(const Tensor& t, const char* name, at::IntArrayRef shape, int64_t dev) {
  if (shape.size() != 4 || t.scalar_type() != at::kBFloat16 || t.sizes() != shape || cuda_index(t) != dev)
    mismatch(t, name, at::kBFloat16, shape, dev, "4-dim ");
  const int64_t H = shape[2], D = shape[3];
  if (H > 1 && t.stride(2) != D) throw Bad(std::string(name) + ": a token's heads must be consecutive");
  const int64_t step = token_stride(t, name, 2);
  return shape[0] * shape[1] > 1 ? step : H * D;
}

// (k_new, v_new, k, v, k_scale, v_scale, page_table, seq_lens, max_seq_len, inv_freq, offset, interleaved,
//  magnitude, stream)
PyObject* kv_write(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 14, [&]() -> PyObject* {
    const Tensor &k_new = ten(a[0], "k_new"), &k = ten(a[2], "k");
    const Tensor *v_new = opt(a[1], "v_new"), *v = opt(a[3], "v"), *ks = opt(a[4], "k_scale"),
                 *vs = opt(a[5], "v_scale"), *table = opt(a[6], "page_table"), *lens = opt(a[7], "seq_lens"),
                 *w = opt(a[9], "inv_freq");
    const int64_t dev = cuda_index(k_new);
    const auto shape = k_new.sizes();
    const int64_t kst = new_tokens(k_new, "k_new", shape, dev);
    if (!v_new != !v) throw Bad("v_new and v: both tensors, or both None to write keys only");
    const int64_t vst = v_new ? new_tokens(*v_new, "v_new", shape, dev) : 0;
    const int B = small(shape[0], "k_new"), n = small(shape[1], "k_new"), H = small(shape[2], "k_new"),
              D = small(shape[3], "k_new");
    const Cache c = check_cache(k, v, ks, vs, table, lens, B, H, D, dev);
    int rot = 0, off = 0, il = 0;
    float mag = 1.f;
    if (w) {
      const int64_t np = w->dim() == 1 ? w->size(0) : 0;
      plain(*w, "inv_freq", at::kDouble, dims(np), dev);
      rot = small(2 * np, "inv_freq");
      off = small(a[10], "offset");
      il = truth(a[11]);
      mag = real(a[12]);
    }
    not_tracked(&k, "k");
    not_tracked(v, "v");
    not_tracked(ks, "k_scale");
    not_tracked(vs, "v_scale");
    on_current(dev);
    Stream st(a[13], dev);
    const int slab = small(c.slab, "k"), cols = small(c.cols, "page_table"), slabs = small(c.slabs, "k");
    const double* wp = ptr<double>(w);
    if (c.paged) {
      const int cap = small(a[8], "max_seq_len");
      if (c.int8)
        call("kv_write_int8_paged", [&] {
          return g_lib.kv_write_int8_paged(ptr(k_new), ptr(v_new), kst, vst, ptr<int>(table), ptr<int>(lens), B, n, H, D,
                                           slab, cols, slabs, cap, wp, off, rot, il, mag, ptr(k), ptr(v), ptr<float>(ks),
                                           ptr<float>(vs), st.raw);
        });
      else
        call("kv_write_paged", [&] {
          return g_lib.kv_write_paged(ptr(k_new), ptr(v_new), kst, vst, ptr<int>(table), ptr<int>(lens), B, n, H, D,
                                      slab, cols, slabs, cap, wp, off, rot, il, mag, ptr(k), ptr(v), st.raw);
        });
    } else if (c.int8) {
      call("kv_write_int8_contig", [&] {
        return g_lib.kv_write_int8_contig(ptr(k_new), ptr(v_new), kst, vst, ptr<int>(lens), B, n, H, D, slab, wp, off,
                                          rot, il, mag, ptr(k), ptr(v), ptr<float>(ks), ptr<float>(vs), st.raw);
      });
    } else {
      call("kv_write_contig", [&] {
        return g_lib.kv_write_contig(ptr(k_new), ptr(v_new), kst, vst, ptr<int>(lens), B, n, H, D, slab, wp, off, rot,
                                     il, mag, ptr(k), ptr(v), st.raw);
      });
    }
    for (const Tensor* t : {&k, v, ks, vs}) written(t);
    Py_RETURN_NONE;
  });
}

// (k, v, k_scale, v_scale, page_table, seq_lens, max_seq_len, n_tokens, starts, k_out, v_out, stream,
//  zero_rest)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 13, [&]() -> PyObject* {
    const Tensor& k = ten(a[0], "k");
    const Tensor *v = opt(a[1], "v"), *ks = opt(a[2], "k_scale"), *vs = opt(a[3], "v_scale"),
                 *table = opt(a[4], "page_table"), *lens = opt(a[5], "seq_lens"), *starts = opt(a[8], "starts"),
                 *ko = opt(a[9], "k_out"), *vo = opt(a[10], "v_out");
    if (k.dim() != 4 || (table && table->dim() != 2)) throw Bad("k, page_table: expected 4 and 2 dims");
    const int64_t dev = cuda_index(k);
    const int B = small(table ? table->size(0) : k.size(0), "k"), H = small(k.size(2), "k"), D = small(k.size(3), "k"),
              n = small(a[7], "n_tokens");
    const Cache c = check_cache(k, v, ks, vs, table, lens, B, H, D, dev);
    if (starts) plain(*starts, "starts", at::kInt, dims(B), dev);
    if (n < 0) throw Bad("n_tokens: negative");
    if (ko) plain(*ko, "k_out", at::kBFloat16, dims(B, n, H, D), dev);
    if (!v && vo) throw Bad("v_out: no v to read");
    if (vo) plain(*vo, "v_out", at::kBFloat16, dims(B, n, H, D), dev);
    not_tracked(ko, "k_out");
    not_tracked(vo, "v_out");
    on_current(dev);
    Stream st(a[11], dev);
    const auto opts = k.options().dtype(at::kBFloat16);
    // outputs made here hold zeros where no token lies; a given one only when the caller asks for it
    const bool fill = truth(a[12]) || (!ko && !vo);
    auto make = [&] { return fill ? at::empty(dims(B, n, H, D), opts) : at::zeros(dims(B, n, H, D), opts); };
    const Tensor kt = ko ? *ko : make();
    const Tensor vt = vo ? *vo : v ? make() : Tensor();
    void* vp = v ? vt.data_ptr() : nullptr;
    const int slab = small(c.slab, "k"), cols = small(c.cols, "page_table"), slabs = small(c.slabs, "k");
    if (!c.paged) {
      call("kv_read_int8_contig", [&] {
        auto f = fill ? g_lib.kv_read_int8_contig_filled : g_lib.kv_read_int8_contig;
        return f(ptr(k), ptr(v), ptr<float>(ks), ptr<float>(vs), ptr<int>(starts),
                                         ptr<int>(lens), B, n, H, D, slab, ptr(kt), vp, st.raw);
      });
    } else {
      const int cap = small(a[6], "max_seq_len");
      if (c.int8)
        call("kv_read_int8_paged", [&] {
          auto f = fill ? g_lib.kv_read_int8_paged_filled : g_lib.kv_read_int8_paged;
          return f(ptr(k), ptr(v), ptr<float>(ks), ptr<float>(vs), ptr<int>(table),
                                          ptr<int>(starts), ptr<int>(lens), B, n, H, D, slab, cols, slabs, cap, ptr(kt),
                                          vp, st.raw);
        });
      else
        call("kv_read_paged", [&] {
          auto f = fill ? g_lib.kv_read_paged_filled : g_lib.kv_read_paged;
          return f(ptr(k), ptr(v), ptr<int>(table), ptr<int>(starts), ptr<int>(lens), B, n, H, D,
                                     slab, cols, slabs, cap, ptr(kt), vp, st.raw);
        });
    }
    written(ko);
    written(vo);
    PyObject* kr = ko ? same(a[9]) : THPVariable_Wrap(kt);
    PyObject* vr = vo || !v ? same(a[10]) : THPVariable_Wrap(vt);
    PyObject* r = kr && vr ? PyTuple_Pack(2, kr, vr) : nullptr;
    Py_XDECREF(kr);
    Py_XDECREF(vr);
    return r;
  });
}

// ---------------------------------------------------------------- latent attention

// (q, cache, page_table, seq_lens, max_seq_len, scale, workspace, out, stream)
PyObject* latent_attn(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 9, [&]() -> PyObject* {
    const Tensor &q = ten(a[0], "q"), &cache = ten(a[1], "cache");
    const Tensor *table = opt(a[2], "page_table"), *lens = opt(a[3], "seq_lens"), *ws = opt(a[6], "workspace"),
                 *given = opt(a[7], "out");
    if (q.dim() != 4 || cache.dim() != 3) throw Bad("q, cache: expected 4 and 3 dims");
    const int64_t dev = cuda_index(q), W = q.size(3), R = W - kLatentRope;
    const int B = small(q.size(0), "q"), n = small(q.size(1), "q"), H = small(q.size(2), "q");
    plain(q, "q", at::kBFloat16, dims(B, n, H, W), dev);
    plain(cache, "cache", at::kBFloat16, dims(table ? cache.size(0) : B, cache.size(1), W), dev);
    const int64_t cols = table && table->dim() == 2 ? table->size(1) : 0;
    if (table) {
      plain(*table, "page_table", at::kInt, dims(B, cols), dev);
      if (!lens) throw Bad("seq_lens: a paged cache needs them");
    }
    if (lens) plain(*lens, "seq_lens", at::kInt, dims(B), dev);
    if (R < 0) throw Bad("q: a row is the latent and 64 rotated elements");
    if (given) plain(*given, "out", at::kBFloat16, dims(B, n, H, R), dev);
    if (ws && (!ws->is_contiguous() || cuda_index(*ws) != dev))
      throw Bad("workspace: expected a contiguous tensor on cuda:" + std::to_string(dev));
    const float scale = real(a[5]);
    not_tracked(given, "out");
    on_current(dev);
    Stream st(a[8], dev);
    const Tensor out = given ? *given : at::empty(dims(B, n, H, R), q.options());
    const char* fn = table ? "latent_attn_paged" : "latent_attn_contig";
    Tensor work;
    if (!ws) {
      const long long bytes = g_lib.latent_workspace_bytes(B, n, H, small(R, "q"), 0);
      if (bytes < 0) throw Failed{fn, (int)-bytes};
      work = at::empty(dims(bytes), q.options().dtype(at::kByte));
    }
    const Tensor& w = ws ? *ws : work;
    const long long size = (long long)w.nbytes();
    const int slab = small(cache.size(1), "cache"), slabs = small(cache.size(0), "cache"),
              columns = small(cols, "page_table");
    if (table) {
      const int cap = small(a[4], "max_seq_len");
      call(fn, [&] {
        return g_lib.latent_attn_paged(ptr(q), ptr(cache), ptr<int>(table), ptr<int>(lens), B, n, H, (int)R, slab,
                                       columns, slabs, cap, scale, ptr(w), size, ptr(out), st.raw);
      });
    } else {
      call(fn, [&] {
        return g_lib.latent_attn_contig(ptr(q), ptr(cache), ptr<int>(lens), B, n, H, (int)R, slab, scale, ptr(w), size,
                                        ptr(out), st.raw);
      });
    }
    written(given);
    return given ? same(a[7]) : THPVariable_Wrap(out);
  });
}

// (token, head) strides of keys or values [B, ctx, H, D] (or [B, ctx, D]): a head's elements
// consecutive, batch entries ctx tokens apart.  Strides that reach no element count as dense.
std::pair<int64_t, int64_t> cache_strides(const Tensor& t, const char* name, at::IntArrayRef want, int64_t dev) {
  if (t.scalar_type() != at::kBFloat16 || t.sizes() != want || cuda_index(t) != dev)
    mismatch(t, name, at::kBFloat16, want, dev, "");
  const auto st = t.strides();
  const int64_t B = want[0], ctx = want[1], H = want.size() == 4 ? want[2] : 1, D = want.back();
  const int64_t head = H > 1 ? st[2] : D;
  const int64_t dense = ((H - 1) * head + D + 7) / 8 * 8;
  const int64_t step = ctx > 1 ? st[1] : B > 1 && ctx == 1 ? st[0] : dense;
  if (ctx > 0 && D > 0 && ((D > 1 && st.back() != 1) || (B > 1 && st[0] != ctx * step))) {
    std::ostringstream s;
    s << name << ": a head's elements must be consecutive and batch entries max_ctx tokens apart, got strides " << st;
    throw Bad(s.str());
  }
  return {step, head};
}

// (q, k_nope, k_rope, v, seq_lens, scale, out, stream)
PyObject* latent_prefill(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const Tensor &q = ten(a[0], "q"), &k = ten(a[1], "k_nope"), &pe = ten(a[2], "k_rope"), &v = ten(a[3], "v");
    const Tensor *lens = opt(a[4], "seq_lens"), *given = opt(a[6], "out");
    if (q.dim() != 4 || k.dim() != 4) throw Bad("q, k_nope: expected 4 dims");
    const int64_t dev = cuda_index(q), W = q.size(3), D = std::max<int64_t>(W - kLatentRope, 0), ctx = k.size(1);
    const int B = small(q.size(0), "q"), n = small(q.size(1), "q"), H = small(q.size(2), "q");
    plain(q, "q", at::kBFloat16, dims(B, n, H, W), dev);
    const auto kst = cache_strides(k, "k_nope", dims(B, ctx, H, D), dev), vst = cache_strides(v, "v", dims(B, ctx, H, D), dev),
               pst = cache_strides(pe, "k_rope", dims(B, ctx, kLatentRope), dev);
    if (kst != vst) {
      std::ostringstream s;
      s << "v: expected the strides of k_nope, got " << v.strides() << " and " << k.strides();
      throw Bad(s.str());
    }
    if (lens) plain(*lens, "seq_lens", at::kInt, dims(B), dev);
    if (given) plain(*given, "out", at::kBFloat16, dims(B, n, H, D), dev);
    const float scale = real(a[5]);
    const int ctxi = small(ctx, "k_nope");
    not_tracked(given, "out");
    on_current(dev);
    Stream st(a[7], dev);
    const Tensor out = given ? *given : at::empty(dims(B, n, H, D), q.options());
    Tensor work;
    const long long bytes = g_lib.latent_prefill_workspace_bytes(B, n, H, (int)D, ctxi, 0);
    if (bytes < 0) throw Failed{"latent_prefill_contig", (int)-bytes};
    if (bytes > 0) work = at::empty(dims(bytes), q.options().dtype(at::kByte));
    call("latent_prefill_contig", [&] {
      return g_lib.latent_prefill_contig(ptr(q), ptr(k), ptr(pe), ptr(v), ptr<int>(lens), B, n, H, (int)D,
                                         ctxi, kst.first, kst.second, pst.first, scale,
                                         bytes > 0 ? ptr(work) : nullptr, bytes, ptr(out), st.raw);
    });
    written(given);
    return given ? same(a[6]) : THPVariable_Wrap(out);
  });
}

// ---------------------------------------------------------------- attention over long caches

// A scale, or None: one over the root of the head's width.
float scale_or(PyObject* o, int64_t D) { return o == Py_None ? (float)std::pow((double)D, -0.5) : real(o); }

// A workspace that the caller gave, or one of these bytes (negative: an error) that is made here.
struct Work {
  Tensor own;
  void* at;
  long long size;
  Work(const Tensor* given, long long bytes, const char* fn, const Tensor& like, int64_t dev) {
    if (given) {
      if (!given->is_contiguous() || cuda_index(*given) != dev)
        throw Bad("workspace: expected a contiguous tensor on cuda:" + std::to_string(dev));
      at = given->data_ptr();
      size = (long long)given->nbytes();
      return;
    }
    if (bytes < 0) throw Failed{fn, (int)-bytes};
    own = at::empty(dims(bytes), like.options().dtype(at::kByte));
    at = bytes ? own.data_ptr() : nullptr;
    size = bytes;
  }
};

// (q, k_prefix, v_prefix, k, v, prefix_table, prefix_len, page_table, seq_lens, max_seq_len, scale, workspace, out,
//  stream)
PyObject* prefix_attn(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 14, [&]() -> PyObject* {
    const Tensor &q = ten(a[0], "q"), &k = ten(a[3], "k"), &v = ten(a[4], "v");
    const Tensor *kp = opt(a[1], "k_prefix"), *vp = opt(a[2], "v_prefix"), *pt = opt(a[5], "prefix_table"),
                 *table = opt(a[7], "page_table"), *lens = opt(a[8], "seq_lens"), *ws = opt(a[11], "workspace"),
                 *given = opt(a[12], "out");
    if (q.dim() != 4 || k.dim() != 4) throw Bad("q, k: expected 4 dims");
    const int64_t dev = cuda_index(q);
    const int B = small(q.size(0), "q"), n = small(q.size(1), "q"), Hq = small(q.size(2), "q"), D = small(q.size(3), "q"),
              H = small(k.size(2), "k");
    plain(q, "q", at::kBFloat16, dims(B, n, Hq, D), dev);
    const Cache c = check_cache(k, &v, nullptr, nullptr, table, lens, B, H, D, dev);
    if (given) plain(*given, "out", at::kBFloat16, dims(B, n, Hq, D), dev);
    int P, cap = 0;
    if (table) {
      P = small(a[6], "prefix_len");
      cap = small(a[9], "max_seq_len");
      if (!pt) throw Bad("prefix_table: expected a tensor");
      if (P < 0) throw Bad("prefix_len: negative");
      const int64_t need = c.slab > 0 ? (P + c.slab - 1) / c.slab : 0;
      if (pt->dim() != 1 || pt->size(0) < need)
        throw Bad("prefix_table: expected one dim of at least " + std::to_string(need) + " pages");
      plain(*pt, "prefix_table", at::kInt, dims(pt->size(0)), dev);
    } else {
      if (!kp || !vp) throw Bad("k_prefix, v_prefix: expected tensors");
      P = kp->dim() == 3 ? small(kp->size(0), "k_prefix") : 0;
      plain(*kp, "k_prefix", at::kBFloat16, dims(P, H, D), dev);
      plain(*vp, "v_prefix", at::kBFloat16, dims(P, H, D), dev);
    }
    const float scale = scale_or(a[10], D);
    not_tracked(given, "out");
    on_current(dev);
    Stream st(a[13], dev);
    const Tensor out = given ? *given : at::empty(dims(B, n, Hq, D), q.options());
    const char* fn = table ? "prefix_attn_paged" : "prefix_attn_contig";
    const Work w(ws, ws ? 0 : g_lib.prefix_attn_workspace_bytes(B, n, Hq, H, D, 0), fn, q, dev);
    const int slab = small(c.slab, "k"), cols = small(c.cols, "page_table"), slabs = small(c.slabs, "k");
    if (table)
      call(fn, [&] {
        return g_lib.prefix_attn_paged(ptr(q), ptr(k), ptr(v), ptr<int>(pt), P, ptr<int>(table), ptr<int>(lens), B, n, Hq,
                                       H, D, slab, cols, slabs, cap, scale, w.at, w.size, ptr(out), st.raw);
      });
    else
      call(fn, [&] {
        return g_lib.prefix_attn_contig(ptr(q), ptr(kp), ptr(vp), ptr(k), ptr(v), ptr<int>(lens), B, n, Hq, H, D, P, slab,
                                        scale, w.at, w.size, ptr(out), st.raw);
      });
    written(given);
    return given ? same(a[12]) : THPVariable_Wrap(out);
  });
}

// (k, page_table, seq_lens, max_seq_len, block_size, n_tokens, out, stream)
PyObject* block_means(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const Tensor& k = ten(a[0], "k");
    const Tensor *table = opt(a[1], "page_table"), *lens = opt(a[2], "seq_lens"), *given = opt(a[6], "out");
    if (k.dim() != 4 || (table && table->dim() != 2)) throw Bad("k, page_table: expected 4 and 2 dims");
    const int64_t dev = cuda_index(k);
    const int B = small(table ? table->size(0) : k.size(0), "k"), H = small(k.size(2), "k"), D = small(k.size(3), "k"),
              block = small(a[4], "block_size");
    if (block <= 0) throw Bad("block_size: expected a positive number");
    const Cache c = check_cache(k, nullptr, nullptr, nullptr, table, lens, B, H, D, dev);
    const int cap = table ? small(a[3], "max_seq_len") : small(c.slab, "k");
    const int64_t room = table ? std::min<int64_t>(std::max(cap, 0), c.cols * c.slab) : cap;
    const int n = a[5] == Py_None ? small(room, "k") : small(a[5], "n_tokens");
    const int64_t blocks = given && given->dim() == 4 ? given->size(2) : (room + block - 1) / block;
    if (given) plain(*given, "out", at::kBFloat16, dims(B, H, blocks, D), dev);
    not_tracked(given, "out");
    on_current(dev);
    Stream st(a[7], dev);
    const Tensor out = given ? *given : at::zeros(dims(B, H, blocks, D), k.options());
    const int slab = small(c.slab, "k"), cols = small(c.cols, "page_table"), slabs = small(c.slabs, "k"),
              nb = small(blocks, "out");
    if (table)
      call("block_means_paged", [&] {
        return g_lib.block_means_paged(ptr(k), ptr<int>(table), ptr<int>(lens), B, n, H, D, slab, cols, slabs, cap, block,
                                       nb, ptr(out), st.raw);
      });
    else
      call("block_means_contig", [&] {
        return g_lib.block_means_contig(ptr(k), ptr<int>(lens), B, n, H, D, slab, block, nb, ptr(out), st.raw);
      });
    written(given);
    return given ? same(a[6]) : THPVariable_Wrap(out);
  });
}

// (q, means, seq_lens, block_size, n_select, first, recent, out, stream)
PyObject* block_select(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 9, [&]() -> PyObject* {
    const Tensor &q = ten(a[0], "q"), &means = ten(a[1], "means");
    const Tensor *lens = opt(a[2], "seq_lens"), *given = opt(a[7], "out");
    if (q.dim() != 4 || means.dim() != 4) throw Bad("q, means: expected 4 dims");
    const int64_t dev = cuda_index(q);
    const int B = small(q.size(0), "q"), n = small(q.size(1), "q"), Hq = small(q.size(2), "q"), D = small(q.size(3), "q"),
              H = small(means.size(1), "means"), blocks = small(means.size(2), "means"), block = small(a[3], "block_size"),
              pick = small(a[4], "n_select"), first = small(a[5], "first"), recent = small(a[6], "recent");
    plain(q, "q", at::kBFloat16, dims(B, n, Hq, D), dev);
    plain(means, "means", at::kBFloat16, dims(B, H, blocks, D), dev);
    if (lens) plain(*lens, "seq_lens", at::kInt, dims(B), dev);
    if (pick < 0) throw Bad("n_select: negative");
    if (given) plain(*given, "out", at::kInt, dims(B, n, H, pick), dev);
    on_current(dev);
    Stream st(a[8], dev);
    const Tensor out = given ? *given : at::empty(dims(B, n, H, pick), q.options().dtype(at::kInt));
    call("block_select", [&] {
      return g_lib.block_select(ptr(q), ptr(means), ptr<int>(lens), B, n, Hq, H, D, block, blocks, pick, first, recent,
                                ptr<int>(out), st.raw);
    });
    written(given);
    return given ? same(a[7]) : THPVariable_Wrap(out);
  });
}

// (q, k, v, blocks, page_table, seq_lens, max_seq_len, block_size, scale, out, stream)
PyObject* sparse_attn(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 11, [&]() -> PyObject* {
    const Tensor &q = ten(a[0], "q"), &k = ten(a[1], "k"), &v = ten(a[2], "v"), &blocks = ten(a[3], "blocks");
    const Tensor *table = opt(a[4], "page_table"), *lens = opt(a[5], "seq_lens"), *given = opt(a[9], "out");
    if (q.dim() != 4 || k.dim() != 4 || blocks.dim() != 4) throw Bad("q, k, blocks: expected 4 dims");
    const int64_t dev = cuda_index(q);
    const int B = small(q.size(0), "q"), n = small(q.size(1), "q"), Hq = small(q.size(2), "q"), D = small(q.size(3), "q"),
              H = small(k.size(2), "k"), pick = small(blocks.size(3), "blocks"), block = small(a[7], "block_size");
    plain(q, "q", at::kBFloat16, dims(B, n, Hq, D), dev);
    const Cache c = check_cache(k, &v, nullptr, nullptr, table, lens, B, H, D, dev);
    plain(blocks, "blocks", at::kInt, dims(B, n, H, pick), dev);
    if (given) plain(*given, "out", at::kBFloat16, dims(B, n, Hq, D), dev);
    const float scale = scale_or(a[8], D);
    not_tracked(given, "out");
    on_current(dev);
    Stream st(a[10], dev);
    const Tensor out = given ? *given : at::empty(dims(B, n, Hq, D), q.options());
    const char* fn = table ? "sparse_attn_paged" : "sparse_attn_contig";
    const int slab = small(c.slab, "k"), cols = small(c.cols, "page_table"), slabs = small(c.slabs, "k"),
              cap = table ? small(a[6], "max_seq_len") : 0;
    if (table)
      call(fn, [&] {
        return g_lib.sparse_attn_paged(ptr(q), ptr(k), ptr(v), ptr<int>(blocks), ptr<int>(table), ptr<int>(lens), B, n, Hq,
                                       H, D, slab, cols, slabs, cap, block, pick, scale, ptr(out), st.raw);
      });
    else
      call(fn, [&] {
        return g_lib.sparse_attn_contig(ptr(q), ptr(k), ptr(v), ptr<int>(blocks), ptr<int>(lens), B, n, Hq, H, D, slab,
                                        block, pick, scale, ptr(out), st.raw);
      });
    written(given);
    return given ? same(a[9]) : THPVariable_Wrap(out);
  });
}

// ---------------------------------------------------------------- weights and eviction

// (q, k, k_scale, weights, page_table, seq_lens, max_seq_len, scale, decay, workspace, out, stream)
PyObject* kv_weights(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 12, [&]() -> PyObject* {
    const Tensor &q = ten(a[0], "q"), &k = ten(a[1], "k");
    const Tensor *ks = opt(a[2], "k_scale"), *prior = opt(a[3], "weights"), *table = opt(a[4], "page_table"),
                 *lens = opt(a[5], "seq_lens"), *ws = opt(a[9], "workspace"), *given = opt(a[10], "out");
    if (q.dim() != 4 || k.dim() != 4) throw Bad("q, k: expected 4 dims");
    const int64_t dev = cuda_index(q);
    const int B = small(q.size(0), "q"), n = small(q.size(1), "q"), Hq = small(q.size(2), "q"), D = small(q.size(3), "q"),
              H = small(k.size(2), "k");
    plain(q, "q", at::kBFloat16, dims(B, n, Hq, D), dev);
    const Cache c = check_cache(k, nullptr, ks, nullptr, table, lens, B, H, D, dev);
    const auto shape = dims(c.slabs, H, c.slab);
    if (prior) plain(*prior, "weights", at::kFloat, shape, dev);
    if (given) plain(*given, "out", at::kFloat, shape, dev);
    const Tensor* kept = given ? given : prior;  // where the sums go, unless they are made here
    not_tracked(kept, given ? "out" : "weights");
    const float scale = scale_or(a[7], D), decay = real(a[8]);
    on_current(dev);
    Stream st(a[11], dev);
    const Tensor out = kept ? *kept : at::zeros(shape, q.options().dtype(at::kFloat));
    const int slab = small(c.slab, "k"), cols = small(c.cols, "page_table"), slabs = small(c.slabs, "k");
    const int cap = table ? small(a[6], "max_seq_len") : slab;
    const int64_t room = table ? std::min<int64_t>(std::max(cap, 0), c.cols * c.slab) : cap;
    const char* fn = table ? (ks ? "kv_weights_int8_paged" : "kv_weights_paged")
                           : (ks ? "kv_weights_int8_contig" : "kv_weights_contig");
    const Work w(ws, ws ? 0 : g_lib.kv_weights_workspace_bytes(B, n, Hq, H, (int)room, 0), fn, q, dev);
    const float* from = ptr<float>(prior);
    call(fn, [&] {
      if (table)
        return ks ? g_lib.kv_weights_int8_paged(ptr(q), ptr(k), ptr<float>(ks), ptr<int>(table), ptr<int>(lens), B, n, Hq, H,
                                                D, slab, cols, slabs, cap, scale, decay, from, w.at, w.size,
                                                ptr<float>(out), st.raw)
                  : g_lib.kv_weights_paged(ptr(q), ptr(k), ptr<int>(table), ptr<int>(lens), B, n, Hq, H, D, slab, cols, slabs,
                                           cap, scale, decay, from, w.at, w.size, ptr<float>(out), st.raw);
      return ks ? g_lib.kv_weights_int8_contig(ptr(q), ptr(k), ptr<float>(ks), ptr<int>(lens), B, n, Hq, H, D, slab, scale,
                                               decay, from, w.at, w.size, ptr<float>(out), st.raw)
                : g_lib.kv_weights_contig(ptr(q), ptr(k), ptr<int>(lens), B, n, Hq, H, D, slab, scale, decay, from, w.at,
                                          w.size, ptr<float>(out), st.raw);
    });
    written(kept);
    return given ? same(a[10]) : prior ? same(a[3]) : THPVariable_Wrap(out);
  });
}

// (k, v, k_scale, v_scale, weights, page_table, seq_lens, max_seq_len, keep, first, recent, kept, new_lens, k_out,
//  v_out, k_scale_out, v_scale_out, weights_out, stream)
PyObject* kv_evict(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 19, [&]() -> PyObject* {
    const Tensor &k = ten(a[0], "k"), &weights = ten(a[4], "weights");
    const Tensor *v = opt(a[1], "v"), *ks = opt(a[2], "k_scale"), *vs = opt(a[3], "v_scale"),
                 *table = opt(a[5], "page_table"), *lens = opt(a[6], "seq_lens"), *kept = opt(a[11], "kept"),
                 *nl = opt(a[12], "new_lens"), *ko = opt(a[13], "k_out"), *vo = opt(a[14], "v_out"),
                 *kso = opt(a[15], "k_scale_out"), *vso = opt(a[16], "v_scale_out"), *wo = opt(a[17], "weights_out");
    if (k.dim() != 4 || (table && table->dim() != 2)) throw Bad("k, page_table: expected 4 and 2 dims");
    const int64_t dev = cuda_index(k);
    const int B = small(table ? table->size(0) : k.size(0), "k"), H = small(k.size(2), "k"), D = small(k.size(3), "k"),
              keep = small(a[8], "keep"), first = small(a[9], "first"), recent = small(a[10], "recent");
    const Cache c = check_cache(k, v, ks, vs, table, lens, B, H, D, dev);
    plain(weights, "weights", at::kFloat, dims(c.slabs, H, c.slab), dev);
    if (keep <= 0) throw Bad("keep: expected a positive number");
    if (kept) plain(*kept, "kept", at::kInt, dims(B, H, keep), dev);
    if (nl) plain(*nl, "new_lens", at::kInt, dims(B), dev);
    int64_t room = 0;
    const auto type = k.scalar_type();
    if (ko) {
      room = ko->dim() == 4 ? ko->size(1) : 0;
      plain(*ko, "k_out", type, dims(B, room, H, D), dev);
      if (!v != !vo) throw Bad("v_out: expected next to k_out, as v");
      if (vo) plain(*vo, "v_out", type, dims(B, room, H, D), dev);
      if (c.int8 && (!kso || !vs != !vso)) throw Bad("k_scale_out, v_scale_out: an int8 cache needs them");
      if (room < keep) throw Bad("k_out: no room for the tokens that are kept");
    } else if (vo || kso || vso || wo) {
      throw Bad("k_out: expected with the other outputs");
    }
    if (kso) plain(*kso, "k_scale_out", at::kFloat, dims(B, H, room), dev);
    if (vso) plain(*vso, "v_scale_out", at::kFloat, dims(B, H, room), dev);
    if (wo) plain(*wo, "weights_out", at::kFloat, dims(B, H, room), dev);
    const Tensor* moved[5] = {ko ? ko : &k, ko ? vo : v, ko ? kso : ks, ko ? vso : vs, ko ? wo : &weights};
    for (const Tensor* t : moved) not_tracked(t, "an output");
    on_current(dev);
    Stream st(a[18], dev);
    const auto ints = k.options().dtype(at::kInt);
    const Tensor kt = kept ? *kept : at::empty(dims(B, H, keep), ints), nt = nl ? *nl : at::empty(dims(B), ints);
    const int slab = small(c.slab, "k"), cols = small(c.cols, "page_table"), slabs = small(c.slabs, "k"),
              cap = table ? small(a[7], "max_seq_len") : 0, oc = small(room, "k_out");
    const char* fn = table ? (c.int8 ? "kv_evict_int8_paged" : "kv_evict_paged")
                           : (c.int8 ? "kv_evict_int8_contig" : "kv_evict_contig");
    call(fn, [&] {
      int *kd = ptr<int>(kt), *nd = ptr<int>(nt);
      float* wd = ptr<float>(weights);
      if (table)
        return c.int8 ? g_lib.kv_evict_int8_paged(ptr(k), ptr(v), ptr<float>(ks), ptr<float>(vs), wd, ptr<int>(table),
                                                  ptr<int>(lens), B, H, D, slab, cols, slabs, cap, keep, first, recent,
                                                  ptr(ko), ptr(vo), ptr<float>(kso), ptr<float>(vso), ptr<float>(wo), oc, kd,
                                                  nd, st.raw)
                      : g_lib.kv_evict_paged(ptr(k), ptr(v), wd, ptr<int>(table), ptr<int>(lens), B, H, D, slab, cols, slabs,
                                             cap, keep, first, recent, ptr(ko), ptr(vo), ptr<float>(wo), oc, kd, nd, st.raw);
      return c.int8 ? g_lib.kv_evict_int8_contig(ptr(k), ptr(v), ptr<float>(ks), ptr<float>(vs), wd, ptr<int>(lens), B, H, D,
                                                 slab, keep, first, recent, ptr(ko), ptr(vo), ptr<float>(kso),
                                                 ptr<float>(vso), ptr<float>(wo), oc, kd, nd, st.raw)
                    : g_lib.kv_evict_contig(ptr(k), ptr(v), wd, ptr<int>(lens), B, H, D, slab, keep, first, recent, ptr(ko),
                                            ptr(vo), ptr<float>(wo), oc, kd, nd, st.raw);
    });
    for (const Tensor* t : moved) written(t);
    written(kept);
    written(nl);
    PyObject* x = kept ? same(a[11]) : THPVariable_Wrap(kt);
    PyObject* y = nl ? same(a[12]) : THPVariable_Wrap(nt);
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
  });
}

// ---------------------------------------------------------------- the library

// (path, DecodeAttnError): the shared library whose entry points the calls above use.
PyObject* open(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 2) {
    PyErr_SetString(PyExc_TypeError, "open(path, error)");
    return nullptr;
  }
  const char* path = PyUnicode_AsUTF8(a[0]);
  if (!path) return nullptr;
  Library l;
  l.handle = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!l.handle) {
    PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
    return nullptr;
  }
#define FIND(name)                                                            \
  l.name = reinterpret_cast<decltype(l.name)>(dlsym(l.handle, #name));        \
  if (!l.name) {                                                              \
    PyErr_Format(PyExc_RuntimeError, "%s has no %s", path, #name);            \
    return nullptr;                                                           \
  }
  FIND(rope_apply)
  FIND(kv_write_contig)
  FIND(kv_write_paged)
  FIND(kv_write_int8_contig)
  FIND(kv_write_int8_paged)
  FIND(kv_read_paged)
  FIND(kv_read_int8_contig)
  FIND(kv_read_int8_paged)
  FIND(kv_read_paged_filled)
  FIND(kv_read_int8_contig_filled)
  FIND(kv_read_int8_paged_filled)
  FIND(latent_attn_contig)
  FIND(latent_attn_paged)
  FIND(latent_workspace_bytes)
  FIND(latent_prefill_contig)
  FIND(latent_prefill_workspace_bytes)
  FIND(prefix_attn_contig)
  FIND(prefix_attn_paged)
  FIND(prefix_attn_workspace_bytes)
  FIND(block_means_contig)
  FIND(block_means_paged)
  FIND(block_select)
  FIND(sparse_attn_contig)
  FIND(sparse_attn_paged)
  FIND(kv_weights_contig)
  FIND(kv_weights_paged)
  FIND(kv_weights_int8_contig)
  FIND(kv_weights_int8_paged)
  FIND(kv_weights_workspace_bytes)
  FIND(kv_evict_contig)
  FIND(kv_evict_paged)
  FIND(kv_evict_int8_contig)
  FIND(kv_evict_int8_paged)
#undef FIND
  g_lib = l;
  Py_INCREF(a[1]);
  Py_XSETREF(g_error, a[1]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(open),         FAST(rope_apply),  FAST(kv_write),     FAST(kv_read),
                           FAST(latent_attn),  FAST(latent_prefill), FAST(prefix_attn), FAST(block_means),
                           FAST(block_select), FAST(sparse_attn), FAST(kv_weights),   FAST(kv_evict),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding_ext", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding_ext() { return PyModule_Create(&g_module); }
