// Argument checks and marshalling of the tree-verification calls, natively.
//
// A decoding step makes dozens of these calls whose kernels take a few
// microseconds each; checked and passed on in Python, one call costs 15 to 20 us
// of host time, here one or two.  Every function takes its arguments by
// position from the wrapper of the same name in __init__.py, checks each
// tensor's type, device, shape and strides (ValueError), makes the tensors'
// device current, takes that device's current stream unless one is given, and
// calls the C ABI through the addresses that bind() received, so that there is
// one loaded copy of the library.  The status comes back as a number.
//
// Scratch that the caller does not give comes from PyTorch's caching allocator
// on the call's stream and goes back to it at once: the allocator gives it out
// again only behind that stream's work.
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/qhl_stage.h"

namespace {

struct Bound {
  decltype(&qhl_qk_norm_rope) norm_rope;
  decltype(&qhl_tree_attention) tree_attention;
  decltype(&qhl_tree_attention_workspace) workspace;
  decltype(&qhl_deltanet_tree) deltanet_tree;
  decltype(&qhl_pages_free) pages_free;
  decltype(&qhl_pages_fork) pages_fork;
  decltype(&qhl_pages_extend) pages_extend;
  decltype(&qhl_pages_commit) pages_commit;
} g_lib = {};

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

std::string describe(const at::Tensor& t) {
  std::ostringstream s;
  s << "got " << t.scalar_type() << " " << t.sizes() << " strides " << t.strides() << " on " << t.device();
  return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

long long integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  return v;
}
int integer32(PyObject* o, const char* name) {
  const long long v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return (int)v;
}
double real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return v;
}

int type_id(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return QHL_F32;
    case at::kHalf: return QHL_F16;
    case at::kBFloat16: return QHL_BF16;
    default: return -1;
  }
}

bool on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// The device of a call, from its first tensor.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be on a CUDA device, " + describe(t));
  return t.get_device();
}

// A contiguous tensor of `type` with these sizes: its address.
template <typename V>
V* dense(PyObject* o, const char* name, int dev, at::ScalarType type, at::IntArrayRef sizes) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || !on(t, dev) || !t.is_contiguous() || t.sizes() != sizes) {
    std::ostringstream s;
    s << name << " must be a contiguous " << type << " tensor " << sizes << " on cuda:" << dev << ", " << describe(t);
    refuse(s.str());
  }
  return static_cast<V*>(t.data_ptr());
}
int* ints(PyObject* o, const char* name, int dev, long long n) { return dense<int>(o, name, dev, at::kInt, {n}); }

// A [rows, heads, dim] tensor of type `type` whose rows may be strided.
struct Heads {
  void* p;
  long long stride, rows;
};
Heads heads_of(PyObject* o, const char* name, int dev, int type, long long heads, long long dim, long long rows) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 3 || !on(t, dev) || type_id(t) != type || t.size(1) != heads || t.size(2) != dim || (rows >= 0 && t.size(0) != rows) ||
      (t.numel() > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != dim)))) {
    std::ostringstream s;
    s << name << " must be a [" << (rows >= 0 ? std::to_string(rows) : std::string("rows")) << ", " << heads << ", " << dim
      << "] tensor of " << (type == QHL_F16 ? "float16" : "bfloat16") << " with contiguous heads on cuda:" << dev << ", " << describe(t);
    refuse(s.str());
  }
  // the stride of one row alone is never used: any that the checks accept will do
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : heads * dim, t.size(0)};
}

// Makes `dev` current for the call's duration and finds its stream.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::CUDAStream current;
  cudaStream_t stream;
  On(int dev, PyObject* given) : current(c10::cuda::getCurrentCUDAStream(dev)) {
    if (c10::cuda::current_device() != dev) guard.set_index(dev);
    stream = given == Py_None ? current.stream() : reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(given));
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse("stream must be a CUDA stream or its address");
    }
  }
};

// Scratch of the call: the caller's tensor, or the allocator's memory.
struct Scratch {
  void* p = nullptr;
  size_t bytes = 0;
  bool own = false;
  Scratch(PyObject* given, int dev, size_t need, cudaStream_t s) {
    if (given == Py_None) {
      p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(need, s);
      bytes = need;
      own = true;
    } else {
      const at::Tensor& t = tensor(given, "workspace");
      if (!on(t, dev) || !t.is_contiguous()) refuse("workspace must be a contiguous tensor on cuda:" + std::to_string(dev) + ", " + describe(t));
      p = t.data_ptr();
      bytes = t.nbytes();
    }
  }
  ~Scratch() {
    if (own) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
};

const qhl_kv_pages* cache(PyObject* o) { return static_cast<const qhl_kv_pages*>(PyLong_AsVoidPtr(o)); }

// Every entry: a fixed number of arguments, C++ errors turned into Python's.
template <int N, typename F>
PyObject* entry(const char* name, Py_ssize_t n, F&& f) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%s takes %d arguments, got %zd", name, N, n);
    return nullptr;
  }
  if (!g_lib.norm_rope) {
    PyErr_SetString(PyExc_RuntimeError, "the CUDA library is not bound");
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(PyExc_MemoryError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// n_q_heads, n_kv_heads, dim, rope_dims, theta, eps, y, pos, gamma_q, gamma_k, q, k, v, q_off, k_off, v_off (-1: q | gate | k | v), stream
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry<17>("qk_norm_rope", n, [&]() {
    const int hq = integer32(a[0], "n_q_heads"), hkv = integer32(a[1], "n_kv_heads"), dim = integer32(a[2], "dim"), rope = integer32(a[3], "rope_dims");
    const double theta = real(a[4], "theta");
    const float eps = (float)real(a[5], "eps");
    const at::Tensor& y = tensor(a[6], "y");
    const int yt = type_id(y);
    if (y.dim() != 2 || yt < 0 || (y.numel() > 0 && y.size(1) > 1 && y.stride(1) != 1))
      refuse("y must be [rows, width] of f32, f16 or bf16 with contiguous rows, " + describe(y));
    const int dev = device_of(y, "y");
    const long long rows = y.size(0), width = y.size(1), qw = (long long)hq * dim, kw = (long long)hkv * dim;
    long long off[3] = {integer(a[13], "offsets"), integer(a[14], "offsets"), integer(a[15], "offsets")};
    if (off[0] == -1 && off[1] == -1 && off[2] == -1) {
      off[0] = 0;
      off[1] = 2 * qw;
      off[2] = 2 * qw + kw;
    }
    if (off[0] < 0 || off[1] < 0 || off[2] < 0 || off[0] + qw > width || off[1] + kw > width || off[2] + kw > width)
      refuse("y rows of " + std::to_string(width) + " elements do not hold " + std::to_string(hq) + " query and " + std::to_string(hkv) +
             " key and value heads at " + std::to_string(off[0]) + ", " + std::to_string(off[1]) + ", " + std::to_string(off[2]));
    const int* pos = ints(a[7], "pos", dev, rows);
    const float* gq = dense<float>(a[8], "gamma_q", dev, at::kFloat, {dim});
    const float* gk = dense<float>(a[9], "gamma_k", dev, at::kFloat, {dim});
    const int dt = type_id(tensor(a[10], "q"));
    if (dt != QHL_F16 && dt != QHL_BF16) refuse("q, k and v must be float16 or bfloat16");
    const Heads q = heads_of(a[10], "q", dev, dt, hq, dim, rows), k = heads_of(a[11], "k", dev, dt, hkv, dim, rows),
                v = heads_of(a[12], "v", dev, dt, hkv, dim, rows);
    if (rows > INT32_MAX || width > INT32_MAX) refuse("y is too large");
    if (rows == 0) return 0;
    // the stride of one row alone is never used: any that the checks accept will do
    const long long stride = rows > 1 ? y.stride(0) : (width + 7) / 8 * 8;
    const On o(dev, a[16]);
    return g_lib.norm_rope(hq, hkv, dim, rope, theta, eps, y.data_ptr(), yt, stride, (int)off[0], (int)off[1],
                           (int)off[2], (int)rows, pos, gq, gk, dt, q.p, q.stride, k.p, k.stride, v.p, v.stride, o.stream);
  });
}

// cache, device, layer, seqs, q_start, parent, max_nodes, q, k_new, v_new, out, lse, scale (None: 1 / sqrt(dim)), workspace, stream
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry<15>("tree_attention", n, [&]() {
    const qhl_kv_pages* kv = cache(a[0]);
    const int dev = integer32(a[1], "device"), layer = integer32(a[2], "layer"), nodes = integer32(a[6], "max_nodes");
    const at::Tensor &qt = tensor(a[7], "q"), &st = tensor(a[3], "seqs");
    if (dev < 0) refuse("the cache must be on a CUDA device");
    if (qt.dim() != 3 || st.dim() != 1) refuse("q must be [n_rows, n_q_heads, dim] and seqs [batch]");
    const long long rows = qt.size(0), hq = qt.size(1), b = st.size(0);
    if (rows > INT32_MAX || hq > INT32_MAX || b > INT32_MAX) refuse("q or seqs is too large");
    const Heads q = heads_of(a[7], "q", dev, kv->dtype, hq, kv->dim, rows), out = heads_of(a[10], "out", dev, kv->dtype, hq, kv->dim, rows);
    const Heads k = heads_of(a[8], "k_new", dev, kv->dtype, kv->kv_heads, kv->dim, rows),
                v = heads_of(a[9], "v_new", dev, kv->dtype, kv->kv_heads, kv->dim, rows);
    if (k.stride != v.stride) refuse("k_new and v_new must have the same strides");
    float* lse = a[11] == Py_None ? nullptr : dense<float>(a[11], "lse", dev, at::kFloat, {rows, hq});
    const int *seqs = ints(a[3], "seqs", dev, b), *start = ints(a[4], "q_start", dev, b + 1), *parent = ints(a[5], "parent", dev, rows);
    const float scale = a[12] == Py_None ? 1.f / std::sqrt((float)kv->dim) : (float)real(a[12], "scale");
    if (rows == 0) return 0;
    const On o(dev, a[14]);
    const size_t need = g_lib.workspace(kv, (int)hq, (int)rows, (int)b, nodes);
    if (need == 0) return (int)STAGE_E_ARG;
    const Scratch w(a[13], dev, need, o.stream);
    return g_lib.tree_attention(kv, layer, (int)hq, (int)rows, (int)b, nodes, seqs, start, parent, q.p, q.stride, k.p, v.p, k.stride, out.p,
                                out.stride, lse, scale, w.p, w.bytes, o.stream);
  });
}

// Hk, Hv, y, q_start, parent, max_nodes, states, state_index, snaps, o, stream
PyObject* deltanet_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry<11>("deltanet_tree", n, [&]() {
    const int hk = integer32(a[0], "Hk"), hv = integer32(a[1], "Hv"), nodes = integer32(a[5], "max_nodes");
    const at::Tensor &y = tensor(a[2], "y"), &st = tensor(a[6], "states"), &ix = tensor(a[7], "state_index");
    if (y.dim() != 2 || st.dim() != 4 || ix.dim() != 1) refuse("y must be [rows, width], states [n, Hv, 128, 128] and state_index [batch]");
    const int dev = device_of(y, "y");
    const long long rows = y.size(0), ns = st.size(0), b = ix.size(0);
    if (rows > INT32_MAX || ns > INT32_MAX || b > INT32_MAX) refuse("y, states or state_index is too large");
    const float* yp = dense<float>(a[2], "y", dev, at::kFloat, {rows, 256LL * hk + 128LL * hv + 2LL * hv});
    const float* sp = dense<float>(a[6], "states", dev, at::kFloat, {ns, hv, 128, 128});
    float* snaps = dense<float>(a[8], "snaps", dev, at::kFloat, {rows, hv, 128, 128});
    float* op = dense<float>(a[9], "o", dev, at::kFloat, {rows, 128LL * hv});
    const int *index = ints(a[7], "state_index", dev, b), *start = ints(a[3], "q_start", dev, b + 1), *parent = ints(a[4], "parent", dev, rows);
    if (rows == 0) return 0;
    const On o(dev, a[10]);
    return g_lib.deltanet_tree(hk, hv, yp, (int)rows, (int)b, nodes, start, parent, sp, (int)ns, index, snaps, op, o.stream);
  });
}

long long requests(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 1 || t.size(0) > INT32_MAX) refuse(std::string(name) + " must be [n], " + describe(t));
  return t.size(0);
}
int cuda_device(PyObject* o) {
  const int dev = integer32(o, "device");
  if (dev < 0) refuse("the cache must be on a CUDA device");
  return dev;
}

// cache, device, seqs, status, stream
PyObject* pages_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry<5>("pages_free", n, [&]() {
    const long long m = requests(a[2], "seqs");
    const int dev = cuda_device(a[1]);
    const int* s = ints(a[2], "seqs", dev, m);
    int* st = ints(a[3], "status", dev, m);
    const On o(dev, a[4]);
    return g_lib.pages_free(cache(a[0]), (int)m, s, st, o.stream);
  });
}

// cache, device, src, dst, status, stream
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry<6>("pages_fork", n, [&]() {
    const long long m = requests(a[2], "src");
    const int dev = cuda_device(a[1]);
    const int *s = ints(a[2], "src", dev, m), *d = ints(a[3], "dst", dev, m);
    int* st = ints(a[4], "status", dev, m);
    const On o(dev, a[5]);
    return g_lib.pages_fork(cache(a[0]), (int)m, s, d, st, o.stream);
  });
}

// cache, device, seqs, add, status, workspace, stream
PyObject* pages_extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry<7>("pages_extend", n, [&]() {
    const long long m = requests(a[2], "seqs");
    const int dev = cuda_device(a[1]);
    const int *s = ints(a[2], "seqs", dev, m), *d = ints(a[3], "add", dev, m);
    int* st = ints(a[4], "status", dev, m);
    const On o(dev, a[6]);
    const Scratch w(a[5], dev, 16 * (size_t)(m > 0 ? m : 1), o.stream);
    return g_lib.pages_extend(cache(a[0]), (int)m, s, d, st, w.p, w.bytes, o.stream);
  });
}

// cache, device, seqs, q_start, path, n_accepted, pos, k_new, v_new, status, stream
PyObject* pages_commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry<11>("pages_commit", n, [&]() {
    const qhl_kv_pages* kv = cache(a[0]);
    const long long b = requests(a[2], "seqs");
    const int dev = cuda_device(a[1]);
    const at::Tensor &pt = tensor(a[4], "path"), &k = tensor(a[7], "k_new"), &v = tensor(a[8], "v_new");
    if (pt.dim() != 2 || pt.size(1) > INT32_MAX) refuse("path must be [batch, most], " + describe(pt));
    for (const at::Tensor* t : {&k, &v})
      if (t->dim() != 4 || !on(*t, dev) || type_id(*t) != kv->dtype || t->size(0) != kv->n_layers || t->size(2) != kv->kv_heads ||
          t->size(3) != kv->dim || t->size(1) > INT32_MAX ||
          (t->numel() > 0 && (t->stride(3) != 1 || (kv->kv_heads > 1 && t->stride(2) != kv->dim))))
        refuse("k_new and v_new must be [" + std::to_string(kv->n_layers) + ", rows, " + std::to_string(kv->kv_heads) + ", " +
               std::to_string(kv->dim) + "] in the cache's type with contiguous heads on its device, " + describe(*t));
    const long long rows = k.size(1);
    if (v.size(1) != rows || (rows > 1 && k.stride(1) != v.stride(1)) || (kv->n_layers > 1 && k.stride(0) != v.stride(0)))
      refuse("k_new and v_new must be alike");
    const long long sr = rows > 1 ? k.stride(1) : (long long)kv->kv_heads * kv->dim, sl = kv->n_layers > 1 ? k.stride(0) : sr;
    const int *s = ints(a[2], "seqs", dev, b), *start = ints(a[3], "q_start", dev, b + 1), *acc = ints(a[5], "n_accepted", dev, b),
              *pos = ints(a[6], "pos", dev, b);
    const int* path = dense<int>(a[4], "path", dev, at::kInt, {b, pt.size(1)});
    int* st = ints(a[9], "status", dev, b);
    const On o(dev, a[10]);
    return g_lib.pages_commit(kv, (int)b, (int)rows, s, start, path, (int)pt.size(1), acc, pos, k.data_ptr(), v.data_ptr(), sl, sr, st, o.stream);
  });
}

// The addresses of the library's functions, in the order of Bound.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t count = sizeof(Bound) / sizeof(void*);
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "bind takes %zd addresses", count);
    return nullptr;
  }
  void* p[count];
  for (Py_ssize_t i = 0; i < count; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  memcpy(&g_lib, p, sizeof(p));
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),       FAST(norm_rope),    FAST(tree_attention), FAST(deltanet_tree), FAST(pages_free),
                         FAST(pages_fork), FAST(pages_extend), FAST(pages_commit),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Native marshalling of the tree-verification calls, " QHL_BUILT_FOR ".", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
