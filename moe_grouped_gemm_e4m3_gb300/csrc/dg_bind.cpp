// dg_bind.cpp — the short path of the Python binding: the argument checks and the C call of the entry points
// that a training or decode step makes, without Python between them.
//
// A step of a small layer runs kernels of a few microseconds, and a call's checks in Python (five attributes
// of every tensor) cost as much: cast of 64x7168 rows 7.4 us of host time a call, 3.0 of them the library's. Each
// function here takes the entry point's arguments, makes the same checks as the Python path (of every tensor
// its type, its shape, that it is a CUDA tensor and that it is contiguous) and calls the library. Where anything is not as it should be it
// returns None and calls nothing: the Python path then looks again and raises the error. So there is one set
// of error messages, and without this module everything works, more slowly. Torch's accessors throw (the sizes of
// a nested tensor, the data of a fake one, the current stream without a driver): every function is called through
// `guarded`, which makes that a None as well, so that no C++ exception reaches the interpreter.
//
// Host code only; compiled against the headers of the torch installation that it runs with (version()).
#include <Python.h>

#include <dlfcn.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <initializer_list>
#include <string>

namespace {

constexpr uint32_t bit(at::ScalarType t) { return 1u << (int)t; }
static_assert((int)at::ScalarType::Float8_e4m3fn < 32 && (int)at::ScalarType::UInt64 < 32, "type masks are 32 bits");
constexpr uint32_t kFp8 = bit(at::ScalarType::Byte) | bit(at::ScalarType::Float8_e4m3fn);
constexpr uint32_t kBf16 = bit(at::ScalarType::BFloat16) | bit(at::ScalarType::Short) | bit(at::ScalarType::UInt16);
constexpr uint32_t kF32 = bit(at::ScalarType::Float);
constexpr uint32_t kI32 = bit(at::ScalarType::Int);
constexpr uint32_t kRng = bit(at::ScalarType::Long) | bit(at::ScalarType::UInt64);

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align4(int64_t x) { return cdiv(x, 4) * 4; }
// Scale entries along an axis of n elements: one a 128, or one packed word a 512.
int64_t groups(int64_t n, bool ue) { return ue ? cdiv(cdiv(n, 128), 4) : cdiv(n, 128); }

using Shape = std::initializer_list<int64_t>;

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// One call's arguments: the first that is not as it should be makes the whole call "not here".
struct Check {
  bool ok = true;

  void* ptr(PyObject* o, uint32_t types, at::IntArrayRef shape) {
    if (!ok) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!t || !t->defined() || t->layout() != at::kStrided || !t->is_cuda() || (int)t->scalar_type() >= 32 ||
        !(types & bit(t->scalar_type())) || t->sizes() != shape || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  void* ptr(PyObject* o, uint32_t types, Shape shape) { return ptr(o, types, at::IntArrayRef(shape.begin(), shape.size())); }
  void* opt(PyObject* o, uint32_t types, Shape shape) { return o == Py_None ? nullptr : ptr(o, types, shape); }
  void* opt(PyObject* o, uint32_t types, at::IntArrayRef shape) { return o == Py_None ? nullptr : ptr(o, types, shape); }

  // The sizes of a tensor of this many dimensions.
  at::IntArrayRef sizes(PyObject* o, size_t dims) {
    const at::Tensor* t = ok ? tensor(o) : nullptr;
    if (!t || !t->defined() || t->layout() != at::kStrided || (size_t)t->dim() != dims) {
      ok = false;
      static const int64_t zeros[3] = {0, 0, 0};
      return at::IntArrayRef(zeros, 3);
    }
    return t->sizes();
  }
  int64_t integer(PyObject* o) {
    if (!ok || !PyLong_CheckExact(o)) return ok = false, 0;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return v;
  }
  double real(PyObject* o) {
    if (!ok || !(PyFloat_CheckExact(o) || PyLong_CheckExact(o))) return ok = false, 0.0;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return v;
  }
  // None: torch's current stream; otherwise anything with a cuda_stream is left to Python, which passes the number.
  void* stream(PyObject* o) {
    if (!ok) return nullptr;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    return reinterpret_cast<void*>(integer(o));
  }
  // A size as the library takes it.
  int size(int64_t v) {
    if (v < 0 || v > INT32_MAX) ok = false;
    return (int)v;
  }
};

PyObject* not_here() { Py_RETURN_NONE; }

// The call itself, with the interpreter's lock released, as ctypes does: a launch waits when the stream's queue is full, and
// a first call may allocate.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... Args>
PyObject* status_of(F f, Args... args) {
  int status;
  {
    Unlocked u;
    status = f(args...);
  }
  return PyLong_FromLong(status);
}

using P = void*;
// The library's entry points, by variant: bit 0 FP32 output, bit 1 packed UE8M0 scales.
int (*g_gated[4])(P, P, P, P, P, P, P, double, int, int, int, P);
int (*g_gated_grouped[4])(P, P, P, P, P, P, P, P, double, int, int, int, int, P);
int (*g_dense[4][4])(P, P, P, P, P, int, int, int, P);   // nt, nn, tn, tt
int (*g_contiguous[2][4])(P, P, P, P, P, P, int, int, int, int, P);   // nt, nn
int (*g_kgrouped[4])(P, P, P, P, P, P, int, int, int, int, P);
int (*g_backward[2])(P, P, P, P, double, P, P, P, P, P, P, int, int, P);
int (*g_cast[2])(P, P, P, P, P, P, P, P, P, int, int, int, P);
int (*g_dropout[2])(P, P, P, P, double, long long, P);
bool g_loaded = false;

bool variant(Check& c, PyObject* o, int most, int* v) {
  const int64_t x = c.integer(o);
  if (!g_loaded || x < 0 || x >= most) c.ok = false;
  *v = (int)x;
  return c.ok;
}

// gated(variant, A, sA, B, sB, m_indices or None (dense), H, GU, rng, p, stream); variant + 4: contiguous
PyObject* gated(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int v;
  if (n != 11 || !variant(c, a[0], 8, &v)) return not_here();
  const bool f32 = v & 1, ue = v & 2, grouped = v & 4;
  const auto as = c.sizes(a[1], 2), bs = c.sizes(a[3], grouped ? 3 : 2);
  if (!c.ok) return not_here();
  const int64_t M = as[0], K = as[1], G = grouped ? bs[0] : 1, N = bs[grouped ? 1 : 0], nk = groups(K, ue);
  if (bs[grouped ? 2 : 1] != K || N % 2) return not_here();
  const uint32_t st = ue ? kI32 : kF32;
  P A = c.ptr(a[1], kFp8, {M, K}), sA = c.ptr(a[2], st, {nk, align4(M)}), B = c.ptr(a[3], kFp8, bs);
  P sB = grouped ? c.ptr(a[4], st, {G, cdiv(N, 128), nk}) : c.ptr(a[4], st, {cdiv(N, 128), nk});
  P idx = grouped ? c.ptr(a[5], kI32, {M}) : nullptr;
  P H = c.ptr(a[6], f32 ? kF32 : kBf16, {M, N / 2}), GU = c.opt(a[7], kBf16, {M, N}), rng = c.opt(a[8], kRng, {2});
  const double p = c.real(a[9]);
  P s = c.stream(a[10]);
  const int m = c.size(M), nn = c.size(N), k = c.size(K), g = c.size(G);
  if (!c.ok) return not_here();
  return grouped ? status_of(g_gated_grouped[v & 3], A, sA, B, sB, idx, H, GU, rng, p, m, nn, k, g, s)
                 : status_of(g_gated[v & 3], A, sA, B, sB, H, GU, rng, p, m, nn, k, s);
}

// dense(variant + 4 · layout (nt, nn, tn, tt), A, sA, B, sB, D, M, N, K, stream)
PyObject* dense(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int v;
  if (n != 10 || !variant(c, a[0], 16, &v)) return not_here();
  const int layout = v >> 2;
  const bool f32 = v & 1, ue = v & 2, a_t = layout >= 2, b_n = layout == 1 || layout == 2;
  const int64_t M = c.integer(a[6]), N = c.integer(a[7]), K = c.integer(a[8]);
  const int m = c.size(M), nn = c.size(N), k = c.size(K);
  if (!c.ok) return not_here();
  const uint32_t st = ue ? kI32 : kF32;
  P A = a_t ? c.ptr(a[1], kFp8, {K, M}) : c.ptr(a[1], kFp8, {M, K}), sA = c.ptr(a[2], st, {groups(K, ue), align4(M)});
  P B = b_n ? c.ptr(a[3], kFp8, {K, N}) : c.ptr(a[3], kFp8, {N, K}), sB = c.ptr(a[4], st, {cdiv(N, 128), groups(K, ue)});
  P D = c.ptr(a[5], f32 ? kF32 : kBf16, {M, N});
  P s = c.stream(a[9]);
  if (!c.ok) return not_here();
  return status_of(g_dense[layout][v & 3], A, sA, B, sB, D, m, nn, k, s);
}

// contiguous(variant + 4 · (B stored [G, K, N]), A, sA, B, sB, m_indices, D, stream)
PyObject* contiguous(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int v;
  if (n != 8 || !variant(c, a[0], 8, &v)) return not_here();
  const bool f32 = v & 1, ue = v & 2, b_n = v & 4;
  const auto as = c.sizes(a[1], 2), bs = c.sizes(a[3], 3);
  if (!c.ok) return not_here();
  const int64_t M = as[0], K = as[1], G = bs[0], N = bs[b_n ? 2 : 1];
  if (bs[b_n ? 1 : 2] != K) return not_here();
  const uint32_t st = ue ? kI32 : kF32;
  P A = c.ptr(a[1], kFp8, {M, K}), sA = c.ptr(a[2], st, {groups(K, ue), align4(M)}), B = c.ptr(a[3], kFp8, bs);
  P sB = c.ptr(a[4], st, {G, cdiv(N, 128), groups(K, ue)}), idx = c.ptr(a[5], kI32, {M});
  P D = c.ptr(a[6], f32 ? kF32 : kBf16, {M, N});
  P s = c.stream(a[7]);
  const int m = c.size(M), nn = c.size(N), k = c.size(K), g = c.size(G);
  if (!c.ok) return not_here();
  return status_of(g_contiguous[b_n][v & 3], A, sA, B, sB, idx, D, m, nn, k, g, s);
}

// k_grouped(variant, A, sA, B, sB, k_offsets, D, stream)
PyObject* k_grouped(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int v;
  if (n != 8 || !variant(c, a[0], 4, &v)) return not_here();
  const bool f32 = v & 1, ue = v & 2;
  const auto as = c.sizes(a[1], 2), bs = c.sizes(a[3], 2), os = c.sizes(a[5], 1);
  if (!c.ok || os[0] < 1) return not_here();
  const int64_t K = as[0], M = as[1], N = bs[1], G = os[0] - 1;
  const uint32_t st = ue ? kI32 : kF32;
  P A = c.ptr(a[1], kFp8, {K, M}), sA = c.ptr(a[2], st, {groups(K, ue), align4(M)}), B = c.ptr(a[3], kFp8, {K, N});
  P sB = c.ptr(a[4], st, {cdiv(N, 128), groups(K, ue)}), off = c.ptr(a[5], kI32, {G + 1});
  P D = c.ptr(a[6], f32 ? kF32 : kBf16, {G, M, N});
  P s = c.stream(a[7]);
  const int m = c.size(M), nn = c.size(N), k = c.size(K), g = c.size(G);
  if (!c.ok) return not_here();
  return status_of(g_kgrouped[v], A, sA, B, sB, off, D, g, m, nn, k, s);
}

// backward(ue8m0, dH, GU, dGUr, sR, dGUc, sC, Hb, sHb, m_indices, rng, p, stream)
PyObject* backward(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int ue;
  if (n != 13 || !variant(c, a[0], 2, &ue)) return not_here();
  const auto hs = c.sizes(a[1], 2);
  if (!c.ok) return not_here();
  const int64_t M = hs[0], I = hs[1];
  const uint32_t st = ue ? kI32 : kF32;
  P dh = c.ptr(a[1], kBf16, {M, I}), gu = c.ptr(a[2], kBf16, {M, 2 * I});
  P qr = c.opt(a[3], kFp8, {M, 2 * I}), sr = c.opt(a[4], st, {groups(2 * I, ue), align4(M)});
  P qc = c.opt(a[5], kFp8, {M, 2 * I}), sc = c.opt(a[6], st, {groups(M, ue), 2 * I});
  P hb = c.opt(a[7], kFp8, {M, I}), sh = c.opt(a[8], st, {cdiv(I, 128), groups(M, ue)});
  P idx = c.opt(a[9], kI32, {M}), rng = c.opt(a[10], kRng, {2});
  const double p = c.real(a[11]);
  P s = c.stream(a[12]);
  const int m = c.size(M), i = c.size(I);
  if (!c.ok) return not_here();
  return status_of(g_backward[ue], dh, gu, idx, rng, p, qr, sr, qc, sc, hb, sh, m, i, s);
}

// cast(ue8m0, X, Xr, sR, Xc, sC, Xb, sB, sBt, m_indices, stream), of one matrix [M, N]
PyObject* cast(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int ue;
  if (n != 11 || !variant(c, a[0], 2, &ue)) return not_here();
  const auto xs = c.sizes(a[1], 2);
  if (!c.ok) return not_here();
  const int64_t M = xs[0], N = xs[1], Mb = cdiv(M, 128), Nb = cdiv(N, 128);
  const uint32_t st = ue ? kI32 : kF32;
  P x = c.ptr(a[1], kBf16, {M, N});
  P qr = c.opt(a[2], kFp8, {M, N}), sr = c.opt(a[3], st, {groups(N, ue), align4(M)});
  P qc = c.opt(a[4], kFp8, {M, N}), sc = c.opt(a[5], st, {groups(M, ue), align4(N)});
  P qb = c.opt(a[6], kFp8, {M, N}), sb = c.opt(a[7], st, {Mb, groups(N, ue)}), sbt = c.opt(a[8], st, {Nb, groups(M, ue)});
  P idx = c.opt(a[9], kI32, {M});
  P s = c.stream(a[10]);
  const int m = c.size(M), nn = c.size(N);
  if (!c.ok) return not_here();
  return status_of(g_cast[ue], x, idx, qr, sr, qc, sc, qb, sb, sbt, 1, m, nn, s);
}

// dropout(X, R, Y, rng, p, stream)
PyObject* dropout(PyObject* const* a, Py_ssize_t n) {
  Check c;
  const at::Tensor* x = n == 6 && g_loaded ? tensor(a[0]) : nullptr;
  if (!x || !x->defined() || x->layout() != at::kStrided) return not_here();
  const bool f32 = x->scalar_type() == at::ScalarType::Float;
  const uint32_t type = f32 ? kF32 : kBf16;
  P px = c.ptr(a[0], type, x->sizes()), pr = c.opt(a[1], type, x->sizes()), py = c.ptr(a[2], type, x->sizes());
  P rng = c.opt(a[3], kRng, {2});
  const double p = c.real(a[4]);
  P s = c.stream(a[5]);
  if (!c.ok) return not_here();
  return status_of(g_dropout[f32], px, pr, py, rng, p, x->numel(), s);
}

// The function as Python calls it: an exception of torch's is one more "not here".
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (...) {
    PyErr_Clear();
    return not_here();
  }
}

template <typename F>
bool find(void* lib, F& f, const std::string& name) {
  f = reinterpret_cast<F>(dlsym(lib, name.c_str()));
  return f != nullptr;
}

// load(path of libdg.so): whether every entry point was found
PyObject* load(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW);
  bool ok = lib != nullptr;
  static const char* const layouts[4] = {"nt", "nn", "tn", "tt"};
  for (int v = 0; ok && v < 4; ++v) {
    const std::string tail = std::string(v & 2 ? "_ue8m0" : "") + (v & 1 ? "_f32" : "");
    ok = find(lib, g_gated[v], "dg_fp8_gemm_nt_swiglu" + tail) && find(lib, g_gated_grouped[v], "dg_fp8_grouped_contiguous_swiglu" + tail) &&
         find(lib, g_contiguous[0][v], "dg_fp8_grouped_contiguous" + tail) && find(lib, g_contiguous[1][v], "dg_fp8_grouped_contiguous_nn" + tail) &&
         find(lib, g_kgrouped[v], "dg_fp8_k_grouped_gemm_tn_contiguous" + tail);
    for (int l = 0; ok && l < 4; ++l) ok = find(lib, g_dense[l][v], std::string("dg_fp8_gemm_") + layouts[l] + tail);
  }
  for (int ue = 0; ok && ue < 2; ++ue)
    ok = find(lib, g_backward[ue], ue ? "dg_swiglu_backward_fp8_ue8m0" : "dg_swiglu_backward_fp8") &&
         find(lib, g_cast[ue], ue ? "dg_cast_fp8_ue8m0" : "dg_cast_fp8") &&
         find(lib, g_dropout[ue], ue ? "dg_dropout_f32" : "dg_dropout_bf16");
  g_loaded = ok;
  return PyBool_FromLong(ok);
}

// The version of torch whose headers this was compiled against.
PyObject* version(PyObject*, PyObject*) { return PyUnicode_FromString(TORCH_VERSION); }

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(gated), FAST(dense), FAST(contiguous), FAST(k_grouped), FAST(backward), FAST(cast), FAST(dropout),
                           {"load", load, METH_O, nullptr}, {"version", version, METH_NOARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_dgbind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dgbind() { return PyModule_Create(&g_module); }
