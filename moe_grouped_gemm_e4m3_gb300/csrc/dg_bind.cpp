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
#include <ATen/ops/empty.h>
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
constexpr uint32_t kByte = bit(at::ScalarType::Byte);
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
  int device = -1;   // of the first tensor; `here` looks whether it is every tensor's and the current one
  bool one_device = true;

  void* ptr(PyObject* o, uint32_t types, at::IntArrayRef shape) {
    if (!ok) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!t || !t->defined() || t->layout() != at::kStrided || !t->is_cuda() || (int)t->scalar_type() >= 32 ||
        !(types & bit(t->scalar_type())) || t->sizes() != shape || !t->is_contiguous()) {
      ok = false;
      return nullptr;
    }
    if (device < 0) device = t->get_device();
    one_device &= device == t->get_device();
    return t->data_ptr();
  }
  void here() { ok = ok && one_device && device == c10::cuda::current_device(); }
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
int (*g_norm[4])(P, P, P, P, P, P, double, P, P, P, P, P, P, int, int, P);   // bit 0 FP32 stream, bit 1 packed scales
int (*g_norm_backward[2])(P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, long long, int, int, P);
int (*g_route[2][2])(P, P, P, P, int, int, double, int, int, int, P);   // forward, backward; FP32, BF16 logits
int (*g_moe[6])(P, P, P, P, P, P, P, P, P, P, long long, int, int, int, int, int, int, P);   // bit 0 FP32 output, then the weights' form
int (*g_mxfp4[2])(P, P, P, P, P, int, int, int, P);
long long (*g_norm_workspace)(int, int);
long long (*g_moe_workspace)(int, int, int);
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

// A workspace: the caller's uint8 tensor, or memory of torch's allocator on the current stream (with another stream given,
// Python sees to it). The tensor is kept until the call has been made; what reuses its memory comes later on the stream.
struct Workspace {
  at::Tensor own;
  P at = nullptr;
  long long bytes = 0;
  void take(Check& c, PyObject* given, PyObject* stream, long long need) {
    if (!c.ok) return;
    if (given != Py_None) {
      const at::Tensor* t = tensor(given);
      if (!t || !t->defined() || t->dim() != 1) {
        c.ok = false;
        return;
      }
      at = c.ptr(given, kByte, t->sizes());
      c.here();
      bytes = t->numel();
    } else if (stream != Py_None) {
      c.ok = false;
    } else if (need > 0) {
      own = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)c.device));
      at = own.data_ptr();
      bytes = need;
    }
  }
};

// norm(ue8m0, X, B, w_after, gate, scale, W, eps, R, Y, Yq, sY, rstd, rstd_after, stream)
PyObject* norm(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int ue;
  if (n != 15 || !variant(c, a[0], 2, &ue)) return not_here();
  const auto xs = c.sizes(a[1], 2);
  if (!c.ok) return not_here();
  const int64_t M = xs[0], N = xs[1];
  const bool f32 = tensor(a[1])->scalar_type() == at::ScalarType::Float;
  const uint32_t t = f32 ? kF32 : kBf16;
  P x = c.ptr(a[1], t, {M, N}), b = c.opt(a[2], t, {M, N}), wa = c.opt(a[3], kF32, {N}), gate = c.opt(a[4], kF32, {M}),
    scale = c.opt(a[5], kF32, {N}), w = c.opt(a[6], kF32, {N});
  const double eps = c.real(a[7]);
  P r = c.opt(a[8], t, {M, N}), y = c.opt(a[9], t, {M, N}), q = c.opt(a[10], kFp8, {M, N});
  P sq = c.opt(a[11], ue ? kI32 : kF32, {groups(N, ue), align4(M)}), rstd = c.opt(a[12], kF32, {M}), after = c.opt(a[13], kF32, {M});
  c.here();
  P s = c.stream(a[14]);
  const int m = c.size(M), nn = c.size(N);
  if (!c.ok) return not_here();
  return status_of(g_norm[f32 + 2 * ue], x, b, wa, gate, scale, w, eps, r, y, q, sq, rstd, after, m, nn, s);
}

// norm_backward(dY, dR, R, B, W, w_after, gate, scale, rstd, rstd_after, dX, dB, dW, dw_after, dgate, dscale, workspace, stream)
PyObject* norm_backward(PyObject* const* a, Py_ssize_t n) {
  Check c;
  if (n != 18 || !g_loaded) return not_here();
  PyObject* first = a[0] != Py_None ? a[0] : a[1];
  const auto xs = c.sizes(first, 2);
  if (!c.ok) return not_here();
  const int64_t M = xs[0], N = xs[1];
  const bool f32 = tensor(first)->scalar_type() == at::ScalarType::Float;
  const uint32_t t = f32 ? kF32 : kBf16;
  P p[16];
  // M x N of the stream's type, N, or M values
  static const char kind[17] = "xxxxnnmnmmxxnnmn";
  for (int i = 0; i < 16; ++i)
    p[i] = kind[i] == 'x' ? c.opt(a[i], t, {M, N}) : c.opt(a[i], kF32, {kind[i] == 'n' ? N : M});
  c.here();
  P s = c.stream(a[17]);
  const int m = c.size(M), nn = c.size(N);
  Workspace ws;
  ws.take(c, a[16], a[17], c.ok && (p[12] || p[13] || p[15]) ? g_norm_workspace(m, nn) : 0);
  if (!c.ok) return not_here();
  return status_of(g_norm_backward[f32], p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11], p[12], p[13], p[14], p[15],
                   ws.at, ws.bytes, m, nn, s);
}

// route(backward, logits, bias or dweights, ids, weights or dlogits, score, renormalize, factor, stream)
PyObject* route(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int back;
  if (n != 9 || !variant(c, a[0], 2, &back)) return not_here();
  const auto ls = c.sizes(a[1], 2), is = c.sizes(a[3], 2);
  if (!c.ok) return not_here();
  const int64_t T = ls[0], E = ls[1], k = is[1];
  const bool bf16 = tensor(a[1])->scalar_type() != at::ScalarType::Float;
  const uint32_t t = bf16 ? kBf16 : kF32;
  P l = c.ptr(a[1], t, {T, E}), ids = c.ptr(a[3], kI32, {T, k});
  P in = back ? c.ptr(a[2], kF32, {T, k}) : c.opt(a[2], kF32, {E}), out = back ? c.ptr(a[4], t, {T, E}) : c.ptr(a[4], kF32, {T, k});
  const int64_t score = c.integer(a[5]);
  if (!PyBool_Check(a[6])) c.ok = false;
  const int renorm = a[6] == Py_True;
  const double factor = c.real(a[7]);
  c.here();
  P s = c.stream(a[8]);
  const int tt = c.size(T), e = c.size(E), kk = c.size(k), how = c.size(score);
  if (!c.ok) return not_here();
  return back ? status_of(g_route[1][bf16], in, l, ids, out, how, renorm, factor, tt, e, kk, s)
              : status_of(g_route[0][bf16], l, in, ids, out, how, renorm, factor, tt, e, kk, s);
}

// moe(variant, A, sA, W1, sW1, W2, sW2, ids, weights, Y, workspace, stream)
PyObject* moe(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int v;
  if (n != 12 || !variant(c, a[0], 6, &v)) return not_here();
  const bool f32 = v & 1, ue = v / 2 == 1, four = v / 2 == 2;
  const auto as = c.sizes(a[1], 2), w1 = c.sizes(a[3], 3), w2 = c.sizes(a[5], 3), is = c.sizes(a[7], 2);
  if (!c.ok) return not_here();
  const int64_t T = as[0], K = as[1], E = w1[0], I = w1[1] / 2, N = w2[1], k = is[1], per = four ? 2 : 1;
  if (w1[1] % 2 || w1[2] * per != K || w2[0] != E || w2[2] * per != I) return not_here();
  const uint32_t st = ue ? kI32 : kF32, qt = four ? kByte : kFp8;
  P A = c.ptr(a[1], kFp8, {T, K}), sA = c.ptr(a[2], st, {groups(K, ue), align4(T)}), W1 = c.ptr(a[3], qt, w1), W2 = c.ptr(a[5], qt, w2);
  P s1 = four ? c.ptr(a[4], kByte, {E, 2 * I, K / 32}) : c.ptr(a[4], st, {E, cdiv(2 * I, 128), groups(K, ue)});
  P s2 = four ? c.ptr(a[6], kByte, {E, N, I / 32}) : c.ptr(a[6], st, {E, cdiv(N, 128), groups(I, ue)});
  P ids = c.ptr(a[7], kI32, {T, k}), w = c.ptr(a[8], kF32, {T, k}), Y = c.ptr(a[9], f32 ? kF32 : kBf16, {T, N});
  c.here();
  P s = c.stream(a[11]);
  const int t = c.size(T), kk = c.size(k), e = c.size(E), K_ = c.size(K), I_ = c.size(I), N_ = c.size(N);
  Workspace ws;
  ws.take(c, a[10], a[11], c.ok ? g_moe_workspace(t, kk, I_) : 0);
  if (!c.ok) return not_here();
  return status_of(g_moe[v], A, sA, W1, s1, W2, s2, ids, w, Y, ws.at, ws.bytes, t, kk, e, K_, I_, N_, s);
}

// mxfp4(FP32 output, A, sA, B, sB, D, stream)
PyObject* mxfp4(PyObject* const* a, Py_ssize_t n) {
  Check c;
  int f32;
  if (n != 7 || !variant(c, a[0], 2, &f32)) return not_here();
  const auto as = c.sizes(a[1], 2), bs = c.sizes(a[3], 2);
  if (!c.ok) return not_here();
  const int64_t M = as[0], K = as[1], N = bs[0];
  if (K % 32) return not_here();
  P A = c.ptr(a[1], kFp8, {M, K}), sA = c.ptr(a[2], kF32, {cdiv(K, 128), align4(M)}), B = c.ptr(a[3], kByte, {N, K / 2}),
    sB = c.ptr(a[4], kByte, {N, K / 32}), D = c.ptr(a[5], f32 ? kF32 : kBf16, {M, N});
  c.here();
  P s = c.stream(a[6]);
  const int m = c.size(M), nn = c.size(N), k = c.size(K);
  if (!c.ok) return not_here();
  return status_of(g_mxfp4[f32], A, sA, B, sB, D, m, nn, k, s);
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
  static const char* const forms[3] = {"", "_ue8m0", "_mxfp4"};
  for (int f = 0; ok && f < 2; ++f) {
    const std::string type = f ? "f32" : "bf16", tail = f ? "_f32" : "";
    ok = find(lib, g_norm[f], "dg_residual_norm_" + type) && find(lib, g_norm[2 + f], "dg_residual_norm_" + type + "_ue8m0") &&
         find(lib, g_norm_backward[f], "dg_residual_norm_backward_" + type) && find(lib, g_route[0][1 - f], "dg_route_topk_" + type) &&
         find(lib, g_route[1][1 - f], "dg_route_topk_backward_" + type) && find(lib, g_mxfp4[f], "dg_fp8_mxfp4_gemm_nt" + tail);
    for (int i = 0; ok && i < 3; ++i) ok = find(lib, g_moe[2 * i + f], std::string("dg_fp8_moe_swiglu") + forms[i] + tail);
  }
  ok = ok && find(lib, g_norm_workspace, "dg_residual_norm_backward_workspace") && find(lib, g_moe_workspace, "dg_fp8_moe_workspace");
  g_loaded = ok;
  return PyBool_FromLong(ok);
}

// The version of torch whose headers this was compiled against.
PyObject* version(PyObject*, PyObject*) { return PyUnicode_FromString(TORCH_VERSION); }

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(gated), FAST(dense), FAST(contiguous), FAST(k_grouped), FAST(backward), FAST(cast), FAST(dropout),
                           FAST(norm), FAST(norm_backward), FAST(route), FAST(moe), FAST(mxfp4),
                           {"load", load, METH_O, nullptr}, {"version", version, METH_NOARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_dgbind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dgbind() { return PyModule_Create(&g_module); }
