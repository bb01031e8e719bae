// Argument marshalling of the Python binding's short calls, compiled: the checks, allocations and the
// call into liblowbit.so of adapter_gemm, adapter_backward, gemm_dx, the 8-bit copies and the vocabulary calls. A call's
// host time with it and in Python: 10.2 and 19.0 us for one token (6 us on the GPU), 17.2 and 30.7 for the
// backward of 77 tokens, 5.6 and 10.9 for the 8-bit copy of 77 x 2560 values.
//
// Each function returns its outputs, or the library's status as an int if that is not 0, or None if
// the arguments are not what a correct call passes: the binding then goes through its own checks,
// which name what is wrong. The library's entry points come as addresses, so that whichever build of
// it is loaded is the one that is called.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "lowbit.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr ScalarType kBf16 = at::kBFloat16, kF16 = at::kHalf, kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte;
constexpr ScalarType kF8 = at::kFloat8_e4m3fn;

struct Unfit {};   // the arguments are left to the binding's own checks

const Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) throw Unfit{};
    return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unfit{};
    }
    return v;
}
template <class F>
F function(PyObject* o) {
    return reinterpret_cast<F>(static_cast<uintptr_t>(integer(o)));
}
void need(bool ok) {
    if (!ok) throw Unfit{};
}
void fits(const Tensor& t, ScalarType type, at::IntArrayRef shape, at::Device dev) {
    need(t.scalar_type() == type && t.device() == dev && t.layout() == at::kStrided && t.sizes() == shape &&
         t.is_contiguous());
}
void* ptr(const Tensor& t) { return t.data_ptr(); }

// A tensor argument that may be None.
struct Maybe {
    Tensor t;
    bool given;
    Maybe(PyObject* o, ScalarType type, at::IntArrayRef shape, at::Device dev) : given(o != Py_None) {
        if (given) {
            t = tensor(o);
            fits(t, type, shape, dev);
        }
    }
    void* ptr() const { return given ? t.data_ptr() : nullptr; }
};
// The same for an output: allocated where it is not given.
Tensor output(PyObject* o, at::IntArrayRef shape, const Tensor& like) {
    if (o == Py_None) return at::empty(shape, like.options());
    const Tensor& t = tensor(o);
    fits(t, kBf16, shape, like.device());
    return t;
}

// x [M][K] with W's words, or dy [M][N] with W^T's.
struct Linear {
    Tensor in, words, scales;
    Maybe zeros;
    int64_t M, N, K;
    int bits, group;
    at::Device dev;

    static int between(PyObject* o, int lo, int hi) {
        const int64_t n = integer(o);
        need(n >= lo && n <= hi);
        return static_cast<int>(n);
    }
    static at::DimVector groups(const Tensor& scales) {
        need(scales.dim() == 2);
        return at::DimVector{scales.size(0), scales.size(1)};
    }
    Linear(PyObject* in_, PyObject* words_, PyObject* scales_, PyObject* zeros_, PyObject* bits_, PyObject* group_,
           bool transposed)
        : in(tensor(in_)), words(tensor(words_)), scales(tensor(scales_)),
          zeros(zeros_, kF16, groups(scales), tensor(in_).device()), bits(between(bits_, 1, 4)),
          group(between(group_, 1, 1 << 20)), dev(in.device()) {
        need(in.is_cuda() && in.dim() == 2 && words.dim() == 2 && bits != 3);
        fits(in, kBf16, in.sizes(), dev);
        M = in.size(0);
        N = scales.size(1);
        K = transposed ? words.size(0) : in.size(1);
        need(K % group == 0 && (!transposed || in.size(1) == N));
        fits(scales, kF16, {K / group, N}, dev);
        if (transposed)
            fits(words, kI32, {K, (N + 127) / 128 * 128 * bits / 32}, dev);
        else
            fits(words, kI32, {N, K * bits / 32}, dev);
    }
};

struct Adapters {
    Tensor a, b, scaling;
    Maybe index;
    int64_t L, R;
    lowbit_adapters c;
    static const Tensor& three(PyObject* o) {
        const Tensor& t = tensor(o);
        need(t.dim() == 3);
        return t;
    }
    Adapters(PyObject* a_, PyObject* b_, PyObject* s_, PyObject* i_, const Linear& l)
        : a(three(a_)), b(tensor(b_)), scaling(tensor(s_)), index(i_, kI32, {l.M}, l.dev), L(a.size(0)), R(a.size(1)) {
        fits(a, kBf16, {L, R, l.K}, l.dev);
        fits(b, kBf16, {L, l.N, R}, l.dev);
        fits(scaling, kF32, {L}, l.dev);
        need(L < (int64_t(1) << 31) && R < (int64_t(1) << 31));
        c.num = static_cast<int>(L);
        c.rank = static_cast<int>(R);
        c.A = ptr(a);
        c.B = ptr(b);
        c.scaling = static_cast<const float*>(ptr(scaling));
        c.index = static_cast<const int32_t*>(index.ptr());
    }
};

// The call's workspace: given, or allocated on the current stream (which the caching allocator ties it
// to, as to the pool of a graph under capture).
struct Workspace {
    Tensor t;
    size_t bytes;
    Workspace(PyObject* given, PyObject* size_fn, const Linear& l, int64_t num, int64_t rank) {
        if (given != Py_None) {
            t = tensor(given);
            need(t.dim() == 1);
            fits(t, kU8, t.sizes(), l.dev);
            bytes = static_cast<size_t>(t.numel());
            return;
        }
        const auto size = function<decltype(&lowbit_adapter_workspace_size)>(size_fn);
        need(num < (int64_t(1) << 31) && rank < (int64_t(1) << 31));
        bytes = size(l.M, l.N, l.K, static_cast<int>(num), static_cast<int>(rank));
        t = at::empty({static_cast<int64_t>(bytes) + 1}, l.in.options().dtype(kU8));
    }
};

template <class F>
lowbit_status without_gil(F call) {
    lowbit_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    return st;
}
void* stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// Runs `body`; None where the arguments do not fit or PyTorch refuses something (the binding's own path
// then meets the same and reports it).
template <class F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F body) {
    if (have != want) {
        PyErr_SetString(PyExc_TypeError, "marshal: wrong number of arguments");
        return nullptr;
    }
    try {
        return body();
    } catch (const Unfit&) {
    } catch (const std::exception&) {
    }
    Py_RETURN_NONE;
}
PyObject* status(lowbit_status st) { return PyLong_FromLong(st); }

// (fn, size_fn, x, packed, scales, zeros, bits, group, a, b, scaling, index, out, p, codes, exps, ws)
PyObject* adapter_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 17, [&]() -> PyObject* {
        const Linear l(v[2], v[3], v[4], v[5], v[6], v[7], false);
        const Adapters ad(v[8], v[9], v[10], v[11], l);
        const c10::cuda::CUDAGuard guard(l.dev);
        const Tensor out = output(v[12], {l.M, l.N}, l.in);
        const Maybe p(v[13], kBf16, {l.M, ad.R}, l.dev);
        need((v[14] == Py_None) == (v[15] == Py_None) && (v[14] == Py_None || l.K % 32 == 0));
        const Maybe codes(v[14], kF8, {l.M, l.K}, l.dev), exps(v[15], kU8, {l.M, l.K / 32}, l.dev);
        const Workspace ws(v[16], v[1], l, ad.L, ad.R);
        const auto fn = function<decltype(&lowbit_adapter_gemm)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(l.M, l.N, l.K, l.bits, l.group, ptr(l.in), static_cast<const uint32_t*>(ptr(l.words)), ptr(l.scales),
                      l.zeros.ptr(), &ad.c, ptr(out), p.ptr(), static_cast<uint8_t*>(codes.ptr()),
                      static_cast<uint8_t*>(exps.ptr()), ptr(ws.t), ws.bytes, stream_of(l.dev));
        });
        return st == LOWBIT_OK ? THPVariable_Wrap(out) : status(st);
    });
}

// (fn, size_fn, dy, packed_t, scales, zeros, bits, group, out, ws)
PyObject* gemm_dx(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const Linear l(v[2], v[3], v[4], v[5], v[6], v[7], true);
        const c10::cuda::CUDAGuard guard(l.dev);
        const Tensor out = output(v[8], {l.M, l.K}, l.in);
        const Workspace ws(v[9], v[1], l, 0, 0);
        const auto fn = function<decltype(&lowbit_gemm_dx)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(l.M, l.N, l.K, l.bits, l.group, ptr(l.in), static_cast<const uint32_t*>(ptr(l.words)), ptr(l.scales),
                      l.zeros.ptr(), ptr(out), ptr(ws.t), ws.bytes, stream_of(l.dev));
        });
        return st == LOWBIT_OK ? THPVariable_Wrap(out) : status(st);
    });
}

// (fn, size_fn, dy, packed_t, scales, zeros, bits, group, a, b, scaling, index, x, codes, exps, p, dx, da, db,
//  need_dx, ws); x or codes and exps are None
PyObject* adapter_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 21, [&]() -> PyObject* {
        const Linear l(v[2], v[3], v[4], v[5], v[6], v[7], true);
        const Adapters ad(v[8], v[9], v[10], v[11], l);
        const Maybe x(v[12], kBf16, {l.M, l.K}, l.dev);
        need(l.K % 32 == 0 && (v[13] == Py_None) == (v[14] == Py_None) && x.given == (v[13] == Py_None));
        const Maybe codes(v[13], kF8, {l.M, l.K}, l.dev), exps(v[14], kU8, {l.M, l.K / 32}, l.dev);
        const Tensor& p = tensor(v[15]);
        fits(p, kBf16, {l.M, ad.R}, l.dev);
        need(v[19] == Py_True || v[19] == Py_False);
        const bool need_dx = v[19] == Py_True;
        need(need_dx || v[16] == Py_None);
        const c10::cuda::CUDAGuard guard(l.dev);
        Tensor dx;
        if (need_dx) dx = output(v[16], {l.M, l.K}, l.in);
        const Tensor da = output(v[17], {ad.L, ad.R, l.K}, l.in), db = output(v[18], {ad.L, l.N, ad.R}, l.in);
        const Workspace ws(v[20], v[1], l, ad.L, ad.R);
        const auto fn = function<decltype(&lowbit_adapter_backward)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(l.M, l.N, l.K, l.bits, l.group, ptr(l.in), static_cast<const uint32_t*>(ptr(l.words)), ptr(l.scales),
                      l.zeros.ptr(), &ad.c, x.ptr(), static_cast<const uint8_t*>(codes.ptr()),
                      static_cast<const uint8_t*>(exps.ptr()), ptr(p), need_dx ? ptr(dx) : nullptr, ptr(da), ptr(db),
                      ptr(ws.t), ws.bytes, stream_of(l.dev));
        });
        if (st != LOWBIT_OK) return status(st);
        PyObject* first = Py_None;
        if (need_dx) first = THPVariable_Wrap(dx);
        else Py_INCREF(Py_None);
        PyObject* r = PyTuple_New(3);
        PyTuple_SET_ITEM(r, 0, first);
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(da));
        PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(db));
        return r;
    });
}

// (fn, x) -> (codes, exps)
PyObject* checkpoint_store(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 2, [&]() -> PyObject* {
        const Tensor& x = tensor(v[1]);
        need(x.is_cuda() && x.dim() == 2 && x.size(1) % 32 == 0);
        fits(x, kBf16, x.sizes(), x.device());
        const int64_t M = x.size(0), K = x.size(1);
        const c10::cuda::CUDAGuard guard(x.device());
        const Tensor codes = at::empty({M, K}, x.options().dtype(kF8)), exps = at::empty({M, K / 32}, x.options().dtype(kU8));
        const auto fn = function<decltype(&lowbit_checkpoint_store)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(ptr(x), M, K, static_cast<uint8_t*>(ptr(codes)), static_cast<uint8_t*>(ptr(exps)), stream_of(x.device()));
        });
        if (st != LOWBIT_OK) return status(st);
        PyObject* r = PyTuple_New(2);
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(codes));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(exps));
        return r;
    });
}

// (fn, codes, exps, out)
PyObject* checkpoint_load(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject* {
        const Tensor &codes = tensor(v[1]), &exps = tensor(v[2]);
        need(codes.is_cuda() && codes.dim() == 2 && codes.size(1) % 32 == 0);
        const int64_t M = codes.size(0), K = codes.size(1);
        fits(codes, kF8, {M, K}, codes.device());
        fits(exps, kU8, {M, K / 32}, codes.device());
        const c10::cuda::CUDAGuard guard(codes.device());
        Tensor out;
        if (v[3] == Py_None) {
            out = at::empty({M, K}, codes.options().dtype(kBf16));
        } else {
            out = tensor(v[3]);
            fits(out, kBf16, {M, K}, codes.device());
        }
        const auto fn = function<decltype(&lowbit_checkpoint_load)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(static_cast<const uint8_t*>(ptr(codes)), static_cast<const uint8_t*>(ptr(exps)), M, K, ptr(out),
                      stream_of(codes.device()));
        });
        return st == LOWBIT_OK ? THPVariable_Wrap(out) : status(st);
    });
}

// ---- a vocabulary ----
// A table [N][K]: weight bf16 (bits 16), or words with scales (and zeros).
struct Table {
    Tensor weight;
    int64_t N, K;
    int bits, group;
    at::Device dev;
    Tensor scales, zeros;
    const void *s = nullptr, *z = nullptr;
    Table(PyObject* w_, PyObject* s_, PyObject* z_, PyObject* b_, PyObject* g_)
        : weight(tensor(w_)), bits(Linear::between(b_, 1, 16)), group(Linear::between(g_, 0, 1 << 20)), dev(weight.device()) {
        need(weight.is_cuda() && weight.dim() == 2);
        if (bits == 16) {
            need(s_ == Py_None && z_ == Py_None);
            fits(weight, kBf16, weight.sizes(), dev);
            N = weight.size(0);
            K = weight.size(1);
            return;
        }
        need((bits == 1 || bits == 2 || bits == 4) && group > 0);
        fits(weight, kI32, weight.sizes(), dev);
        N = weight.size(0);
        K = weight.size(1) * 32 / bits;
        need(K % group == 0 && s_ != Py_None);
        scales = tensor(s_);
        fits(scales, kF16, {K / group, N}, dev);
        s = ptr(scales);
        if (z_ != Py_None) {
            zeros = tensor(z_);
            fits(zeros, kF16, {K / group, N}, dev);
            z = ptr(zeros);
        }
    }
};
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unfit{};
    }
    return v;
}
int64_t rows_of(PyObject* vocab, const Table& t) {
    const int64_t v = vocab == Py_None ? t.N : integer(vocab);
    need(v >= 1 && v <= t.N);
    return v;
}
// A workspace given, or allocated on the current stream.
struct Bytes {
    Tensor t;
    size_t bytes;
    template <class F>
    Bytes(PyObject* given, const Tensor& like, F size) {
        if (given != Py_None) {
            t = tensor(given);
            need(t.dim() == 1);
            fits(t, kU8, t.sizes(), like.device());
            bytes = static_cast<size_t>(t.numel());
            return;
        }
        bytes = size();
        t = at::empty({static_cast<int64_t>(bytes) + 1}, like.options().dtype(kU8));
    }
};
Tensor fp32_output(PyObject* o, int64_t M, const Tensor& like) {
    if (o == Py_None) return at::empty({M}, like.options().dtype(kF32));
    const Tensor& t = tensor(o);
    fits(t, kF32, {M}, like.device());
    return t;
}
const int32_t* ints(const Tensor& t) { return static_cast<const int32_t*>(ptr(t)); }
PyObject* two(PyObject* a, PyObject* b) {
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, a);
    PyTuple_SET_ITEM(r, 1, b);
    return r;
}

// (fn, tokens, weight, scales, zeros, bits, group, multiplier, out)
PyObject* embedding(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const Table t(v[2], v[3], v[4], v[5], v[6]);
        const Tensor& tokens = tensor(v[1]);
        need(tokens.dim() == 1);
        const int64_t T = tokens.size(0);
        fits(tokens, kI32, {T}, t.dev);
        const float multiplier = static_cast<float>(number(v[7]));
        const c10::cuda::CUDAGuard guard(t.dev);
        Tensor out;
        if (v[8] == Py_None) {
            out = at::empty({T, t.K}, t.weight.options().dtype(kBf16));
        } else {
            out = tensor(v[8]);
            fits(out, kBf16, {T, t.K}, t.dev);
        }
        const auto fn = function<decltype(&lowbit_embedding)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(T, t.N, t.K, t.bits, t.group, ints(tokens), ptr(t.weight), t.s, t.z, multiplier, ptr(out), stream_of(t.dev));
        });
        return st == LOWBIT_OK ? THPVariable_Wrap(out) : status(st);
    });
}

// (fn, size_fn, tokens, dy, rows, first, multiplier, out, ws)
PyObject* embedding_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const Tensor &tokens = tensor(v[2]), &dy = tensor(v[3]);
        need(dy.is_cuda() && dy.dim() == 2);
        const int64_t T = dy.size(0), K = dy.size(1), rows = integer(v[4]), first = integer(v[5]);
        fits(dy, kBf16, {T, K}, dy.device());
        fits(tokens, kI32, {T}, dy.device());
        need(rows >= 0 && first >= 0);
        const float multiplier = static_cast<float>(number(v[6]));
        const c10::cuda::CUDAGuard guard(dy.device());
        const Tensor out = output(v[7], {rows, K}, dy);
        const Bytes ws(v[8], dy, [&] { return function<decltype(&lowbit_embedding_workspace_size)>(v[1])(T, rows, K); });
        const auto fn = function<decltype(&lowbit_embedding_backward)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(T, K, first, rows, ints(tokens), ptr(dy), multiplier, ptr(out), ptr(ws.t), ws.bytes, stream_of(dy.device()));
        });
        return st == LOWBIT_OK ? THPVariable_Wrap(out) : status(st);
    });
}

// (fn, size_fn, x, labels, weight, scales, zeros, bits, group, vocab, loss, lse, ws)
PyObject* cross_entropy(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const Table t(v[4], v[5], v[6], v[7], v[8]);
        const Tensor &x = tensor(v[2]), &labels = tensor(v[3]);
        need(x.dim() == 2);
        const int64_t M = x.size(0), vocab = rows_of(v[9], t);
        fits(x, kBf16, {M, t.K}, t.dev);
        fits(labels, kI32, {M}, t.dev);
        const c10::cuda::CUDAGuard guard(t.dev);
        const Tensor loss = fp32_output(v[10], M, x), lse = fp32_output(v[11], M, x);
        const Bytes ws(v[12], x, [&] {
            return function<decltype(&lowbit_cross_entropy_workspace_size)>(v[1])(M, vocab, t.K, t.bits, 0);
        });
        const auto fn = function<decltype(&lowbit_cross_entropy)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(M, vocab, t.N, t.K, t.bits, t.group, ptr(x), ptr(t.weight), t.s, t.z, ints(labels), static_cast<float*>(ptr(loss)),
                      static_cast<float*>(ptr(lse)), ptr(ws.t), ws.bytes, stream_of(t.dev));
        });
        return st == LOWBIT_OK ? two(THPVariable_Wrap(loss), THPVariable_Wrap(lse)) : status(st);
    });
}

// (fn, size_fn, grad, x, labels, lse, weight, scales, zeros, bits, group, vocab, need_dw, dx, dw, ws)
PyObject* cross_entropy_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject* {
        const Table t(v[6], v[7], v[8], v[9], v[10]);
        const Tensor &grad = tensor(v[2]), &x = tensor(v[3]), &labels = tensor(v[4]), &lse = tensor(v[5]);
        need(x.dim() == 2);
        const int64_t M = x.size(0), vocab = rows_of(v[11], t);
        fits(x, kBf16, {M, t.K}, t.dev);
        fits(labels, kI32, {M}, t.dev);
        fits(grad, kF32, {M}, t.dev);
        fits(lse, kF32, {M}, t.dev);
        need(v[12] == Py_True || v[12] == Py_False);
        const bool need_dw = v[12] == Py_True;
        need(need_dw ? t.bits == 16 : v[14] == Py_None);
        const c10::cuda::CUDAGuard guard(t.dev);
        const Tensor dx = output(v[13], {M, t.K}, x);
        Tensor dw;
        if (need_dw) dw = output(v[14], {t.N, t.K}, x);
        const Bytes ws(v[15], x, [&] {
            return function<decltype(&lowbit_cross_entropy_workspace_size)>(v[1])(M, vocab, t.K, t.bits, need_dw ? 2 : 1);
        });
        const auto fn = function<decltype(&lowbit_cross_entropy_backward)>(v[0]);
        const lowbit_status st = without_gil([&] {
            return fn(M, vocab, t.N, t.K, t.bits, t.group, ptr(x), ptr(t.weight), t.s, t.z, ints(labels), static_cast<const float*>(ptr(lse)),
                      static_cast<const float*>(ptr(grad)), ptr(dx), need_dw ? ptr(dw) : nullptr, ptr(ws.t), ws.bytes, stream_of(t.dev));
        });
        if (st != LOWBIT_OK) return status(st);
        PyObject* second = Py_None;
        if (need_dw) second = THPVariable_Wrap(dw);
        else Py_INCREF(Py_None);
        return two(THPVariable_Wrap(dx), second);
    });
}

#define LOWBIT_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LOWBIT_METHOD(adapter_gemm),     LOWBIT_METHOD(gemm_dx),         LOWBIT_METHOD(adapter_backward),
                         LOWBIT_METHOD(checkpoint_store), LOWBIT_METHOD(checkpoint_load),
                         LOWBIT_METHOD(embedding), LOWBIT_METHOD(embedding_backward), LOWBIT_METHOD(cross_entropy),
                         LOWBIT_METHOD(cross_entropy_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject* m = PyModule_Create(&module);
    // the PyTorch whose headers this was compiled with: the binding uses it with no other
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", LOWBIT_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
