// Argument marshalling of the Python binding's short calls, compiled: the checks, allocations and the
// call into liblowbit.so of adapter_gemm, adapter_backward, gemm_dx and the 8-bit copies. A call's host
// time with it and in Python: 10.2 and 19.0 us for one token (6 us on the GPU), 17.2 and 30.7 for the
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

#define LOWBIT_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LOWBIT_METHOD(adapter_gemm),     LOWBIT_METHOD(gemm_dx),         LOWBIT_METHOD(adapter_backward),
                         LOWBIT_METHOD(checkpoint_store), LOWBIT_METHOD(checkpoint_load), {nullptr, nullptr, 0, nullptr}};
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
