"""Refusals of the adapter, gradient and 8-bit copy entry points, without a GPU: every check runs
before anything is launched."""
import ctypes

import pytest
import torch

import bit_weight_only_w2_b200 as lb

A = 1 << 20   # a fake 256-byte-aligned address: never dereferenced, checks fail first
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return lb.load()


def adapters(**kw):
    d = dict(num=4, rank=16, A=A, B=A, scaling=A, index=A)
    d.update(kw)
    return lb.Adapters(*[d[k] for k in ("num", "rank", "A", "B", "scaling", "index")])


BASE = dict(M=16, N=256, K=256, bits=2, gs=64, X=A, W=A, scales=A, zeros=None, Y=A, ws=A, ws_bytes=BIG)
LINEAR = [
    (dict(bits=3), 1), (dict(gs=0), 1), (dict(K=100), 1), (dict(zeros=A), 1), (dict(bits=4), 1), (dict(M=-1), 1),
    (dict(X=None), 1), (dict(W=None), 1), (dict(X=A + 2), 2), (dict(W=A + 4), 2), (dict(Y=A + 8), 2),
    (dict(gs=32), 3), (dict(N=100), 3), (dict(bits=1, K=192), 3),
    (dict(ws=None), 8), (dict(ws=A + 16), 8), (dict(ws_bytes=64), 8),
]
SETS = [
    (dict(num=0), 1), (dict(num=-1), 1), (dict(rank=0), 1), (dict(A=None), 1), (dict(B=None), 1),
    (dict(scaling=None), 1), (dict(A=A + 2), 2), (dict(B=A + 8), 2), (dict(index=A + 2), 2), (dict(scaling=A + 1), 2),
    (dict(num=4097), 3), (dict(rank=12), 3), (dict(rank=136), 3),
]


def forward(lib, ad, P=None, codes=None, exps=None, **kw):
    d = dict(BASE, **kw)
    return lib.lowbit_adapter_gemm(d["M"], d["N"], d["K"], d["bits"], d["gs"], d["X"], d["W"], d["scales"], d["zeros"],
                                   ctypes.byref(ad) if ad is not None else None, d["Y"], P, codes, exps, d["ws"],
                                   d["ws_bytes"], None)


def backward(lib, ad, X=A, codes=None, exps=None, P=A, dX=A, dA=A, dB=A, **kw):
    d = dict(BASE, **kw)
    return lib.lowbit_adapter_backward(d["M"], d["N"], d["K"], d["bits"], d["gs"], A, d["W"], d["scales"], d["zeros"],
                                       ctypes.byref(ad) if ad is not None else None, X, codes, exps, P, dX, dA, dB,
                                       d["ws"], d["ws_bytes"], None)


def dx(lib, **kw):
    d = dict(BASE, **kw)
    return lib.lowbit_gemm_dx(d["M"], d["N"], d["K"], d["bits"], d["gs"], d["X"], d["W"], d["scales"], d["zeros"],
                              d["Y"], d["ws"], d["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", LINEAR)
def test_linear_arguments(lib, kw, want):
    assert forward(lib, adapters(), **kw) == want
    assert dx(lib, **kw) == want
    if not {"X", "Y"} & set(kw):
        assert backward(lib, adapters(), **kw) == want


@pytest.mark.parametrize("kw,want", SETS)
def test_adapter_sets(lib, kw, want):
    assert forward(lib, adapters(**kw)) == want
    assert backward(lib, adapters(**kw)) == want


def test_missing_adapters(lib):
    assert forward(lib, None) == 1
    assert backward(lib, None) == 1


def test_kept_copies(lib):
    assert forward(lib, adapters(), P=A + 2) == 2
    assert forward(lib, adapters(), codes=A) == 1          # codes without exponents
    assert forward(lib, adapters(), exps=A) == 1
    assert forward(lib, adapters(), codes=A + 8, exps=A) == 2


def test_backward_arguments(lib):
    assert backward(lib, adapters(), X=None) == 1                          # neither x nor its copy
    assert backward(lib, adapters(), codes=A, exps=A) == 1                 # both
    assert backward(lib, adapters(), X=None, codes=A) == 1
    assert backward(lib, adapters(), P=None) == 1
    assert backward(lib, adapters(), dA=None) == 1
    assert backward(lib, adapters(), dB=None) == 1
    assert backward(lib, adapters(), dX=A + 4) == 2
    assert backward(lib, adapters(), dB=A + 4) == 2
    assert backward(lib, adapters(), P=A + 4) == 2


def test_empty_problems(lib):
    assert forward(lib, adapters(), M=0, X=None, Y=None, ws=None) == 0
    assert forward(lib, adapters(), N=0) == 0
    assert dx(lib, M=0, X=None, Y=None, ws=None) == 0
    assert forward(lib, adapters(rank=12), M=0) == 3       # still checked


def test_workspace_size(lib):
    size = lib.lowbit_adapter_workspace_size
    assert size(-1, 256, 256, 1, 16) == 0 and size(1, 256, 256, 4097, 16) == 0 and size(1, 256, 256, 1, 129) == 0
    assert size(1, 256, 256, 1, 0) == 0 and size(0, 256, 256, 0, 0) == 0
    for args in ((100, 256, 1024, 3, 16), (4608, 9728, 2560, 64, 64)):
        need = size(*args)
        assert need % 256 == 0 and need >= args[0] * max(args[1], args[2]) * 2
        M, N, K, L, R = args
        # the forward needs no more than the size says, and a byte less than its own need is refused
        assert forward(lib, adapters(num=L, rank=R), M=M, N=N, K=K, ws_bytes=M * K * 2) == 8
        assert size(M + 1, N, K, L, R) >= need


def test_transpose_arguments(lib):
    assert lib.lowbit_transposed_words(1032, 1024, 4) == 1024 * 1152 // 8
    assert lib.lowbit_transposed_words(8, 64, 2) == 64 * 128 // 16
    assert lib.lowbit_transposed_words(8, 65, 2) == 0 and lib.lowbit_transposed_words(8, 64, 3) == 0
    assert lib.lowbit_transpose(A, 8, 64, 3, A, None) == 1
    assert lib.lowbit_transpose(None, 8, 64, 2, A, None) == 1
    assert lib.lowbit_transpose(A, 8, 64, 2, A + 4, None) == 2
    assert lib.lowbit_transpose(None, 0, 64, 2, None, None) == 0


def test_checkpoint_arguments(lib):
    for fn in (lambda x, M, K, c, e: lib.lowbit_checkpoint_store(x, M, K, c, e, None),
               lambda x, M, K, c, e: lib.lowbit_checkpoint_load(c, e, M, K, x, None)):
        assert fn(A, 4, 48, A, A) == 1 and fn(A, -1, 64, A, A) == 1
        assert fn(None, 4, 64, A, A) == 1 and fn(A, 4, 64, None, A) == 1 and fn(A, 4, 64, A, None) == 1
        assert fn(A + 8, 4, 64, A, A) == 2 and fn(A, 4, 64, A + 8, A) == 2
        assert fn(None, 0, 64, None, None) == 0


def test_binding_refuses_before_the_library():
    bf = dict(dtype=torch.bfloat16)
    x, packed = torch.zeros(4, 128, **bf), torch.zeros(16, 8, dtype=torch.int32)
    scales = torch.zeros(2, 16, dtype=torch.float16)
    a, b, s = torch.zeros(2, 8, 128, **bf), torch.zeros(2, 16, 8, **bf), torch.zeros(2)
    good = dict(x=x, packed=packed, scales=scales, zeros=None, bits=2, group_size=64, a=a, b=b, scaling=s)
    with pytest.raises(ValueError, match="CUDA"):
        lb.adapter_gemm(**good)
    for name, bad in (("a", a.float()), ("a", a[:, :, :64].contiguous()), ("b", b[:1].contiguous()), ("b", b.transpose(1, 2)),
                      ("scaling", s.double()), ("scaling", torch.zeros(3)), ("x", x.half()), ("x", x.t())):
        with pytest.raises(ValueError):
            lb.adapter_gemm(**dict(good, **{name: bad}))
    with pytest.raises(ValueError):
        lb.checkpoint_empty(4, 48, "cpu")
    with pytest.raises(ValueError):
        lb.transpose_packed(packed, 64, 2)
    ck = lb.checkpoint_empty(4, 128, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lb.checkpoint_load(ck)
    with pytest.raises(ValueError):
        lb.checkpoint_store(x.half())
