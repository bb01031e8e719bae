"""Refusals and workspace sizes of the vocabulary entry points, without a GPU: every check runs before
anything is launched."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb

A = 1 << 20   # a fake 256-byte-aligned address: never dereferenced, checks fail first
BIG = 1 << 50
BASE = dict(M=17, vocab=250, N=256, K=256, bits=2, gs=64, X=A, W=A, scales=A, zeros=None, labels=A, loss=A, lse=A, grad=A, dX=A,
            dW=None, ws=A, ws_bytes=BIG)
DENSE = dict(bits=16, gs=0, scales=None)


@pytest.fixture(scope="module")
def lib():
    return lb.load()


def forward(lib, **kw):
    d = dict(BASE, **kw)
    return lib.lowbit_cross_entropy(*[d[k] for k in ("M", "vocab", "N", "K", "bits", "gs", "X", "W", "scales", "zeros", "labels",
                                                     "loss", "lse", "ws", "ws_bytes")], None)


def backward(lib, **kw):
    d = dict(BASE, **kw)
    return lib.lowbit_cross_entropy_backward(*[d[k] for k in ("M", "vocab", "N", "K", "bits", "gs", "X", "W", "scales", "zeros",
                                                              "labels", "lse", "grad", "dX", "dW", "ws", "ws_bytes")], None)


def lookup(lib, T=5, Y=A, tokens=A, **kw):
    d = dict(BASE, **kw)
    return lib.lowbit_embedding(T, d["N"], d["K"], d["bits"], d["gs"], tokens, d["W"], d["scales"], d["zeros"], 1.0, Y, None)


def lookup_backward(lib, T=5, K=256, first=0, rows=16, tokens=A, dY=A, dE=A, ws=A, ws_bytes=BIG):
    return lib.lowbit_embedding_backward(T, K, first, rows, tokens, dY, 1.0, dE, ws, ws_bytes, None)


TABLES = [
    (dict(bits=3), 1), (dict(bits=8), 1), (dict(gs=0), 1), (dict(K=100), 1), (dict(K=0), 1), (dict(zeros=A), 1), (dict(bits=4), 1),
    (dict(W=None), 1), (dict(scales=None), 1), (dict(W=A + 4), 2), (dict(scales=A + 2), 2), (dict(bits=4, zeros=A + 8), 2),
    (dict(gs=32), 3), (dict(N=252), 3), (dict(bits=1, K=192), 3), (dict(N=1 << 31), 3),
    (dict(bits=16), 1), (dict(DENSE, zeros=A), 1), (dict(DENSE, W=None), 1), (dict(DENSE, W=A + 8), 2), (dict(DENSE, K=100), 3),
    (dict(DENSE, K=1 << 31), 3),
]
LOSSES = [
    (dict(M=-1), 1), (dict(vocab=0), 1), (dict(vocab=-5), 1), (dict(vocab=257), 1), (dict(X=None), 1), (dict(labels=None), 1),
    (dict(X=A + 2), 2), (dict(labels=A + 2), 2), (dict(M=1 << 31), 3), (dict(lse=None), 1), (dict(lse=A + 2), 2),
    (dict(ws=None), 8), (dict(ws=A + 16), 8), (dict(ws_bytes=64), 8),
]


@pytest.mark.parametrize("kw,want", TABLES)
def test_tables(lib, kw, want):
    assert forward(lib, **kw) == want
    assert backward(lib, **kw) == want
    assert lookup(lib, **kw) == want


@pytest.mark.parametrize("kw,want", LOSSES)
def test_loss_arguments(lib, kw, want):
    assert forward(lib, **kw) == want
    assert backward(lib, **kw) == want
    assert forward(lib, **DENSE, **kw) == want
    assert backward(lib, **DENSE, dW=A, **kw) == want


def test_outputs(lib):
    assert forward(lib, loss=None) == 1 and forward(lib, loss=A + 1) == 2
    assert backward(lib, grad=None) == 1 and backward(lib, grad=A + 2) == 2
    assert backward(lib, dX=None) == 1 and backward(lib, dX=A + 8) == 2
    assert backward(lib, dW=A) == 3                        # a packed table is frozen
    assert backward(lib, **DENSE, dW=A + 8) == 2


def test_lookup_arguments(lib):
    for kw, want in ((dict(T=-1), 1), (dict(tokens=None), 1), (dict(Y=None), 1), (dict(tokens=A + 2), 2), (dict(Y=A + 8), 2),
                     (dict(T=1 << 31), 3)):
        assert lookup(lib, **kw) == want
        assert lookup(lib, **DENSE, **kw) == want


def test_lookup_gradient_arguments(lib):
    for kw, want in ((dict(T=-1), 1), (dict(K=0), 1), (dict(first=-1), 1), (dict(rows=-1), 1), (dict(tokens=None), 1),
                     (dict(dY=None), 1), (dict(dE=None), 1), (dict(tokens=A + 1), 2), (dict(dY=A + 8), 2), (dict(dE=A + 4), 2),
                     (dict(K=100), 3), (dict(T=1 << 31), 3), (dict(rows=1 << 31), 3), (dict(first=1 << 31), 3), (dict(K=1 << 23), 3),
                     (dict(ws=None), 8), (dict(ws=A + 8), 8), (dict(T=9999, ws_bytes=4096), 8)):
        assert lookup_backward(lib, **kw) == want


def test_empty_problems(lib):
    assert forward(lib, M=0, X=None, W=None, labels=None, loss=None, lse=None, ws=None) == 0
    assert backward(lib, M=0, X=None, W=None, labels=None, lse=None, grad=None, dX=None, ws=None) == 0
    assert forward(lib, M=0, gs=32) == 3                   # still checked
    assert lookup(lib, T=0, tokens=None, Y=None, W=None) == 0
    assert lookup_backward(lib, rows=0, dE=None, ws=None) == 0


def test_workspace_size_of_invalid_arguments(lib):
    size, emb = lib.lowbit_cross_entropy_workspace_size, lib.lowbit_embedding_workspace_size
    for bad in ((-1, 8, 64, 2, 0), (1, 0, 64, 2, 0), (1, 8, 0, 2, 0), (1, 8, 64, 3, 0), (1, 8, 64, 2, 3), (1, 8, 64, 2, -1),
                (1 << 31, 8, 64, 2, 0), (1, 1 << 31, 64, 2, 1)):
        assert size(*bad) == 0
    assert emb(-1, 8, 64) == 0 and emb(1, -1, 64) == 0 and emb(1, 8, -1) == 0 and emb(1 << 31, 8, 64) == 0
    assert size(0, 8, 64, 2, 0) % 256 == 0 and emb(0, 0, 0) % 256 == 0


@pytest.mark.parametrize("bits", [2, 16])
@pytest.mark.parametrize("backward", [0, 1, 2])
@pytest.mark.parametrize("vocab,K", [(1, 128), (1000, 640), (32768, 2560), (131072, 4096), (200001, 128)])
def test_workspace_of_a_larger_batch_serves_a_smaller_one(lib, bits, backward, vocab, K):
    """The size never falls as the batch grows, through every choice of tile, piece and slices."""
    size = lib.lowbit_cross_entropy_workspace_size
    sizes = [size(M, vocab, K, bits, backward) for M in [*range(0, 700), *range(700, 40000, 61), 16383, 16384, 16385]]
    assert all(s % 256 == 0 for s in sizes)
    sizes[-3:] = []
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert size(16384, vocab, K, bits, backward) <= size(16385, vocab, K, bits, backward)


@pytest.mark.parametrize("rows", [1, 24, 300, 131072])
@pytest.mark.parametrize("K", [8, 2560])
def test_workspace_of_more_tokens_serves_fewer(lib, rows, K):
    size = lib.lowbit_embedding_workspace_size
    sizes = [size(T, rows, K) for T in [*range(0, 5000), *range(5000, 100000, 331)]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_binding_refuses_before_the_library():
    bf = dict(dtype=torch.bfloat16)
    x, w = torch.zeros(4, 128, **bf), torch.zeros(16, 8, dtype=torch.int32)
    s, labels = torch.zeros(2, 16, dtype=torch.float16), torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    good = dict(x=x, labels=labels, weight=w, scales=s, zeros=None, bits=2, group_size=64)
    with pytest.raises(ValueError, match="CUDA"):
        lb.cross_entropy(**good)
    with pytest.raises(ValueError, match="CUDA"):
        lb.embedding(labels, w, s, None, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        lb.embedding_backward(labels, x, 3)
    for name, bad in (("x", x.half()), ("x", x.t()), ("x", x[:, :64].contiguous()), ("labels", labels.long()), ("labels", labels[:3]),
                      ("weight", w.long()), ("weight", w[0]), ("scales", s.float()), ("scales", s[:1]), ("scales", None), ("bits", 3),
                      ("bits", 16), ("zeros", s.t()), ("group_size", 0), ("group_size", 96)):
        with pytest.raises(ValueError):
            lb.cross_entropy(**dict(good, **{name: bad}))
        with pytest.raises(ValueError):
            lb.cross_entropy_backward(f, lse=f, **dict(good, **{name: bad}))
        if name in ("weight", "scales", "bits", "zeros", "group_size"):
            with pytest.raises(ValueError):
                lb.embedding(labels, **{k: v for k, v in dict(good, **{name: bad}).items() if k not in ("x", "labels")})
    with pytest.raises(ValueError):
        lb.embedding(labels.long(), w, s, None, 2, 64)
    for bad in (dict(tokens=labels.long()), dict(tokens=labels[:2]), dict(dy=x.float()), dict(dy=x[0])):
        with pytest.raises(ValueError):
            lb.embedding_backward(**dict(dict(tokens=labels, dy=x, rows=3), **bad))


def test_sizes_whose_tiles_would_pass_32_bits(lib):
    """A vocabulary (or K) that ends within a tile or a block's stride of 2^31 is refused: its last indices would not fit."""
    last = (1 << 31) - (1 << 16)
    size = lib.lowbit_cross_entropy_workspace_size
    for N in (last + 8, (1 << 31) - 1024, (1 << 31) - 8):
        for kw in (dict(bits=2), DENSE):
            for M in (1, 17, 300):
                assert forward(lib, N=N, vocab=N, K=64, M=M, **kw) == 3
                assert backward(lib, N=N, vocab=N, K=64, M=M, **kw) == 3
            assert size(1, N, 64, kw["bits"], 0) == size(1, N, 64, kw["bits"], 1) == 0
        assert forward(lib, **DENSE, N=8, vocab=8, K=N) == 3 and backward(lib, **DENSE, N=8, vocab=8, K=N) == 3
        assert size(1, 8, N, 16, 0) == 0
    # the largest that is taken goes on to the checks of the workspace; a table may be longer than its vocabulary
    assert forward(lib, N=last, vocab=last, K=64, ws=None) == 8 and size(1, last, 64, 2, 0) == 4 * last
    assert forward(lib, N=(1 << 31) - 8, vocab=last, K=64, ws=None) == 8
