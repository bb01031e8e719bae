"""Token embeddings, the cross entropy over a vocabulary and their gradients, against 64-bit references."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import check
from tests._vocab import Loss, Table, embedding_grad_ref, embedding_ref, inputs

pytestmark = pytest.mark.gpu

FORMATS = [(16, 0), (1, 128), (2, 64), (2, 128), (4, 64), (4, 128)]
# (M, K, rows of the table, vocabulary): one token, tiles of 128 and of 256 filled and not, K of half a stage of
# words, vocabularies that end inside a tile and before the table does
SIZES = [(1, 128, 8, 8), (1, 640, 1000, 997), (16, 256, 504, 500), (127, 192, 136, 129), (128, 384, 128, 128),
         (129, 64, 264, 257), (300, 1280, 1008, 1003), (513, 128, 4104, 4099), (256, 512, 512, 512)]


def sizes_of(bits, gs):
    return [s for s in SIZES if bits == 16 or s[1] % max(gs, 128 if bits == 1 else gs) == 0]


CASES = [(b, g, *s) for b, g in FORMATS for s in sizes_of(b, g)] + [(16, 0, 5, 8, 3, 2), (16, 0, 200, 1288, 1003, 1001),
                                                                    (16, 0, 33, 72, 50, 50)]


@pytest.mark.parametrize("bits,gs,M,K,N,V", CASES)
def test_cross_entropy_and_gradients(bits, gs, M, K, N, V):
    table = Table(N, K, bits, gs)
    x, labels, grad = inputs(M, K, V)
    loss, lse = lb.cross_entropy(x, labels, *table.args(), vocab=V)
    torch.cuda.synchronize()
    assert lb.device_status() == 0
    ref = Loss(x, labels, table, V)
    check(lse, ref.lse, ref.e_lse, "lse")
    check(loss, ref.loss, ref.e_loss, "loss")
    dx, dw = lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V, need_dw=bits == 16)
    torch.cuda.synchronize()
    assert lb.device_status() == 0
    (rx, ex), (rw, ew) = ref.gradients(grad, lse)
    check(dx, rx, ex, "dx")
    if bits == 16:
        check(dw[:V], rw, ew, "dw")
        assert not dw[V:].any()
    else:
        assert dw is None
    none = ~ref.valid
    assert not loss[none].any() and not dx[none].any()


@pytest.mark.parametrize("bits,gs", FORMATS)
@pytest.mark.parametrize("T,K,N,multiplier", [(1, 128, 8, 1.0), (3, 256, 1000, 0.3), (77, 2560, 520, 1.0), (1000, 1152, 72, 34.0)])
def test_embedding(bits, gs, T, K, N, multiplier):
    table = Table(N, K, bits, gs)
    tokens = torch.randint(-2, N + 2, (T,), device="cuda", dtype=torch.int32)
    y = lb.embedding(tokens, *table.args(), multiplier=multiplier)
    check(y, *embedding_ref(tokens, table, multiplier), "y")


@pytest.mark.parametrize("T,K,first,rows,multiplier", [
    (1, 8, 0, 1, 1.0), (5, 64, 3, 2, 1.0), (77, 2560, 100, 24, 0.5), (1000, 200, 0, 50, 1.0), (1025, 1032, 7, 300, 3.0),
    (2049, 128, 0, 255, 1.0), (5000, 136, 0, 256, 1.0), (16385, 128, 0, 70000, 1.0), (32768, 64, 10, 1000, 1.0),
    (32769, 64, 10, 1000, 1.0), (100003, 72, 0, 66000, 1.0)])
def test_embedding_backward(T, K, first, rows, multiplier):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + K)
    u = torch.rand(T, generator=g, device="cuda")
    tokens = (first - 2 + (rows + 4) * u ** 3).int()     # low ones many times over, some outside the rows
    dy = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    out = torch.full((rows, K), float("nan"), device="cuda", dtype=torch.bfloat16)
    got = lb.embedding_backward(tokens, dy, rows, first=first, multiplier=multiplier, out=out)
    assert got is out
    check(out, *embedding_grad_ref(tokens, dy, first, rows, multiplier), "dtable")
    again = lb.embedding_backward(tokens, dy, rows, first=first, multiplier=multiplier)
    assert torch.equal(out, again)
