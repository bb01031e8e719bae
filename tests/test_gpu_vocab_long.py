"""The vocabulary operators where their inputs are cut up: gradients whose G takes several pieces, more tokens than the forward
takes at a time, and embedding gradients of more tokens than one launch sums up the sort's counts of."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import check
from tests._vocab import Loss, Table, embedding_grad_ref, inputs
from tests.test_gpu_vocab_edges import guarded

pytestmark = pytest.mark.gpu

PIECE = 256 << 20   # bytes of a term of G that are formed at a time


# (M, vocabulary, pieces): the last piece shorter than the others, more slices than one for dX or one, at most 128 tokens (whose
# pieces are long), and more than the forward's 16384
@pytest.mark.parametrize("bits,gs", [(1, 128), (2, 64), (4, 64), (4, 128), (16, 0)])
@pytest.mark.parametrize("M,V,pieces", [(2048, 70001, 2), (1500, 200003, 3), (300, 450001, 2), (100, 1400011, 2), (17003, 8203, 2)])
def test_gradients_in_pieces(bits, gs, M, V, pieces):
    K = 128
    assert -(-M * V * 2 // PIECE) == pieces
    table = Table((V + 7) // 8 * 8, K, bits, gs)
    x, labels, grad = inputs(M, K, V)
    loss, lse = lb.cross_entropy(x, labels, *table.args(), vocab=V)
    dw_too = bits == 16
    ws, ok = guarded((lb.cross_entropy_workspace_size(M, V, K, bits, 2 if dw_too else 1),), torch.uint8, 9)
    dx, ok_dx = guarded((M, K), torch.bfloat16)
    dw, ok_dw = guarded((table.N, K), torch.bfloat16) if dw_too else (None, lambda: True)
    lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V, need_dw=dw_too, dx=dx, dw=dw, ws=ws)
    torch.cuda.synchronize()
    assert lb.device_status() == 0 and ok() and ok_dx() and ok_dw()
    again = lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V, need_dw=dw_too)
    assert torch.equal(again[0], dx) and (dw is None or torch.equal(again[1], dw))
    del ws, again
    ref = Loss(x, labels, table, V)
    check(lse, ref.lse, ref.e_lse, "lse")
    check(loss, ref.loss, ref.e_loss, "loss")
    (rx, ex), (rw, ew) = ref.gradients(grad, lse)
    check(dx, rx, ex, "dx")
    if dw_too:
        check(dw[:V], rw, ew, "dw")
        assert not dw[V:].any()


@pytest.mark.parametrize("bits,gs", [(2, 64), (16, 0)])
def test_the_pieces_of_a_label(bits, gs):
    """A gradient of the labels alone (every other weight far below them): each token's dX is minus its label's row, to the
    rounding of G, from whichever piece the label lies in, its first and last rows too."""
    M, V, K = 2048, 70001, 128
    table = Table((V + 7) // 8 * 8, K, bits, gs)
    piece = 35072                                       # half of the vocabulary, in tiles of 256 rows
    at = [0, 255, 256, piece - 1, piece, piece + 1, piece + 255, V - 1, V - 2]
    labels = torch.tensor(at, device="cuda", dtype=torch.int32).repeat(M // len(at) + 1)[:M]
    x, _, _ = inputs(M, K, V)
    lse = torch.full((M,), 200.0, device="cuda")       # exp(l - 200): nothing is left of the others
    one = torch.ones(M, device="cuda")
    dx, dw = lb.cross_entropy_backward(one, x, labels, lse, *table.args(), vocab=V, need_dw=bits == 16)
    want = -table.rows()[labels.long()]
    check(dx, want, 2.0 ** -8 * want.abs(), "dx")
    if bits == 16:
        sums = torch.zeros(table.N, K, device="cuda", dtype=torch.float64).index_add_(0, labels.long(), -x.double())
        mag = torch.zeros_like(sums).index_add_(0, labels.long(), x.double().abs())
        check(dw, sums, 2.0 ** -8 * sums.abs() + 2 * M * 2.0 ** -24 * mag, "dw")


# one digit, two and three; the most tokens whose tiles' counts the moves sum up themselves, one more, and many more
@pytest.mark.parametrize("T", [131072, 131073, 300001])
@pytest.mark.parametrize("K,first,rows", [(8, 0, 300), (72, 11, 300), (72, 0, 70000), (8, 5, 70001), (8, 0, 600000)])
def test_embedding_gradient_of_many_tokens(T, K, first, rows):
    g = torch.Generator(device="cuda").manual_seed(T + K + rows)
    tokens = (first - 50 + (rows + 100) * torch.rand(T, generator=g, device="cuda", dtype=torch.float64) ** 2).int()   # low ones more often
    assert bool((tokens < first).any()) and bool((tokens >= first + rows).any())
    dy = torch.randn(T, K, generator=g, dtype=torch.bfloat16, device="cuda")
    ws, ok = guarded((lb.embedding_workspace_size(T, rows, K),), torch.uint8, 9)
    out, ok_out = guarded((rows, K), torch.bfloat16)
    lb.embedding_backward(tokens, dy, rows, first=first, multiplier=0.7, out=out, ws=ws)
    torch.cuda.synchronize()
    assert ok() and ok_out()
    check(out, *embedding_grad_ref(tokens, dy, first, rows, 0.7), "dtable")
    again = lb.embedding_backward(tokens, dy, rows, first=first, multiplier=0.7)
    assert torch.equal(out, again)


@pytest.mark.parametrize("T", [131072, 140001])
def test_the_order_of_a_sum(T):
    """A row's sum runs in the tokens' order (rows of 16 tokens here, two to a run): behind 1 each 2^-24, half a step, is lost
    to the even neighbour, and -1 leaves nothing; in front of 1 and -1 all fourteen are kept."""
    rows, K, per = 8192, 8, 16
    n = rows * per
    tokens = torch.arange(rows, device="cuda", dtype=torch.int32).repeat(per)       # row r's tokens: r, r + rows, ...
    tokens = torch.cat([tokens, torch.full((T - n,), -1, device="cuda", dtype=torch.int32)])
    dy = torch.full((T, K), 2.0 ** -24, device="cuda", dtype=torch.bfloat16)
    dy[:rows], dy[n - rows:n] = 1.0, -1.0
    assert not lb.embedding_backward(tokens, dy, rows, multiplier=2.0 ** 24).any()
    dy[:rows], dy[n - 2 * rows:n - rows] = 2.0 ** -24, 1.0
    assert (lb.embedding_backward(tokens, dy, rows, multiplier=2.0 ** 24) == 14).all()
