"""Accuracy of the cross entropy over a vocabulary where a rounding could show: zeros of uint4 rows anywhere in fp16's
range, and what a reader of the entry points' documentation would count on."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import check
from tests._vocab import H32, HB16, Loss, Table

pytestmark = pytest.mark.gpu


def zero_bound(ref, x, table, V):
    """What the two fp16 values of a uint4 weight may be off, summed over K: 2^-22 (|q - z| + |z| + 25) s + 2^-24."""
    gs = table.gs
    z = table.zeros.double()[:, :V].T.repeat_interleave(gs, 1)
    s = table.scales.double()[:, :V].T.repeat_interleave(gs, 1)
    q = table.codes.double()[:V]
    return x.double().abs() @ (2.0 ** -22 * ((q - z).abs() + z.abs() + 25) * s + 2.0 ** -24).T


@pytest.mark.parametrize("M", [1, 16, 17, 128, 129])
@pytest.mark.parametrize("gs", [64, 128])
def test_zeros_anywhere(M, gs):
    """Zero points of either sign, far outside the codes' range and between fp16's coarse steps. All of x has one sign, so
    that what is cut off a zero adds up over K instead of cancelling."""
    K, N, V = 256, 264, 261
    table = Table(N, K, 4, gs)
    odd = [-9.0078125, -8.0078125, -15.9921875, -31.984375, -120.0625, -0.0078125, 7.99609375, 31.984375, 120.0625, 1000.5, -1000.5,
           -1999.0, 1999.0, 0.0, 15.0, -3.3]
    table.zeros.copy_(torch.tensor(odd, device="cuda").repeat(K // gs * N // 16 + 1)[:K // gs * N].view(K // gs, N).half())
    # logits of some 10 whatever the zero: the scale falls with it
    table.scales.copy_((2.0 / K / (8 + table.zeros.float().abs())).half())
    g = torch.Generator(device="cuda").manual_seed(M)
    x = (0.5 + torch.rand(M, K, generator=g, device="cuda")).bfloat16()
    labels = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    grad = torch.randn(M, generator=g, device="cuda")
    loss, lse = lb.cross_entropy(x, labels, *table.args(), vocab=V)
    dx, _ = lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V)
    torch.cuda.synchronize()
    assert lb.device_status() == 0
    ref = Loss(x, labels, table, V)
    more = zero_bound(ref, x, table, V)
    ref.el = ref.el + more
    check(lse, ref.lse, ref.e_lse + more.amax(1), "lse")
    check(loss, ref.loss, ref.e_loss + 2 * more.amax(1), "loss")
    (rx, ex), _ = ref.gradients(grad, lse)
    check(dx, rx, ex, "dx")


@pytest.mark.parametrize("M", [17, 128, 129])
@pytest.mark.parametrize("z", [-9.0078125, -15.9921875, -120.0625, 31.984375, 1000.5])
def test_weights_of_one_zero(M, z):
    """One row against zeros: x has a single value per token, so each logit difference is one weight; weights are off by at
    most the two values' bound, and by what fp32 takes from a sum of one product and zeros."""
    K, N = 128, 72
    table = Table(N, K, 4, 64)
    table.zeros.fill_(z)
    table.scales.fill_(1.0)
    x = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    at = torch.arange(M, device="cuda") % K
    x[torch.arange(M, device="cuda"), at] = 2.0 ** -3
    labels = (torch.arange(M, device="cuda") * 7 % N).int()
    loss, lse = lb.cross_entropy(x, labels, *table.args())
    target = (lse.double() - loss.double())
    w = table.rows()
    want = x.double() @ w.T
    want = want[torch.arange(M, device="cuda"), labels.long()]
    q = table.codes.double()[labels.long(), at]
    weight = 2.0 ** -3 * (2.0 ** -22 * ((q - z).abs() + abs(z) + 25) + 2.0 ** -24)
    # the sum's own rounding and what scales it (2^-24 of 8 steps), lse and loss in fp32
    check(target, want, weight + 2.0 ** -24 * (8 * want.abs() + 2 * lse.double().abs() + 2 * loss.double().abs()), "target")


def half_step(v):
    """Half a step of bf16 at v >= 0."""
    return torch.exp2(torch.floor(torch.log2(v.clamp_min(2.0 ** -126))) - 8)


@pytest.mark.parametrize("M,K,N,V,labelled,repeat", [
    (513, 128, 4000, 4000, 513, 1), (1024, 256, 20000, 20000, 900, 1), (1024, 136, 20000, 19999, 1020, 2), (2049, 72, 9000, 8990, 900, 3),
    (4133, 128, 70000, 70000, 4097, 1), (1500, 64, 300, 290, 1111, 1), (700, 128, 5000, 4099, 3, 1), (640, 64, 260, 257, 0, 1)])
def test_dw_of_many_tokens(M, K, N, V, labelled, repeat):
    """The mean over the labelled tokens, a factor that bf16 does not hold: at the labels G is -1 / labelled and a little, and
    enters dW as two bf16 values, so a row that a label makes up is off by its own rounding (half a step, taken exactly). Nothing
    else of G is larger than 2 / V of that, and is rounded to 2^-8; p's error as Loss counts it; fp32 sums of 2 M products."""
    table = Table(N, K, 16, norm=1.0)
    g = torch.Generator(device="cuda").manual_seed(M + V)
    x = (torch.randn(M, K, generator=g, device="cuda") / 64).bfloat16()     # tokens that know nothing: p near 1 / V
    labels = torch.randint(0, max(V // repeat, 1), (M,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.randperm(M, generator=g, device="cuda")[labelled:]
    labels[out] = torch.tensor([-100, V, 2 ** 31 - 1], device="cuda", dtype=torch.int32).repeat(M)[:len(out)]
    x[out[:5]] = float("nan")
    grad = torch.full((M,), 1.0 / max(labelled, 1), device="cuda")
    lse = lb.cross_entropy(x, labels, *table.args(), vocab=V)[1]
    dx, dw = lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V, need_dw=True)
    torch.cuda.synchronize()
    assert lb.device_status() == 0
    x = torch.where(((labels >= 0) & (labels < V))[:, None], x, 0.0).bfloat16()
    ref = Loss(x, labels, table, V)
    l = torch.where(ref.valid, lse, 0.0).double()[:, None]
    p = torch.where(ref.valid[:, None], (ref.l - l).exp(), 0.0)
    assert p.max() <= 2 / V
    hot = torch.zeros_like(p)
    hot[torch.arange(M, device="cuda"), ref.label] = 1.0
    f = torch.where(ref.valid, grad, 0.0).double()[:, None]
    G = f * (p - hot)
    ep = p * torch.expm1(1.01 * (ref.el + 1.4427 * 3 * (ref.l.abs() + l.abs()) * H32) + 2.0 ** -21) + H32
    eG = 1.01 * f * ep + torch.where(hot > 0, 2.0 ** -16 + 2 * H32, HB16 + 2 * H32) * G.abs()
    want = G.T @ x.double()
    e = eG.T @ x.double().abs() + (2 * M + 16) * H32 * (G.abs().T @ x.double().abs())
    check(dw[:V], want, e + half_step(want.abs() + e), "dw")
    assert not dw[V:].any() and not dx[out].any()
    (rx, ex), _ = ref.gradients(torch.where(ref.valid, grad, 0.0), torch.where(ref.valid, lse, 0.0))
    check(dx, rx, ex, "dx")
    again = lb.cross_entropy_backward(grad, torch.where(ref.valid[:, None], x, 7.0), labels, lse, *table.args(), vocab=V, need_dw=True)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


FORMATS = [(16, 0), (1, 128), (2, 64), (4, 64)]


@pytest.mark.parametrize("bits,gs", FORMATS)
@pytest.mark.parametrize("M,K", [(509, 1280), (509, 2560), (77, 2560), (300, 8192), (77, 8192)])
def test_error_in_the_norm(bits, gs, M, K):
    """What the tensor cores cut off a sum over n = K / 16 steps is 0.26 n 2^-24 of it on average, and made up for; a fifth of
    that is its spread over the tokens, which is left, with two roundings to fp32 (2^-23) and nothing that adds up over tokens."""
    V = 6007
    table = Table(6008, K, bits, gs, seed=3)
    g = torch.Generator(device="cuda").manual_seed(K + M)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    labels = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse = lb.cross_entropy(x, labels, *table.args(), vocab=V)
    l = x.double() @ table.rows()[:V].T
    want = torch.logsumexp(l, 1)
    left = 0.26 * (K / 16) * 2.0 ** -24 / 5 + 2.0 ** -23
    assert float((lse.double() - want).norm() / want.norm()) <= left
    want = want - l.gather(1, labels.long()[:, None])[:, 0]
    assert float((loss.double() - want).norm() / want.norm()) <= left


@pytest.mark.parametrize("bits,gs", FORMATS)
@pytest.mark.parametrize("M", [40, 200])
@pytest.mark.parametrize("K", [2560, 8192])
@pytest.mark.parametrize("large", ["first", "last", "spread"])
def test_a_few_large_columns(bits, gs, M, K, large):
    """Four columns of x that carry the logit, and small ones of the same sign. Last, they lose nothing, and the factor that
    makes up for the usual loss stays: 0.26 K / 16 2^-24, and a tenth for what the small ones lose among themselves. First or
    in between, each step of the small ones may lose on the whole sum: at most half of what K fp32 additions may. (One row:
    lse is its logit, rounded once, and scaled once.)"""
    table = Table(8, K, bits, gs)
    at = {"first": torch.arange(4), "last": torch.arange(K - 4, K), "spread": torch.arange(4) * (K // 4) + 7}[large].cuda()
    if bits == 16:
        table.weight.copy_(table.weight.abs())
        table.weight[:, at] = 0.05
    else:
        table.codes.copy_(torch.full_like(table.codes, 13 if bits == 4 else 1))
        table.weight = lb.pack(table.codes, bits)
    g = torch.Generator(device="cuda").manual_seed(K)
    x = 1e-3 + 2e-3 * torch.rand(M, K, generator=g, device="cuda")
    x[:, at] = K / 50 * (1 + torch.rand(M, 4, generator=g, device="cuda"))
    x = x.bfloat16()
    labels = torch.full((M,), -1, device="cuda", dtype=torch.int32)
    _, lse = lb.cross_entropy(x, labels, *table.args(), vocab=1)
    w = table.rows()[0]
    assert bool((w >= 0).all())
    want = x.double() @ w
    bound = (0.36 * K / 16 * 2.0 ** -24 if large == "last" else K * 2.0 ** -25) + 2.0 ** -22
    if bits == 4:   # the weights' two fp16 values: 2^-22 (|q - z| + |z| + 25) s, of weights of 4 s and more with |z| <= 9
        bound = bound + 2.0 ** -22 * (4 + 9 + 25) / 4
    check(lse, want, bound * want, "lse")


def test_the_factor_of_very_long_rows():
    """Behind K = 65536 the factor grows no more: a single product, which loses nothing, is off by 0.26 * 4096 * 2^-24 at most."""
    K, M = 1 << 20, 20
    w = torch.zeros(8, K, device="cuda", dtype=torch.bfloat16)
    x = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    w[:, -1], x[:, -1] = 1.0, torch.arange(1, M + 1, device="cuda").bfloat16()
    _, lse = lb.cross_entropy(x, torch.zeros(M, device="cuda", dtype=torch.int32), w, vocab=1)
    want = x[:, -1].double()
    check(lse, want, (0.26 * 4096 * 2.0 ** -24 + 2.0 ** -22) * want, "lse")
