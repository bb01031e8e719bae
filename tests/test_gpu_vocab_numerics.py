"""Accuracy of the cross entropy over a vocabulary where a rounding could show: zeros of uint4 rows anywhere in fp16's
range, and what a reader of the entry points' documentation would count on."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import check
from tests._vocab import Loss, Table

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
