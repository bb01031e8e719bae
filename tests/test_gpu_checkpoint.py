"""The 8-bit activation copy on the GPU, against its definition in 64 bits: every output is determined
exactly (a power-of-two scale, one rounding), so codes, exponents and loaded values are compared bit
for bit."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import checkpoint_ref

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=12345.0), torch.nan_to_num(b, nan=12345.0)) and torch.equal(a.isnan(), b.isnan())


def check(x):
    ck = lb.checkpoint_store(x)
    codes, exps, values = checkpoint_ref(x)
    assert torch.equal(ck.exps.cpu(), exps)
    assert same(ck.codes.double().cpu(), codes)
    # -0 keeps its sign
    assert torch.equal(torch.signbit(ck.codes.float().cpu())[codes == 0], torch.signbit(x.float().cpu())[codes == 0])
    got = lb.checkpoint_load(ck)
    assert same(got.cpu(), values.to(torch.bfloat16))


@pytest.mark.parametrize("M,K", [(1, 32), (1, 96), (3, 64), (7, 2560), (77, 320), (256, 1024), (1000, 352), (5, 9728)])
def test_sizes(M, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(M * 7 + K)
    x = torch.randn(M, K, generator=g, device="cuda")
    check((x * torch.exp2(torch.randint(-20, 20, (M, 1), generator=g, device="cuda").float())).bfloat16())


def test_every_bf16_value():
    """Each finite bf16 value next to 31 others of the same or smaller size, so that every exponent and
    every rounding of e4m3 occurs; subnormal blocks too."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    bits = torch.cat([bits, bits | 0x8000])
    bits = torch.where(bits >= 0x8000, bits - 0x10000, bits).to(torch.int16)
    x = bits.view(torch.bfloat16).cuda()
    check(x.reshape(-1, 32).contiguous())          # neighbours: the same binade
    check(x.reshape(32, -1).t().contiguous())      # far apart: most fall below the block's range


def test_special_values():
    inf, nan, big, tiny = float("inf"), float("nan"), 3.3895e38, 9.2e-41
    rows = [[0.0] * 32, [-0.0] * 32, [nan] * 32, [inf, -inf] * 16, [big, -big, 1.0, tiny] * 8, [tiny] * 32,
            [1.0, inf, 2.0, nan] * 8, [448.0] * 32, [449.0] * 32, [464.0, 448.0] * 16, [1.75, 1.7578125] * 16,
            [nan, -0.0, 0.0, inf] * 8]
    check(torch.tensor(rows, dtype=torch.float32).bfloat16().cuda())
    wide = torch.zeros(4, 64, device="cuda").bfloat16()
    wide[1, 40] = inf                               # only its own block is affected
    wide[1, 3] = 1.0
    check(wide)


def test_outputs_given_and_empty():
    x = torch.randn(9, 64, device="cuda").bfloat16()
    ck = lb.checkpoint_empty(9, 64, "cuda")
    assert lb.checkpoint_store(x, out=ck) is ck
    out = torch.empty_like(x)
    assert lb.checkpoint_load(ck, out=out) is out
    assert torch.equal(out, lb.checkpoint_load(lb.checkpoint_store(x)))
    e = lb.checkpoint_store(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert lb.checkpoint_load(e).shape == (0, 64)


def test_error_bound():
    """|x - copy| <= 2^-4 |x|, or half a step of e4m3's smallest values, 2^-10 of the block's scale."""
    x = torch.randn(64, 4096, device="cuda").bfloat16()
    ck = lb.checkpoint_store(x)
    scale = torch.exp2(ck.exps.double() - 127).repeat_interleave(32, 1)
    off = (lb.checkpoint_load(ck).double() - x.double()).abs()
    assert (off <= torch.maximum(x.double().abs() * 2.0 ** -4, scale * 2.0 ** -10)).all()
