"""Adapters beside the packed linear, their gradients and the 8-bit activation copy on the GPU,
against 64-bit references with bounds counted from the roundings (tests/_adapters.py)."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import Problem, backward_ref, check, checkpoint_ref, forward_ref

pytestmark = pytest.mark.gpu

FORMATS = [(1, 64), (1, 128), (2, 64), (2, 128), (4, 64), (4, 128)]

# (M, K, N, L, R, index): every token tile, ragged M, odd multiples of 8 in N, K past a multiple of
# 128, ranks that do not fill their slot, more adapters than a tile has tokens, no adapter at all
CASES = [
    (1, 128, 8, 1, 8, None),
    (1, 256, 72, 3, 16, "last"),
    (5, 384, 264, 3, 24, "holes"),
    (16, 1024, 1032, 16, 16, "random"),
    (17, 256, 136, 2, 8, "random"),
    (33, 640, 256, 5, 40, "sorted"),
    (64, 256, 512, 7, 64, "holes"),
    (77, 512, 200, 4, 128, "random"),
    (130, 256, 384, 300, 16, "random"),
    (200, 384, 256, 1, 72, None),
    (257, 256, 512, 3, 32, "sorted"),
    (300, 512, 264, 9, 96, "holes"),
    (513, 256, 256, 70, 64, "random"),
    (530, 128, 768, 2, 128, "none"),
]


def run_forward(pr, keep=True):
    p = torch.full((pr.M, pr.R), 7.0, dtype=torch.bfloat16, device="cuda") if keep else None
    ck = lb.checkpoint_empty(pr.M, pr.K, "cuda") if keep else None
    y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), p=p, checkpoint=ck)
    assert lb.device_status() == 0
    return y, p, ck


@pytest.mark.parametrize("bits,gs", FORMATS)
@pytest.mark.parametrize("M,K,N,L,R,index", CASES)
def test_forward(M, K, N, L, R, index, bits, gs):
    pr = Problem(M, K, N, bits, gs, L, R, index)
    y, p, ck = run_forward(pr)
    ry, ey, rp, ep = forward_ref(pr)
    check(p, rp, ep, "p")
    check(y, ry, ey, "y")
    codes, exps, _ = checkpoint_ref(pr.x)
    assert torch.equal(ck.exps.cpu(), exps) and torch.equal(ck.codes.double().cpu(), codes)
    assert torch.equal(run_forward(pr, keep=False)[0], y)


@pytest.mark.parametrize("bits,gs", FORMATS)
@pytest.mark.parametrize("M,K,N,L,R,index", CASES)
def test_backward(M, K, N, L, R, index, bits, gs):
    pr = Problem(M, K, N, bits, gs, L, R, index)
    for x, value in ((pr.x, pr.x), (lb.checkpoint_store(pr.x), None)):
        value = lb.checkpoint_load(x) if value is None else value
        dx, da, db = lb.adapter_backward(pr.dy, x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
        assert lb.device_status() == 0
        (rx, ex), (ra, ea), (rb, eb) = backward_ref(pr, value)
        check(dx, rx, ex, "dx")
        check(da, ra, ea, "da")
        check(db, rb, eb, "db")


@pytest.mark.parametrize("bits,gs", FORMATS)
@pytest.mark.parametrize("M,K,N", [(1, 128, 8), (19, 256, 136), (50, 640, 1032), (100, 384, 264), (300, 256, 512),
                                   (513, 1152, 200)])
def test_gemm_dx(M, K, N, bits, gs):
    pr = Problem(M, K, N, bits, gs, 1, 8, "none")
    (rx, ex), _, _ = backward_ref(pr, pr.x)
    dx = lb.gemm_dx(pr.dy, pr.packed_t, *pr.args())
    assert lb.device_status() == 0
    check(dx, rx, ex, "dx")


@pytest.mark.parametrize("bits,K", [(2, 192), (4, 320), (4, 64)])
def test_k_of_half_a_block(bits, K):
    """K a multiple of 64 but not of 128: W^T's last row tile is partly outside."""
    pr = Problem(90, K, 264, bits, 64, 3, 16, "random")
    y, p, _ = run_forward(pr)
    ry, ey, rp, ep = forward_ref(pr)
    check(y, ry, ey, "y")
    for (r, e), got in zip(backward_ref(pr, pr.x),
                           lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())):
        check(got, r, e, "gradient")


@pytest.mark.parametrize("N,K", [(8, 64), (72, 192), (128, 128), (264, 320), (1032, 256)])
@pytest.mark.parametrize("bits", [1, 2, 4])
def test_transpose(N, K, bits):
    if bits == 1 and K % 32:
        pytest.skip("not a binary size")
    lo, hi = {1: (0, 2), 2: (-1, 2), 4: (0, 16)}[bits]
    codes = torch.randint(lo, hi, (N, K), device="cuda").to(torch.int8)
    if bits == 1:
        codes = codes * 2 - 1
    wide = torch.full((K, (N + 127) // 128 * 128), {1: -1, 2: -1, 4: 0}[bits], dtype=torch.int8, device="cuda")
    wide[:, :N] = codes.T
    got = lb.transpose_packed(lb.pack(codes, bits), K, bits)
    assert got.numel() == lb.transposed_words(N, K, bits)
    assert torch.equal(got, lb.pack(wide, bits))


@pytest.mark.parametrize("bits,gs", FORMATS)
@pytest.mark.parametrize("M,L,R,index", [(500, 3, 32, "sorted"), (511, 40, 64, "holes"), (400, 1, 8, None)])
def test_split_pairs(M, L, R, index, bits, gs):
    """Sizes that run K slices over clusters of CTA pairs, in both directions."""
    pr = Problem(M, 3200, 2560, bits, gs, L, R, index)
    y, p, _ = run_forward(pr)
    ry, ey, rp, ep = forward_ref(pr)
    check(p, rp, ep, "p")
    check(y, ry, ey, "y")
    pr = Problem(M, 2560, 3200, bits, gs, L, R, index)
    got = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
    assert lb.device_status() == 0
    for (r, e), g in zip(backward_ref(pr, pr.x), got):
        check(g, r, e, "gradient")
    assert torch.equal(lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())[0], got[0])
