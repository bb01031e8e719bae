"""Adapters, gradients and 8-bit copies on the GPU at the edges of what the entry points take, against the
64-bit references of tests/_adapters.py."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import Problem, backward_ref, check, forward_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K,L,R,M,largest", [(4096, 4096, 256, 128, 147, 148), (1024, 512, 64, 32, 256, 257),
                                               (1032, 640, 300, 64, 88, 768), (264, 256, 4096, 128, 19, 64)])
def test_workspace_of_a_larger_batch(N, K, L, R, M, largest):
    """A batch on the workspace of a larger one gets what it gets on its own, and leaves what lies behind."""
    pr = Problem(M, K, N, 2, 64, L, R, "random")
    size = lb.adapter_workspace_size(largest, N, K, L, R)
    ws = torch.full((size + 256,), 9, dtype=torch.uint8, device="cuda")
    y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), ws=ws[:size])
    got = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args(), ws=ws[:size])
    assert lb.device_status() == 0 and (ws[size:] == 9).all()
    assert torch.equal(y, lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args()))
    ry, ey, _, _ = forward_ref(pr)
    check(y, ry, ey, "y")
    for (r, e), g in zip(backward_ref(pr, pr.x), got):
        check(g, r, e, "gradient")


def test_a_linear_without_rows():
    pr = Problem(20, 256, 8, 2, 64, 2, 16)
    none = dict(packed=pr.packed[:0], scales=pr.scales[:, :0].contiguous(), zeros=None, bits=2, group_size=64, a=pr.a,
                b=pr.b[:, :0].contiguous(), scaling=pr.scaling, index=pr.index)
    assert lb.adapter_gemm(pr.x, **none).shape == (20, 0)
    with pytest.raises(lb.LowbitError, match="UNSUPPORTED"):
        lb.adapter_gemm(pr.x, **none, p=pr.p)
    with pytest.raises(lb.LowbitError, match="UNSUPPORTED"):
        lb.adapter_gemm(pr.x, **none, checkpoint=lb.checkpoint_empty(20, 256, "cuda"))
    dy, wt = pr.dy[:, :0].contiguous(), pr.packed_t[:, :0].contiguous()
    assert not lb.gemm_dx(dy, wt, none["scales"], None, 2, 64).any()      # a sum over nothing
    with pytest.raises(lb.LowbitError, match="UNSUPPORTED"):
        lb.adapter_backward(dy, pr.x, pr.p, wt, none["scales"], None, 2, 64, pr.a, none["b"], pr.scaling, pr.index)


def test_a_linear_of_many_rows():
    """More than 65535 row tiles of 128, in both directions."""
    pr = Problem(20, 64, (1 << 23) + 136, 2, 64, 2, 8, "random")
    y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args())
    ry, ey, _, _ = forward_ref(pr)
    check(y, ry, ey, "y")
    del y, ry, ey
    got = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
    assert lb.device_status() == 0
    for (r, e), g in zip(backward_ref(pr, pr.x), got):
        check(g, r, e, "gradient")


@pytest.mark.parametrize("compiled", [True, False])
def test_a_pair_as_checkpoint(compiled, monkeypatch):
    """A plain (codes, exps) pair is taken with the compiled marshalling and without it, and checked."""
    if not compiled:
        calls = object.__new__(lb._Marshalled)
        calls.lib = lb.load()
        calls.adapter_gemm = lambda *args: None
        monkeypatch.setattr(lb, "_marshalled", calls)
    pr = Problem(20, 256, 136, 2, 64, 2, 16)
    want = lb.checkpoint_empty(20, 256, "cuda")
    y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), checkpoint=want)
    codes, exps = torch.zeros_like(want.codes), torch.zeros_like(want.exps)
    assert torch.equal(lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), checkpoint=(codes, exps)), y)
    assert torch.equal(codes.view(torch.uint8), want.codes.view(torch.uint8)) and torch.equal(exps, want.exps)
    with pytest.raises(ValueError, match="checkpoint"):
        lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), checkpoint=(codes[1:], exps))


@pytest.mark.parametrize("M,K,N,L,R,index", [(9, 256, 136, 3, 24, "holes"), (17, 256, 136, 4096, 16, "random"),
                                             (150, 384, 264, 5, 128, "sorted"), (900, 256, 520, 40, 32, "holes"),
                                             (900, 512, 264, 1, 64, None), (2100, 192, 264, 300, 8, "random")])
@pytest.mark.parametrize("eight", [False, True])
def test_index_checks(M, K, N, L, R, index, eight):
    """The build with device-side index checks: none fires, through every kernel of the entry points (up to
    16 tokens, P by the copy pass and by a kernel of its own, x in bf16 and in 8 bits, far more adapters than
    the batch uses), and the results are the release build's."""
    pr = Problem(M, K, N, 2, 64, L, R, index)

    def run():
        p, ck = torch.empty(M, R, dtype=torch.bfloat16, device="cuda"), lb.checkpoint_empty(M, K, "cuda")
        y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), p=p, checkpoint=ck)
        g = lb.adapter_backward(pr.dy, ck if eight else pr.x, p, pr.packed_t, *pr.args(), *pr.adapter_args())
        assert lb.device_status() == 0
        return y, p, ck.codes.view(torch.uint8), ck.exps, *g, lb.gemm_dx(pr.dy, pr.packed_t, *pr.args())

    want = run()
    release = lb._lib
    try:
        lb._lib = lb.load_debug()
        assert lb._lib.lowbit_debug_checks_enabled() == 1
        got = run()
    finally:
        lb._lib = release
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ry, ey, _, _ = forward_ref(pr)
    check(want[0], ry, ey, "y")


@pytest.mark.parametrize("M", [9, 40, 300])
@pytest.mark.parametrize("K,N", [(9216, 136), (256, 9216)])
def test_adapters_past_32_bits(M, K, N):
    """More than 2^31 values in A and dA, or in B and dB: the first and the last adapter in use, the others
    without tokens."""
    L, R = 1830, 128
    pr = Problem(M, K, N, 2, 64, 2, R, "random")
    assert L * R * max(K, N) > 1 << 31
    a, b = (torch.zeros(L, *t.shape[1:], dtype=torch.bfloat16, device="cuda") for t in (pr.a, pr.b))
    scaling, ends = torch.ones(L, device="cuda"), [0, L - 1]
    a[ends], b[ends], scaling[ends] = pr.a, pr.b, pr.scaling
    index = pr.index * (L - 1)
    y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), a, b, scaling, index)
    ry, ey, _, _ = forward_ref(pr)
    check(y, ry, ey, "y")
    dx, da, db = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), a, b, scaling, index)
    assert lb.device_status() == 0
    for (r, e), g, name in zip(backward_ref(pr, pr.x), (dx, da[ends], db[ends]), ("dx", "da", "db")):
        check(g, r, e, name)
    assert not da[1:-1].any() and not db[1:-1].any()
