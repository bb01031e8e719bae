"""The compiled argument marshalling (_marshal.so): it takes exactly the calls that the binding's own
checks take, makes the same library call, and leaves everything else to those checks."""
import pytest
import torch

import bit_weight_only_w2_b200 as lb
from bit_weight_only_w2_b200 import _marshal
from tests._adapters import Problem

gpu = pytest.mark.gpu


def test_built_for_this_torch():
    assert _marshal.torch_version == torch.__version__.split("+")[0]


def test_everything_else_is_left_to_the_binding():
    """Host tensors, things that are no tensors, numbers out of range: None, and nothing raised."""
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 4, dtype=torch.int32)
    s, a, b = torch.zeros(1, 8, dtype=torch.float16), torch.zeros(1, 8, 64).bfloat16(), torch.zeros(1, 8, 8).bfloat16()
    one = torch.ones(1)
    c = lb._calls()
    rest = (None,) * 6
    assert c.adapter_gemm(x, w, s, None, 2, 64, a, b, one, *rest) is None
    for bad in (None, 3, "x", [1.0]):
        assert c.adapter_gemm(bad, w, s, None, 2, 64, a, b, one, *rest) is None
        assert c.gemm_dx(x, bad, s, None, 2, 64, None, None) is None
        assert c.adapter_backward(x, w, s, None, 2, 64, a, bad, one, None, x, None, None, x, None, None, None, True,
                                  None) is None
        assert c.checkpoint_store(bad) is None
        assert c.checkpoint_load(bad, x, None) is None
    for bits, group in ((2.0, 64), (None, 64), (2, 1 << 70), (2, 0), (3, 64), ((1 << 32) + 2, 64)):
        assert c.adapter_gemm(x, w, s, None, bits, group, a, b, one, *rest) is None
    with pytest.raises(TypeError):
        c.gemm_dx(x, w)


class Python:
    """Calls inside take the binding's own checks and its ctypes call."""

    def __enter__(self):
        self.saved = lb._calls()
        other = object.__new__(lb._Marshalled)
        other.lib = self.saved.lib
        for name in ("adapter_gemm", "gemm_dx", "adapter_backward", "checkpoint_store", "checkpoint_load"):
            setattr(other, name, lambda *args: None)
        lb._marshalled = other

    def __exit__(self, *exc):
        lb._marshalled = self.saved


def calls(pr):
    """Every entry point and every way to give its outputs."""
    empty = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    ad = pr.adapter_args()
    M, K, N, L, R = pr.M, pr.K, pr.N, pr.L, pr.R
    ws = torch.empty(lb.adapter_workspace_size(M, N, K, L, R), dtype=torch.uint8, device="cuda")
    out = []
    for given in (False, True):
        p, ck = (empty(M, R), lb.checkpoint_empty(M, K, "cuda")) if given else (None, None)
        opt = lambda *s: empty(*s) if given else None
        w = ws if given else None
        y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *ad, out=opt(M, N), p=p, checkpoint=ck, ws=w)
        dx = lb.gemm_dx(pr.dy, pr.packed_t, *pr.args(), out=opt(M, K), ws=w)
        st = lb.checkpoint_store(pr.x, lb.checkpoint_empty(M, K, "cuda") if given else None)
        ld = lb.checkpoint_load(st, opt(M, K))
        x = st if given else pr.x
        g = lb.adapter_backward(pr.dy, x, pr.p, pr.packed_t, *pr.args(), *ad, dx=opt(M, K), da=opt(L, R, K),
                                db=opt(L, N, R), ws=w)
        h = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *ad, need_dx=False)
        assert type(st) is lb.Checkpoint and h[0] is None
        out += [y, dx, st.codes, st.exps, ld, *g, *h[1:]] + ([p, *ck] if given else [])
    return out


@gpu
@pytest.mark.parametrize("M,K,N,L,R,index", [(1, 256, 72, 3, 16, "last"), (17, 384, 136, 1, 8, None), (150, 256, 264, 5, 24, "holes"),
                                             (0, 256, 264, 2, 16, "random")])
@pytest.mark.parametrize("bits", [1, 4])
def test_same_results_as_the_binding(M, K, N, L, R, index, bits):
    pr = Problem(M, K, N, bits, 64, L, R, index)
    got = calls(pr)
    with Python():
        want = calls(pr)
    assert len(got) == len(want) and lb.device_status() == 0
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@gpu
def test_outputs_given_are_returned():
    pr = Problem(20, 256, 136, 2, 64, 2, 16)
    y, dx = torch.empty_like(pr.dy), torch.empty_like(pr.x)
    ad = pr.adapter_args()
    assert lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *ad, out=y) is y
    assert lb.gemm_dx(pr.dy, pr.packed_t, *pr.args(), out=dx) is dx
    assert lb.checkpoint_load(lb.checkpoint_store(pr.x), dx) is dx
    da, db = torch.empty_like(pr.a), torch.empty_like(pr.b)
    r = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *ad, dx=dx, da=da, db=db)
    assert r[0] is dx and r[1] is da and r[2] is db


@gpu
def test_a_tensor_that_does_not_fit_is_refused_by_name():
    """One argument at a time: wrong type, shape, layout or device. The compiled calls leave each to the
    binding, which raises."""
    pr = Problem(20, 256, 136, 4, 64, 2, 16)
    p, ck = pr.p, lb.checkpoint_empty(20, 256, "cuda")
    ws = torch.empty(lb.adapter_workspace_size(20, 136, 256, 2, 16), dtype=torch.uint8, device="cuda")
    fwd = dict(x=pr.x, packed=pr.packed, scales=pr.scales, zeros=pr.zeros, bits=4, group_size=64, a=pr.a, b=pr.b,
               scaling=pr.scaling, index=pr.index, out=torch.empty_like(pr.dy), p=p, ws=ws)
    bwd = dict(dy=pr.dy, x=pr.x, p=p, packed_t=pr.packed_t, scales=pr.scales, zeros=pr.zeros, bits=4, group_size=64,
               a=pr.a, b=pr.b, scaling=pr.scaling, index=pr.index, dx=torch.empty_like(pr.x), da=torch.empty_like(pr.a),
               db=torch.empty_like(pr.b), ws=ws)
    dx = dict(dy=pr.dy, packed_t=pr.packed_t, scales=pr.scales, zeros=pr.zeros, bits=4, group_size=64,
              out=torch.empty_like(pr.x), ws=ws)
    for fn, kw in ((lb.adapter_gemm, fwd), (lb.adapter_backward, bwd), (lb.gemm_dx, dx)):
        fn(**kw)
        for name, t in kw.items():
            if not isinstance(t, torch.Tensor):
                continue
            wide = torch.stack([t, t], -1)[..., 0]
            assert name == "scaling" or wide.numel() < 2 or not wide.is_contiguous()
            bad = [t.double(), t.cpu(), wide, t[None]] + ([t[:-1]] if name != "ws" else [])
            for b in bad:
                with pytest.raises(ValueError):
                    fn(**dict(kw, **{name: b}))
        with pytest.raises(lb.LowbitError, match="WORKSPACE"):
            fn(**dict(kw, ws=ws[:64]))
    for part in (lb.Checkpoint(ck.codes[:-1], ck.exps), lb.Checkpoint(ck.codes, ck.exps[:, :-1].contiguous()),
                 lb.Checkpoint(ck.codes.cpu(), ck.exps)):
        with pytest.raises(ValueError):
            lb.adapter_gemm(**fwd, checkpoint=part)
        with pytest.raises(ValueError):
            lb.adapter_backward(**dict(bwd, x=part))
        with pytest.raises(ValueError):
            lb.checkpoint_load(part)
    with pytest.raises(ValueError, match="need_dx"):
        lb.adapter_backward(**bwd, need_dx=False)
    assert lb.adapter_backward(**dict(bwd, dx=None), need_dx=0)[0] is None
    assert lb.adapter_backward(**bwd, need_dx=1)[0] is bwd["dx"]
