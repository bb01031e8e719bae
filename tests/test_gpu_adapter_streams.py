"""Calls of several streams at once: kernels of different calls share the SMs, which shifts the timing of
every warp. Each result has to be, bit for bit, what the call gives alone."""
import random
import threading

import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import Problem

pytestmark = pytest.mark.gpu

NAMES = ("y", "p", "copy", "plain y", "dx", "da", "db", "da without dx", "db without dx", "gemm_dx")


def step(pr):
    p, ck = torch.empty(pr.M, pr.R, dtype=torch.bfloat16, device="cuda"), lb.checkpoint_empty(pr.M, pr.K, "cuda")
    y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), p=p, checkpoint=ck)
    ws = torch.empty(lb.workspace_size(pr.M, pr.K), dtype=torch.uint8, device="cuda")
    plain = lb.gemm(pr.x, pr.packed, *pr.args(), ws=ws)
    return (y, p, ck.codes.view(torch.uint8), plain,
            *lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args()),
            *lb.adapter_backward(pr.dy, pr.x, p, pr.packed_t, *pr.args(), *pr.adapter_args(), need_dx=False)[1:],
            lb.gemm_dx(pr.dy, pr.packed_t, *pr.args()))


def run(prs, passes, streams=4, in_a_row=6):
    want = [step(pr) for pr in prs]
    torch.cuda.synchronize()
    bad = []

    def work(seed):
        rng = random.Random(seed)
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(passes // (streams * in_a_row)):
                ids = [rng.randrange(len(prs)) for _ in range(in_a_row)]
                got = [step(prs[i]) for i in ids]
                torch.cuda.current_stream().synchronize()
                for i, out in zip(ids, got):
                    bad.extend((i, n) for n, a, b in zip(NAMES, out, want[i]) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(s,)) for s in range(streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert lb.device_status() == 0
    assert not bad, (len(bad), bad[:8])


def test_weight_stages_are_kept_until_decoded():
    """Unsplit 64-token tiles of uint4 weights: some rows of a tile came from a weight stage that had been
    refilled, once in some thousand passes."""
    run([Problem(457, 2176, 1480, 4, 64, 1, 96, None), Problem(272, 1408, 2664, 4, 128, 3, 8, "holes")], 12000)


def test_mixed_calls():
    """Every code width, token tile and kernel of the entry points side by side."""
    cases = [(7, 1536, 2832, 4, 64, 300, 8, "holes"), (161, 768, 464, 1, 128, 17, 128, "random"),
             (16, 1280, 1976, 2, 64, 17, 48, "holes"), (55, 2176, 1032, 2, 64, 64, 32, "sorted"),
             (255, 2560, 808, 1, 64, 1, 64, "holes"), (792, 2176, 1864, 4, 64, 64, 88, "holes"),
             (428, 1408, 2752, 4, 64, 17, 120, "sorted"), (608, 1792, 1680, 2, 64, 300, 96, "holes"),
             (33, 2688, 744, 4, 64, 3, 48, None), (1541, 1408, 744, 4, 128, 1, 128, "sorted"),
             (512, 2560, 2560, 2, 128, 2, 16, "sorted"), (64, 512, 9728, 4, 64, 5, 16, "random")]
    run([Problem(*c) for c in cases], 4800)


@pytest.mark.parametrize("call", ["forward", "forward of few tokens", "gradients", "gemm_dx", "gemm", "gemm of few tokens"])
def test_first_cuda_work_of_a_thread(call):
    """A host thread that has no CUDA context yet, with buffers whose tensor maps are new: everything given,
    so that no allocation binds one first."""
    pr = Problem(9 if "few" in call else 90, 256, 264, 2, 64, 3, 16, "random")
    size = max(lb.adapter_workspace_size(pr.M, pr.N, pr.K, pr.L, pr.R), lb.workspace_size(pr.M, pr.K))
    kept = []
    for _ in range(3):
        x, dy = pr.x.clone(), pr.dy.clone()
        y, dx, da, db = (torch.empty_like(t) for t in (dy, x, pr.a, pr.b))
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        calls = {"forward": lambda: lb.adapter_gemm(x, pr.packed, *pr.args(), *pr.adapter_args(), out=y, ws=ws),
                 "gradients": lambda: lb.adapter_backward(dy, x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args(), dx=dx,
                                                          da=da, db=db, ws=ws),
                 "gemm_dx": lambda: lb.gemm_dx(dy, pr.packed_t, *pr.args(), out=dx, ws=ws),
                 "gemm": lambda: lb.gemm(x, pr.packed, *pr.args(), out=y, ws=ws)}
        failed = []

        def work():
            try:
                calls[call.split(" of ")[0]]()
            except Exception as e:
                failed.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        assert not failed, failed
        kept.append((x, dy, y, dx, da, db, ws))   # (the next round's buffers lie elsewhere)
    assert lb.device_status() == 0
