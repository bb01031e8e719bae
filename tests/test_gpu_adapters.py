"""Adapters beside the packed linear, their gradients and the 8-bit activation copy on the GPU,
against 64-bit references with bounds counted from the roundings (tests/_adapters.py)."""
import subprocess
import sys
import threading

import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import H32, HB16, Problem, backward_ref, check, checkpoint_ref, forward_ref

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


@pytest.mark.parametrize("M", [9, 16, 40, 100, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_adapters_stay_apart(M, value):
    """An adapter with an infinity or NaN gives its own tokens non-finite results and changes no other bit."""
    pr = Problem(M, 512, 264, 2, 64, 4, 16, "random")
    own = pr.rows() == 1
    y0, p0, _ = run_forward(pr)
    g0 = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
    for name, at in (("b", (1, 100, 3)), ("a", (1, 5, 300)), ("scaling", (1,))):
        t = getattr(pr, name)
        kept = t.clone()
        t[at] = value
        y, p, _ = run_forward(pr)
        assert torch.equal(y[~own], y0[~own]) and torch.equal(p[~own], p0[~own])
        assert (~torch.isfinite(y[own])).any(1).all()
        dx, da, db = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
        assert torch.equal(dx[~own], g0[0][~own]) and (~torch.isfinite(dx[own])).any(1).all()
        for got, want in ((da, g0[1]), (db, g0[2])):
            assert torch.equal(got[[0, 2, 3]], want[[0, 2, 3]])
        assert torch.equal(db, g0[2])                    # (dB does not read the adapter at all)
        setattr(pr, name, kept)


@pytest.mark.parametrize("M", [7, 16, 60, 300])
def test_not_finite_tokens_stay_apart(M):
    """A token whose input is not finite affects its own row and, in the backward, its adapter's gradients."""
    pr = Problem(M, 256, 264, 4, 64, 3, 24, "random")
    y0, p0, _ = run_forward(pr)
    g0 = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
    bad = M // 2
    others = torch.arange(M, device="cuda") != bad
    a_bad = int(pr.rows()[bad])
    rest = [l for l in range(3) if l != a_bad]
    for value in (float("nan"), float("inf")):
        pr.x[bad, 17] = value
        y, p, _ = run_forward(pr)
        assert torch.equal(y[others], y0[others]) and torch.equal(p[others], p0[others])
        assert not torch.isfinite(y[bad]).all()
        pr.dy[bad, 3] = value
        dx, da, db = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
        assert torch.equal(dx[others], g0[0][others]) and not torch.isfinite(dx[bad]).all()
        assert torch.equal(da[rest], g0[1][rest]) and torch.equal(db[rest], g0[2][rest])


def test_no_adapter_is_the_plain_product():
    """Tokens without an adapter get what the linear alone gives, to the last bit of a shared tile choice."""
    for M in (12, 80, 300):
        pr = Problem(M, 512, 512, 2, 128, 2, 16, "none")
        y, p, _ = run_forward(pr)
        assert not p.any()
        ry, ey, _, _ = forward_ref(pr)
        check(y, ry, ey, "y")
        dx, da, db = lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
        assert not da.any() and not db.any()
        assert torch.equal(dx, lb.gemm_dx(pr.dy, pr.packed_t, *pr.args()))


def test_gradients_against_differences():
    """Directional derivatives of sum(y * dy) by central differences in 64 bits of the reference forward,
    against the gradients of the kernels along the same directions."""
    pr = Problem(60, 256, 136, 2, 64, 3, 16, "holes")
    p = run_forward(pr)[1]
    pr.p = p
    dx, da, db = lb.adapter_backward(pr.dy, pr.x, p, pr.packed_t, *pr.args(), *pr.adapter_args())
    w, rows, dy = pr.weights(), pr.rows(), pr.dy.double()

    def loss(x, a, b):
        y = x @ w.T
        for l in range(pr.L):
            m = (rows == l).nonzero().flatten()
            y[m] += float(pr.scaling[l]) * (x[m] @ a[l].T) @ b[l].T
        return (y * dy).sum()

    x, a, b = pr.x.double(), pr.a.double(), pr.b.double()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for i, (t, grad) in enumerate(((x, dx), (a, da), (b, db))):
        v = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)
        args = [x, a, b]
        h = 2.0 ** -10
        args[i] = t + h * v
        up = loss(*args)
        args[i] = t - h * v
        slope = (up - loss(*args)) / (2 * h)       # exact: the loss is at most quadratic in each
        want = (grad.double() * v).sum()
        # each gradient entry is off by at most its own rounding 2^-8 and the 2^-8 of dp or p behind it
        assert abs(want - slope) <= 2 * 2.0 ** -8 * (grad.double().abs() * v.abs()).sum() + 1e-9 * slope.abs()


def test_streams_devices_and_graphs():
    """The calls on a side stream, and captured twice into graphs that replay in turn on new inputs."""
    prs = [Problem(M, 512, 264, 2, 64, 3, 16, "random", seed=i) for i, M in enumerate((10, 90, 300))]
    want = []
    for pr in prs:
        y, p, ck = run_forward(pr)
        want.append((y, p, *lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args())))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for pr, w in zip(prs, want):
            y, p, ck = run_forward(pr)
            got = (y, p, *lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args()))
            assert all(torch.equal(a, b) for a, b in zip(got, w))
    torch.cuda.current_stream().wait_stream(side)

    graphs = []
    for pr in prs:
        g = torch.cuda.CUDAGraph()
        out = {}
        with torch.cuda.graph(g):
            p = torch.empty(pr.M, pr.R, dtype=torch.bfloat16, device="cuda")
            ck = lb.checkpoint_empty(pr.M, pr.K, "cuda")
            y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), p=p, checkpoint=ck)
            out["got"] = (y, p, *lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args()))
        graphs.append((g, out))
    for turn in range(2):
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out["got"], w))
        # the same graphs on other values in the same buffers
        for pr in prs:
            pr.x.copy_(torch.randn_like(pr.x) if turn == 0 else pr.x)
            if turn == 0:
                pr.index.copy_(torch.randint(-1, 3, (pr.M,), device="cuda", dtype=torch.int32))
        if turn == 0:
            want = []
            for pr in prs:
                y, p, ck = run_forward(pr)
                want.append((y, p, *lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args())))
    assert lb.device_status() == 0


def test_results_repeat():
    for M, L, index in ((16, 5, "random"), (203, 64, "random"), (700, 3, "sorted")):
        pr = Problem(M, 1024, 520, 4, 64, L, 32, index)
        first = None
        for _ in range(4):
            y, p, ck = run_forward(pr)
            got = (y, p, ck.codes.view(torch.uint8), *lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args()))
            assert first is None or all(torch.equal(a, b) for a, b in zip(got, first))
            first = got


def test_buffers_given_and_rows_behind():
    """Outputs in given buffers; memory behind each is left as it was; a workspace of exactly the stated size."""
    for M in (3, 50, 270):
        pr = Problem(M, 256, 264, 2, 64, 3, 24, "random")
        rows = lambda n, k: torch.full((n + 8, k), 7.0, dtype=torch.bfloat16, device="cuda")
        y, p, dx, db = rows(M, 264), rows(M, 24), rows(M, 256), rows(3 * 264, 24)
        da = rows(3 * 24, 256)
        n = lb.adapter_workspace_size(M, 264, 256, 3, 24)
        ws = torch.full((n + 256,), 9, dtype=torch.uint8, device="cuda")
        lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), out=y[:M], p=p[:M], ws=ws[:n])
        lb.adapter_backward(pr.dy, pr.x, p[:M], pr.packed_t, *pr.args(), *pr.adapter_args(), dx=dx[:M],
                            da=da[:72].view(3, 24, 256), db=db[:3 * 264].view(3, 264, 24), ws=ws[:n])
        assert torch.equal(y[:M], run_forward(pr)[0])
        for t, m in ((y, M), (p, M), (dx, M), (da, 72), (db, 3 * 264)):
            assert (t[m:] == 7).all()
        assert (ws[n:] == 9).all()
        with pytest.raises(lb.LowbitError):
            lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), ws=ws[:M * 256 * 2])


def test_empty_batches():
    pr = Problem(5, 256, 264, 2, 64, 3, 24, "random")
    none = lambda k: torch.empty(0, k, dtype=torch.bfloat16, device="cuda")
    idx = torch.empty(0, dtype=torch.int32, device="cuda")
    y = lb.adapter_gemm(none(256), pr.packed, *pr.args(), pr.a, pr.b, pr.scaling, idx)
    assert y.shape == (0, 264)
    dx, da, db = lb.adapter_backward(none(264), none(256), none(24), pr.packed_t, *pr.args(), pr.a, pr.b, pr.scaling, idx)
    assert dx.shape == (0, 256) and not da.any() and not db.any()
    assert lb.gemm_dx(none(264), pr.packed_t, *pr.args()).shape == (0, 256)
    assert lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args(), need_dx=False)[0] is None


def test_injected_failures_reach_the_caller():
    lib = lb.load()
    for M in (8, 100):
        pr = Problem(M, 256, 264, 2, 64, 3, 24, "random")
        want = run_forward(pr)[0]
        for what in (1, 2):
            assert lib.lowbit_test_fail_next(what) == 0
            with pytest.raises(lb.LowbitError, match="CUDA"):
                lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args())
            assert lib.lowbit_test_fail_next(what) == 0
            with pytest.raises(lb.LowbitError, match="CUDA"):
                lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())
        assert lib.lowbit_test_fail_next(2) == 0
        with pytest.raises(lb.LowbitError, match="CUDA"):
            lb.checkpoint_store(pr.x)
        assert torch.equal(run_forward(pr)[0], want)


def test_debug_build():
    """The same calls on the build with device-side index checks: no check fires, and the same results."""
    pr = Problem(150, 512, 264, 2, 64, 5, 24, "holes")
    y, p, ck = run_forward(pr)
    g = lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args())
    release = lb._lib
    try:
        lb._lib = lb.load_debug()
        y2, p2, ck2 = run_forward(pr)
        g2 = lb.adapter_backward(pr.dy, ck2, p2, pr.packed_t, *pr.args(), *pr.adapter_args())
        assert lb.device_status() == 0
    finally:
        lb._lib = release
    assert torch.equal(y, y2) and torch.equal(p, p2) and all(torch.equal(a, b) for a, b in zip(g, g2))


@pytest.mark.parametrize("R", [8, 32, 64, 128])
@pytest.mark.parametrize("index", ["sorted", "random"])
def test_gradients_over_many_tiles(R, index):
    """More tiles than SMs, so that a CTA goes through several, of the 8-bit and the bf16 operand, with long
    and empty segments; tokens that follow one another and tokens that do not."""
    pr = Problem(2500, 4096, 5120, 2, 128, 4, R, index)
    idx = pr.index.clone()
    idx[idx == 2] = 3                     # an adapter without tokens
    pr.index = idx
    for x in (pr.x, lb.checkpoint_store(pr.x)):
        value = lb.checkpoint_load(x) if isinstance(x, lb.Checkpoint) else x
        got = lb.adapter_backward(pr.dy, x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args(), need_dx=False)
        assert lb.device_status() == 0
        _, (ra, ea), (rb, eb) = backward_ref(pr, value)
        check(got[1], ra, ea, "da")
        check(got[2], rb, eb, "db")


@pytest.mark.parametrize("M,L,index", [(600, 1, None), (2100, 1, "holes"), (2100, 2, "last"), (2100, 3, None),
                                       (1100, 2, "random")])
@pytest.mark.parametrize("R", [16, 40, 64, 128])
def test_gradients_of_many_tokens(M, L, index, R):
    """Few tiles and many tokens; the same bits every time."""
    pr = Problem(M, 320, 264, 4, 64, L, R, index)
    for x in (pr.x, lb.checkpoint_store(pr.x)):
        value = lb.checkpoint_load(x) if isinstance(x, lb.Checkpoint) else x
        calls = [lb.adapter_backward(pr.dy, x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args()) for _ in range(3)]
        assert lb.device_status() == 0
        for (r, e), got in zip(backward_ref(pr, value), calls[0]):
            check(got, r, e, "gradient")
        assert all(torch.equal(a, b) for c in calls[1:] for a, b in zip(c, calls[0]))


def test_two_threads_on_two_streams():
    """Calls of two host threads on streams of their own at once, each against its own results alone."""
    prs = [Problem(M, 1024, 776, 2, 64, 5, 32, "random", seed=M) for M in (14, 410)]
    want, bad = [], []
    for pr in prs:
        y, p, ck = run_forward(pr)
        want.append((y, *lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args())))
    torch.cuda.synchronize()

    def work(pr, w):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                p = torch.empty(pr.M, pr.R, dtype=torch.bfloat16, device="cuda")
                ck = lb.checkpoint_empty(pr.M, pr.K, "cuda")
                y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), p=p, checkpoint=ck)
                got = (y, *lb.adapter_backward(pr.dy, ck, p, pr.packed_t, *pr.args(), *pr.adapter_args()))
                if not all(torch.equal(a, b) for a, b in zip(got, w)):
                    bad.append(pr.M)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=a) for a in zip(prs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and lb.device_status() == 0


@pytest.mark.parametrize("M", [12, 300])
def test_first_call_under_capture(M):
    """A process whose first calls of these entry points are captured."""
    code = f"""
import torch, bit_weight_only_w2_b200 as lb
from tests._adapters import Problem, forward_ref, check
pr = Problem({M}, 512, 264, 2, 64, 3, 16, "random")
p = torch.empty(pr.M, pr.R, dtype=torch.bfloat16, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), p=p)
    dx, da, db = lb.adapter_backward(pr.dy, pr.x, p, pr.packed_t, *pr.args(), *pr.adapter_args())
g.replay()
torch.cuda.synchronize()
ry, ey, rp, ep = forward_ref(pr)
check(y, ry, ey, "y")
check(p, rp, ep, "p")
eager = lb.adapter_backward(pr.dy, pr.x, p, pr.packed_t, *pr.args(), *pr.adapter_args())
assert all(torch.equal(a, b) for a, b in zip(eager, (dx, da, db)))
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_offsets_past_32_bits():
    """More than 2^31 values in x, dx and the 8-bit copy, and 2^32 bytes in each: rows at both ends and
    across the borders, and the gradients of an adapter whose tokens are those rows."""
    M, K, N = 234057, 9216, 136
    pr = Problem(48, K, N, 2, 64, 2, 16)
    border = (1 << 31) // K
    rows = torch.cat([torch.arange(0, 8), torch.arange(border // 2 - 4, border // 2 + 4),
                      torch.arange(border - 8, border + 16), torch.arange(M - 8, M)]).cuda()
    assert len(rows) == pr.M and M * K > 1 << 31
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    dy = torch.full((M, N), 0.01, dtype=torch.bfloat16, device="cuda")
    index = torch.zeros(M, dtype=torch.int32, device="cuda")
    x[rows], dy[rows], index[rows] = pr.x, pr.dy, 1
    p, ck = torch.empty(M, 16, dtype=torch.bfloat16, device="cuda"), lb.checkpoint_empty(M, K, "cuda")
    y = lb.adapter_gemm(x, pr.packed, *pr.args(), pr.a, pr.b, pr.scaling, index, p=p, checkpoint=ck)
    pr.index = torch.ones(pr.M, dtype=torch.int32, device="cuda")
    ry, ey, rp, ep = forward_ref(pr)
    check(p[rows], rp, ep, "p")
    check(y[rows], ry, ey, "y")
    codes, exps, _ = checkpoint_ref(pr.x)
    assert torch.equal(ck.exps[rows].cpu(), exps) and torch.equal(ck.codes[rows].double().cpu(), codes)
    again = lb.checkpoint_store(x)
    assert torch.equal(again.codes.view(torch.uint8), ck.codes.view(torch.uint8)) and torch.equal(again.exps, ck.exps)
    del again
    pr.p, kept = p[rows], lb.checkpoint_load(lb.Checkpoint(ck.codes[rows].contiguous(), ck.exps[rows].contiguous()))
    assert torch.equal(lb.checkpoint_load(ck)[rows], kept)
    for inp, seen in ((x, pr.x), (ck, kept)):
        dx, da, db = lb.adapter_backward(dy, inp, p, pr.packed_t, *pr.args(), pr.a, pr.b, pr.scaling, index)
        (rdx, edx), (rda, eda), (rdb, edb) = backward_ref(pr, seen)
        check(dx[rows], rdx, edx, "dx")
        check(da[1], rda[1], eda[1], "da")
        check(db[1], rdb[1], edb[1], "db")
    assert lb.device_status() == 0


@pytest.mark.parametrize("graph", [False, True])
def test_calls_in_a_row_on_one_workspace(graph):
    """Kernels of neighbouring calls overlap at their ends: a row of calls of different lengths on one
    workspace gives what the same calls give one by one."""
    prs = [Problem(1200, 2048, 2048, 2, 64, 1, 8, None), Problem(90, 512, 264, 4, 64, 3, 64), Problem(40, 256, 1032, 1, 128, 2, 16),
           Problem(700, 384, 4096, 2, 128, 4, 128, "holes")]
    size = max(lb.adapter_workspace_size(pr.M, pr.N, pr.K, pr.L, pr.R) for pr in prs)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def row(between):
        out = []
        for pr in prs + prs[::-1]:
            for call in (lambda: [lb.adapter_gemm(pr.x, pr.packed, *pr.args(), *pr.adapter_args(), ws=ws)],
                         lambda: list(lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args(), ws=ws)),
                         lambda: [lb.gemm_dx(pr.dy, pr.packed_t, *pr.args(), ws=ws)],
                         lambda: list(lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args(), ws=ws)),
                         lambda: list(lb.adapter_backward(pr.dy, pr.x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args(),
                                                          need_dx=False, ws=ws))[1:]):
                out += call()
                between()
        return out

    want = row(torch.cuda.synchronize)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = row(lambda: None)
    for _ in range(10):
        if graph:
            for t in got:
                t.zero_()
            g.replay()
        else:
            got = row(lambda: None)
        assert lb.device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M,L,index", [(3, 1, None), (65, 2, "sorted"), (40, 7, "random")])
@pytest.mark.parametrize("R", [8, 24, 64, 128])
@pytest.mark.parametrize("eight", [False, True])
def test_da_is_rounded_once(M, L, index, R, eight):
    """dA within half a step of bf16, where a few large channels and few tokens leave nothing to average
    dp's rounding: dp comes in two terms (2^-16)."""
    pr = Problem(M, 256, 264, 2, 64, L, R, index)
    pr.x[:, 5::100] *= 16
    x = lb.checkpoint_store(pr.x) if eight else pr.x
    seen = (lb.checkpoint_load(x) if eight else x).double()
    da = lb.adapter_backward(pr.dy, x, pr.p, pr.packed_t, *pr.args(), *pr.adapter_args())[1]
    assert lb.device_status() == 0
    rows, h = pr.rows(), HB16
    for l in range(L):
        m = (rows == l).nonzero().flatten()
        dy, b, sc, n = pr.dy[m].double(), pr.b[l].double(), float(pr.scaling[l]), len(m)
        dp = sc * (dy @ b)
        f = (pr.N + 2) * H32 * sc * (dy.abs() @ b.abs())
        pe = f + h * h * (dp.abs() + f)
        ref = dp.T @ seen[m]
        e = pe.T @ seen[m].abs() + 2 * n * H32 * (1 + h) * (dp.abs().T @ seen[m].abs())
        check(da[l], ref, e + h * (ref.abs() + e), "da")
