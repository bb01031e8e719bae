"""Vocabulary operators on the GPU at the edges of what the entry points take: empty and ignored inputs, values that are
not finite, buffers and what lies behind them, graphs, streams, long offsets, and a run of them together."""
import threading

import pytest
import torch

import bit_weight_only_w2_b200 as lb
from tests._adapters import check
from tests._vocab import H32, HB16, Loss, Table, embedding_grad_ref, embedding_ref, inputs

pytestmark = pytest.mark.gpu

BF16 = dict(dtype=torch.bfloat16, device="cuda")


def loss_step(table, x, labels, grad, V):
    loss, lse = lb.cross_entropy(x, labels, *table.args(), vocab=V)
    dx, dw = lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V, need_dw=table.bits == 16)
    return (loss, lse, dx) if dw is None else (loss, lse, dx, dw)


def check_loss(table, x, labels, grad, V, got):
    ref = Loss(x, labels, table, V)
    check(got[1], ref.lse, ref.e_lse, "lse")
    check(got[0], ref.loss, ref.e_loss, "loss")
    (rx, ex), (rw, ew) = ref.gradients(grad, got[1])
    check(got[2], rx, ex, "dx")
    if len(got) > 3:
        check(got[3][:V], rw, ew, "dw")


@pytest.mark.parametrize("bits,gs", [(1, 128), (2, 64), (4, 64), (16, 0)])
@pytest.mark.parametrize("rest", [1, 9, 16, 100, 300])
def test_tokens_behind_the_first_sixteen_thousand(bits, gs, rest):
    """The forward takes 16384 tokens at a time; what is left may be as few as any kernel takes."""
    M, K, V = 16384 + rest, 128, 131
    table = Table(136, K, bits, gs)
    x, labels, _ = inputs(M, K, V)
    loss, lse = lb.cross_entropy(x, labels, *table.args(), vocab=V)
    assert lb.device_status() == 0
    ref = Loss(x, labels, table, V)
    check(lse, ref.lse, ref.e_lse, "lse")
    check(loss, ref.loss, ref.e_loss, "loss")


@pytest.mark.parametrize("bits,gs", [(2, 64), (16, 0)])
def test_nothing_to_do(bits, gs):
    table = Table(64, 128, bits, gs)
    x, labels, f = torch.empty(0, 128, **BF16), torch.empty(0, device="cuda", dtype=torch.int32), torch.empty(0, device="cuda")
    loss, lse = lb.cross_entropy(x, labels, *table.args())
    assert loss.shape == lse.shape == (0,)
    dw = torch.full((64, 128), float("nan"), **BF16) if bits == 16 else None
    dx, got = lb.cross_entropy_backward(f, x, labels, lse, *table.args(), need_dw=bits == 16, dw=dw)
    assert dx.shape == (0, 128) and got is dw and (dw is None or not dw.any())
    assert lb.embedding(labels, *table.args()).shape == (0, 128)
    de = torch.full((5, 128), float("nan"), **BF16)
    assert not lb.embedding_backward(labels, x, 5, out=de).any()
    assert lb.embedding_backward(labels, x, 0).shape == (0, 128)
    tokens, dy = torch.zeros(3, device="cuda", dtype=torch.int32), torch.ones(3, 128, **BF16)
    assert lb.embedding_backward(tokens, dy, 0).shape == (0, 128)


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("bits,gs", [(1, 128), (2, 64), (4, 64), (16, 0)])
def test_no_label_at_all(bits, gs, M):
    """Every label outside the vocabulary: a lse, no loss, no gradient, even from rows that are not finite."""
    K, V = 256, 197
    table = Table(200, K, bits, gs)
    x, _, grad = inputs(M, K, V)
    labels = torch.tensor([-100, V, 2 ** 31 - 1, -1, -2 ** 31, 199], device="cuda").repeat(M // 6 + 1)[:M].int()
    got = loss_step(table, x, labels, grad, V)
    check_loss(table, x, labels, grad, V, got)
    assert not got[0].any() and all(not g.any() for g in got[2:])
    x[1] = float("inf")
    x[2, 7] = float("nan")
    grad[0] = float("nan")
    got = loss_step(table, x, labels, grad, V)
    assert not got[0].any() and all(not g.any() for g in got[2:])
    (table.weight if bits == 16 else table.scales)[0, 3] = float("inf")
    got = loss_step(table, x, labels, grad, V)
    assert not got[2].any()


@pytest.mark.parametrize("M", [1, 7, 16, 90, 300])
@pytest.mark.parametrize("bits,gs", [(1, 128), (2, 64), (4, 64), (16, 0)])
def test_not_finite(bits, gs, M):
    """A token whose x is not finite has a loss and gradient that are not; the others' are as without it. Rows behind the
    vocabulary take no part, whatever they hold."""
    K, N, V = 384, 264, 257
    table = Table(N, K, bits, gs)
    x, labels, grad = inputs(M, K, V, ignored=0)
    labels = labels % V
    want = loss_step(table, x, labels, grad, V)
    if bits == 16:
        table.weight[V:] = float("nan")
    else:
        table.scales[:, V:] = float("inf")
        table.weight[V:] = -1
    got = loss_step(table, x, labels, grad, V)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[M // 2, 5] = bad
        got = loss_step(table, y, labels, grad, V)
        assert lb.device_status() == 0
        keep = torch.arange(M, device="cuda") != M // 2
        assert not torch.isfinite(got[0][~keep]).any() and not torch.isfinite(got[2][~keep]).all()
        for a, b in zip(got[:3], want):
            assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("M", [5, 16, 100, 257])
@pytest.mark.parametrize("bits,gs", [(2, 64), (4, 128), (16, 0)])
def test_one_row_and_far_logits(bits, gs, M):
    """A vocabulary of one row (loss and gradients are zero), and logits far from zero on both sides."""
    K = 128
    table = Table(8, K, bits, gs)
    x, labels, grad = inputs(M, K, 1)
    labels = torch.zeros_like(labels)
    got = loss_step(table, x, labels, grad, 1)
    check_loss(table, x, labels, grad, 1, got)
    far = Table(504, K, bits, gs, norm=200.0)
    for sign in (1.0, -1.0):
        x, labels, grad = inputs(M, K, 500)
        x = sign * x.abs()
        got = loss_step(far, x, labels, grad, 500)
        assert torch.isfinite(got[0]).all()
        check_loss(far, x, labels, grad, 500, got)


def guarded(shape, dtype, fill=7.0):
    """A tensor inside a larger one, and what has to stay as it is around it (256 bytes each side)."""
    n = 1
    for s in shape:
        n *= s
    pad = 256 // torch.empty(0, dtype=dtype).element_size()
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return whole[pad:pad + n].view(shape), lambda: bool((whole[:pad] == fill).all() and (whole[pad + n:] == fill).all())


@pytest.mark.parametrize("bits,gs", [(1, 128), (2, 128), (4, 64), (16, 0)])
@pytest.mark.parametrize("M,larger", [(1, 1), (16, 17), (13, 128), (77, 129), (128, 200), (200, 16385), (300, 300)])
def test_buffers_and_workspaces_of_a_larger_batch(bits, gs, M, larger):
    K, N, V = 256, 1000, 997
    table = Table(N, K, bits, gs)
    x, labels, grad = inputs(M, K, V)
    want = loss_step(table, x, labels, grad, V)
    loss, ok1 = guarded((M,), torch.float32)
    lse, ok2 = guarded((M,), torch.float32)
    dx, ok3 = guarded((M, K), torch.bfloat16)
    dw, ok4 = guarded((N, K), torch.bfloat16) if bits == 16 else (None, lambda: True)
    ws, ok5 = guarded((lb.cross_entropy_workspace_size(larger, V, K, bits, 0),), torch.uint8, 9)
    r = lb.cross_entropy(x, labels, *table.args(), vocab=V, loss=loss, lse=lse, ws=ws)
    assert r[0] is loss and r[1] is lse
    ws, ok6 = guarded((lb.cross_entropy_workspace_size(larger, V, K, bits, 2 if bits == 16 else 1),), torch.uint8, 9)
    r = lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V, need_dw=bits == 16, dx=dx, dw=dw, ws=ws)
    assert r[0] is dx and r[1] is dw
    got = (loss, lse, dx) if dw is None else (loss, lse, dx, dw)
    assert lb.device_status() == 0 and all(ok() for ok in (ok1, ok2, ok3, ok4, ok5, ok6))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(lb.LowbitError, match="WORKSPACE"):
        lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V, ws=ws[:256])
    with pytest.raises(ValueError):   # a packed table's dW; a buffer for one that is not asked for
        lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), vocab=V, need_dw=bits != 16, dw=dw)
    with pytest.raises(ValueError):
        lb.cross_entropy(x, labels, *table.args(), vocab=N + 1)


@pytest.mark.parametrize("T,rows,larger", [(5, 24, 5), (1000, 24, 4097), (1500, 700, 2049), (5000, 700, 200000)])
def test_lookup_buffers(T, rows, larger):
    K = 264
    g = torch.Generator(device="cuda").manual_seed(T)
    tokens = torch.randint(90, 110 + rows, (T,), generator=g, device="cuda", dtype=torch.int32)
    dy = torch.randn(T, K, generator=g, **BF16)
    de, ok1 = guarded((rows, K), torch.bfloat16)
    ws, ok2 = guarded((lb.embedding_workspace_size(larger, rows, K),), torch.uint8, 9)
    lb.embedding_backward(tokens, dy, rows, first=100, out=de, ws=ws)
    check(de, *embedding_grad_ref(tokens, dy, 100, rows, 1.0), "de")
    table = Table(100 + rows, K, 16)
    y, ok3 = guarded((T, K), torch.bfloat16)
    assert lb.embedding(tokens, *table.args(), multiplier=3.0, out=y) is y
    check(y, *embedding_ref(tokens, table, 3.0), "y")
    assert ok1() and ok2() and ok3()
    if T > 4096:
        with pytest.raises(lb.LowbitError, match="WORKSPACE"):
            lb.embedding_backward(tokens, dy, rows, first=100, ws=ws[:512])


@pytest.mark.parametrize("T,K,rows", [(100003, 72, 5000), (20000, 1032, 300)])
def test_one_token_over_and_over(T, K, rows):
    """Nearly all tokens the same row: its sum runs over every run of the sorted list."""
    g = torch.Generator(device="cuda").manual_seed(T)
    tokens = torch.full((T,), 17, device="cuda", dtype=torch.int32)
    tokens[:: 1001] = 16
    tokens[1:: 1003] = rows - 1
    dy = torch.randn(T, K, generator=g, **BF16)
    check(lb.embedding_backward(tokens, dy, rows), *embedding_grad_ref(tokens, dy, 0, rows, 1.0), "de")
    dy[5] = float("inf")
    tokens[5] = 3
    de = lb.embedding_backward(tokens, dy, rows)
    assert (de[3] == float("inf")).all() and torch.isfinite(de[:3]).all() and torch.isfinite(de[4:]).all()


class Step:
    """The two ends of a training step around one frozen ternary linear: embeddings from a table of its own, the linear,
    a head, and the gradients back to both tables."""

    def __init__(self, M, K, H, V, head_bits, seed=0):
        self.M, self.V, self.mult = M, V, 1.5
        self.embed, self.linear = Table(V, K, 16, seed=seed), Table(H, K, 2, 64, seed=seed, norm=1.0)
        self.head = Table((V + 7) // 8 * 8, H, head_bits, 0 if head_bits == 16 else 64, seed=seed)
        g = torch.Generator(device="cuda").manual_seed(M + V + seed)
        self.tokens = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
        _, self.labels, _ = inputs(M, 8, V, seed=seed)
        self.grad = torch.full((M,), 1.0 / M, device="cuda")
        self.linear_t = lb.transpose_packed(self.linear.weight, K, 2)

    def run(self):
        e = lb.embedding(self.tokens, *self.embed.args(), multiplier=self.mult)
        h = lb.gemm(e, *self.linear.args())
        loss, lse = lb.cross_entropy(h, self.labels, *self.head.args(), vocab=self.V)
        dh, dw = lb.cross_entropy_backward(self.grad, h, self.labels, lse, *self.head.args(), vocab=self.V,
                                           need_dw=self.head.bits == 16)
        de = lb.gemm_dx(dh, self.linear_t, self.linear.scales, None, 2, 64)
        dtable = lb.embedding_backward(self.tokens, de, self.V, multiplier=self.mult)
        return [t for t in (e, h, loss, lse, dh, dw, de, dtable) if t is not None]


@pytest.mark.parametrize("M,K,H,V,bits", [(6, 128, 256, 50, 16), (77, 256, 384, 203, 4), (200, 256, 128, 1001, 16),
                                          (40, 128, 128, 500, 2)])
def test_a_step_against_autograd(M, K, H, V, bits):
    """Each call of the run against 64 bits on what it was handed, and the whole against autograd in 64 bits: per token, the
    roundings of e and h (half a step each) move a logit by at most |dh| max |w| = D, so its loss by 2 D and its softmax by
    e^(2 D) - 1; norms of the products carry that, and the roundings of G, dh, de and dtable, to the end (2 % on top for
    products of these and fp32 sums)."""
    st = Step(M, K, H, V, bits)
    out = st.run()
    assert lb.device_status() == 0
    names = dict(zip(("e", "h", "loss", "lse", "dh") + (("dw",) if bits == 16 else ()) + ("de", "dtable"), out))
    W, head = st.linear.rows(), st.head.rows()[:V]
    check(names["e"], *embedding_ref(st.tokens, st.embed, st.mult), "e")
    product = lambda a, b, n: (a @ b, n * H32 * (a.abs() @ b.abs()) * (1 + HB16) + HB16 * (a @ b).abs())
    check(names["h"], *product(names["e"].double(), W.T, K), "h")
    check_loss(st.head, names["h"], st.labels, st.grad, V, [names[n] for n in ("loss", "lse", "dh") + (("dw",) if bits == 16 else ())])
    check(names["de"], *product(names["dh"].double(), W, H), "de")
    check(names["dtable"], *embedding_grad_ref(st.tokens, names["de"], 0, V, st.mult), "dtable")

    table, head_ = st.embed.rows().requires_grad_(), head.clone().requires_grad_()
    e = table[st.tokens.long()] * st.mult
    h = e @ W.T
    logits = h @ head_.T
    valid = (st.labels >= 0) & (st.labels < V)
    lse = torch.logsumexp(logits, 1)
    loss = torch.where(valid, lse - logits.gather(1, torch.where(valid, st.labels, 0).long()[:, None])[:, 0], 0.0)
    dh, de = torch.autograd.grad((loss * st.grad).sum(), (h, e), retain_graph=True)
    (loss * st.grad).sum().backward()
    e, h, loss = e.detach(), h.detach(), loss.detach()
    norm2 = lambda a: torch.linalg.matrix_norm(a, 2)
    D = 1.02 * HB16 * (e.norm(dim=1) * norm2(W) + h.norm(dim=1)) * head.norm(dim=1).max()
    assert ((names["loss"].double() - loss).abs() <= 2 * D + 1e-5).all()
    p = torch.softmax(logits.detach(), 1) * st.grad[:, None]
    p[~valid] = 0
    hot = torch.zeros_like(p)
    hot[valid, st.labels[valid].long()] = st.grad.double()[valid]
    off = 1.02 * ((torch.expm1(2 * D)[:, None] * p).norm() + HB16 * (p + hot).norm()) * norm2(head) + 1.02 * HB16 * dh.norm()
    assert float((names["dh"].double() - dh).norm()) <= off
    off = 1.02 * (off * norm2(W) + HB16 * de.norm())
    assert float((names["de"].double() - de).norm()) <= off
    off = 1.02 * (st.mult * off * torch.bincount(st.tokens.long()).max().double().sqrt() + HB16 * table.grad.norm())
    assert float((names["dtable"].double() - table.grad).norm()) <= off


@pytest.mark.parametrize("bits,gs", [(4, 64), (16, 0)])
@pytest.mark.parametrize("M", [4, 40, 140])
def test_gradient_against_differences(bits, gs, M):
    """Central differences of the calls' own losses along directions d: the difference's own errors are the two losses' over
    2 h, and the third derivative's, which is the difference of the 64-bit losses less their derivative."""
    K, V, h = 128, 120, 2.0 ** -5
    table = Table(V, K, bits, gs)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.randint(-32, 33, (M, K), generator=g, device="cuda") / 32).bfloat16()    # (x +- h d is exact in bf16)
    labels = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    one = torch.ones(M, device="cuda")
    loss, lse = lb.cross_entropy(x, labels, *table.args())
    dx, _ = lb.cross_entropy_backward(one, x, labels, lse, *table.args())
    ref = Loss(x, labels, table, V)
    (rx, ex), _ = ref.gradients(one, lse)
    for _ in range(3):
        d = torch.randint(-1, 2, (M, K), generator=g, device="cuda").double()
        up, down = ((x.double() + s * h * d).bfloat16() for s in (1, -1))
        assert torch.equal(up.double() - down.double(), 2 * h * d)
        a, b = (lb.cross_entropy(y, labels, *table.args())[0].double() for y in (up, down))
        ra, rb = Loss(up, labels, table, V), Loss(down, labels, table, V)
        third = ((ra.loss - rb.loss) / (2 * h) - (rx * d).sum(1)).abs()
        bound = (ra.e_loss + rb.e_loss) / (2 * h) + third + (ex * d.abs()).sum(1)
        check((a - b) / (2 * h), (dx.double() * d).sum(1), bound + 1e-12, "difference")


@pytest.mark.parametrize("bits", [16, 4])
def test_captured(bits):
    """A step captured into a graph and replayed on new inputs, beside eager calls and a second graph of the same step."""
    st, other = Step(130, 256, 128, 700, bits), Step(130, 256, 128, 700, bits, seed=1)
    want = [st.run(), other.run()]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        st.run()
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=stream):
                out = st.run()
            graphs.append((gr, out))
    torch.cuda.current_stream().wait_stream(stream)
    first = (st.tokens.clone(), st.labels.clone(), st.embed.weight.clone(), st.head.weight.clone())
    second = (other.tokens, other.labels, other.embed.weight, other.head.weight)
    both = [[st.linear, st.head], [other.linear, other.head]]
    pieces = [[[t.clone() for t in (b.weight, b.scales, b.zeros) if t is not None] for b in pair] for pair in both]
    lt = [st.linear_t.clone(), other.linear_t.clone()]
    for i in (0, 1, 1, 0):
        for to, new in zip((st.tokens, st.labels, st.embed.weight, st.head.weight), (first, second)[i]):
            to.copy_(new)
        for t, new in zip(both[0], pieces[i]):
            for a, b in zip([v for v in (t.weight, t.scales, t.zeros) if v is not None], new):
                a.copy_(b)
        st.linear_t.copy_(lt[i])
        for gr, out in graphs:
            gr.replay()
            eager = st.run()
            torch.cuda.synchronize()
            assert lb.device_status() == 0
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
            assert all(torch.equal(a, b) for a, b in zip(eager, want[i]))


def test_calls_of_several_streams():
    """Steps of four streams at once: each result is, bit for bit, what the step gives alone."""
    steps = [Step(5, 128, 256, 1000, 4), Step(33, 256, 128, 3001, 16), Step(77, 256, 256, 5003, 4), Step(300, 384, 128, 2001, 2),
             Step(700, 128, 384, 9001, 16), Step(16, 256, 256, 777, 2)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for i in range(60):
                j = (i * (k + 1) + k) % len(steps)
                got = steps[j].run()
                torch.cuda.current_stream().synchronize()
                bad.extend((j, n) for n, (a, b) in enumerate(zip(got, want[j])) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert lb.device_status() == 0 and not bad, bad[:8]


@pytest.mark.parametrize("bits,gs", [(2, 64), (16, 0)])
def test_first_cuda_work_of_a_thread(bits, gs):
    M, K, V = 40, 128, 264
    table = Table(V, K, bits, gs)
    x, labels, grad = inputs(M, K, V)
    want = loss_step(table, x, labels, grad, V)[0]
    loss, lse, y = torch.empty_like(want), torch.empty_like(want), torch.empty_like(x)
    ws = torch.empty(lb.cross_entropy_workspace_size(M, V, K, bits, 0), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            lb.embedding(labels, *table.args(), out=y)
            lb.cross_entropy(x, labels, *table.args(), loss=loss, lse=lse, ws=ws)
        except Exception as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed and torch.equal(loss, want)
    check(y, *embedding_ref(labels, table, 1.0), "y")


@pytest.mark.parametrize("bits,gs", [(4, 64), (16, 0)])
def test_without_the_compiled_marshalling(bits, gs, monkeypatch):
    st = Step(50, 128, 256, 300, bits)
    want = st.run()
    calls = object.__new__(lb._Marshalled)
    calls.lib = lb.load()
    for name in ("embedding", "embedding_backward", "cross_entropy", "cross_entropy_backward", "gemm_dx"):
        setattr(calls, name, lambda *args: None)
    monkeypatch.setattr(lb, "_marshalled", calls)
    got = st.run()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_arguments_that_do_not_fit_are_refused_by_name():
    M, K, N = 20, 128, 72
    table = Table(N, K, 4, 64)
    x, labels, grad = inputs(M, K, N)
    f = lambda: torch.zeros(M, device="cuda")
    ws = torch.empty(lb.cross_entropy_workspace_size(M, N, K, 4, 1), dtype=torch.uint8, device="cuda")
    t = dict(weight=table.weight, scales=table.scales, zeros=table.zeros, bits=4, group_size=64)
    fwd = dict(t, x=x, labels=labels, loss=f(), lse=f(), ws=ws)
    bwd = dict(t, grad=grad, x=x, labels=labels, lse=f(), dx=torch.empty_like(x), ws=ws)
    look = dict(t, tokens=labels, out=torch.empty_like(x))
    back = dict(tokens=labels, dy=x, rows=9, out=torch.empty(9, K, **BF16), ws=ws)
    for fn, kw in ((lb.cross_entropy, fwd), (lb.cross_entropy_backward, bwd), (lb.embedding, look), (lb.embedding_backward, back)):
        fn(**kw)
        for name, v in kw.items():
            if not isinstance(v, torch.Tensor):
                continue
            wide = torch.stack([v, v], -1)[..., 0]
            for b in [v.double(), v.cpu(), wide, v[None]] + ([v[:-1]] if name not in ("ws", "tokens", "weight") else []):
                with pytest.raises(ValueError):
                    fn(**dict(kw, **{name: b}))
    for fn, kw in ((lb.cross_entropy, fwd), (lb.cross_entropy_backward, bwd), (lb.embedding, look)):
        for name, b in (("scales", None), ("bits", 16), ("bits", 3), ("group_size", 48)):
            with pytest.raises(ValueError):
                fn(**dict(kw, **{name: b}))
        with pytest.raises(lb.LowbitError, match="INVALID"):
            fn(**dict(kw, zeros=None))
    for name, b in (("rows", -1), ("first", -2)):
        with pytest.raises(ValueError):
            lb.embedding_backward(**dict(back, out=None, **{name: b}))


def test_past_32_bits():
    """More than 2^31 values in a table, its gradients and the embeddings."""
    K, N = 4096, 600008
    assert N * K > 1 << 31
    w = torch.zeros(N, K, **BF16)
    at = torch.tensor([0, 1, 524287, 524288, 599999, 600007], device="cuda")
    rows = Table(6, K, 16)
    w[at] = rows.weight
    tokens = at.int().repeat(100001)[:N - 2]
    y = lb.embedding(tokens, w)
    for lo in range(0, N - 2, 60000):
        assert torch.equal(y[lo:lo + 60000], rows.weight.repeat(10000, 1)[:y[lo:lo + 60000].shape[0]])
    small = tokens[:1200]
    de = lb.embedding_backward(small, y[:1200], N)
    r, e = embedding_grad_ref(torch.arange(6, device="cuda").repeat(200), y[:1200], 0, 6, 1.0)
    check(de[at], r, e, "de")
    assert int((de != 0).any(1).sum()) == 6
    del y, de
    # a logit of zero for all rows but six
    M = 5
    x, _, grad = inputs(M, K, 6)
    labels = at[[5, 4, 2, 0, 3]].int()
    loss, lse = lb.cross_entropy(x, labels, w)
    l = x.double() @ rows.rows().T
    full = torch.cat([l, torch.zeros(M, 1, device="cuda", dtype=torch.float64)], 1)
    full[:, 6] += torch.log(torch.tensor(float(N - 6), dtype=torch.float64))
    want = torch.logsumexp(full, 1)
    s = K * H32 * (x.double().abs() @ rows.rows().abs().T).amax(1)
    check(lse, want, s + 2.0 ** -14, "lse")   # (sums of 600008 terms: 413 steps of 2^-24, and the arguments)
    dx, dw = lb.cross_entropy_backward(grad, x, labels, lse, w, need_dw=True)
    assert lb.device_status() == 0
    p = (l - lse.double()[:, None]).exp()
    hot = torch.zeros_like(p)
    hot[torch.arange(M, device="cuda"), torch.tensor([5, 4, 2, 0, 3], device="cuda")] = 1
    G = grad.double()[:, None] * (p - hot)
    eG = (HB16 + 2 * s.amax() + 2.0 ** -15) * (grad.double().abs()[:, None] * (p + hot))
    check(dx, G @ rows.rows(), (1 + HB16) * (eG @ rows.rows().abs()) + HB16 * (G @ rows.rows()).abs() +
          N * H32 * (G.abs() @ rows.rows().abs()), "dx")
    check(dw[at], G.T @ x.double(), (1 + HB16) * (eG.T @ x.double().abs()) + 2 * HB16 * (G.T @ x.double()).abs(), "dw")
    other = grad.double()[:, None] * (-lse.double()).exp()[:, None] * x.double()
    got = dw[[2, 300000, 524289, 600000]].double()
    check(got, other.sum(0).expand(4, K), (2.0 ** -7 + 2.0 ** -15) * other.abs().sum(0).expand(4, K), "dw of the others")


@pytest.mark.parametrize("V", [500, 40000])
def test_same_results_every_time(V):
    """No result depends on timing: twenty calls, while another stream keeps the GPU busy."""
    table = Table((V + 7) // 8 * 8, 256, 2, 64)
    x, labels, grad = inputs(700, 256, V)
    tokens = labels.abs() % 300
    want = loss_step(table, x, labels, grad, V) + (lb.embedding_backward(tokens, x, 300),)
    side = torch.cuda.Stream()
    a = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            a @ a
        got = loss_step(table, x, labels, grad, V) + (lb.embedding_backward(tokens, x, 300),)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("T,K,first,rows", [(1, 8, 0, 4000), (7, 1240, 3, 4001), (200, 1032, 0, 3000), (256, 136, 50, 20011),
                                            (256, 2560, 0, 3276), (256, 2560, 0, 3278), (257, 136, 5, 2000)])
@pytest.mark.parametrize("spread", [1, 6])
def test_few_tokens_of_a_table(T, K, first, rows, spread):
    """Tokens spread out and on few rows (some by a warp, some by eight), zeros in all other rows."""
    g = torch.Generator(device="cuda").manual_seed(T + K)
    tokens = (first - 2 + (rows + 4) * torch.rand(T, generator=g, device="cuda") ** spread).int()
    dy = torch.randn(T, K, generator=g, **BF16)
    de, ok = guarded((rows, K), torch.bfloat16)
    lb.embedding_backward(tokens, dy, rows, first=first, multiplier=0.7, out=de)
    check(de, *embedding_grad_ref(tokens, dy, first, rows, 0.7), "de")
    assert ok()


@pytest.mark.parametrize("bits,gs", [(1, 128), (2, 64), (4, 64), (16, 0)])
@pytest.mark.parametrize("M,K,V", [(3, 128, 43000), (90, 256, 30001), (300, 128, 60000), (140, 384, 9001)])
def test_many_slices(bits, gs, M, K, V):
    """Few tiles of dX whose reduction over a long vocabulary is cut into many slices."""
    table = Table((V + 7) // 8 * 8, K, bits, gs)
    x, labels, grad = inputs(M, K, V)
    check_loss(table, x, labels, grad, V, loss_step(table, x, labels, grad, V))


@pytest.mark.parametrize("M,K,V", [(1, 128, 1000), (40, 264, 5000), (300, 512, 3003)])
def test_the_label_is_most_of_the_gradient(M, K, V):
    """Tokens that know nothing (all p near 1 / V): dX is the label's row and little else, and G's rounding to bf16 there
    does not show: |G| of the others is at most 2 / V of it, so dX is off by its own rounding and 2^-8 2 sum |w| / V."""
    table = Table(V, K, 16, norm=1.0)
    x, labels, grad = inputs(M, K, V)
    x = (x.float() / 64).bfloat16()
    loss, lse = lb.cross_entropy(x, labels, *table.args())
    dx, _ = lb.cross_entropy_backward(grad, x, labels, lse, *table.args())
    ref = Loss(x, labels, table, V)
    (rx, _), _ = ref.gradients(grad, lse)
    p = (ref.l - lse.double()[:, None]).exp()
    assert p.max() <= 2 / V
    f = torch.where(ref.valid, grad, 0.0).double().abs()[:, None]
    w = ref.w.abs()
    sums = f * (w.sum(0) / V * 2 + w[ref.label])
    e = HB16 * f * 2 / V * w.sum(0) + (V + 16) * H32 * sums + 2.0 ** -20 * f * w[ref.label]
    check(dx, rx, e + HB16 * (rx.abs() + e), "dx")


@pytest.mark.parametrize("M,K,V", [(1, 128, 1000), (3, 264, 5003), (65, 128, 999), (512, 136, 2000)])
def test_dw_of_few_tokens(M, K, V):
    """G enters dW as two bf16 values, so a row that one token makes up is off by its own rounding: p's error in fp32 (as
    Loss counts it), 2^-16 of G, fp32 sums of 2 M products, and one rounding."""
    table = Table(V, K, 16)
    x, labels, grad = inputs(M, K, V)
    lse = lb.cross_entropy(x, labels, *table.args())[1]
    _, dw = lb.cross_entropy_backward(grad, x, labels, lse, *table.args(), need_dw=True)
    ref = Loss(x, labels, table, V)
    l = lse.double()[:, None]
    p = (ref.l - l).exp()
    hot = torch.zeros_like(p)
    hot[torch.arange(M, device="cuda"), ref.label] = 1.0
    f = torch.where(ref.valid, grad, 0.0).double()[:, None]
    G = f * (p - hot)
    ep = p * torch.expm1(1.01 * (ref.el + 1.4427 * 3 * (ref.l.abs() + l.abs()) * H32) + 2.0 ** -21) + H32
    eG = 1.01 * f.abs() * ep + (2.0 ** -16 + 2 * H32) * G.abs()
    xs = torch.where(ref.valid[:, None], x.double(), 0.0)
    want = G.T @ xs
    e = eG.T @ xs.abs() + (2 * M + 16) * H32 * (G.abs().T @ xs.abs())
    check(dw, want, e + HB16 * (want.abs() + e), "dw")
