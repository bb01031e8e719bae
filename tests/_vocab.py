"""Seeded problems and 64-bit references for the vocabulary operators, with error bounds counted from the
roundings each of them makes."""
from __future__ import annotations

import torch

import bit_weight_only_w2_b200 as lb

H16 = 2.0 ** -11                             # half a step of fp16, relative
HB16 = torch.finfo(torch.bfloat16).eps / 2   # 2^-8: half a step of bf16
H32 = 2.0 ** -24
LOG2E = 1.4426950408889634


class Table:
    """Rows [N][K] of a vocabulary on the GPU: bf16 (bits 16), or codes, words and scales."""

    def __init__(self, N, K, bits, gs=0, seed=0, device="cuda", norm=2.0):
        g = torch.Generator(device=device)
        g.manual_seed(7919 * N + 31 * K + bits + 1000003 * seed)
        self.N, self.K, self.bits, self.gs = N, K, bits, gs
        self.scales = self.zeros = self.codes = None
        if bits == 16:
            self.weight = (torch.randn(N, K, generator=g, device=device) * (norm / K ** 0.5)).bfloat16()
            return
        lo, hi = {1: (0, 2), 2: (-1, 2), 4: (0, 16)}[bits]
        self.codes = torch.randint(lo, hi, (N, K), generator=g, device=device).to(torch.int8)
        if bits == 1:
            self.codes = self.codes * 2 - 1
        spread = {1: 1.0, 2: 0.8, 4: 4.7}[bits]
        self.scales = ((0.5 + torch.rand(K // gs, N, generator=g, device=device)) * (norm / spread / K ** 0.5)).half()
        self.zeros = (6 + 3 * torch.rand(K // gs, N, generator=g, device=device)).half() if bits == 4 else None
        self.weight = lb.pack(self.codes, bits)

    def args(self):
        return self.weight, self.scales, self.zeros, self.bits, self.gs

    def rows(self):
        """The rows in 64 bits."""
        if self.bits == 16:
            return self.weight.double()
        q = self.codes.double()
        if self.zeros is not None:
            q = q - self.zeros.double().T.repeat_interleave(self.gs, 1)
        return q * self.scales.double().T.repeat_interleave(self.gs, 1)


def inputs(M, K, V, seed=0, device="cuda", ignored=0.2):
    """(x, labels, grad): some labels outside the vocabulary, written as several values."""
    g = torch.Generator(device=device)
    g.manual_seed(104729 * M + 13 * K + V + 1000003 * seed)
    x = torch.randn(M, K, generator=g, device=device).bfloat16()
    labels = torch.randint(0, V, (M,), generator=g, device=device)
    if M > 1:
        u = torch.rand(M, generator=g, device=device)
        labels = torch.where(u < ignored / 3, -100, torch.where(u < 2 * ignored / 3, V, torch.where(u < ignored, -2 ** 31, labels)))
    grad = torch.randn(M, generator=g, device=device)
    return x, labels.to(torch.int32), grad


class Loss:
    """The cross entropy of x over the first V rows of a table in 64 bits, and how far off fp32 sums may be."""

    def __init__(self, x, labels, table, V):
        self.x, self.table, self.V = x.double(), table, V
        self.w = table.rows()[:V]
        self.valid = (labels >= 0) & (labels < V)
        self.label = torch.where(self.valid, labels, 0).long()
        self.l = self.x @ self.w.T
        K = x.shape[1]
        s = self.x.abs() @ self.w.abs().T
        self.el = K * H32 * s           # fp32 sums of K products
        if table.bits != 16:            # X's fp16 copy: 2^-25 of fp16 on rows scaled to 2^15 .. 2^16
            self.el = self.el + (2.0 ** -40 * self.x.abs().amax(1))[:, None] * self.w.abs().sum(1)[None, :]
        if table.bits == 4:
            # weights as two fp16 values, the second rounded: it is at most 2^-11 of the first and 2^-7 (2^-6 for
            # |z| > 8) of s, so 2^-11 of that, and 2^-25 of its smallest step
            step = table.scales.double()[:, :V].T.repeat_interleave(table.gs, 1)
            self.el = self.el + 2.0 ** -22 * s + 2.0 ** -17 * (self.x.abs() @ step.T) + 2.0 ** -25 * self.x.abs().sum(1)[:, None]
            if len(x) <= 16:
                # few tokens: sums of x (q - 8), less (z - 8) times a sum of x, both times s
                q = (table.codes.double()[:V] - 8).abs() + (table.zeros.double()[:, :V].T - 8).abs().repeat_interleave(table.gs, 1)
                self.el = self.el + K * H32 * (self.x.abs() @ (q * step).T)
        self.lse = torch.logsumexp(self.l, 1)
        self.target = self.l.gather(1, self.label[:, None])[:, 0]
        self.loss = torch.where(self.valid, self.lse - self.target, 0.0)
        # the exponentials: 2^x to 2^-22, its argument in fp32 twice (tile, and joining tiles), then sums of 64 terms
        # a thread, a tile's and its joins
        top = self.l.abs().amax(1)
        args = 2 * LOG2E * 3 * top * H32
        sums = (80 + 2 * V / 128 / 32 + 40) * H32 + 3 * 2.0 ** -22
        self.e_lse = self.el.amax(1) + args + sums + 4 * H32 * (self.lse.abs() + top)
        self.e_loss = torch.where(self.valid, self.e_lse + self.el.gather(1, self.label[:, None])[:, 0] +
                                  2 * H32 * (self.loss.abs() + self.lse.abs()), 0.0)

    def gradients(self, grad, lse):
        """((dx, bound), (dw, bound)) for the lse that the call was given."""
        lse = lse.double()
        M, V = self.l.shape
        p = (self.l - lse[:, None]).exp()
        f = torch.where(self.valid, grad, 0.0).double()[:, None]
        hot = torch.zeros_like(p)
        hot[torch.arange(M, device=p.device), self.label] = 1.0
        G = f * (p - hot)
        # p: the logit's error, the argument's and 2^x's; p - 1 in fp32; then one rounding of G
        arg = LOG2E * 3 * (self.l.abs() + lse.abs()[:, None]) * H32
        ep = p * torch.expm1(1.01 * (self.el + arg) + 2.0 ** -21) + H32
        dense = self.table.bits == 16
        half = HB16 if dense else H16
        eG = f.abs() * ep * (1 + half) + (half + 2 * H32) * G.abs() + f.abs() * (0 if dense else 2.0 ** -40)
        w = self.w
        dx = G @ w
        ex = eG @ w.abs() + (V + 16) * H32 * (G.abs() @ w.abs())
        if self.table.bits == 4:   # q - z and its product with s, each rounded to fp16
            ex = ex + (2 * H16 + H16 * H16) * (G.abs() @ w.abs()) + 2.0 ** -25 * G.abs().sum(1)[:, None]
        ex = ex + HB16 * (dx.abs() + ex)
        x = torch.where(self.valid[:, None], self.x, 0.0)
        dw = G.T @ x
        ew = eG.T @ x.abs() + (M + 16) * H32 * (G.abs().T @ x.abs())
        ew = ew + HB16 * (dw.abs() + ew)
        return (dx, ex), (dw, ew)


def embedding_ref(tokens, table, multiplier):
    """(y, bound): a value, its products with scale and multiplier in fp32, and one rounding to bf16."""
    w = table.rows()
    t = tokens.long()
    has = (t >= 0) & (t < table.N)
    y = torch.where(has[:, None], w[torch.where(has, t, 0)], 0.0) * multiplier
    return y, (HB16 + 4 * H32) * y.abs()


def embedding_grad_ref(tokens, dy, first, rows, multiplier):
    """(sums, bound): n - 1 additions in fp32, the multiplier's product, and one rounding to bf16."""
    at = tokens.long() - first
    at = torch.where((at >= 0) & (at < rows), at, rows)
    out = torch.zeros(rows + 1, dy.shape[1], dtype=torch.float64, device=dy.device)
    mag, n = out.clone(), torch.zeros(rows + 1, 1, dtype=torch.float64, device=dy.device)
    out.index_add_(0, at, dy.double())
    mag.index_add_(0, at, dy.double().abs())
    n.index_add_(0, at, torch.ones(len(at), 1, dtype=torch.float64, device=dy.device))
    m = abs(multiplier)
    e = (n[:-1] + 1) * H32 * mag[:-1] * m
    y = out[:-1] * multiplier
    return y, e + HB16 * (y.abs() + e)
