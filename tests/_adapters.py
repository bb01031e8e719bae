"""Seeded problems and 64-bit references for the adapter, gradient and 8-bit copy tests, with
error bounds counted from the roundings each operator makes."""
from __future__ import annotations

import torch

import bit_weight_only_w2_b200 as lb

H16 = 2.0 ** -11    # half a step of fp16, relative
HB16 = torch.finfo(torch.bfloat16).eps / 2   # 2^-8: half a step of bf16
H32 = 2.0 ** -24


class Problem:
    """Inputs on the GPU: codes, packed words both ways, scales (and zeros), x, dy, adapters, p."""

    def __init__(self, M, K, N, bits, gs, L, R, index="random", seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(1000003 * seed + 7919 * M + 31 * K + N + bits)
        rnd = lambda *s: torch.randn(*s, generator=g, device=device)
        uni = lambda *s: torch.rand(*s, generator=g, device=device)
        self.M, self.K, self.N, self.bits, self.gs, self.L, self.R = M, K, N, bits, gs, L, R
        if bits == 1:
            self.codes = (torch.randint(0, 2, (N, K), generator=g, device=device) * 2 - 1).to(torch.int8)
        elif bits == 2:
            self.codes = torch.randint(-1, 2, (N, K), generator=g, device=device).to(torch.int8)
        else:
            self.codes = torch.randint(0, 16, (N, K), generator=g, device=device).to(torch.int8)
        self.scales = (0.005 + 0.015 * uni(K // gs, N)).half()
        self.zeros = (6 + 3 * uni(K // gs, N)).half() if bits == 4 else None
        self.packed = lb.pack(self.codes, bits)
        self.packed_t = lb.transpose_packed(self.packed, K, bits)
        self.x = rnd(M, K).bfloat16()
        self.dy = (0.05 * rnd(M, N)).bfloat16()
        self.a = (rnd(L, R, K) / K ** 0.5).bfloat16()
        self.b = (0.1 * rnd(L, N, R)).bfloat16()
        self.scaling = 0.5 + uni(L)
        if index is None:
            self.index = None
        else:
            v = torch.randint(0, L, (M,), generator=g, device=device)
            if index == "sorted":
                v = v.sort().values
            elif index == "none":
                v = torch.full_like(v, -1)
            elif index == "holes":     # some tokens without one, written as several out-of-range values
                hole = torch.randint(0, 5, (M,), generator=g, device=device)
                v = torch.where(hole == 0, -1, torch.where(hole == 1, L, torch.where(hole == 2, -2 ** 31, v)))
            elif index == "last":      # every token on the last adapter
                v = torch.full_like(v, L - 1)
            self.index = v.to(torch.int32)
        self.p = torch.where(self.rows()[:, None] >= 0, rnd(M, R), 0.0).bfloat16()

    def rows(self):
        """The adapter of each token, -1 for none."""
        if self.index is None:
            return torch.zeros(self.M, dtype=torch.int64, device=self.x.device)
        v = self.index.long()
        return torch.where((v >= 0) & (v < self.L), v, -1)

    def weights(self):
        s = self.scales.double().T.repeat_interleave(self.gs, 1)
        q = self.codes.double()
        if self.zeros is not None:
            q = q - self.zeros.double().T.repeat_interleave(self.gs, 1)
        return q * s

    def adapter_args(self):
        return self.a, self.b, self.scaling, self.index

    def args(self):
        return self.scales, self.zeros, self.bits, self.gs


def forward_ref(pr):
    """(y, y's bound, p, p's bound) in 64 bits. p is a K-long fp32 sum rounded to bf16; y adds its R
    products and the K of the packed weights in fp32 and rounds once; uint4 weights are fp16."""
    x, w = pr.x.double(), pr.weights()
    y, s = x @ w.T, x.abs() @ w.abs().T
    e = (pr.K * H32 + (H16 if pr.bits == 4 else 0)) * s
    p = torch.zeros(pr.M, pr.R, dtype=torch.float64, device=x.device)
    pe = torch.zeros_like(p)
    rows = pr.rows()
    for l in range(pr.L):
        m = (rows == l).nonzero().flatten()
        if not len(m):
            continue
        a, b, sc = pr.a[l].double(), pr.b[l].double(), float(pr.scaling[l])
        p[m] = sc * (x[m] @ a.T)
        f = (pr.K + 2) * H32 * sc * (x[m].abs() @ a.abs().T)
        pe[m] = f + HB16 * (p[m].abs() + f)
        y[m] += p[m] @ b.T
        e[m] += pe[m] @ b.abs().T + (pr.K + pr.R) * H32 * (p[m].abs() @ b.abs().T)
    return y, e + HB16 * (y.abs() + e), p, pe


def backward_ref(pr, x):
    """[(value, bound)] of dx, da, db in 64 bits for the input `x` (what the backward was given)."""
    dy, w, x = pr.dy.double(), pr.weights(), x.double()
    dx, s = dy @ w, dy.abs() @ w.abs()
    e = (pr.N * H32 + (2 * H16 + H16 * H16 if pr.bits == 4 else 0)) * s
    da, db = torch.zeros_like(pr.a, dtype=torch.float64), torch.zeros_like(pr.b, dtype=torch.float64)
    ea, eb = torch.zeros_like(da), torch.zeros_like(db)
    rows = pr.rows()
    for l in range(pr.L):
        m = (rows == l).nonzero().flatten()
        if not len(m):
            continue
        a, b, sc = pr.a[l].double(), pr.b[l].double(), float(pr.scaling[l])
        dp = sc * (dy[m] @ b)
        f = (pr.N + 2) * H32 * sc * (dy[m].abs() @ b.abs())
        pe = f + HB16 * (dp.abs() + f)
        dx[m] += dp @ a
        e[m] += pe @ a.abs() + (pr.N + pr.R) * H32 * (dp.abs() @ a.abs())
        n = len(m)
        da[l] = dp.T @ x[m]
        fa = pe.T @ x[m].abs() + n * H32 * (dp.abs().T @ x[m].abs())
        ea[l] = fa + HB16 * (da[l].abs() + fa)
        p = pr.p[m].double()
        db[l] = dy[m].T @ p
        fb = n * H32 * (dy[m].abs().T @ p.abs())
        eb[l] = fb + HB16 * (db[l].abs() + fb)
    return (dx, e + HB16 * (dx.abs() + e)), (da, ea), (db, eb)


def check(got, ref, bound, what):
    # 2^-126: a value below fp32's normal range
    off = (got.double() - ref).abs()
    bad = ~(off <= bound + 2.0 ** -126)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        worst = (off / (bound + 2.0 ** -126)).max().item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound (worst {worst:.3g}), first at "
                             f"{at}: got {got[tuple(at)].item()}, want {ref[tuple(at)].item()}")


def checkpoint_ref(x):
    """(codes as fp64 values, exponent bytes, loaded values) from the definition, in 64 bits on the CPU."""
    v = x.double().cpu().reshape(x.shape[0], -1, 32)
    finite = torch.isfinite(v)
    top = torch.where(finite, v.abs(), 0.0).amax(-1)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0)), torch.tensor(-127.0))
    e = torch.where((top > 0) & (top > 448.0 * torch.exp2(e)), e + 1, e)          # log2 rounded down
    e = torch.where((top > 0) & (top <= 448.0 * torch.exp2(e - 1)), e - 1, e).clamp_min(-127)
    scaled = v / torch.exp2(e)[:, :, None]
    mag = scaled.abs().clamp_min(2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(mag)) - 3)                            # e4m3: 3 mantissa bits
    codes = torch.round(scaled / step) * step                                      # torch.round: half to even
    codes = torch.where(finite, codes, float("nan"))
    return codes.reshape(x.shape), (e + 127).to(torch.uint8), (codes * torch.exp2(e)[:, :, None]).reshape(x.shape)
