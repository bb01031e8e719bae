"""Operators around a frozen low-bit linear, as cases to measure: adapters of many requests beside
the packed projection, the gradients of both, and the 8-bit copy of the input they are formed from.

    forward   y = x W^T + scaling_a (x A_a^T) B_a^T     a = the adapter of each token (or none)
    dx        dx = dy W                                 the frozen linear's input gradient
    backward  dx = dy W + dp A_a,  dp = scaling_a dy B_a,  dA_a = sum dp^T x,  dB_a = sum dy^T p
    store     x -> 8-bit codes and one power-of-two exponent per 32 values
    load      the values those stand for, in bf16

W[N][K] is decoded from packed codes (binary, ternary or uint4 words and fp16 group scales). `run`
computes each in plain torch operations in 32 bits, or, with `own` set, through this package.
"""
import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one request's token in a small projection: nothing but latency
        dict(name="forward_one_token", op="forward", M=1, K=2560, N=2560, bits=4, group=64, adapters=8, rank=16,
             requests=1, save=False),
        # a decode step of 16 requests, each with an adapter of its own, on the text encoder's up projection
        dict(name="forward_16_requests", op="forward", M=16, K=2560, N=9728, bits=4, group=64, adapters=32, rank=16,
             requests=16, save=False),
        # a larger decode batch: 203 tokens, 64 adapters in no order, some tokens with none
        dict(name="forward_203_requests", op="forward", M=203, K=4096, N=4096, bits=2, group=128, adapters=64,
             rank=32, requests=203, save=False),
        # a training step's forward over the tokens of several images and prompts, one adapter per
        # concept, ragged; keeps p and the 8-bit copy of x for the backward
        dict(name="forward_train", op="forward", M=4173, K=9216, N=9216, bits=2, group=128, adapters=3, rank=64,
             requests=7, save=True),
        # the input gradient of a linear without adapters: a padded prompt, and an image
        dict(name="dx_512", op="dx", M=512, K=2560, N=9728, bits=4, group=64),
        dict(name="dx_image", op="dx", M=4608, K=9216, N=9216, bits=1, group=128),
        # fine-tuning one small adapter on one prompt, x kept in bf16
        dict(name="backward_prompt", op="backward", M=77, K=2560, N=2560, bits=4, group=64, adapters=1, rank=8,
             requests=1, save=False),
        # several adapters trained at once on ragged prompts
        dict(name="backward_ragged", op="backward", M=1537, K=2560, N=9728, bits=2, group=64, adapters=5, rank=32,
             requests=11, save=True),
        # the backward that belongs to forward_train, from the 8-bit copy
        dict(name="backward_train", op="backward", M=4173, K=9216, N=9216, bits=2, group=128, adapters=3, rank=64,
             requests=7, save=True),
        # the 8-bit copy by itself: one prompt, and an image's widest activations, stored and read back
        dict(name="store_prompt", op="store", M=77, K=2560),
        dict(name="store_image", op="store", M=4608, K=12288),
        dict(name="load_image", op="load", M=4608, K=12288),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["forward", "forward", "forward", "dx", "backward", "backward", "store", "load"])
    K = 128 * _log(rng, 2, 72)
    if op in ("store", "load"):
        return dict(op=op, M=_log(rng, 1, 4608), K=K)
    bits = rng.choice([1, 2, 4])
    case = dict(op=op, M=_log(rng, 1, 4173) if op == "forward" else _log(rng, 33, 4173), K=K, N=8 * _log(rng, 32, 1152),
                bits=bits, group=rng.choice([64, 128]))
    if op == "dx":
        return case
    M = case["M"]
    adapters = _log(rng, 1, 64)
    # one token per request (a decode batch), or requests of many tokens
    requests = M if M <= 512 and op == "forward" and rng.random() < 0.6 else min(M, _log(rng, 1, 24))
    case.update(adapters=adapters, rank=rng.choice([8, 16, 24, 32, 48, 64] if adapters > 8 else [8, 16, 24, 32, 64, 128]),
                requests=1 if adapters == 1 else requests, save=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _activations(g, M, K):
    """Normal values with a few channels an order of magnitude larger, as transformer inputs have."""
    x = torch.randn(M, K, generator=g, device=DEV)
    wide = 1.0 + 15.0 * (torch.rand(K, generator=g, device=DEV) < 0.01).float()
    return (x * wide).to(torch.bfloat16)


def _index(case, seed):
    """The adapter of each token: requests of consecutive tokens, about one in ten without an adapter."""
    r = np.random.RandomState(seed % (1 << 31))
    M, n = case["M"], case["requests"]
    cuts = np.sort(r.choice(np.arange(1, M), n - 1, replace=False)) if n > 1 else np.zeros(0, np.int64)
    owner = np.searchsorted(cuts, np.arange(M), side="right")
    of = r.randint(0, case["adapters"], n)
    if n > 1:
        of[r.rand(n) < 0.1] = -1
    return torch.from_numpy(of[owner].astype(np.int32)).to(DEV)


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    M, K = case["M"], case["K"]
    s = {"x": _activations(g, M, K)}
    if case["op"] in ("store", "load"):
        return s
    N, bits, G = case["N"], case["bits"], K // case["group"]
    if bits == 1:
        codes = torch.randint(0, 2, (N, K), generator=g, device=DEV, dtype=torch.int8) * 2 - 1
    elif bits == 2:
        u = torch.rand(N, K, generator=g, device=DEV)
        codes = (u >= 0.7).to(torch.int8) - (u < 0.3).to(torch.int8)
    else:
        codes = torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=torch.int8)
    s["codes"] = codes
    s["scales"] = (0.005 + 0.015 * torch.rand(G, N, generator=g, device=DEV)).half()
    s["zeros"] = (6.0 + 3.0 * torch.rand(G, N, generator=g, device=DEV)).half() if bits == 4 else None
    s["dy"] = (torch.randn(M, N, generator=g, device=DEV) * 0.05).to(torch.bfloat16)
    if case["op"] == "dx":
        return s
    L, R = case["adapters"], case["rank"]
    s["a"] = (torch.randn(L, R, K, generator=g, device=DEV) / K ** 0.5).to(torch.bfloat16)
    s["b"] = (torch.randn(L, N, R, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    s["scaling"] = 0.5 + torch.rand(L, generator=g, device=DEV)
    s["index"] = _index(case, seed) if L > 1 else None
    s["p"] = torch.randn(M, R, generator=g, device=DEV).to(torch.bfloat16)
    if s["index"] is not None:
        s["p"][s["index"] < 0] = 0
    return s


def _word_columns(W, bits):
    """Column held by offset i of word j of a row of W words: blocks of four words interleave
    column pairs (2- and 4-bit rows), the remaining words hold consecutive columns."""
    cpw = 32 // bits
    j = torch.arange(W, device=DEV)[:, None]
    i = torch.arange(cpw, device=DEV)[None, :]
    block = (j < W // 4 * 4) if bits != 1 else torch.zeros_like(j, dtype=torch.bool)
    inner = 4 * cpw * (j // 4) + 8 * (i // 2) + 2 * (j % 4) + i % 2
    return torch.where(block, inner, j * cpw + i)


def _positions(bits):
    i = torch.arange(32 // bits, device=DEV)
    return (i % 2) * 16 + (i // 2) * bits


def _pack(fields, bits):
    """Fields [rows][columns] -> words [rows][columns * bits / 32] (int32)."""
    cols = _word_columns(fields.shape[1] * bits // 32, bits)
    words = fields[:, cols.reshape(-1)].reshape(fields.shape[0], *cols.shape)
    total = (words.to(torch.int64) << _positions(bits)).sum(-1)
    return torch.where(total >= 1 << 31, total - (1 << 32), total).to(torch.int32)


def _fields(codes, bits):
    return (codes > 0).to(torch.uint8) if bits == 1 else (codes + 1).to(torch.uint8) if bits == 2 else codes.to(torch.uint8)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    if case["op"] == "load" or (case["op"] == "backward" and case["save"]):
        s["kept"] = _store(s["x"])
    if "codes" in s:
        fields = _fields(s.pop("codes"), case["bits"])
        if case["op"] == "forward":
            s["packed"] = _pack(fields, case["bits"])
            del s["dy"], s["p"]
        else:   # the words of W^T, whose rows are filled up to a multiple of 128 columns with zero fields
            wide = torch.zeros(case["K"], -(-case["N"] // 128) * 128, dtype=torch.uint8, device=DEV)
            wide[:, :case["N"]] = fields.T
            s["packed_t"] = _pack(wide, case["bits"])
    return s


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------
def _codes(words, bits):
    """Words [rows][W] -> the code values, fp32 [rows][W * 32 / bits]."""
    cols = _word_columns(words.shape[1], bits).reshape(-1)
    fields = ((words[:, :, None] >> _positions(bits).to(torch.int32)) & ((1 << bits) - 1)).reshape(words.shape[0], -1)
    out = torch.empty(fields.shape, dtype=torch.float32, device=words.device)
    out[:, cols] = fields.float()
    return out * 2 - 1 if bits == 1 else out - 1 if bits == 2 else out


def _weights(s):
    """W [N][K] in fp32, from whichever words the state holds."""
    case = s["case"]
    q = _codes(s["packed"], case["bits"]) if "packed" in s else _codes(s["packed_t"], case["bits"])[:, :case["N"]].T
    scale = s["scales"].float().T.repeat_interleave(case["group"], 1)
    if s["zeros"] is not None:
        q = q - s["zeros"].float().T.repeat_interleave(case["group"], 1)
    return q * scale


def _chosen(s, M):
    """[M][L] of 0 / 1: the adapter of each token."""
    L = s["a"].shape[0]
    index = s["index"] if s["index"] is not None else torch.zeros(M, dtype=torch.int32, device=DEV)
    return index[:, None] == torch.arange(L, device=DEV)[None, :]


def _store(x):
    """The 8-bit form of x: e4m3 values of x / 2^e, e the smallest exponent that brings the largest
    finite value of each 32 to at most 448 (kept as e + 127; 0 for a block of zeros)."""
    M, K = x.shape
    v = x.float().reshape(M, K // 32, 32)
    finite = torch.isfinite(v)
    largest = torch.where(finite, v.abs(), 0.0).amax(-1)
    mant, exp = torch.frexp(largest)                      # largest = mant * 2^exp, mant in [0.5, 1)
    e = exp - 9 + (mant > 0.875).int()
    kept = torch.where(largest > 0, (e + 127).clamp(0, 254), 0)
    half = ((127 - kept) // 2)[:, :, None]
    rest = (127 - kept)[:, :, None] - half
    scaled = torch.where(finite, torch.ldexp(torch.ldexp(v, half), rest), float("nan"))
    return scaled.reshape(M, K).to(torch.float8_e4m3fn), kept.to(torch.uint8)


def _load(codes, exps):
    M, K = codes.shape
    e = exps.int()[:, :, None] - 127
    v = codes.float().reshape(M, K // 32, 32)
    return torch.ldexp(torch.ldexp(v, e // 2), e - e // 2).reshape(M, K)


def _forward(s):
    x = s["x"].float()
    L, R, K = s["a"].shape
    p = (x @ s["a"].float().reshape(L * R, K).T).reshape(-1, L, R) * s["scaling"][:, None]
    p = torch.where(_chosen(s, x.shape[0])[:, :, None], p, 0.0)
    y = x @ _weights(s).T + p.reshape(-1, L * R) @ s["b"].float().permute(0, 2, 1).reshape(L * R, -1)
    if not s["case"]["save"]:
        return {"y": y.to(torch.bfloat16)}
    codes, exps = _store(s["x"])
    return {"y": y.to(torch.bfloat16), "p": p.sum(1).to(torch.bfloat16), "codes": codes, "exps": exps}


def _backward(s):
    dy = s["dy"].float()
    x = _load(*s["kept"]) if s["case"]["save"] else s["x"].float()
    L, R, K = s["a"].shape
    N = dy.shape[1]
    sel = _chosen(s, dy.shape[0])[:, :, None]
    dp = (dy @ s["b"].float().permute(1, 0, 2).reshape(N, L * R)).reshape(-1, L, R) * s["scaling"][:, None]
    dp = torch.where(sel, dp, 0.0).reshape(-1, L * R)
    p = torch.where(sel, s["p"].float()[:, None, :], 0.0).reshape(-1, L * R)
    dx = dy @ _weights(s) + dp @ s["a"].float().reshape(L * R, K)
    da = (dp.T @ x).reshape(L, R, K)
    db = (dy.T @ p).reshape(N, L, R).permute(1, 0, 2)
    return {"dx": dx.to(torch.bfloat16), "da": da.to(torch.bfloat16), "db": db.to(torch.bfloat16).contiguous()}


def _plain(s):
    op = s["case"]["op"]
    if op == "forward":
        return _forward(s)
    if op == "backward":
        return _backward(s)
    if op == "dx":
        return {"dx": (s["dy"].float() @ _weights(s)).to(torch.bfloat16)}
    if op == "store":
        codes, exps = _store(s["x"])
        return {"codes": codes, "exps": exps}
    return {"x": _load(*s["kept"]).to(torch.bfloat16)}


# ---------------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------------
def _own(s):
    import bit_weight_only_w2_b200 as lb

    case = s["case"]
    op = case["op"]
    if op == "store":
        kept = lb.checkpoint_store(s["x"])
        return {"codes": kept.codes, "exps": kept.exps}
    if op == "load":
        return {"x": lb.checkpoint_load(lb.Checkpoint(*s["kept"]))}
    bits, group = case["bits"], case["group"]
    if op == "dx":
        return {"dx": lb.gemm_dx(s["dy"], s["packed_t"], s["scales"], s["zeros"], bits, group)}
    if op == "backward":
        x = lb.Checkpoint(*s["kept"]) if case["save"] else s["x"]
        dx, da, db = lb.adapter_backward(s["dy"], x, s["p"], s["packed_t"], s["scales"], s["zeros"], bits, group,
                                         s["a"], s["b"], s["scaling"], s["index"])
        return {"dx": dx, "da": da, "db": db}
    if not case["save"]:
        return {"y": lb.adapter_gemm(s["x"], s["packed"], s["scales"], s["zeros"], bits, group, s["a"], s["b"],
                                     s["scaling"], s["index"])}
    p = torch.empty(case["M"], case["rank"], dtype=torch.bfloat16, device=DEV)
    kept = lb.checkpoint_empty(case["M"], case["K"], DEV)
    y = lb.adapter_gemm(s["x"], s["packed"], s["scales"], s["zeros"], bits, group, s["a"], s["b"], s["scaling"],
                        s["index"], p=p, checkpoint=kept)
    return {"y": y, "p": p, "codes": kept.codes, "exps": kept.exps}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    M, K = case["M"], case["K"]
    eight = M * K + M * K // 32
    if case["op"] in ("store", "load"):
        return {"bytes": M * K * 2 + eight, "flops": M * K}
    N, bits = case["N"], case["bits"]
    nbytes = N * K * bits // 8 + K // case["group"] * N * (4 if bits == 4 else 2) + M * (K + N) * 2
    flops = 2 * M * N * K
    if case["op"] == "dx":
        return {"bytes": nbytes, "flops": flops}
    L, R = case["adapters"], case["rank"]
    used = min(L, case["requests"])
    if case["op"] == "forward":
        nbytes += used * R * (K + N) * 2 + M * 4 + (M * R * 2 + eight if case["save"] else 0)
        flops += 2 * M * R * (K + N)
    else:   # also x (in 8 bits or bf16) and p, and every adapter's gradient
        nbytes += (used + L) * R * (K + N) * 2 + M * 4 + M * R * 2 + (eight if case["save"] else M * K * 2)
        flops += 2 * 2 * M * R * (K + N)
    return {"bytes": nbytes, "flops": flops}


def _exact_load(s):
    codes, exps = s["kept"]
    return codes.double() * torch.exp2(exps.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    x = s["x"].double()
    if op in ("store", "load"):
        kept = _store(s["x"])
        if op == "load":
            return {"x": _exact_load({"kept": kept})}
        return {"codes": x * torch.exp2(127 - kept[1].double()).repeat_interleave(32, 1), "exps": None}
    w = s["codes"].double()
    scale = s["scales"].double()
    for g in range(scale.shape[0]):   # one group of columns at a time
        cols = slice(g * case["group"], (g + 1) * case["group"])
        if s["zeros"] is not None:
            w[:, cols] -= s["zeros"][g].double()[:, None]
        w[:, cols] *= scale[g][:, None]
    dy = s["dy"].double()
    if op == "dx":
        return {"dx": dy @ w}
    L, R, K = s["a"].shape
    index = s["index"] if s["index"] is not None else torch.zeros(case["M"], dtype=torch.int32, device=DEV)
    a, b = s["a"].double(), s["b"].double()
    if op == "forward":
        y, p = x @ w.T, torch.zeros(case["M"], R, dtype=torch.float64, device=DEV)
        for l in range(L):
            rows = (index == l).nonzero().flatten()
            p[rows] = x[rows] @ a[l].T * s["scaling"][l].double()
            y[rows] += p[rows] @ b[l].T
        if not case["save"]:
            return {"y": y}
        kept = _store(s["x"])
        return {"y": y, "p": p, "codes": x * torch.exp2(127 - kept[1].double()).repeat_interleave(32, 1), "exps": None}
    if case["save"]:
        x = _exact_load({"kept": _store(s["x"])})
    dx, da, db = dy @ w, torch.zeros_like(a), torch.zeros_like(b)
    for l in range(L):
        rows = (index == l).nonzero().flatten()
        dp = dy[rows] @ b[l] * s["scaling"][l].double()
        dx[rows] += dp @ a[l]
        da[l] = dp.T @ x[rows]
        db[l] = dy[rows].T @ s["p"][rows].double()
    return {"dx": dx, "da": da, "db": db}
