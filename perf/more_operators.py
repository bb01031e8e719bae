"""The two ends of a model around low-bit linears, as cases to measure: the lookup of token embeddings
and its gradient, and the softmax cross entropy over the vocabulary and its gradient.

    embed        y_t = multiplier E[token_t]                       (tokens outside the table: zeros)
    embed_grad   dE_v = multiplier * the sum of dy_t over token_t = v
    loss         l = x W^T,  lse_m = log sum_v exp l_mv,  loss_m = lse_m - l_m[label_m]
    loss_grad    G_mv = g_m (exp(l_mv - lse_m) - [v = label_m]),  dx = G W,  dW = G^T x

Rows whose label is outside the vocabulary have no loss and no gradient. A table (E or W, [rows][K]) is
bf16 (`bits` 16), or packed binary, ternary or uint4 words with fp16 group scales (and zeros); rows behind
the vocabulary, which fill a packed table up to a multiple of eight, take no part. `run` computes each in
plain torch operations in 32 bits, or, with `own` set, through this package.
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
        # scoring one token, a small vocabulary, the table in 4 bits: the words are read once
        dict(name="loss_one_token", op="loss", M=1, K=2560, V=32768, bits=4, group=64),
        # a decode batch scored against a large bf16 head: the head is read once
        dict(name="loss_16_tokens", op="loss", M=16, K=2560, V=131072, bits=16, group=0),
        # one long prompt, an odd vocabulary, the head in 4 bits
        dict(name="loss_prompt", op="loss", M=509, K=2560, V=100003, bits=4, group=64),
        # a training step's tokens over the largest head
        dict(name="loss_train", op="loss", M=4096, K=2560, V=131072, bits=16, group=0),
        # fine-tuning adapters under a frozen head on one padded prompt
        dict(name="loss_grad_prompt", op="loss_grad", M=77, K=2560, V=32768, bits=4, group=64, dw=False),
        # several ragged prompts at once, a frozen ternary head
        dict(name="loss_grad_ragged", op="loss_grad", M=1537, K=4096, V=50009, bits=2, group=128, dw=False),
        # the backward that belongs to loss_train, the head trained too
        dict(name="loss_grad_train", op="loss_grad", M=4096, K=2560, V=131072, bits=16, group=0, dw=True),
        # one token of a decode step from a packed table: nothing but latency
        dict(name="embed_one_token", op="embed", T=1, K=2560, V=131072, bits=4, group=64, multiplier=1.0),
        # a batch of long prompts from a bf16 table, scaled by sqrt(K)
        dict(name="embed_prompts", op="embed", T=32749, K=4096, V=131072, bits=16, group=0, multiplier=64.0),
        # the same from a packed ternary table
        dict(name="embed_prompts_packed", op="embed", T=16384, K=2560, V=65536, bits=2, group=128, multiplier=1.0),
        # training a few added concept tokens on ragged prompts
        dict(name="embed_grad_concepts", op="embed_grad", T=1537, K=2560, V=131072, first=131048, rows=24, share=0.1,
             multiplier=1.0),
        # training the whole table on a batch of long prompts
        dict(name="embed_grad_table", op="embed_grad", T=32768, K=2560, V=131072, first=0, rows=131072, share=1.0,
             multiplier=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["loss", "loss", "loss_grad", "loss_grad", "embed", "embed_grad"])
    bits = rng.choice([1, 2, 4, 16, 16])
    K = 8 * _log(rng, 16, 512) if bits == 16 else 128 * _log(rng, 1, 32)
    group = 0 if bits == 16 else rng.choice([64, 128])
    V = _log(rng, 500, 131072)
    if op == "embed":
        return dict(op=op, T=_log(rng, 1, 32749), K=K, V=V, bits=bits, group=group, multiplier=rng.choice([1.0, K ** 0.5]))
    if op == "embed_grad":
        if rng.random() < 0.5:
            first, rows, share = 0, V, 1.0
        else:
            rows = _log(rng, 1, V // 2)
            first, share = V - rows, rng.random()
        K = 8 * _log(rng, 16, 320)
        return dict(op=op, T=_log(rng, 1, 32768), K=K, V=V, first=first, rows=rows, share=share,
                    multiplier=rng.choice([1.0, K ** 0.5]))
    M = min(_log(rng, 1, 4096), 4096 * 2560 * 131072 // (V * K))
    case = dict(op=op, M=M, K=K, V=V, bits=bits, group=group)
    if op == "loss_grad":
        case["dw"] = bits == 16 and rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _table(case, g):
    """A table of V rows: bf16, or random codes in packed words (rows filled up to a multiple of eight)."""
    V, K, bits = case["V"], case["K"], case["bits"]
    if bits == 16:
        return {"weight": (torch.randn(V, K, generator=g, device=DEV) * (2.2 / K ** 0.5)).to(torch.bfloat16),
                "scales": None, "zeros": None}
    N = (V + 7) // 8 * 8
    words = torch.randint(-2 ** 31, 2 ** 31, (N, K * bits // 32), generator=g, device=DEV, dtype=torch.int32)
    if bits == 2:   # fields of 0, 1, 2: a 3 becomes a 1 (the code 0)
        words = words & ~((words & (words >> 1) & 0x55555555) << 1)
    # scales that give the rows a norm of about two, as a head's logits have on normalised inputs
    spread = {1: 1.0, 2: 0.5 ** 0.5, 4: 4.7}[bits]
    groups = K // case["group"]
    scales = ((0.5 + torch.rand(groups, N, generator=g, device=DEV)) * (2.2 / (spread * K ** 0.5))).half()
    zeros = (6.0 + 3.0 * torch.rand(groups, N, generator=g, device=DEV)).half() if bits == 4 else None
    return {"weight": words, "scales": scales, "zeros": zeros}


def _tokens(case, g, n, V):
    """Token ids, the lower the more frequent (log-uniform, as words are)."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    return (torch.exp(u * float(np.log(V + 1.0))) - 1.0).long().clamp_(0, V - 1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": dict(case)}
    K, V = case["K"], case["V"]
    if case["op"] == "embed_grad":
        T = case["T"]
        tokens = _tokens(case, g, T, max(1, case["first"]) if case["first"] else V)
        if case["first"]:
            chosen = torch.rand(T, generator=g, device=DEV) < case["share"]
            inside = torch.randint(case["first"], case["first"] + case["rows"], (T,), generator=g, device=DEV,
                                   dtype=torch.int32)
            tokens = torch.where(chosen, inside, tokens)
        s["tokens"] = tokens
        s["dy"] = (torch.randn(T, K, generator=g, device=DEV) * 0.05).to(torch.bfloat16)
        return s
    s.update(_table(case, g))
    if case["op"] == "embed":
        s["tokens"] = _tokens(case, g, case["T"], V)
        return s
    M = case["M"]
    s["labels"] = _tokens(case, g, M, V)
    # normalised inputs that lean to their label's row, some more than others
    lean = 3.0 * torch.rand(M, 1, generator=g, device=DEV)
    x = torch.randn(M, K, generator=g, device=DEV) + lean * _rows(s, s["labels"].long())
    s["x"] = x.to(torch.bfloat16)
    if M > 1:   # about one token in ten belongs to a prompt that is not trained on
        s["labels"] = torch.where(torch.rand(M, generator=g, device=DEV) < 0.1, -100, s["labels"])
    if case["op"] == "loss_grad":
        s["grad"] = torch.full((M,), 1.0 / M, device=DEV)
        s["lse"] = _plain(dict(s, case=dict(case, op="loss")))["lse"]
    return s


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------
def _layout(W, bits):
    """(word, shift) of each column of a row of W words: blocks of four words interleave column pairs
    (2- and 4-bit rows), the remaining words hold consecutive columns."""
    cpw = 32 // bits
    j = torch.arange(W, device=DEV)[:, None]
    i = torch.arange(cpw, device=DEV)[None, :]
    block = (j < W // 4 * 4) if bits != 1 else torch.zeros_like(j, dtype=torch.bool)
    cols = torch.where(block, 4 * cpw * (j // 4) + 8 * (i // 2) + 2 * (j % 4) + i % 2, j * cpw + i)
    word, shift = torch.empty(W * cpw, dtype=torch.long, device=DEV), torch.empty(W * cpw, dtype=torch.int32, device=DEV)
    word[cols.reshape(-1)] = j.expand_as(cols).reshape(-1)
    shift[cols.reshape(-1)] = ((i % 2) * 16 + (i // 2) * bits).expand_as(cols).reshape(-1).to(torch.int32)
    return word, shift


def _decode(words, scales, zeros, bits, group):
    """Rows of words [n][W] and their scales [n][K / group] -> fp32 [n][K]."""
    word, shift = _layout(words.shape[1], bits)
    q = ((words[:, word] >> shift) & ((1 << bits) - 1)).float()
    q = q * 2 - 1 if bits == 1 else q - 1 if bits == 2 else q
    if zeros is not None:
        q = q - zeros.float().repeat_interleave(group, 1)
    return q * scales.float().repeat_interleave(group, 1)


def _rows(s, ids):
    """Rows `ids` of the table in fp32."""
    case = s["case"]
    if case["bits"] == 16:
        return s["weight"][ids].float()
    z = s["zeros"][:, ids].T if s["zeros"] is not None else None
    return _decode(s["weight"][ids], s["scales"][:, ids].T, z, case["bits"], case["group"])


def _weights(s):
    """The vocabulary's rows in fp32."""
    case, V = s["case"], s["case"]["V"]
    if case["bits"] == 16:
        return s["weight"].float()
    z = s["zeros"][:, :V].T if s["zeros"] is not None else None
    return _decode(s["weight"][:V], s["scales"][:, :V].T, z, case["bits"], case["group"])


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return {"y": (_rows(s, s["tokens"].long()) * case["multiplier"]).to(torch.bfloat16)}
    if op == "embed_grad":
        first, rows = case["first"], case["rows"]
        at = s["tokens"].long() - first
        ids, order = torch.where((at >= 0) & (at < rows), at, rows).sort(stable=True)
        # sums over runs of the sorted tokens, as differences of prefix sums (of long sums: in 64 bits)
        sums = torch.cat([torch.zeros(1, case["K"], dtype=torch.float64, device=DEV),
                          s["dy"][order].double().cumsum(0)])
        ends = torch.searchsorted(ids, torch.arange(rows + 1, device=DEV))
        total = sums[ends[1:]] - sums[ends[:-1]]
        return {"dtable": (total * case["multiplier"]).to(torch.bfloat16)}
    w, x = _weights(s), s["x"].float()
    logits = x @ w.T
    valid = (s["labels"] >= 0) & (s["labels"] < case["V"])
    label = torch.where(valid, s["labels"], 0).long()
    if op == "loss":
        top = logits.amax(1, keepdim=True)
        lse = top[:, 0] + (logits - top).exp().sum(1).log()
        return {"loss": torch.where(valid, lse - logits.gather(1, label[:, None])[:, 0], 0.0), "lse": lse}
    p = (logits - s["lse"][:, None]).exp()
    p[torch.arange(case["M"], device=DEV), label] -= 1.0
    G = torch.where(valid, s["grad"], 0.0)[:, None] * p
    out = {"dx": (G @ w).to(torch.bfloat16)}
    if case["dw"]:
        out["dw"] = (G.T @ x).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------------
def _own(s):
    import bit_weight_only_w2_b200 as lb

    case = s["case"]
    op = case["op"]
    if op == "embed_grad":
        return {"dtable": lb.embedding_backward(s["tokens"], s["dy"], case["rows"], first=case["first"],
                                                multiplier=case["multiplier"])}
    table = (s["weight"], s["scales"], s["zeros"], case["bits"], case["group"])
    if op == "embed":
        return {"y": lb.embedding(s["tokens"], *table, multiplier=case["multiplier"])}
    if op == "loss":
        loss, lse = lb.cross_entropy(s["x"], s["labels"], *table, vocab=case["V"])
        return {"loss": loss, "lse": lse}
    dx, dw = lb.cross_entropy_backward(s["grad"], s["x"], s["labels"], s["lse"], *table, vocab=case["V"],
                                       need_dw=case["dw"])
    return {"dx": dx, "dw": dw} if case["dw"] else {"dx": dx}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    K, V = case["K"], case["V"]
    if case["op"] == "embed_grad":
        T = case["T"]
        return {"bytes": T * 4 + T * case["share"] * K * 2 + case["rows"] * K * 2, "flops": T * case["share"] * K}
    bits = case["bits"]
    row = K * bits / 8 + (0 if bits == 16 else K // case["group"] * (4 if bits == 4 else 2))
    if case["op"] == "embed":
        T = case["T"]
        return {"bytes": T * 4 + min(T, V) * row + T * K * 2, "flops": T * K}
    M = case["M"]
    if case["op"] == "loss":
        return {"bytes": V * row + M * K * 2 + M * 12, "flops": 2 * M * V * K}
    # the logits are formed again, then a product for each gradient
    return {"bytes": V * row + 2 * M * K * 2 + M * 12 + (V * K * 2 if case["dw"] else 0),
            "flops": (3 if case["dw"] else 2) * 2 * M * V * K}


def _exact_rows(s, lo, hi):
    """Rows lo .. hi - 1 of the table in 64 bits, column by column of the words' layout."""
    case = s["case"]
    w = s["weight"][lo:hi]
    bits, K = case["bits"], case["K"]
    if bits == 16:
        return w.double()
    per = 32 // bits
    W = w.shape[1]
    out = torch.empty(hi - lo, K, dtype=torch.float64, device=DEV)
    for pair in range(per // 2):
        for half in range(2):
            field = ((w.long() >> (16 * half + bits * pair)) & ((1 << bits) - 1)).double()
            whole = W // 4 * 4 if bits != 1 else 0
            for q in range(4):   # word q of each block of four
                if whole:
                    out[:, 8 * pair + 2 * q + half:4 * per * (whole // 4):4 * per] = field[:, q:whole:4]
            out[:, per * whole + 2 * pair + half::per] = field[:, whole:]
    out = 2 * out - 1 if bits == 1 else out - 1 if bits == 2 else out
    out = out.reshape(hi - lo, K // case["group"], case["group"])
    if s["zeros"] is not None:
        out -= s["zeros"][:, lo:hi].T.double()[:, :, None]
    return (out * s["scales"][:, lo:hi].T.double()[:, :, None]).reshape(hi - lo, K)


def exact(case, seed):
    s = prepare(case, seed)
    op, K, V = case["op"], case["K"], case["V"]
    if op == "embed_grad":
        out = torch.zeros(case["rows"] + 1, K, dtype=torch.float64, device=DEV)
        at = s["tokens"].long() - case["first"]
        at = torch.where((at >= 0) & (at < case["rows"]), at, case["rows"])
        out.index_add_(0, at, s["dy"].double())
        return {"dtable": out[:-1] * case["multiplier"]}
    step = 8192
    if op == "embed":
        out = torch.zeros(case["T"], K, dtype=torch.float64, device=DEV)
        for lo in range(0, V, step):
            hi = min(V, lo + step)
            here = ((s["tokens"] >= lo) & (s["tokens"] < hi)).nonzero().flatten()
            out[here] = _exact_rows(s, lo, hi)[s["tokens"][here].long() - lo]
        return {"y": out * case["multiplier"]}
    x, labels = s["x"].double(), s["labels"].long()
    valid = (labels >= 0) & (labels < V)
    if op == "loss":
        parts, target = [], torch.zeros(case["M"], dtype=torch.float64, device=DEV)
        for lo in range(0, V, step):
            l = x @ _exact_rows(s, lo, min(V, lo + step)).T
            parts.append(torch.logsumexp(l, 1))
            here = (valid & (labels >= lo) & (labels < lo + step)).nonzero().flatten()
            target[here] = l[here, labels[here] - lo]
        lse = torch.logsumexp(torch.stack(parts), 0)
        return {"loss": torch.where(valid, lse - target, 0.0), "lse": lse}
    g = torch.where(valid, s["grad"], 0.0).double()
    dx = torch.zeros_like(x)
    dw = torch.zeros(V, K, dtype=torch.float64, device=DEV) if case["dw"] else None
    for lo in range(0, V, step):
        hi = min(V, lo + step)
        w = _exact_rows(s, lo, hi)
        G = (x @ w.T - s["lse"].double()[:, None]).exp()
        here = (valid & (labels >= lo) & (labels < hi)).nonzero().flatten()
        G[here, labels[here] - lo] -= 1.0
        G *= g[:, None]
        dx += G @ w
        if dw is not None:
            dw[lo:hi] = G.T @ x
    return {"dx": dx, "dw": dw} if case["dw"] else {"dx": dx}
