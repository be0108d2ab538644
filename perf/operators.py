"""Cases of the block-scaled FP8 operators, with their plain forms.

Four operators, each on the inputs that a program has in hand before the call:

  quant    FP8 e4m3 codes with one scale per 128 x 128 block of a weight, or
           per token and 128 values of an activation;
  linear   a 16-bit activation quantized per token and 128 values, times a
           block-scaled FP8 weight;
  grouped  the same for tokens sorted by expert, each run of rows against its
           own expert's weight (the prefill side of a mixture of experts);
  moe      the router's choice (top-k of the logits) and the whole expert layer
           for a few tokens: gate and up projections, SwiGLU, the down
           projection and the weighted sum.

`own` chooses between the plain form (torch operations in fp32) and the
library's kernels.  A scale is max(fl32(absmax / 448), 1e-8) and a code is
e4m3(fl32(x / scale)), round to nearest even.
"""
import math

import torch

own = False

BLOCK = 128
FP8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A weight as it is converted once, when a checkpoint is loaded.
        {"name": "quant weight 8192x8192", "op": "quant", "what": "weight", "m": 8192, "k": 8192, "dtype": "bf16"},
        # A training step's master weight, kept in fp32, with ragged last blocks.
        {"name": "quant weight fp32 ragged", "op": "quant", "what": "weight", "m": 1552, "k": 2080, "dtype": "fp32"},
        # Activations that several projections share, so they are quantized on their own.
        {"name": "quant act 4096x8192", "op": "quant", "what": "act", "m": 4096, "k": 8192, "dtype": "bf16"},
        # One token of one sequence through a q_proj-sized layer: latency.
        {"name": "linear 1 token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16", "bias": False},
        # A decode batch of 48 sequences through an FFN-up-sized layer.
        {"name": "linear 48 tokens", "op": "linear", "m": 48, "n": 14336, "k": 4096, "dtype": "bf16", "bias": False},
        # A chunk of a prompt, in fp16 with a bias, no size a multiple of 128.
        {"name": "linear ragged", "op": "linear", "m": 333, "n": 4112, "k": 2080, "dtype": "fp16", "bias": True},
        # Prefill through the largest dense layer measured here.
        {"name": "linear 4096x8192x8192", "op": "linear", "m": 4096, "n": 8192, "k": 8192, "dtype": "bf16", "bias": False},
        # Prefill of a mixture of experts, tokens spread as a router spreads them.
        {"name": "grouped 16 experts", "op": "grouped", "m": 4096, "experts": 16, "n": 2048, "k": 4096, "skew": 0.3, "dtype": "bf16"},
        # Many small experts, some without a token, a ragged reduction.
        {"name": "grouped ragged", "op": "grouped", "m": 777, "experts": 40, "n": 1040, "k": 1440, "skew": 1.0, "dtype": "fp16"},
        # One token through two of sixteen experts: latency and the weights' bytes.
        {"name": "moe 1 token", "op": "moe", "m": 1, "experts": 16, "top_k": 2, "hidden": 4096, "inter": 2048,
         "scoring": "softmax", "pad": 0, "dtype": "bf16"},
        # A decode batch over many small experts.
        {"name": "moe 16 tokens", "op": "moe", "m": 16, "experts": 128, "top_k": 8, "hidden": 4096, "inter": 768,
         "scoring": "sigmoid", "pad": 0, "dtype": "bf16"},
        # A full batch, padded by three rows, over every expert; a ragged hidden size.
        {"name": "moe 64 tokens", "op": "moe", "m": 64, "experts": 32, "top_k": 4, "hidden": 2880, "inter": 1408,
         "scoring": "softmax", "pad": 3, "dtype": "fp16"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread evenly over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "grouped", "moe", "moe"])
    if op == "quant":
        return {"op": op, "what": rng.choice(["weight", "act"]), "m": _log(rng, 16, 8192, 16),
                "k": _log(rng, 128, 8192, 32), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 64, 8192, 16), "k": _log(rng, 128, 8192, 32),
                "dtype": rng.choice(["bf16", "fp16"]), "bias": rng.random() < 0.5}
    if op == "grouped":
        return {"op": op, "m": _log(rng, 1, 4096), "experts": _log(rng, 1, 64), "n": _log(rng, 128, 2048, 16),
                "k": _log(rng, 128, 4096, 32), "skew": round(rng.uniform(0.0, 1.5), 2),
                "dtype": rng.choice(["bf16", "fp16"])}
    experts = _log(rng, 4, 128)
    m = _log(rng, 1, 64)
    hidden = _log(rng, 512, 4096, 32)
    return {"op": op, "m": m, "experts": experts, "top_k": min(experts, rng.randint(1, 8)), "hidden": hidden,
            "inter": _log(rng, 128, min(1408, (400 << 20) // (experts * hidden) // 128 * 128), 128),
            "scoring": rng.choice(["softmax", "sigmoid"]), "pad": rng.choice([0, 0, min(3, m - 1)]),
            "dtype": rng.choice(["bf16", "fp16"])}


def work(case):
    """Each input read once, each output written once; experts that some token chose."""
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    up = lambda v: -(-v // BLOCK)  # noqa: E731
    if c["op"] == "quant":
        scales = (up(c["m"]) if c["what"] == "weight" else c["m"]) * up(c["k"])
        return {"bytes": c["m"] * c["k"] * (size + 1) + 4 * scales, "flops": 2 * c["m"] * c["k"]}
    if c["op"] in ("linear", "grouped"):
        m, n, k = c["m"], c["n"], c["k"]
        experts = 1
        if c["op"] == "grouped":
            experts = sum(x > 0 for x in _counts(c))
        return {"bytes": m * k * size + experts * (n * k + 4 * up(n) * up(k)) + 2 * m * n, "flops": 2 * m * n * k}
    tokens, h, i = c["m"] - c["pad"], c["hidden"], c["inter"]
    active = c["experts"] * (1 - (1 - c["top_k"] / c["experts"]) ** tokens)
    return {"bytes": active * 3 * h * i * (1 + 4 / BLOCK ** 2) + c["m"] * (h * (size + 2) + 4 * c["experts"]),
            "flops": 6 * tokens * c["top_k"] * h * i}


# ---------------------------------------------------------------- inputs

def _counts(c):
    """Tokens of each expert: shares spread by exp(skew x normal), from the case alone."""
    g = torch.Generator().manual_seed(c["m"] * 1000003 + c["experts"])
    share = torch.exp(c["skew"] * torch.randn(c["experts"], generator=g))
    edge = torch.round(torch.cumsum(share, 0) / share.sum() * c["m"]).to(torch.int64)
    edge[-1] = c["m"]
    return torch.diff(edge, prepend=torch.zeros(1, dtype=torch.int64)).tolist()


def _scale(amax):
    """max(fl32(amax / 448), 1e-8); by a tensor, as a division by a number may be a product with its reciprocal."""
    return (amax / torch.full_like(amax, 448.0)).clamp_min(1e-8)


def _blocks(W):
    """Codes and scales of a stack of weights [experts, n, k], 128 x 128 values at a time."""
    e, n, k = W.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    P = torch.nn.functional.pad(W.float(), (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(e, nb, BLOCK, kb, BLOCK)
    S = _scale(P.abs().amax(dim=(2, 4)))
    Q = (P / S[:, :, None, :, None]).to(FP8).view(e, nb * BLOCK, kb * BLOCK)
    return Q[:, :n, :k].contiguous(), S


def _weights(g, experts, n, k):
    """A stack of quantized weights of the size that trained layers have, made a few experts at a time."""
    at = max(1, (1 << 27) // (n * k))
    parts = [_blocks((torch.randn(min(at, experts - e), n, k, generator=g, device="cuda") * 0.02).bfloat16())
             for e in range(0, experts, at)]
    return torch.cat([p[0].view(torch.uint8) for p in parts]).view(FP8), torch.cat([p[1] for p in parts])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": dict(c)}
    if c["op"] == "quant":
        X = rand(c["m"], c["k"])
        if c["what"] == "weight":
            X *= 0.02
        else:
            X = torch.where(rand(c["m"], c["k"]) > 3.0, X * 100.0, X)
        s["X"] = X.to(DTYPES[c["dtype"]])
        return s
    k = c["hidden"] if c["op"] == "moe" else c["k"]
    X = rand(c["m"], k)
    s["X"] = torch.where(rand(c["m"], k) > 3.0, X * 100.0, X).to(DTYPES[c["dtype"]])  # a few large values, as hidden states have
    if c["op"] == "linear":
        W, S = _weights(g, 1, c["n"], k)
        s["W"], s["S"] = W[0], S[0]
        s["bias"] = rand(c["n"]) if c["bias"] else None
    elif c["op"] == "grouped":
        s["W"], s["S"] = _weights(g, c["experts"], c["n"], k)
        counts = torch.tensor([0] + _counts(c))
        s["offsets"] = torch.cumsum(counts, 0).to(torch.int32).cuda()
    else:
        s["W13"], s["S13"] = _weights(g, c["experts"], 2 * c["inter"], k)
        s["W2"], s["S2"] = _weights(g, c["experts"], k, c["inter"])
        s["logits"] = 1.5 * rand(c["m"], c["experts"])
        if c["pad"]:  # padding rows choose no expert
            s["logits"][c["m"] - c["pad"]:] = -math.inf
    return s


# ---------------------------------------------------------------- plain forms

def _act(X):
    """Codes and scales of an activation: groups of 128 along the last axis, the last one padded with zeros."""
    k = X.shape[-1]
    kb = -(-k // BLOCK)
    P = torch.nn.functional.pad(X.float(), (0, kb * BLOCK - k)).unflatten(-1, (kb, BLOCK))
    S = _scale(P.abs().amax(-1))
    return (P / S[..., None]).to(FP8).flatten(-2)[..., :k], S


def _act_value(X):
    Q, S = _act(X)
    return Q.float() * S.repeat_interleave(BLOCK, -1)[..., :X.shape[-1]]


def _value(W, S):
    """The values that a stack of block-scaled codes stands for."""
    n, k = W.shape[-2:]
    return W.float() * S.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]


def _choose(logits, top_k, scoring):
    """The top_k largest logits, the lowest index first among equals; -inf is never chosen (-1, weight 0)."""
    L = logits.float()
    top, ids = torch.sort(L, dim=-1, descending=True, stable=True)
    top, ids = top[:, :top_k], ids[:, :top_k]
    none = top == -math.inf
    if scoring == "softmax":
        p = torch.exp(top - top[:, :1])
    else:
        p = 1.0 / (1.0 + torch.exp(-top))
    p = torch.where(none, 0.0, p)
    total = p.sum(-1, keepdim=True)
    return torch.where(none, -1, ids).to(torch.int32), torch.where(none, 0.0, p / total)


def _swiglu(gu):
    gate, up = gu.chunk(2, -1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _layer(x, ids, weights, s, c):
    """Every chosen expert's output, weighted and summed over a token's choices."""
    m, experts = x.shape[0], c["experts"]
    if ids.numel() < experts:  # fewer choices than experts: each choice on its own
        e = ids.clamp_min(0).flatten().long()
        gu = torch.matmul(_value(s["W13"].view(torch.uint8)[e].view(FP8), s["S13"][e]),
                          x.repeat_interleave(ids.shape[1], 0)[:, :, None])[:, :, 0]
        y = torch.matmul(_value(s["W2"].view(torch.uint8)[e].view(FP8), s["S2"][e]), _act_value(_swiglu(gu))[:, :, None])[:, :, 0]
        return (y.view(m, ids.shape[1], -1) * weights[:, :, None]).sum(1)
    gu = torch.matmul(x, _value(s["W13"], s["S13"]).transpose(1, 2))  # every token through every expert
    y = torch.matmul(_act_value(_swiglu(gu)), _value(s["W2"], s["S2"]).transpose(1, 2))
    gates = torch.zeros(m, experts, device=x.device).scatter_add_(1, ids.clamp_min(0).long(), weights)
    return (y * gates.T[:, :, None]).sum(0)


def run(state):
    s = state
    c = s["case"]
    X = s["X"]
    if own:
        from bit_quantized_b200 import q8
        if c["op"] == "quant":
            q = q8.q8_quantize_weight_block(X) if c["what"] == "weight" else q8.q8_quantize_act_block(X)
            return {"codes": q.codes, "scale": q.scale}
        if c["op"] == "linear":
            return q8.q8_linear_fp8_block_dynamic(X, q8.QWeightBlock(s["W"], s["S"]), bias=s["bias"])
        if c["op"] == "grouped":
            return q8.q8_linear_fp8_block_grouped(q8.q8_quantize_act_block(X), q8.QWeightBlock(s["W"], s["S"]), s["offsets"])
        ids, weights = q8.q8_moe_route(s["logits"], c["top_k"], scoring=c["scoring"])
        y = q8.q8_moe_fp8_block(X, ids, weights, q8.QWeightBlock(s["W13"], s["S13"]), q8.QWeightBlock(s["W2"], s["S2"]))
        return {"ids": ids, "weights": weights, "y": y}
    if c["op"] == "quant":
        if c["what"] == "weight":
            Q, S = _blocks(X[None])
            return {"codes": Q[0], "scale": S[0]}
        Q, S = _act(X)
        return {"codes": Q.contiguous(), "scale": S.T.contiguous()}  # scales: one row per group of 128
    x = _act_value(X)
    if c["op"] == "linear":
        y = torch.matmul(x, _value(s["W"], s["S"]).T)
        return (y if s["bias"] is None else y + s["bias"]).bfloat16()
    if c["op"] == "grouped":
        # each expert's rows, padded to the longest expert's, as one batched product
        off = s["offsets"].long()
        count = torch.diff(off)
        row = torch.arange(X.shape[0], device=X.device)
        e = torch.searchsorted(off, row, right=True) - 1
        at = row - off[e]
        P = torch.zeros(c["experts"], max(_counts(c)), c["k"], device=X.device)
        P[e, at] = x
        return torch.matmul(P, _value(s["W"], s["S"]).transpose(1, 2))[e, at].bfloat16()
    ids, weights = _choose(s["logits"], c["top_k"], c["scoring"])
    return {"ids": ids, "weights": weights, "y": _layer(x, ids, weights, s, c).bfloat16()}


# ---------------------------------------------------------------- in 64 bits

def _e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even: 4 significant bits, the smallest step 2^-9, at most 448."""
    _, exponent = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (exponent - 4).clamp_min(-9))
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _quantized(x, dims):
    """Codes and scales in 64 bits; scale and quotient are rounded to 32 bits, as the definition says."""
    S = (x.abs().amax(dim=dims, keepdim=True) / 448.0).float().double()
    S = torch.maximum(S, torch.tensor(1e-8, dtype=torch.float32, device=x.device).double())
    return _e4m3((x / S).float().double()), S


def _groups(x):
    """x along its last axis in groups of 128: the values of their codes."""
    k = x.shape[-1]
    cut = k // BLOCK * BLOCK
    whole = x[..., :cut].reshape(*x.shape[:-1], cut // BLOCK, BLOCK)
    Q, S = _quantized(whole, (-1,))
    out = [(Q * S).reshape(*x.shape[:-1], cut)]
    if cut < k:
        Q, S = _quantized(x[..., cut:], (-1,))
        out.append(Q * S)
    return torch.cat(out, -1)


def _wide(W, S):
    n, k = W.shape
    row, col = torch.arange(n, device=W.device) // BLOCK, torch.arange(k, device=W.device) // BLOCK
    return W.double() * S.double()[row][:, col]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    x = s["X"].double()
    if c["op"] == "quant":
        down = BLOCK if c["what"] == "weight" else 1
        m, k = c["m"], c["k"]
        mb, kb = -(-m // down), -(-k // BLOCK)
        P = torch.zeros(mb * down, kb * BLOCK, dtype=torch.float64, device=x.device)
        P[:m, :k] = x
        Q, S = _quantized(P.view(mb, down, kb, BLOCK), (1, 3))
        S = S[:, 0, :, 0]
        return {"codes": Q.view(mb * down, kb * BLOCK)[:m, :k], "scale": S if down > 1 else S.T.contiguous()}
    x = _groups(x)
    if c["op"] == "linear":
        y = x @ _wide(s["W"], s["S"]).T
        return y if s["bias"] is None else y + s["bias"].double()
    if c["op"] == "grouped":
        off = s["offsets"].tolist()
        return torch.cat([x[off[e]:off[e + 1]] @ _wide(s["W"][e], s["S"][e]).T for e in range(c["experts"])])
    L = s["logits"].double().cpu()
    weights = torch.zeros(c["m"], c["top_k"], dtype=torch.float64)
    y = torch.zeros(c["m"], c["hidden"], dtype=torch.float64, device=x.device)
    chosen = {}
    for t in range(c["m"]):
        order = sorted((e for e in range(c["experts"]) if L[t, e] > -math.inf), key=lambda e: (-float(L[t, e]), e))[:c["top_k"]]
        p = [math.exp(float(L[t, e] - L[t, order[0]])) if c["scoring"] == "softmax" else 1.0 / (1.0 + math.exp(-float(L[t, e])))
             for e in order]
        for j, e in enumerate(order):
            weights[t, j] = p[j] / sum(p)
            chosen.setdefault(e, []).append((t, p[j] / sum(p)))
    for e, pairs in sorted(chosen.items()):
        rows = torch.tensor([t for t, _ in pairs], device=x.device)
        gu = x[rows] @ _wide(s["W13"][e], s["S13"][e]).T
        gate, up = gu[:, :c["inter"]], gu[:, c["inter"]:]
        h = _groups(gate / (1.0 + torch.exp(-gate)) * up)
        y[rows] += (h @ _wide(s["W2"][e], s["S2"][e]).T) * torch.tensor([[w] for _, w in pairs], dtype=torch.float64, device=x.device)
    return {"ids": None, "weights": weights.to(x.device), "y": y}
