"""Cases of the block-scaled FP8 operators: the activation pass, the linear
and the mixture-of-experts layer for a few tokens.

All three work on E4M3 codes with one fp32 scale per block of 128: weights
[N, K] in blocks of 128 x 128, activations [M, K] per token and 128 features.

  quantize  A = max(max |x| over the block, 2^-100), s = fp32(A / 448),
            r = fp32(448 / A), code = E4M3(fp32(x r)), nearest even
  linear    Y = sum_g sx[g, m] sw[n / 128, g] sum_{k in g} qx qw + bias, from X
            in bf16 (the pass above included)
  moe       router logits X Wr^T, the top_k largest (ties to the lowest
            expert), softmax weights, per chosen expert
            (silu(X Wg) * (X Wu)) Wd, their weighted sum; FP8 weights, bf16
            activations

`run` computes them in plain torch operations, or calls the framework's entry
points where `own` is true.
"""

import math

import torch
import torch.nn.functional as F

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -100


def listed():
    return [
        # one activation pass of a short batch (latency) and of a video model's tokens (bandwidth)
        {"name": "quantize few tokens", "op": "quantize", "M": 16, "K": 5120},
        {"name": "quantize video", "op": "quantize", "M": 32760, "K": 5120},
        # one conditioning vector through a projection: the weight is read once
        {"name": "linear one token", "op": "linear", "M": 1, "K": 5120, "N": 5120, "bias": True, "out": "bf16"},
        # a few sequences decoded together, a wide up-projection
        {"name": "linear few tokens", "op": "linear", "M": 13, "K": 2048, "N": 12288, "bias": False, "out": "bf16"},
        # a ragged prompt into a head of odd width, K ending inside a block, fp32 output
        {"name": "linear ragged", "op": "linear", "M": 333, "K": 1936, "N": 1000, "bias": True, "out": "f32"},
        # image and text tokens of one 1024 x 1024 picture through an MLP up-projection
        {"name": "linear image", "op": "linear", "M": 4608, "K": 5120, "N": 12288, "bias": True, "out": "bf16"},
        # a video model's attention projection, the largest
        {"name": "linear video", "op": "linear", "M": 32760, "K": 5120, "N": 5120, "bias": True, "out": "bf16"},
        # one token decoded
        {"name": "moe one token", "op": "moe", "T": 1, "H": 2048, "I": 768, "E": 64, "k": 8, "renorm": True},
        # eight sequences decoded together
        {"name": "moe eight tokens", "op": "moe", "T": 8, "H": 4096, "I": 1408, "E": 64, "k": 4, "renorm": True},
        # a ragged batch on odd sizes, weights of the softmax over all experts
        {"name": "moe ragged", "op": "moe", "T": 23, "H": 1072, "I": 400, "E": 40, "k": 3, "renorm": False},
        # a full batch that reaches nearly every expert
        {"name": "moe full batch", "op": "moe", "T": 64, "H": 4096, "I": 1408, "E": 128, "k": 8, "renorm": True},
    ]


def _log(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "moe", "moe"])
    if op == "quantize":
        return {"op": op, "M": _log(rng, 1, 32760), "K": _log(rng, 64, 5120, 16)}
    if op == "linear":
        K, N = _log(rng, 64, 12288, 16), _log(rng, 64, 12288, 8)
        M = _log(rng, 1, min(32760, 32760 * 5120 * 5120 // (K * N)))
        return {"op": op, "M": M, "K": K, "N": N, "bias": rng.random() < 0.5,
                "out": rng.choice(["bf16", "bf16", "f32"])}
    E = _log(rng, 4, 128)
    return {"op": op, "T": _log(rng, 1, 64), "H": _log(rng, 128, 4096, 16), "I": _log(rng, 64, 1408, 16), "E": E,
            "k": rng.randint(1, min(8, E)), "renorm": rng.random() < 0.5}


# ------------------------------------------------------------- the inputs --

def _blocks(n):
    return -(-n // BLOCK)


def _quantize_weight(w):
    """Codes and scales of bf16 weights [..., N, K], one scale per 128 x 128."""
    N, K = w.shape[-2:]
    gn, gk = _blocks(N), _blocks(K)
    p = F.pad(w, (0, gk * BLOCK - K, 0, gn * BLOCK - N)).unflatten(-1, (gk, BLOCK)).unflatten(-3, (gn, BLOCK))
    a = p.abs().amax(dim=(-3, -1)).double().clamp_min(TINY)
    s, r = (a / E4M3_MAX).float(), (E4M3_MAX / a).float()
    q = (p.float() * r[..., :, None, :, None]).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).flatten(-2).flatten(-3, -2)[..., :N, :K].contiguous()
    return q.view(torch.float8_e4m3fn), s


def _tokens(gen, M, K):
    """Activations of unit spread with a few outlier channels, as the
    quantized linears of this repository meet them."""
    x = torch.randn((M, K), generator=gen, device="cuda")
    picks = torch.randint(0, K, (max(1, K // 200),), generator=gen, device="cuda")
    x[:, picks] *= 20.0
    return x.bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    empty = lambda dtype, *shape: torch.empty(shape, device="cuda", dtype=dtype)  # noqa: E731
    state = dict(case)
    if case["op"] == "moe":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        state["X"] = randn(T, H)
        state["wr"] = randn(E, H) * (2.0 / math.sqrt(H))
        state["w13"], state["s13"] = _quantize_weight(randn(E, 2, I, H).mul_(1.0 / math.sqrt(H)))
        state["w2"], state["s2"] = _quantize_weight(randn(E, H, I).mul_(1.0 / math.sqrt(I)))
        state["Y"] = empty(torch.bfloat16, T, H)
        state["idx"], state["gate"] = empty(torch.int32, T, k), empty(torch.float32, T, k)
        state["workspace"] = empty(torch.uint8, 8 * T * k * (I + 128) + 16 * T * E + 65536)
        return state
    M, K = case["M"], case["K"]
    state["X"] = _tokens(gen, M, K)
    if case["op"] == "quantize":
        state["qx"], state["sx"] = empty(torch.float8_e4m3fn, M, K), empty(torch.float32, _blocks(K), M)
        return state
    N = case["N"]
    state["qw"], state["sw"] = _quantize_weight(randn(N, K).mul_(0.02))
    state["b"] = randn(N).mul_(0.01) if case["bias"] else None
    state["Y"] = empty(torch.bfloat16 if case["out"] == "bf16" else torch.float32, M, N)
    state["workspace"] = empty(torch.uint8, M * K + 4 * M * _blocks(K) + 65536)
    return state


# --------------------------------------------------------- the plain form --

def _quantize(X):
    M, K = X.shape
    x = F.pad(X.float(), (0, _blocks(K) * BLOCK - K)).view(M, -1, BLOCK)
    a = x.abs().amax(2).double().clamp_min(TINY)
    s, r = (a / E4M3_MAX).float(), (E4M3_MAX / a).float()
    q = (x * r[:, :, None]).to(torch.float8_e4m3fn)
    return q, s


def _widen(q, s):
    """fp32 weights of codes [..., N, K] and scales [..., N / 128, K / 128]."""
    N, K = q.shape[-2:]
    return q.float() * s.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]


def _linear(c):
    q, s = _quantize(c["X"])
    x = (q.float() * s[:, :, None]).flatten(1)[:, : c["K"]]
    y = x @ _widen(c["qw"], c["sw"]).t()
    if c["b"] is not None:
        y = y + c["b"].float()
    return y.to(c["Y"].dtype)


def _moe(c):
    T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
    logits = c["X"].double() @ c["wr"].double().t()
    top, idx = (v[:, :k] for v in torch.sort(logits, dim=1, descending=True, stable=True))
    e = torch.exp((top - top[:, :1]).float())
    all_e = e if c["renorm"] else torch.exp((logits - top[:, :1]).float())
    gate = e / all_e.sum(1, keepdim=True)
    x = c["X"].float()
    if T * k < E:  # the chosen experts' weights, gathered
        at = idx.reshape(-1)
        w13, w2 = _widen(c["w13"][at], c["s13"][at]), _widen(c["w2"][at], c["s2"][at])
        x = x.repeat_interleave(k, 0)[:, None, :]  # [T k, 1, H]
        g, u = torch.bmm(x, w13[:, 0].mT.contiguous()), torch.bmm(x, w13[:, 1].mT.contiguous())
        o = torch.bmm(g * torch.sigmoid(g) * u, w2.mT.contiguous()).view(T, k, H)
        y = (o * gate[:, :, None]).sum(1)
    else:  # every expert on every token
        w13, w2 = _widen(c["w13"], c["s13"]), _widen(c["w2"], c["s2"])
        gu = x @ w13.view(E * 2 * I, H).t()
        g, u = gu.view(T, E, 2, I).unbind(2)
        share = torch.zeros((T, E), device=x.device).scatter_(1, idx, gate)
        h = g * torch.sigmoid(g) * u * share[:, :, None]
        y = h.view(T, E * I) @ w2.transpose(0, 1).reshape(H, E * I).t()
    return {"y": y.bfloat16(), "experts": idx.int(), "weights": gate}


def run(state):
    c = state
    if own:
        from bit_quantized_linear_amd import binding as b

        if c["op"] == "quantize":
            b.svdq_fp8_quantize_act(c["X"], c["qx"], c["sx"])
            return {"codes": c["qx"], "scales": c["sx"]}
        if c["op"] == "linear":
            b.svdq_fp8_linear(c["X"], c["qw"], c["sw"], c["b"], c["workspace"], c["Y"])
            return c["Y"]
        b.svdq_fp8_moe_layer(c["X"], c["wr"], c["w13"], c["s13"], c["w2"], c["s2"], c["Y"], c["idx"], c["gate"],
                             c["workspace"], renormalize=c["renorm"])
        return {"y": c["Y"], "experts": c["idx"], "weights": c["gate"]}
    if c["op"] == "quantize":
        q, s = _quantize(c["X"])
        return {"codes": q.flatten(1)[:, : c["K"]].contiguous(), "scales": s.t().contiguous()}
    return _linear(c) if c["op"] == "linear" else _moe(c)


def work(case):
    """Each input read once, each output written once; the experts that a
    batch of T tokens reaches, k of E each, as many as it does on average."""
    if case["op"] == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": 3 * M * K + 4 * M * _blocks(K), "flops": 2 * M * K}
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        wide = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * M * K + N * K + 4 * _blocks(N) * _blocks(K) + (2 * N if case["bias"] else 0) + wide * M * N,
                "flops": 2 * M * N * K}
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    reached = E * (1 - (1 - k / E) ** T)
    return {"bytes": reached * 3 * H * I + 2 * E * H + 4 * T * H + 8 * T * k,
            "flops": T * k * 6 * H * I + 2 * T * E * H}


# -------------------------------------------- the definition, in 64 bits --

def _e4m3(v):
    """The E4M3 values nearest to v (64 bits, |v| < 464), ties to even."""
    step = torch.exp2(torch.frexp(v)[1].sub(1).clamp_min(-6).double() - 3)
    return torch.round(v / step) * step


def _codes64(X):
    """E4M3 values [M, K] and scales [M, blocks] of bf16 X, 64 bits between
    the roundings that the definition names."""
    M, K = X.shape
    values, scales = [], []
    for k in range(0, K, BLOCK):
        x = X[:, k: k + BLOCK].double()
        a = torch.maximum(x.abs().max(1).values, torch.tensor(TINY, dtype=torch.float64, device=x.device))
        r = torch.div(E4M3_MAX, a).float().double()
        scales.append(torch.div(a, E4M3_MAX).float().double())
        values.append(_e4m3((x * r[:, None]).float().double()))
    return torch.cat(values, 1), torch.stack(scales, 1)


def _wide64(q, s):
    rows = torch.arange(q.shape[-2], device=q.device) // BLOCK
    cols = torch.arange(q.shape[-1], device=q.device) // BLOCK
    return q.double() * s.double()[..., rows, :][..., cols]


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "moe":
        T, k = c["T"], c["k"]
        x = c["X"].double()
        logits = torch.stack([(x * w.double()).sum(1) for w in c["wr"]], 1)
        weights = torch.softmax(logits, 1)
        key, chosen = logits.clone(), []
        for _ in range(k):  # the first of the largest, k times
            best = key.max(1, keepdim=True).values
            chosen.append((key == best).int().argmax(1))
            key[torch.arange(T, device=x.device), chosen[-1]] = -math.inf
        idx = torch.stack(chosen, 1)
        gate = weights.gather(1, idx)
        if c["renorm"]:
            gate = gate / gate.sum(1, keepdim=True)
        y = torch.zeros((T, c["H"]), dtype=torch.float64, device=x.device)
        for e in idx.unique().tolist():
            t, j = (idx == e).nonzero(as_tuple=True)
            up = _wide64(c["w13"][e], c["s13"][e])
            g, u = x[t] @ up[0].t(), x[t] @ up[1].t()
            o = (g / (1 + torch.exp(-g)) * u) @ _wide64(c["w2"][e], c["s2"][e]).t()
            y[t] += gate[t, j][:, None] * o
        return {"y": y, "experts": idx, "weights": gate}
    values, scales = _codes64(c["X"])
    if c["op"] == "quantize":
        return {"codes": values, "scales": scales.t().contiguous()}
    cols = torch.arange(c["K"], device=values.device) // BLOCK
    y = (values * scales[:, cols]) @ _wide64(c["qw"], c["sw"]).t()
    return y + c["b"].double() if c["b"] is not None else y
