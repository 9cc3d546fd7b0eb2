"""Cases of the operators around a decoder block's block-scaled FP8 linears: the
norm that feeds them, rotary positions, and attention over a cache of 8-bit keys
and values.

  norm    h = X + residual, y = h / sqrt(mean(h^2) + eps) * w; per token and 128
          features A = max(max |y|, 2^-100), scale = A / 448, code = E4M3(y 448 / A)
  rope    pair j of a head is turned by positions[t, axis of j] * freqs[j]; the
          pairs are (2 j, 2 j + 1) or (j, j + R / 2); axis a has sections[a]
          consecutive pairs
  append  new keys and values into pages of 64 tokens: E4M3 codes, keys [64, D] and
          values [D, 64] per page and head, and per page and head one scale for
          each, the least power of two s with max |x| <= 448 s; a page that is
          filled further keeps its scale or, where the new tokens need a larger
          one, has its codes rounded to that
  attention  softmax(scale Q K^T) V over a sequence's pages, for its newest
          tokens; query heads share key heads in consecutive groups; causal, with
          a window or without

`run` computes them in plain torch operations, or calls the framework's entry
points where `own` is true.
"""

import math

import torch
import torch.nn.functional as F

own = False

BLOCK = 128
PAGE = 64
E4M3_MAX = 448.0
TINY = 2.0 ** -100
EPS = 1e-6


def listed():
    return [
        # the sum and norm before a projection of eight sequences decoded together (latency)
        {"name": "norm few tokens", "op": "norm", "M": 8, "K": 4096, "residual": True, "bf16": False},
        # a ragged prompt, K ending inside a block, a bf16 copy for a layer that takes bf16
        {"name": "norm ragged", "op": "norm", "M": 333, "K": 1936, "residual": False, "bf16": True},
        # a video model's tokens (bandwidth)
        {"name": "norm video", "op": "norm", "M": 32760, "K": 5120, "residual": True, "bf16": False},
        # query and key heads of sixteen sequences decoded together, positions up to a million
        {"name": "rope decode", "op": "rope", "T": 16, "H": 40, "D": 128, "R": 128, "sections": "64", "interleaved": False,
         "far": 1000000},
        # a video model's query and key heads, turned by time, height and width
        {"name": "rope video", "op": "rope", "T": 32760, "H": 80, "D": 128, "R": 128, "sections": "22 21 21",
         "interleaved": True, "far": 64},
        # one token each of sixteen sequences into their last pages
        {"name": "append decode", "op": "append", "B": 16, "new": 1, "past": 4100, "ragged": True, "Hk": 8, "D": 128},
        # three latent frames of a video after eighteen others
        {"name": "append video", "op": "append", "B": 1, "new": 4680, "past": 28080, "ragged": False, "Hk": 40, "D": 128},
        # the next token of one long text
        {"name": "attention one token", "op": "attention", "B": 1, "new": 1, "past": 32759, "ragged": False, "Hq": 32,
         "Hk": 8, "D": 128, "causal": True, "window": 0, "lse": False},
        # a batch of decoded sequences of many lengths
        {"name": "attention decode", "op": "attention", "B": 32, "new": 1, "past": 8191, "ragged": True, "Hq": 32, "Hk": 8,
         "D": 128, "causal": True, "window": 0, "lse": False},
        # a few drafted tokens each, to be checked, in a model whose layer sees a window
        {"name": "attention draft", "op": "attention", "B": 5, "new": 4, "past": 2000, "ragged": True, "Hq": 14, "Hk": 2,
         "D": 64, "causal": True, "window": 1000, "lse": True},
        # prompts of three sequences, two of them after a shared prefix
        {"name": "attention prompts", "op": "attention", "B": 3, "new": 2777, "past": 1500, "ragged": True, "Hq": 32,
         "Hk": 8, "D": 128, "causal": True, "window": 0, "lse": True},
        # three latent frames of a video over all frames so far, every head with its own keys, the largest
        {"name": "attention video", "op": "attention", "B": 1, "new": 4680, "past": 28080, "ragged": False, "Hq": 40,
         "Hk": 40, "D": 128, "causal": False, "window": 0, "lse": False},
    ]


def _log(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "rope", "append", "attention", "attention", "attention"])
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 32760), "K": _log(rng, 64, 5120, 16), "residual": rng.random() < 0.7,
                "bf16": rng.random() < 0.3}
    if op == "rope":
        D = rng.choice([64, 80, 128, 128])
        R = rng.choice([D, D, D // 2 // 16 * 16])
        axes = rng.choice([1, 3, 3])
        cut = sorted(rng.randint(0, R // 2) for _ in range(axes - 1))
        sections = [b - a for a, b in zip([0] + cut, cut + [R // 2])]
        return {"op": op, "T": _log(rng, 1, 32760), "H": _log(rng, 1, 80), "D": D, "R": R,
                "sections": " ".join(map(str, sections)), "interleaved": rng.random() < 0.5, "far": _log(rng, 16, 1000000)}
    Hk, D = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([64, 128, 128])
    if op == "append":
        B = _log(rng, 1, 32)
        return {"op": op, "B": B, "new": _log(rng, 1, 32760 // B), "past": _log(rng, 1, 32760 // B), "ragged": True,
                "Hk": Hk, "D": D}
    case = {"op": op, "ragged": True, "Hq": Hk * rng.choice([1, 2, 4, 5, 7, 8]), "Hk": Hk, "D": D,
            "causal": rng.random() < 0.8, "window": 0, "lse": rng.random() < 0.5}
    if rng.random() < 0.5:  # decoded tokens
        case["B"] = _log(rng, 1, 64)
        case["new"] = rng.choice([1, 1, 1, 2, 4])
        case["past"] = _log(rng, 16, min(32760, 262144 // case["B"]))
    else:
        case["B"] = rng.randint(1, 4)
        case["new"] = _log(rng, 16, 4680)
        case["past"] = _log(rng, 1, 8192)
    if case["causal"] and rng.random() < 0.3:
        case["window"] = _log(rng, 16, 4096)
    return case


# ------------------------------------------------------------- the inputs --

def _plan(case):
    """New tokens and tokens before them of each sequence; the first has the
    case's own sizes, the others of a ragged batch between a fifth and all."""
    part = lambda b, g: 0.2 + 0.8 * (b * g % 1.0) if case["ragged"] and b else 1.0  # noqa: E731
    return [(max(1, round(case["new"] * part(b, 0.618034))), round(case["past"] * part(b, 0.754878)))
            for b in range(case["B"])]


def _pages(n):
    return -(-n // PAGE)


def _codes(gen, *shape):
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for i in range(0, shape[0], 64):
        part = torch.randn((min(64, shape[0] - i),) + shape[1:], generator=gen, device="cuda")
        out[i: i + 64] = part.mul_(64.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return out


def _cache(state, gen):
    """Pages in an order of their own, a few of them free, and the plan's tensors;
    the entries of the page table behind a sequence's last page are -1."""
    plan = _plan(state)
    used = [_pages(new + past) for new, past in plan]
    total, widest = sum(used) + 3, max(used)
    order = torch.randperm(total, generator=gen, device="cuda").tolist()
    rows, at = [], 0
    for n in used:
        rows.append(order[at: at + n] + [-1] * (widest - n))
        at += n
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = [0]
    for new, _ in plan:
        starts.append(starts[-1] + new)
    Hk, D = state["Hk"], state["D"]
    scale = lambda: torch.exp2(torch.randint(-7, -5, (total, Hk), generator=gen, device="cuda").float())  # noqa: E731
    state.update(plan=plan, rows=rows, table=whole(rows), starts=whole(starts), lengths=whole([n + p for n, p in plan]),
                 kc=_codes(gen, total, Hk, PAGE, D), vc=_codes(gen, total, Hk, D, PAGE), ks=scale(), vs=scale())
    return starts[-1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    empty = lambda dtype, *shape: torch.empty(shape, device="cuda", dtype=dtype)  # noqa: E731
    state = dict(case)
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        state["X"] = randn(M, K)
        state["r"] = None
        if case["residual"]:  # a residual stream has a few channels far above the others
            state["r"] = randn(M, K)
            state["r"][:, torch.randint(0, K, (max(1, K // 200),), generator=gen, device="cuda")] *= 20.0
        state["w"] = randn(K).mul_(0.1).add_(1.0)
        state["total"] = empty(torch.bfloat16, M, K) if case["residual"] else None
        state["Y"] = empty(torch.bfloat16, M, K) if case["bf16"] else None
        state["qx"], state["sx"] = empty(torch.float8_e4m3fn, M, K), empty(torch.float32, -(-K // BLOCK), M)
        return state
    if case["op"] == "rope":  # the query and key heads of rows that hold the values' heads as well
        T, H, D, R = (case[n] for n in ("T", "H", "D", "R"))
        state["sections"] = [int(s) for s in case["sections"].split()]
        state["X"] = randn(T, H + max(1, H // 4), D)[:, :H]
        state["positions"] = torch.randint(0, case["far"], (T, len(state["sections"])), generator=gen, device="cuda",
                                           dtype=torch.int32)
        freqs = []
        for n in state["sections"]:  # each axis has frequencies from 1 down to 1 / 10000
            freqs += [10000.0 ** (-i / max(1, n)) for i in range(n)]
        state["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
        state["Y"] = empty(torch.bfloat16, T, H, D)
        return state
    T = _cache(state, gen)
    Hk, D = case["Hk"], case["D"]
    if case["op"] == "append":  # rows of a projection: queries, keys, values
        rows = randn(T, 3 * Hk, D)
        state["k"], state["v"] = rows[:, Hk: 2 * Hk], rows[:, 2 * Hk:]
        return state
    Hq = case["Hq"]
    state["q"] = randn(T, Hq, D).mul_(2.0)
    state["scale"] = 1.0 / math.sqrt(D)
    state["O"] = empty(torch.bfloat16, T, Hq, D)
    state["L"] = empty(torch.float32, T, Hq) if case["lse"] else None
    state["workspace"] = empty(torch.uint8, 64 << 20)
    return state


# --------------------------------------------------------- the plain form --

def _norm(c):
    x = c["X"].float()
    if c["r"] is not None:
        x = x + c["r"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * c["w"].float()
    M, K = y.shape
    g = F.pad(y, (0, -K % BLOCK)).view(M, -1, BLOCK)
    a = g.abs().amax(2).clamp_min(TINY)
    q = (g * (E4M3_MAX / a)[:, :, None]).to(torch.float8_e4m3fn).flatten(1)[:, :K].contiguous()
    out = {"codes": q, "scales": (a / E4M3_MAX).t().contiguous()}
    if c["r"] is not None:
        out["sum"] = x.bfloat16()
    if c["bf16"]:
        out["y"] = y.bfloat16()
    return out


def _rope(c):
    axis = torch.repeat_interleave(torch.arange(len(c["sections"])), torch.tensor(c["sections"]))
    angle = c["positions"].double()[:, axis.to(c["positions"].device)] * c["freqs"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    x, R = c["X"].float(), c["R"]
    if c["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., R:]], -1).bfloat16()


def _append_one(x, codes, scales, pages, past, across):
    """x [n, Hk, D] into codes [pages, Hk, 64, D] (or [pages, Hk, D, 64]: across) from token `past` on."""
    n = x.shape[0]
    first, last = past // PAGE, (past + n - 1) // PAGE
    at = past - first * PAGE
    p = torch.tensor(pages[first: last + 1], device=x.device)
    x = F.pad(x.float().permute(1, 2, 0), (at, (last + 1) * PAGE - past - n))  # [Hk, D, tokens]
    x = x.unflatten(2, (-1, PAGE)).permute(2, 0, 3, 1)  # [pages, Hk, 64, D]
    m, e = torch.frexp(x.abs().amax((2, 3)).clamp_min(TINY))
    s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875))
    old = codes[p].float()
    if across:
        old = old.mT
    if at:
        s[0] = torch.maximum(s[0], scales[p[0]])
        old[0, :, :at] *= (scales[p[0]] / s[0])[:, None, None]
    token = torch.arange(first * PAGE, (last + 1) * PAGE, device=x.device).view(-1, 1, PAGE, 1)
    new = torch.where((token >= past) & (token < past + n), x / s[:, :, None, None], old).to(torch.float8_e4m3fn)
    codes.view(torch.uint8)[p] = (new.mT if across else new).contiguous().view(torch.uint8)
    scales[p] = s


def _append(c):
    t = 0
    for (new, past), pages in zip(c["plan"], c["rows"]):
        _append_one(c["k"][t: t + new], c["kc"], c["ks"], pages, past, False)
        _append_one(c["v"][t: t + new], c["vc"], c["vs"], pages, past, True)
        t += new
    return {"keys": c["kc"], "key scales": c["ks"], "values": c["vc"], "value scales": c["vs"]}


def _attention(c):
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    group = Hq // Hk
    out, lse, t = [], [], 0
    for (new, past), pages in zip(c["plan"], c["rows"]):
        n = new + past
        p = torch.tensor(pages[: _pages(n)], device=c["q"].device)
        k = (c["kc"][p].float() * c["ks"][p][:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :n]  # [Hk, n, D]
        v = (c["vc"][p].float() * c["vs"][p][:, :, None, None]).permute(1, 0, 3, 2).flatten(1, 2)[:, :n]
        q = c["q"][t: t + new].float().transpose(0, 1) * c["scale"]
        hidden = None
        if c["causal"]:
            ahead = torch.arange(n, device=q.device) - torch.arange(past, n, device=q.device)[:, None]
            hidden = ahead > 0
            if c["window"]:
                hidden |= ahead <= -c["window"]
        o, l = [], []  # noqa: E741
        step = max(1, (1 << 30) // (new * n * group))  # key heads at a time
        for h in range(0, Hk, step):
            kh, vh = k[h: h + step], v[h: h + step]
            s = torch.bmm(q[h * group: (h + step) * group].reshape(kh.shape[0], group * new, D), kh.mT.contiguous())
            s = s.view(-1, new, n)
            if hidden is not None:
                s.masked_fill_(hidden, -math.inf)
            top = s.amax(2, keepdim=True)
            e = s.sub_(top).exp_()
            total = e.sum(2, keepdim=True)
            o.append(torch.bmm(e.view(kh.shape[0], group * new, n), vh).view(-1, new, D) / total)
            l.append((top + total.log())[:, :, 0])
        out.append(torch.cat(o).transpose(0, 1))
        lse.append(torch.cat(l).t())
        t += new
    out = torch.cat(out).bfloat16()
    return {"o": out, "lse": torch.cat(lse).contiguous()} if c["lse"] else out


def run(state):
    c = state
    if own:
        from bit_quantized_linear_amd import binding as b

        if c["op"] == "norm":
            b.svdq_fp8_norm_quantize(c["X"], c["r"], c["w"], EPS, c["total"], c["Y"], c["qx"], c["sx"])
            out = {"codes": c["qx"], "scales": c["sx"], "sum": c["total"], "y": c["Y"]}
            return {n: t for n, t in out.items() if t is not None}
        if c["op"] == "rope":
            b.svdq_rope(c["X"], c["positions"], c["freqs"], c["sections"], c["Y"], interleaved=c["interleaved"])
            return c["Y"]
        if c["op"] == "append":
            b.svdq_kv8_append(c["k"], c["v"], c["starts"], c["lengths"], c["table"], c["kc"], c["ks"], c["vc"], c["vs"])
            return {"keys": c["kc"], "key scales": c["ks"], "values": c["vc"], "value scales": c["vs"]}
        b.svdq_kv8_attention(c["q"], c["kc"], c["ks"], c["vc"], c["vs"], c["starts"], c["lengths"], c["table"], c["scale"],
                             c["O"], c["L"], c["workspace"], causal=c["causal"], window=c["window"])
        return {"o": c["O"], "lse": c["L"]} if c["lse"] else c["O"]
    return {"norm": _norm, "rope": _rope, "append": _append, "attention": _attention}[c["op"]](c)


def work(case):
    """Each input read once, each output written once; of the cache, what some
    query sees, and the products of the pairs that are not masked."""
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        wide = 2 + (4 if case["residual"] else 0) + (2 if case["bf16"] else 0)
        return {"bytes": (wide + 1) * M * K + 2 * K + 4 * M * -(-K // BLOCK), "flops": 6 * M * K}
    if case["op"] == "rope":
        T, H, D, R = (case[n] for n in ("T", "H", "D", "R"))
        return {"bytes": 4 * T * H * D + 4 * T * len(case["sections"].split()) + 4 * R, "flops": 3 * T * H * R}
    Hk, D = case["Hk"], case["D"]
    plan = _plan(case)
    if case["op"] == "append":
        T = sum(new for new, _ in plan)
        return {"bytes": 6 * T * Hk * D + sum(16 * Hk * (_pages(n + p) - p // PAGE) for n, p in plan), "flops": 4 * T * Hk * D}
    Hq, T, seen, pairs = case["Hq"], 0, 0, 0
    for new, past in plan:
        n, w = new + past, case["window"]
        T += new
        if not case["causal"]:
            seen, pairs = seen + n, pairs + new * n
        elif not w:
            seen, pairs = seen + n, pairs + new * past + new * (new + 1) // 2
        else:
            seen += n - max(0, past + 1 - w)
            pairs += sum(min(w, past + 1 + i) for i in range(new))
    return {"bytes": 4 * T * Hq * D + 2 * seen * Hk * D + 8 * Hk * seen / PAGE + (4 * T * Hq if case["lse"] else 0),
            "flops": 4 * pairs * Hq * D}


# -------------------------------------------- the definition, in 64 bits --

def _values64(codes):
    """The numbers that E4M3 bytes stand for."""
    b = codes.view(torch.uint8).long()
    e, m = b >> 3 & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where(b >= 128, -v, v)


def _e4m3(v):
    """The E4M3 values nearest to v (64 bits, |v| < 464), ties to even."""
    step = torch.exp2(torch.frexp(v)[1].sub(1).clamp_min(-6).double() - 3)
    return torch.round(v / step) * step


def _norm64(c):
    h = c["X"].double() + (0 if c["r"] is None else c["r"].double())
    M, K = h.shape
    y = c["w"].double() * h / ((h * h).sum(1, keepdim=True) / K + EPS).sqrt()
    codes, scales = torch.empty_like(y), []
    for k in range(0, K, BLOCK):
        part = y[:, k: k + BLOCK]
        a = part.abs().max(1).values.clamp(min=TINY)
        codes[:, k: k + BLOCK] = _e4m3(part * (E4M3_MAX / a)[:, None])
        scales.append(a / E4M3_MAX)
    out = {"codes": codes, "scales": torch.stack(scales)}
    if c["r"] is not None:
        out["sum"] = h
    if c["bf16"]:
        out["y"] = y
    return out


def _rope64(c):
    y, R, j = c["X"].double(), c["R"], 0
    out = y.clone()
    for axis, n in enumerate(c["sections"]):
        for _ in range(n):
            a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + R // 2)
            z = torch.polar(torch.ones((), dtype=torch.float64, device=y.device).expand(y.shape[0]),
                            c["positions"][:, axis].double() * c["freqs"][j])[:, None]
            z = torch.complex(y[..., a], y[..., b]) * z
            out[..., a], out[..., b] = z.real, z.imag
            j += 1
    return out


def _append64(c):
    out, new_at = {}, 0
    kept = {"keys": (c["k"], c["kc"], c["ks"]), "values": (c["v"], c["vc"], c["vs"])}
    values = {n: _values64(t[1]) for n, t in kept.items()}
    values["values"] = values["values"].transpose(2, 3).contiguous()
    scales = {n: t[2].double() for n, t in kept.items()}
    for (new, past), pages in zip(c["plan"], c["rows"]):
        for name, (x, _, _) in kept.items():
            for g in range(past // PAGE, (past + new - 1) // PAGE + 1):
                low, high = max(past, g * PAGE), min(past + new, (g + 1) * PAGE)
                t = x[new_at + low - past: new_at + high - past].double().transpose(0, 1)  # [Hk, tokens, D]
                need = t.abs().amax((1, 2)).clamp(min=TINY)
                s = torch.exp2(torch.ceil(torch.log2(need / E4M3_MAX)))
                s = torch.where(s * E4M3_MAX < need, s * 2, s)
                s = torch.where(s * E4M3_MAX / 2 >= need, s / 2, s)
                page, head = values[name][pages[g]], scales[name][pages[g]]
                if low > g * PAGE:
                    s = torch.maximum(s, head)
                    page[:, : low - g * PAGE] = _e4m3(page[:, : low - g * PAGE] * (head / s)[:, None, None])
                page[:, low - g * PAGE: high - g * PAGE] = _e4m3(t / s[:, None, None])
                head.copy_(s)
        new_at += new
    out["keys"], out["key scales"] = values["keys"], scales["keys"]
    out["values"], out["value scales"] = values["values"].transpose(2, 3).contiguous(), scales["values"]
    return out


def _attention64(c):
    group, t = c["Hq"] // c["Hk"], 0
    o = torch.zeros(c["q"].shape, dtype=torch.float64, device=c["q"].device)
    lse = torch.zeros(c["q"].shape[:2], dtype=torch.float64, device=c["q"].device)
    for (new, past), pages in zip(c["plan"], c["rows"]):
        n = new + past
        p = torch.tensor(pages[: _pages(n)], device=o.device)
        at = torch.arange(n, device=o.device)
        query = torch.arange(past, n, device=o.device)[:, None]
        mask = torch.zeros((new, n), dtype=torch.float64, device=o.device)
        if c["causal"]:
            mask[at > query] = -math.inf
            if c["window"]:
                mask[at <= query - c["window"]] = -math.inf
        for h in range(c["Hq"]):
            k = _values64(c["kc"][p, h // group]) * c["ks"][p, h // group].double()[:, None, None]  # [pages, 64, D]
            v = _values64(c["vc"][p, h // group]) * c["vs"][p, h // group].double()[:, None, None]  # [pages, D, 64]
            s = c["scale"] * (c["q"][t: t + new, h].double() @ k.flatten(0, 1)[:n].t()) + mask
            lse[t: t + new, h] = torch.logsumexp(s, 1)
            o[t: t + new, h] = torch.softmax(s, 1) @ v.transpose(1, 2).flatten(0, 1)[:n]
        t += new
    return {"o": o, "lse": lse} if c["lse"] else o


def exact(case, seed):
    c = prepare(case, seed)
    return {"norm": _norm64, "rope": _rope64, "append": _append64, "attention": _attention64}[case["op"]](c)
