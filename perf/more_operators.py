"""Routing by groups and products in 8 bits, as measured cases.

Two operators of an expert-parallel layer and the format between them: the
router by groups (sigmoid or softmax scores, a bias that balances the load and
takes part in the choice only, experts of the best groups, renormalised and
scaled weights, and its gradient), 8-bit rows and weights (E4M3 codes with a
power-of-two scale for each block of 128 values of a row, or 128 x 128 of a
weight), and the products grouped by expert on them, forward and for the rows'
gradient.  ``own`` chooses between the plain form, written with elementary torch
operations, and this package's calls.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # A decode step of sixteen sequences: one router call, all latency.
        {"name": "route_groups_decode", "op": "route", "tokens": 16, "experts": 256, "k": 8,
         "groups": 8, "top_groups": 4, "group_best": 2, "scores": "sigmoid", "bias": True,
         "renorm": True, "scale": 2.5, "dtype": "fp32", "padding": 0.0, "backward": False},
        # A training step's router with its gradient and some padding tokens.
        {"name": "route_groups_train", "op": "route", "tokens": 32768, "experts": 256, "k": 8,
         "groups": 8, "top_groups": 4, "group_best": 2, "scores": "sigmoid", "bias": True,
         "renorm": True, "scale": 2.5, "dtype": "fp32", "padding": 0.01, "backward": True},
        # Softmax scores without a bias, groups of 20 experts by their best one, a ragged batch.
        {"name": "route_groups_softmax", "op": "route", "tokens": 4099, "experts": 160, "k": 6,
         "groups": 8, "top_groups": 3, "group_best": 1, "scores": "softmax", "bias": False,
         "renorm": False, "scale": 16.0, "dtype": "bf16", "padding": 0.0, "backward": True},
        # Rows to 8 bits and back: what a dispatch in 8 bits does to its payload.
        {"name": "fp8_rows", "op": "rows", "rows": 16384, "kdim": 7168, "dtype": "bf16"},
        # Rows that no vector load is aligned to, in 32 bits.
        {"name": "fp8_rows_odd", "op": "rows", "rows": 4099, "kdim": 1001, "dtype": "fp32"},
        # The weights of a projection, as a training step converts them after each update.
        {"name": "fp8_weights", "op": "weights", "experts": 16, "n": 2048, "kdim": 7168,
         "dtype": "bf16"},
        # Sixteen tokens, top-2 of 8 experts: the weights are read for a few rows each.
        {"name": "gmm_fp8_decode", "op": "gmm", "tokens": 16, "k": 2, "experts": 8, "n": 2048,
         "kdim": 7168, "dtype": "bf16", "skew": 0.5, "backward": False},
        # A batch of decodes: a dozen rows for each of many experts.
        {"name": "gmm_fp8_batch", "op": "gmm", "tokens": 192, "k": 4, "experts": 64, "n": 2048,
         "kdim": 2048, "dtype": "bf16", "skew": 0.5, "backward": False},
        # A ragged prompt over 64 experts, some of them with no row at all.
        {"name": "gmm_fp8_prompt", "op": "gmm", "tokens": 2731, "k": 2, "experts": 64, "n": 2048,
         "kdim": 2048, "dtype": "fp16", "skew": 0.7, "backward": False},
        # A training step of one projection: forward and the rows' gradient.
        {"name": "gmm_fp8_train", "op": "gmm", "tokens": 8192, "k": 2, "experts": 16, "n": 2048,
         "kdim": 7168, "dtype": "bf16", "skew": 0.3, "backward": True},
        # Widths that are no whole number of blocks, in both directions.
        {"name": "gmm_fp8_odd", "op": "gmm", "tokens": 513, "k": 3, "experts": 7, "n": 1001,
         "kdim": 523, "dtype": "fp16", "skew": 0.5, "backward": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "rows", "weights", "gmm", "gmm", "gmm"])
    if op == "route":
        groups = rng.choice([1, 2, 4, 4, 8, 8])
        size = _log(rng, 2, 64 if groups == 8 else 512 // groups)
        top_groups = rng.randint(1, groups)
        return {"op": op, "tokens": _log(rng, 1, 32768), "experts": groups * size,
                "k": rng.randint(1, min(8, top_groups * size)), "groups": groups,
                "top_groups": top_groups, "group_best": rng.choice([1, 2]),
                "scores": rng.choice(["sigmoid", "sigmoid", "softmax"]),
                "bias": rng.random() < 0.6, "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5, 16.0]), "dtype": rng.choice(sorted(DT)),
                "padding": rng.choice([0.0, 0.05]), "backward": rng.random() < 0.5}
    if op == "rows":
        return {"op": op, "rows": _log(rng, 1, 16384), "kdim": _log(rng, 16, 7168),
                "dtype": rng.choice(sorted(DT))}
    experts = _log(rng, 1, 64)
    kdim, n = _log(rng, 32, 7168), _log(rng, 32, 4096)
    if rng.random() < 0.6:  # widths of models, against any width
        kdim, n = max(64, kdim // 64 * 64), max(64, n // 64 * 64)
    if op == "weights":
        dtype = rng.choice(sorted(DT))
        experts = max(1, min(experts, (7 << 26) // (SIZE[dtype] * n * kdim)))
        return {"op": op, "experts": experts, "n": n, "kdim": kdim, "dtype": dtype}
    k = rng.randint(1, min(4, experts))
    # The weights stay under 2^28 values, the products under those of 16384 x 2048 x 7168.
    experts = max(k, min(experts, (1 << 28) // (n * kdim)))
    tokens = _log(rng, 1, min(16384, (7 << 35) // (n * kdim)) // k)
    return {"op": op, "tokens": tokens, "k": k, "experts": experts, "n": n,
            "kdim": kdim, "dtype": rng.choice(["bf16", "fp16"]),
            "skew": round(rng.uniform(0.0, 1.0), 3), "backward": rng.random() < 0.5}


# ------------------------------------------------------------------ the inputs

def _choose(gen, dev, tokens, experts, k, skew):
    """k distinct experts for each token, some experts liked more than others."""
    bias = skew * torch.randn(experts, generator=gen, device=dev)
    score = torch.randn(tokens, experts, generator=gen, device=dev) + bias
    return score.sort(dim=1, descending=True, stable=True).indices[:, :k]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"op": case["op"], "dt": dt}
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        logits = (1.5 * randn(T, E) + 0.5 * randn(E)).to(dt)
        if case["padding"]:
            pad = torch.rand(T, generator=gen, device=dev) < case["padding"]
            logits[pad] = float("-inf")
        bias = None
        if case["bias"]:  # sums of small steps up and down, as a balancing rule leaves them
            step = 0.001 if case["scores"] == "sigmoid" else 0.02 / E
            bias = (60 * randn(E)).round() * step
        s.update({c: case[c] for c in ("k", "groups", "top_groups", "group_best", "scores", "renorm",
                                       "scale", "backward")}, logits=logits, bias=bias)
        if case["backward"]:
            s["dweights"] = randn(T, k)
    elif case["op"] == "rows":
        # Rows of very different size, as activations have.
        s.update(x=(randn(case["rows"], case["kdim"]) * randn(case["rows"], 1).exp()).to(dt))
    elif case["op"] == "weights":
        E, N, K = (case[c] for c in ("experts", "n", "kdim"))
        w = torch.empty(E, N, K, dtype=dt, device=dev)
        for e in range(E):
            w[e] = randn(N, K) * randn(N, 1).exp() / math.sqrt(K)
        s.update(w=w)
    else:
        T, k, E, N, K = (case[c] for c in ("tokens", "k", "experts", "n", "kdim"))
        chosen = _choose(gen, dev, T, E, k, case["skew"]).reshape(-1)
        counts = torch.bincount(chosen, minlength=E).to(torch.int32)
        index = (chosen.sort(stable=True).indices // k).to(torch.int32)
        s.update(x=randn(T, K).to(dt), index=index, counts=counts, most=int(counts.max()), kdim=K,
                 backward=case["backward"])
        # Weights as a checkpoint holds them: codes and scales, zeros past a row's
        # end.  Their values are those of trained weights: about 1 / sqrt(K).
        B = -(-K // 128)
        codes = torch.zeros(E, N, B * 128, dtype=torch.float8_e4m3fn, device=dev)
        for e in range(E):
            codes[e, :, :K] = (96 * randn(N, K)).clamp(-448, 448).to(torch.float8_e4m3fn)
        mid = 127 - round(math.log2(96 * math.sqrt(K)))
        scales = torch.randint(mid - 1, mid + 2, (E, -(-N // 128), -(-B // 4) * 4), generator=gen,
                               device=dev, dtype=torch.uint8)
        scales[:, :, B:] = 0
        s.update(codes=codes, scales=scales)
        if case["backward"]:
            s["dy"] = randn(T * k, N).to(dt)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from all_movement_amd import moe
    if s["op"] == "route":
        r = moe.route_grouped(s["logits"], s["k"], scores=s["scores"], bias=s["bias"],
                              groups=s["groups"], top_groups=s["top_groups"],
                              group_best=s["group_best"], renormalize=s["renorm"],
                              scale=s["scale"])
        out = [r.experts, r.weights, r.counts, r.order, r.place]
        if s["backward"]:
            out.append(moe.route_grouped_backward(s["logits"], r.experts, r.weights, s["dweights"],
                                                  scores=s["scores"], renormalize=s["renorm"],
                                                  scale=s["scale"]))
        return out
    if s["op"] == "rows":
        codes, scales = moe.fp8_quantize(s["x"])
        return [moe.fp8_dequantize(codes, scales, s["x"].shape[1], s["dt"])]
    if s["op"] == "weights":
        codes, scales = moe.fp8_quantize_weights(s["w"])
        return [moe.fp8_dequantize_weights(codes, scales, s["w"].shape[2], s["dt"])]
    codes, scales = moe.fp8_quantize(s["x"])
    out = [moe.gmm_fp8(codes, scales, s["codes"], s["scales"], s["counts"], index=s["index"],
                       dtype=s["dt"])]
    if s["backward"]:
        codes, scales = moe.fp8_quantize(s["dy"])
        out.append(moe.gmm_fp8_dx(codes, scales, s["codes"], s["scales"], s["counts"],
                                  cols=s["kdim"], dtype=s["dt"]))
    return out


def _run_plain(s):
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "rows":
        return [_plain_fp8(s["x"].float(), 1).to(s["dt"])]
    if s["op"] == "weights":
        out = torch.empty_like(s["w"])
        for e in range(out.shape[0]):  # an expert at a time: in 32 bits it is twice as large
            out[e] = _plain_fp8(s["w"][e].float(), 128).to(s["dt"])
        return [out]
    counts = s["counts"].long()
    e = torch.repeat_interleave(torch.arange(counts.numel(), device=counts.device), counts,
                                output_size=s["index"].numel())
    slot = torch.arange(e.numel(), device=e.device) - (counts.cumsum(0) - counts)[e]
    w = s["codes"].float()[:, :, :s["kdim"]]
    step = _two32(s["scales"])
    step = step.repeat_interleave(128, 1)[:, :w.shape[1]]
    w = w * step.repeat_interleave(128, 2)[:, :, :s["kdim"]]
    rows = _plain_fp8(s["x"].float(), 1)[s["index"].long()]
    # Each expert's rows filled up to the largest's.
    padded = torch.zeros(w.shape[0], s["most"], rows.shape[1], device=w.device)
    padded[e, slot] = rows
    out = [torch.bmm(padded, w.transpose(1, 2))[e, slot].to(s["dt"])]
    if s["backward"]:
        padded = torch.zeros(w.shape[0], s["most"], w.shape[1], device=w.device)
        padded[e, slot] = _plain_fp8(s["dy"].float(), 1)
        out.append(torch.bmm(padded, w)[e, slot].to(s["dt"]))
    return out


def _two32(scales):
    """2^(s - 127) of scale bytes, in 32 bits."""
    s = scales.int()
    return torch.where(s > 0, s << 23, 1 << 22).view(torch.float32)


def _plain_fp8(x, tall):
    """The values that blocks of tall x 128 take in 8 bits."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x, (0, -cols % 128, 0, -rows % tall))
    b = b.view(b.shape[0] // tall, tall, -1, 128)
    top = b.abs().amax((1, 3), keepdim=True)
    # The least power of two that 448 times reaches the largest magnitude.
    field = ((top.view(torch.int32) + 0x1fffff) >> 23) - 8
    field = field.clamp(min=0)
    codes = (b * ((254 - field) << 23).view(torch.float32)).to(torch.float8_e4m3fn)
    values = codes.float() * _two32(field)
    return values.view(-1, values.shape[2] * 128)[:rows, :cols]


def _plain_route(s):
    """Scores and choice in 64 bits: near ones would change places in 32."""
    l, k, G = s["logits"].double(), s["k"], s["groups"]
    T, E = l.shape
    free = l > float("-inf")
    if s["scores"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        top = torch.where(free, l, -1e300).amax(1, keepdim=True)
        score = torch.where(free, torch.exp(l - top), 0.0)
        score = score / score.sum(1, keepdim=True).clamp(min=1e-300)
    c = score if s["bias"] is None else score + s["bias"].double()
    c = torch.where(free, c, float("-inf"))
    best = c.view(T, G, -1).sort(dim=2, descending=True).values[:, :, :s["group_best"]]
    some = best[:, :, :1] > float("-inf")
    best = torch.where(best > float("-inf"), best, 0.0).sum(2)
    best = torch.where(some[:, :, 0], best, float("-inf"))
    taken = best.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
    allowed = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, taken, True)
    allowed = allowed.repeat_interleave(E // G, 1)
    by = (l if s["bias"] is None else c).masked_fill(~(allowed & free), float("-inf"))
    chosen = by.sort(dim=1, descending=True, stable=True)
    here = chosen.values[:, :k] > float("-inf")
    experts = torch.where(here, chosen.indices[:, :k], -1)
    at = chosen.indices[:, :k]
    picked = torch.where(here, score.gather(1, at), 0.0)
    total = picked.sum(1, keepdim=True) if s["renorm"] else torch.ones_like(picked[:, :1])
    share = picked / torch.where(total > 0, total, 1.0)
    flat = torch.where(here, at, E).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=l.device)
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    by = flat.sort(stable=True)
    row = by.values < E
    order = torch.where(row, by.indices // k, -1).to(torch.int32)
    place = torch.empty(T * k, dtype=torch.int32, device=l.device)
    place[by.indices] = torch.where(row, torch.arange(T * k, device=l.device), -1).to(torch.int32)
    out = [experts.to(torch.int32), (s["scale"] * share).float(), counts[:E], order,
           place.view(T, k)]
    if s["backward"]:
        g = torch.where(here, s["scale"] * s["dweights"].double(), 0.0)
        if s["renorm"]:
            g = g - (share * g).sum(1, keepdim=True)
            g = torch.where(here, g, 0.0)
        d = torch.zeros(T, E + 1, dtype=torch.float64, device=l.device)
        if s["scores"] == "sigmoid":
            d.scatter_(1, flat.view(T, k), share * g / (1 + torch.exp(l.gather(1, at))))
            d = d[:, :E]
        elif s["renorm"]:
            d.scatter_(1, flat.view(T, k), share * g)
            d = d[:, :E]
        else:
            d.scatter_(1, flat.view(T, k), g)
            d = score * (d[:, :E] - (share * g).sum(1, keepdim=True))
        out.append(d.to(s["dt"]))
    return out


# ------------------------------------------------------------------ what a pass costs

def work(case):
    z = SIZE[case["dtype"]]
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        nbytes = T * E * z + T * k * 16 + E * 8
        flops = T * E * 6 + T * k * 4
        if case["backward"]:
            nbytes += T * E * z + T * k * 4
            flops += T * E + T * k * 6
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "rows":
        n, B = case["rows"] * case["kdim"], -(-case["kdim"] // 128)
        # in, to 8 bits and scales, and back out
        return {"bytes": 2 * n * z + 2 * (n + case["rows"] * B), "flops": 3 * n}
    E, N, K = (case[c] for c in ("experts", "n", "kdim"))
    if case["op"] == "weights":
        n = E * N * K
        return {"bytes": 2 * n * z + 2 * (n + n // 16384), "flops": 3 * n}
    T, R = case["tokens"], case["tokens"] * case["k"]
    used = min(E, R)  # experts that can have a row
    nbytes, flops = T * K * z + used * N * K + R * N * z + R * 4 + E * 4, 2 * R * N * K + 3 * T * K
    if case["backward"]:
        nbytes += R * N * z + R * K * z
        flops += 2 * R * N * K + 3 * R * N
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "rows":
        return [_exact_fp8(s["x"])]
    if case["op"] == "weights":
        return [torch.stack([_exact_fp8(w, 128) for w in s["w"]])]
    K, N = case["kdim"], case["n"]
    x = _exact_fp8(s["x"])[s["index"].long()]
    y = torch.zeros(x.shape[0], N, dtype=torch.float64, device=x.device)
    back = case["backward"]
    dy = _exact_fp8(s["dy"]) if back else None
    dx = torch.zeros_like(x)
    at = 0
    for e, m in enumerate(s["counts"].tolist()):
        if m:
            w = s["codes"][e, :, :K].double()
            step = torch.exp2(s["scales"][e].double() - 127)
            w *= step[torch.arange(N, device=w.device) // 128][
                :, torch.arange(K, device=w.device) // 128]
            y[at:at + m] = x[at:at + m] @ w.T
            if back:
                dx[at:at + m] = dy[at:at + m] @ w
        at += m
    return [y, dx] if back else [y]


def _exact_fp8(x, tall=1):
    """Each block's values over its unit, rounded to the nearest multiple of 2^-9
    and to three bits after the first, ties to even."""
    rows, cols = x.shape
    out = torch.empty(rows, cols, dtype=torch.float64, device=x.device)
    for r in range(0, rows, 4096):
        b = x[r:r + 4096].double()
        n = b.shape[0]
        b = torch.nn.functional.pad(b, (0, -cols % 128, 0, -n % tall)).view(
            -(-n // tall), tall, -1, 128)
        top = b.abs().amax((1, 3), keepdim=True)
        m, e = torch.frexp(top)  # top = m 2^e, m in [1/2, 1)
        e = (e - 9 + (m > 448 / 512).int()).clamp(min=-127)
        e = torch.where(top > 0, e, -127).double()
        a = b / torch.exp2(e)
        unit = torch.exp2((torch.frexp(a).exponent - 4).clamp(min=-9).double())
        q = torch.round(a / unit) * unit * torch.exp2(e)
        out[r:r + 4096] = q.reshape(-1, q.shape[2] * 128)[:n, :cols]
    return out


def _exact_route(case, s):
    x, k, G = s["logits"].double(), case["k"], case["groups"]
    T, E = x.shape
    used = x != float("-inf")
    if case["scores"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.softmax(torch.where(used.any(1, keepdim=True), x, 0.0), 1)
    p = p * used
    c = p + (0.0 if s["bias"] is None else s["bias"].double())
    none = torch.full_like(c, float("-inf"))
    c = torch.where(used, c, none)
    left, score = c.clone().view(T, G, E // G), torch.zeros(T, G, device=x.device).double()
    for j in range(min(case["group_best"], E // G)):
        most, at = left.max(2, keepdim=True)
        score += torch.where(most[:, :, 0] > float("-inf"), most[:, :, 0], 0.0)
        left = left.scatter(2, at, float("-inf"))
    score = torch.where(used.view(T, G, -1).any(2), score, float("-inf"))
    ok = torch.zeros(T, G, dtype=torch.bool, device=x.device)
    for j in range(case["top_groups"]):
        ok.scatter_(1, torch.where(ok, float("-inf"), score).argmax(1, keepdim=True), True)
    free = used & ok[:, :, None].expand(T, G, E // G).reshape(T, E)
    left = torch.where(free, x if s["bias"] is None else c, none)
    chosen = torch.zeros_like(x)
    w, g = torch.zeros(T, k, device=x.device).double(), torch.zeros_like(x)
    for j in range(k):
        most, _ = left.max(1, keepdim=True)
        at = left.argmax(1, keepdim=True)
        here = most > float("-inf")
        w[:, j:j + 1] = p.gather(1, at) * here
        chosen.scatter_add_(1, at, here.double())
        if case["backward"]:
            g.scatter_add_(1, at, s["dweights"][:, j:j + 1].double() * here)
        left = left.scatter(1, at, float("-inf"))
    total = w.sum(1, keepdim=True)
    scale = case["scale"] / torch.where(total > 0, total, 1.0) if case["renorm"] else case["scale"]
    out = [None, w * scale, None, None, None]
    if case["backward"]:
        # By the scores first, then by the logits.
        ds = scale * g
        if case["renorm"]:
            mean = (p * chosen * g).sum(1, keepdim=True) / torch.where(total > 0, total, 1.0)
            ds = scale * chosen * (g - mean)
        if case["scores"] == "sigmoid":
            out.append(ds * p * torch.sigmoid(-x))
        else:
            out.append(p * (ds - (p * ds).sum(1, keepdim=True)))
    return out
