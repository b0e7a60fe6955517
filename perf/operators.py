"""The operators around an expert-parallel exchange, as measured cases.

Four operators: the top-k router (experts, weights, the gather list of the
exchange, and its gradient), the products grouped by expert with ragged sizes
(forward, both gradients), the weighted return of the experts' rows to their
tokens (and its gradients), and the microscaled 4-bit format (quantisation and
the grouped product on it).  ``own`` chooses between the plain form, written
with elementary torch operations in 32 bits, and this package's calls.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # A decode step of eight sequences: one router call, all latency.
        {"name": "route_decode", "op": "route", "tokens": 8, "experts": 64, "k": 2, "dtype": "bf16",
         "renorm": True, "padding": 0.0, "backward": False},
        # A training step's router: many experts, padding tokens, the gradient too.
        {"name": "route_train", "op": "route", "tokens": 32768, "experts": 256, "k": 8,
         "dtype": "fp32", "renorm": False, "padding": 0.01, "backward": True},
        # Sixteen tokens, top-2 of 8 experts: the weights are read for a few rows each.
        {"name": "gmm_decode", "op": "gmm", "tokens": 16, "k": 2, "experts": 8, "n": 2048,
         "kdim": 7168, "dtype": "bf16", "skew": 0.5, "backward": False},
        # A ragged prompt over 64 experts, some of them with no row at all.
        {"name": "gmm_prompt", "op": "gmm", "tokens": 2731, "k": 2, "experts": 64, "n": 2048,
         "kdim": 2048, "dtype": "fp16", "skew": 0.7, "backward": False},
        # A training step of one projection: forward, input and weight gradients.
        {"name": "gmm_train", "op": "gmm", "tokens": 8192, "k": 2, "experts": 16, "n": 2048,
         "kdim": 7168, "dtype": "bf16", "skew": 0.3, "backward": True},
        # Odd widths: rows that no vector load is aligned to, in every direction.
        {"name": "gmm_odd", "op": "gmm", "tokens": 513, "k": 3, "experts": 7, "n": 1001,
         "kdim": 523, "dtype": "fp16", "skew": 0.5, "backward": True},
        # The return of a decode step.
        {"name": "combine_decode", "op": "combine", "tokens": 16, "k": 2, "width": 7168,
         "dtype": "bf16", "dropped": 0.0, "backward": False},
        # The return of a training step and its gradients.
        {"name": "combine_train", "op": "combine", "tokens": 8192, "k": 8, "width": 7168,
         "dtype": "bf16", "dropped": 0.0, "backward": True},
        # Odd width, 32-bit rows, tokens whose slots were dropped.
        {"name": "combine_odd", "op": "combine", "tokens": 4099, "k": 3, "width": 1023,
         "dtype": "fp32", "dropped": 0.2, "backward": True},
        # Rows to 4 bits and back: what a dispatch in 4 bits does to its payload.
        {"name": "mx4_round_trip", "op": "mx4", "rows": 16384, "kdim": 7168, "dtype": "bf16"},
        # A decode step on 4-bit weights; the rows are quantised in the call.
        {"name": "gmm_mx4_decode", "op": "gmm_mx4", "tokens": 16, "k": 2, "experts": 8, "n": 2048,
         "kdim": 7168, "dtype": "bf16", "skew": 0.5},
        # A prompt on 4-bit weights.
        {"name": "gmm_mx4_prompt", "op": "gmm_mx4", "tokens": 8192, "k": 2, "experts": 16,
         "n": 2048, "kdim": 7168, "dtype": "bf16", "skew": 0.3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "gmm", "gmm", "combine", "mx4", "gmm_mx4"])
    if op == "route":
        experts = _log(rng, 4, 512)
        return {"op": op, "tokens": _log(rng, 1, 32768), "experts": experts,
                "k": rng.randint(1, min(8, experts)), "dtype": rng.choice(sorted(DT)),
                "renorm": rng.random() < 0.5, "padding": rng.choice([0.0, 0.05]),
                "backward": rng.random() < 0.5}
    if op == "combine":
        return {"op": op, "tokens": _log(rng, 1, 8192), "k": rng.randint(1, 8),
                "width": _log(rng, 16, 7168), "dtype": rng.choice(sorted(DT)),
                "dropped": rng.choice([0.0, 0.3]), "backward": rng.random() < 0.5}
    if op == "mx4":
        return {"op": op, "rows": _log(rng, 1, 16384), "kdim": _log(rng, 16, 7168),
                "dtype": rng.choice(sorted(DT))}
    experts = _log(rng, 1, 64)
    kdim, n = _log(rng, 32, 7168), _log(rng, 32, 4096)
    if rng.random() < 0.6:  # widths of models, against any width
        kdim, n = max(64, kdim // 64 * 64), max(64, n // 64 * 64)
    k = rng.randint(1, min(4, experts))
    tokens = _log(rng, 1, 16384 // k)
    # The weights stay under 1 GiB in 16 bits.
    experts = max(k, min(experts, (1 << 29) // (n * kdim)))
    case = {"op": op, "tokens": tokens, "k": k, "experts": experts, "n": n, "kdim": kdim,
            "dtype": rng.choice(["bf16", "fp16"]), "skew": round(rng.uniform(0.0, 1.0), 3)}
    if op == "gmm":
        case["backward"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ the inputs

def _choose(gen, dev, tokens, experts, k, skew):
    """k distinct experts for each token, some experts liked more than others."""
    bias = skew * torch.randn(experts, generator=gen, device=dev)
    score = torch.randn(tokens, experts, generator=gen, device=dev) + bias
    return score.sort(dim=1, descending=True, stable=True).indices[:, :k]


def _kept(case):
    return max(1, round(case["tokens"] * case["k"] * (1 - case["dropped"])))


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
        s.update(logits=logits, k=k, renorm=case["renorm"], backward=case["backward"])
        if case["backward"]:
            s["dweights"] = randn(T, k)
    elif case["op"] == "combine":
        T, k, H = case["tokens"], case["k"], case["width"]
        # The rows stand in an order by expert: a permutation of the slots kept.
        rank = torch.rand(T * k, generator=gen, device=dev).argsort()
        rows = _kept(case)
        place = torch.full((T * k,), -1, dtype=torch.int32, device=dev)
        place[rank[:rows]] = torch.arange(rows, dtype=torch.int32, device=dev)
        weights = torch.rand(T, k, generator=gen, device=dev) + 0.05
        s.update(y=randn(rows, H).to(dt), place=place.view(T, k),
                 weights=weights / weights.sum(1, keepdim=True), backward=case["backward"])
        if case["backward"]:
            s["dout"] = randn(T, H).to(dt)
    elif case["op"] == "mx4":
        # Rows of very different size, as activations have.
        s.update(x=(randn(case["rows"], case["kdim"]) * randn(case["rows"], 1).exp()).to(dt))
    else:
        T, k, E, N, K = (case[c] for c in ("tokens", "k", "experts", "n", "kdim"))
        chosen = _choose(gen, dev, T, E, k, case["skew"]).reshape(-1)
        counts = torch.bincount(chosen, minlength=E).to(torch.int32)
        index = (chosen.sort(stable=True).indices // k).to(torch.int32)
        s.update(x=randn(T, K).to(dt), index=index, counts=counts, most=int(counts.max()))
        if case["op"] == "gmm":
            s.update(w=(randn(E, N, K) / math.sqrt(K)).to(dt), backward=case["backward"])
            if case["backward"]:
                s["dy"] = randn(T * k, N).to(dt)
        else:
            # Weights as a checkpoint holds them: codes, two to a byte, and scales.
            blocks = -(-K // 32)
            codes = torch.randint(0, 256, (E, N, blocks * 16), generator=gen, device=dev,
                                  dtype=torch.uint8)
            if K % 32:  # the codes past the row's end are zero
                last = torch.arange(blocks * 32, device=dev) < K
                codes = codes & (last[0::2] * 15 + last[1::2] * 240).to(torch.uint8)
            # Steps of 2^-9 to 2^-6: the values of trained weights.
            scales = torch.randint(118, 122, (E, N, blocks), generator=gen, device=dev,
                                   dtype=torch.uint8)
            s.update(codes=codes, scales=scales)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from all_movement_amd import moe
    if s["op"] == "route":
        r = moe.route(s["logits"], s["k"], renormalize=s["renorm"])
        out = [r.experts, r.weights, r.counts, r.order, r.place]
        if s["backward"]:
            out.append(moe.route_backward(s["logits"], r.experts, r.weights, s["dweights"],
                                          renormalize=s["renorm"]))
        return out
    if s["op"] == "combine":
        out = [moe.combine(s["y"], s["place"], s["weights"])]
        if s["backward"]:
            out += moe.combine_backward(s["dout"], s["y"], s["place"], s["weights"])
        return out
    if s["op"] == "mx4":
        codes, scales = moe.mx4_quantize(s["x"])
        return [moe.mx4_dequantize(codes, scales, s["x"].shape[1], s["dt"])]
    if s["op"] == "gmm":
        out = [moe.gmm(s["x"], s["w"], s["counts"], index=s["index"])]
        if s["backward"]:
            out.append(moe.gmm_dx(s["dy"], s["w"], s["counts"]))
            out.append(moe.gmm_dw(s["dy"], s["x"], s["counts"], index=s["index"]))
        return out
    codes, scales = moe.mx4_quantize(s["x"])
    return [moe.gmm_mx4(codes, scales, s["codes"], s["scales"], s["counts"], index=s["index"],
                        dtype=s["dt"])]


def _run_plain(s):
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "combine":
        return _plain_combine(s)
    if s["op"] == "mx4":
        values, _ = _plain_mx4(s["x"].float())
        return [values.to(s["dt"])]
    if s["op"] == "gmm":
        return _plain_gmm(s)
    x, _ = _plain_mx4(s["x"].float())
    w = _plain_mx4_values(s["codes"], s["scales"], x.shape[1])
    e, slot = _plain_places(s)
    return [_plain_product(x[s["index"].long()], w, e, slot, s["most"]).to(s["dt"])]


def _plain_route(s):
    logits, k = s["logits"].float(), s["k"]
    T, E = logits.shape
    free = logits > float("-inf")
    top = logits.sort(dim=1, descending=True, stable=True)  # equal ones stay in order
    taken = top.values[:, :k] > float("-inf")
    experts = torch.where(taken, top.indices[:, :k], -1)
    most = torch.where(free[:, :1] | taken[:, :1], top.values[:, :1], 0.0)
    p = torch.exp(logits - most)
    picked = torch.where(taken, torch.exp(top.values[:, :k] - most), 0.0)
    total = (picked if s["renorm"] else p).sum(1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    weights = picked / total
    flat = torch.where(experts < 0, E, experts).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=logits.device)
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    by = flat.sort(stable=True)
    here = by.values < E
    order = torch.where(here, by.indices // k, -1).to(torch.int32)
    place = torch.empty(T * k, dtype=torch.int32, device=logits.device)
    place[by.indices] = torch.where(here, torch.arange(T * k, device=logits.device),
                                    -1).to(torch.int32)
    out = [experts.to(torch.int32), weights, counts[:E], order, place.view(T, k)]
    if s["backward"]:
        dw = torch.where(taken, s["dweights"], 0.0)
        mean = (weights * dw).sum(1, keepdim=True)
        d = torch.zeros(T, E + 1, device=logits.device)
        d.scatter_(1, flat.view(T, k), weights * dw)
        if s["renorm"]:
            w = torch.zeros(T, E + 1, device=logits.device)
            w.scatter_(1, flat.view(T, k), weights)
            d = d[:, :E] - w[:, :E] * mean
        else:
            d = d[:, :E] - (p / total) * mean
        out.append(d.to(s["dt"]))
    return out


def _plain_combine(s):
    place, w = s["place"].long(), s["weights"]
    here = place >= 0
    rows = s["y"][place.clamp(min=0)].float()
    w = torch.where(here, w, 0.0)
    out = [(rows * w[:, :, None]).sum(1).to(s["dt"])]
    if s["backward"]:
        dout = s["dout"].float()
        dy = torch.empty_like(s["y"])
        dy[place[here]] = (w[:, :, None] * dout[:, None, :]).to(s["dt"])[here]
        out += [dy, torch.where(here, (rows * dout[:, None, :]).sum(2), 0.0)]
    return out


def _plain_places(s):
    counts = s["counts"].long()
    e = torch.repeat_interleave(torch.arange(counts.numel(), device=counts.device), counts,
                                output_size=s["index"].numel())
    first = counts.cumsum(0) - counts
    return e, torch.arange(e.numel(), device=e.device) - first[e]


def _plain_product(rows, w, e, slot, most):
    """rows[r] @ w[e(r)]^T, each expert's rows filled up to the largest's."""
    padded = torch.zeros(w.shape[0], most, rows.shape[1], device=w.device)
    padded[e, slot] = rows
    return torch.bmm(padded, w.transpose(1, 2))[e, slot]


def _plain_gmm(s):
    e, slot = _plain_places(s)
    x, w = s["x"].float()[s["index"].long()], s["w"].float()
    out = [_plain_product(x, w, e, slot, s["most"]).to(s["dt"])]
    if s["backward"]:
        dy = torch.zeros(w.shape[0], s["most"], w.shape[1], device=w.device)
        dy[e, slot] = s["dy"].float()
        out.append(torch.bmm(dy, w)[e, slot].to(s["dt"]))
        padded = torch.zeros(w.shape[0], s["most"], w.shape[2], device=w.device)
        padded[e, slot] = x
        out.append(torch.bmm(dy.transpose(1, 2), padded).to(s["dt"]))
    return out


def _plain_mx4(x):
    """The values that blocks of 32 take in 4 bits, and their exponents."""
    rows, K = x.shape
    blocks = torch.nn.functional.pad(x, (0, -K % 32)).view(rows, -1, 32)
    exponent = torch.frexp(blocks.abs().amax(2)).exponent - 3
    exponent = torch.where(blocks.abs().amax(2) > 0, exponent, -127).clamp(-127, 127)
    up = ((127 - exponent) << 23).view(torch.float32)[:, :, None]
    a = blocks.abs() * up
    q = 0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
    q += (a > 2.5).float() + (a >= 3.5).float() + 2.0 * (a > 5.0).float()
    values = torch.copysign(q, blocks) / up
    return values.view(rows, -1)[:, :K], exponent


def _plain_mx4_values(codes, scales, K):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], dim=-1).int()
    step = (scales.int() << 23).view(torch.float32)
    values = table[both].view(*scales.shape, 32) * step[..., None]
    return values.flatten(2)[..., :K]


# ------------------------------------------------------------------ what a pass costs

def work(case):
    z = SIZE[case["dtype"]]
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        nbytes = T * E * z + T * k * 16 + E * 4
        flops = T * E * 3 + T * k * 2
        if case["backward"]:
            nbytes += T * E * z + T * k * 4
            flops += T * E * 4
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "combine":
        T, k, H = case["tokens"], case["k"], case["width"]
        rows = _kept(case)
        nbytes, flops = rows * H * z + T * H * z + T * k * 8, 2 * rows * H
        if case["backward"]:
            nbytes += rows * H * z + T * H * z + T * k * 4
            flops += 3 * rows * H
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "mx4":
        n = case["rows"] * case["kdim"]
        # in, to 4 bits and scales, and back out
        return {"bytes": 2 * n * z + 2 * (n // 2 + n // 32), "flops": 3 * n}
    T, k, E, N, K = (case[c] for c in ("tokens", "k", "experts", "n", "kdim"))
    R = T * k
    used = min(E, R)  # experts that can have a row
    if case["op"] == "gmm":
        nbytes, flops = T * K * z + used * N * K * z + R * N * z + R * 4 + E * 4, 2 * R * N * K
        if case["backward"]:
            nbytes += R * N * z + R * K * z + E * N * K * z
            flops *= 3
        return {"bytes": nbytes, "flops": flops}
    blocks = -(-K // 32)
    return {"bytes": T * K * z + used * N * blocks * 17 + R * N * z + R * 4 + E * 4,
            "flops": 2 * R * N * K + 3 * T * K}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "combine":
        T, k = s["place"].shape
        y, w = s["y"].double(), s["weights"].double()
        out = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device)
        dy, dw = torch.zeros_like(y), torch.zeros_like(w)
        for j in range(k):
            t = (s["place"][:, j] >= 0).nonzero().view(-1)
            r = s["place"][t, j].long()
            out[t] += w[t, j, None] * y[r]
            if s["backward"]:
                d = s["dout"][t].double()
                dy[r] = w[t, j, None] * d
                dw[t, j] = (d * y[r]).sum(1)
        return [out, dy, dw] if s["backward"] else [out]
    if case["op"] == "mx4":
        return [_exact_mx4(s["x"])]
    K = case["kdim"]
    if case["op"] == "gmm":
        x, w = s["x"].double(), s["w"]
    else:
        x, w = _exact_mx4(s["x"]), None
    rows = x[s["index"].long()]
    y = torch.zeros(rows.shape[0], case["n"], dtype=torch.float64, device=rows.device)
    dx = torch.zeros_like(rows)
    back = case.get("backward", False)
    dw = torch.zeros_like(w, dtype=torch.float64) if back else None
    at = 0
    for e, m in enumerate(s["counts"].tolist()):
        if m:
            if w is not None:
                we = w[e].double()
            else:
                c = torch.stack([s["codes"][e] % 16, s["codes"][e] // 16], -1).flatten(1).long()
                mag, sign = c % 8, 1 - 2 * (c // 8)
                small = mag.double() / 2  # below 2 the steps are halves
                large = (2 + mag % 2) * _two(mag // 2 - 2)
                step = _two(s["scales"][e].long() - 127).repeat_interleave(32, 1)
                we = (sign * torch.where(mag < 4, small, large) * step)[:, :K]
            part = slice(at, at + m)
            y[part] = rows[part] @ we.T
            if back:
                d = s["dy"][part].double()
                dx[part] = d @ we
                dw[e] = d.T @ rows[part]
        at += m
    return [y, dx, dw] if back else [y]


def _exact_route(case, s):
    x, k = s["logits"].double(), case["k"]
    T, E = x.shape
    used = (x != float("-inf")).any(1)
    safe = torch.where(used[:, None], x, 0.0)
    p = torch.softmax(safe, 1) * used[:, None]
    # By the value, equal ones by their number.
    at = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
    sel = torch.gather(p, 1, at) * (torch.gather(x, 1, at) != float("-inf"))
    q = sel / sel.sum(1, keepdim=True).clamp(min=1e-300) if case["renorm"] else sel
    out = [None, q, None, None, None]
    if case["backward"]:
        g = torch.zeros(T, E, dtype=torch.float64, device=x.device)
        g.scatter_(1, at, s["dweights"].double())
        if case["renorm"]:
            p = torch.zeros_like(p).scatter_(1, at, q)
        g = torch.where(p > 0, g, 0.0)
        out.append(p * (g * (torch.zeros_like(p).scatter_(1, at, 1.0))
                        - (q * torch.gather(g, 1, at)).sum(1, keepdim=True)))
    return out


def _two(e):
    """2^e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_mx4(x):
    x = x.double()
    rows, K = x.shape
    b = torch.nn.functional.pad(x, (0, -K % 32)).view(rows, -1, 32)
    top = b.abs().amax(2, keepdim=True)
    shared = (torch.frexp(top).exponent - 1 - 2).clamp(min=-127)
    unit = _two(shared)
    a = b.abs() / unit
    binade = (torch.frexp(a).exponent - 1).clamp(min=0)
    step = _two(binade - 1)
    q = (torch.round(a / step) * step).clamp(max=6.0) * unit * torch.sign(b)
    return torch.where(top > 0, q, 0.0).view(rows, -1)[:, :K]
