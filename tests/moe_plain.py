"""Plain 64-bit forms of the operators around the exchange (CPU, numpy loops and
torch in float64), written from the definitions in include/a2av_moe.h."""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def step(dtype) -> float:
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def gmm(x, w, counts, index=None):
    """y, and the sums of magnitudes that rounding errors scale with."""
    x, w = x.double().cpu(), w.double().cpu()
    rows = x if index is None else x[index.cpu().long()]
    y = torch.zeros(rows.shape[0], w.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(y)
    at = 0
    for e, m in enumerate(counts.tolist()):
        y[at:at + m] = rows[at:at + m] @ w[e].T
        mag[at:at + m] = rows[at:at + m].abs() @ w[e].abs().T
        at += m
    return y[:at], mag[:at]


def gmm_dx(dy, w, counts):
    dy, w = dy.double().cpu(), w.double().cpu()
    dx = torch.zeros(dy.shape[0], w.shape[2], dtype=torch.float64)
    mag = torch.zeros_like(dx)
    at = 0
    for e, m in enumerate(counts.tolist()):
        dx[at:at + m] = dy[at:at + m] @ w[e]
        mag[at:at + m] = dy[at:at + m].abs() @ w[e].abs()
        at += m
    return dx[:at], mag[:at]


def gmm_dw(dy, x, counts, index=None):
    dy, x = dy.double().cpu(), x.double().cpu()
    rows = x if index is None else x[index.cpu().long()]
    dw = torch.zeros(counts.numel(), dy.shape[1], x.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(dw)
    at = 0
    for e, m in enumerate(counts.tolist()):
        dw[e] = dy[at:at + m].T @ rows[at:at + m]
        mag[e] = dy[at:at + m].abs().T @ rows[at:at + m].abs()
        at += m
    return dw, mag


def assert_sums(got, want, mag, terms: int):
    """Sums of ``terms`` products held in FP32, rounded once to got's dtype:
    one step per addition of the sum of magnitudes, half a step of the result
    (and, below the normal numbers, half of the smallest one)."""
    got = got.double().cpu()
    dt = assert_sums.dtype
    tol = (terms + 2) * 2.0 ** -23 * mag + step(dt) * want.abs()
    tol += torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    off = (got - want).abs()
    assert bool(torch.isfinite(got).all()), "values that are no numbers"
    worst = (off - tol).max().item() if off.numel() else 0.0
    assert worst <= 0, f"off by {off.max().item():g}, {worst:g} past the tolerance"


def check_sums(got, want, mag, terms: int):
    assert_sums.dtype = got.dtype
    assert_sums(got, want, mag, terms)


def route(logits: np.ndarray, k: int, renorm: bool):
    """experts, weights, counts, order, place of the definition, in float64."""
    T, E = logits.shape
    experts = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        # NaN above every number, the lowest number first among equals
        rank = sorted((e for e in range(E) if l[e] != -math.inf),
                      key=lambda e: (0, 0.0, e) if math.isnan(l[e]) else (1, -l[e], e))
        chosen = rank[:k]
        if not chosen:
            continue
        experts[t, :len(chosen)] = chosen
        top = l[chosen[0]]
        with np.errstate(invalid="ignore"):
            p = np.exp(l - top)
            p[l == -math.inf] = 0.0
            total = p[chosen].sum() if renorm else p.sum()
            weights[t, :len(chosen)] = p[chosen] / total
    counts = np.bincount(experts[experts >= 0], minlength=E).astype(np.int32)
    order = np.full(T * k, -1, np.int32)
    place = np.full(T * k, -1, np.int32)
    flat = experts.reshape(-1)
    at = 0
    for e in range(E):
        for s in np.nonzero(flat == e)[0]:
            order[at], place[s] = s // k, at
            at += 1
    return experts, weights, counts, order, place.reshape(T, k)


def route_back(logits, experts, weights, dweights, renorm: bool):
    l = logits.astype(np.float64)
    T, E = l.shape
    out = np.zeros((T, E))
    for t in range(T):
        g, q = np.zeros(E), np.zeros(E)
        mean = 0.0
        for j, e in enumerate(experts[t]):
            if e >= 0:
                g[e] = dweights[t, j]
                mean += float(weights[t, j]) * float(dweights[t, j])
                if renorm:
                    q[e] = weights[t, j]
        if not renorm:
            free = l[t] > -math.inf
            if free.any():
                p = np.where(free, np.exp(l[t] - l[t][free].max()), 0.0)
                q = p / p.sum()
        out[t] = q * (g - mean)
    return out


def mx4(x: np.ndarray):
    """codes (one per value), scale bytes and values (float64) of rows."""
    rows, cols = x.shape
    B = -(-cols // 32)
    full = np.zeros((rows, B * 32))
    full[:, :cols] = x
    codes = np.zeros((rows, B * 32), np.uint8)
    scales = np.zeros((rows, B), np.uint8)
    values = np.zeros((rows, B * 32))
    grid = np.array(E2M1)
    for r in range(rows):
        for b in range(B):
            v = full[r, b * 32:(b + 1) * 32]
            if not np.isfinite(v).all():
                scales[r, b] = 255
                values[r, b * 32:(b + 1) * 32] = math.nan
                continue
            top = np.abs(v).max()
            s = 0 if top == 0 else max(0, math.frexp(top)[1] - 1 - 2 + 127)
            scales[r, b] = s
            unit = math.ldexp(1.0, s - 127)
            a = np.minimum(np.abs(v) / unit, 6.0)
            d = np.abs(a[:, None] - grid[None, :])
            # The nearest, of two equally near the one with the even code.
            near = d.min(axis=1)
            first = d.argmin(axis=1)
            tie = (first + 1 < 8) & (d[np.arange(32), np.minimum(first + 1, 7)] == near)
            c = np.where(tie & (first % 2 == 1), first + 1, first)
            sign = np.signbit(v)
            codes[r, b * 32:(b + 1) * 32] = c + 8 * sign
            values[r, b * 32:(b + 1) * 32] = np.where(sign, -1, 1) * grid[c] * unit
    return codes, scales, values[:, :cols]


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def unpack_values(codes, scales, cols: int):
    """float64 values of packed codes [..., 16 B] and scales [..., B]."""
    c = torch.stack([codes.cpu() & 15, codes.cpu() >> 4], -1).flatten(-2).long()
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64)
    s = torch.tensor([math.nan if i == 255 else math.ldexp(1.0, i - 127) for i in range(256)],
                     dtype=torch.float64)
    return (table[c] * s[scales.cpu().long()].repeat_interleave(32, -1))[..., :cols]
