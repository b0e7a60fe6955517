"""A mixture-of-experts layer on one MI355X, from logits to gradients.

Two paths, as a program would run them:

``expert_parallel``  P virtual ranks with E / P experts each.  Every rank routes
    its tokens, the exchange gathers and delivers their rows, each rank
    multiplies what it received with its experts' weights, a second exchange
    brings the rows back, and the weighted return makes tokens of them.
``training_step``    one rank, forward and backward: the gradients of the tokens,
    of both weights and of the router's logits.

``python examples/moe_layer.py [--mx4]`` runs both, checks them against a dense
float64 layer and prints the errors.  With ``--mx4`` the products of the first
path run on 4-bit rows and weights, and the error is that of the format.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from all_movement_amd import a2av, moe  # noqa: E402


def silu(x):
    return torch.nn.functional.silu(x)


def products(rows, w, counts, index=None, mx4=False):
    """rows (gathered by ``index``) times the weight of their expert."""
    if not mx4:
        return moe.gmm(rows, w, counts, index=index, check=True)
    E, N, K = w.shape
    codes, scales = moe.mx4_quantize(w.view(E * N, K))  # a program keeps these
    B = scales.shape[1]
    return moe.gmm_mx4(*moe.mx4_quantize(rows), codes.view(E, N, 16 * B), scales.view(E, N, B),
                       counts, index=index, dtype=rows.dtype, check=True)


def expert_parallel(x, logits, w1, w2, k: int, mx4: bool = False):
    """x [P, T, H] bf16, logits [P, T, E], w1 [E, F, H], w2 [E, H, F]: the layer's
    output [P, T, H], rank by rank on one GPU."""
    P, T, H = x.shape
    E = logits.shape[2]
    local = E // P
    dev = x.device
    routes = [moe.route(logits[s], k) for s in range(P)]
    counts = torch.stack([r.counts for r in routes])            # [source, expert]
    to_rank = counts.view(P, P, local).sum(2, dtype=torch.int32)  # rows s -> d
    words = H // 2                                               # a bf16 row as 32-bit words

    # There: each source's gather list is its router's order.
    most = P * T * k                                             # rows a rank may receive
    there = a2av.Exchange(P, T * H * 2, most * H * 2, P)
    received = torch.empty(P, most, H, dtype=x.dtype, device=dev)
    signal = torch.zeros(P, P, dtype=torch.int32, device=dev)
    recv_counts = torch.empty(P, P, dtype=torch.int32, device=dev)
    there.run(x, received, signal, to_rank * words, recv_counts, P, a2av.FP32,
              index=torch.stack([r.order for r in routes]), row_elems=words, check=True)

    # A rank's rows stand by source and, of one source, by expert: its products
    # take them by expert, whatever the source.
    out_rows = torch.empty(P, most, H, dtype=x.dtype, device=dev)
    back_lists = torch.zeros(P, most, dtype=torch.int32, device=dev)
    for d in range(P):
        mine = counts[:, d * local:(d + 1) * local].contiguous()  # [source, expert of d]
        n = int(mine.sum())
        expert = torch.arange(local, device=dev).repeat(P).repeat_interleave(mine.view(-1).long())
        by_expert = expert.sort(stable=True).indices.to(torch.int32)
        per_expert = mine.sum(0, dtype=torch.int32)
        w = slice(d * local, (d + 1) * local)
        h = products(received[d, :max(n, 1)], w1[w], per_expert, by_expert, mx4)
        out_rows[d, :n] = products(silu(h), w2[w], per_expert, None, mx4)
        back_lists[d, by_expert.long()] = torch.arange(n, dtype=torch.int32, device=dev)

    # Back: the rows in the order they came, so that every source has its own in
    # its router's order again.
    back = a2av.Exchange(P, most * H * 2, T * k * H * 2, P)
    returned = torch.zeros(P, T * k, H, dtype=x.dtype, device=dev)
    back.run(out_rows, returned, signal, to_rank.t().contiguous() * words, recv_counts, P,
             a2av.FP32, index=back_lists, row_elems=words, check=True)
    there.close()
    back.close()
    return torch.stack([moe.combine(returned[s], r.place, r.weights, check=True)
                        for s, r in enumerate(routes)])


def training_step(x, logits, w1, w2, dout, k: int):
    """x [T, H], logits [T, E], dout [T, H]: (out, dx, dlogits, dw1, dw2)."""
    r = moe.route(logits, k, renormalize=False)
    h = moe.gmm(x, w1, r.counts, index=r.order)
    a = silu(h)
    y = moe.gmm(a, w2, r.counts)
    out = moe.combine(y, r.place, r.weights)

    dy, dweights = moe.combine_backward(dout, y, r.place, r.weights)
    dw2 = moe.gmm_dw(dy, a, r.counts)
    da = moe.gmm_dx(dy, w2, r.counts)
    s = torch.sigmoid(h.float())
    dh = (da.float() * (s * (1 + h.float() * (1 - s)))).to(h.dtype)
    dw1 = moe.gmm_dw(dh, x, r.counts, index=r.order)
    dx = moe.combine(moe.gmm_dx(dh, w1, r.counts), r.place)  # the gather's gradient
    dlogits = moe.route_backward(logits, r.experts, r.weights, dweights, renormalize=False)
    return out, dx, dlogits, dw1, dw2


def dense(x, logits, w1, w2, k: int, renormalize: bool):
    """The layer in float64 with autograd, every expert on every token."""
    p = torch.softmax(logits, -1)
    top = logits.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    chosen = torch.zeros_like(p).scatter(-1, top, 1.0)
    w = p * chosen
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    h = silu(torch.einsum("...h,efh->...ef", x, w1))
    return torch.einsum("...ef,ehf,...e->...h", h, w2, w)


def inputs(P: int, T: int, E: int, H: int, F: int, seed: int = 0, device="cuda:0"):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).to(torch.bfloat16).to(device)

    return (randn(P, T, H), randn(P, T, E).float(), randn(E, F, H, scale=H ** -0.5),
            randn(E, H, F, scale=F ** -0.5), randn(P, T, H))


def relative(a, b) -> float:
    return float((a.double().cpu() - b.cpu()).norm() / b.cpu().norm())


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--mx4", action="store_true")
    a = ap.parse_args()
    P, T, E, H, F, k = 4, 96, 8, 256, 512, 2
    x, logits, w1, w2, dout = inputs(P, T, E, H, F)
    out = expert_parallel(x, logits, w1, w2, k, a.mx4)
    wide = [t.double().cpu() for t in (x, logits, w1, w2)]
    print("expert parallel, %d ranks: relative error %.2g" % (P, relative(out, dense(*wide, k, True))))
    got = training_step(x[0], logits[0], w1, w2, dout[0], k)
    leaves = [t.clone().requires_grad_() for t in (wide[0][0], wide[1][0], wide[2], wide[3])]
    want = dense(*leaves, k, False)
    grads = torch.autograd.grad(want, leaves, dout[0].double().cpu())
    for name, g, w in zip(("out", "dx", "dlogits", "dw1", "dw2"), got, (want.detach(), *grads)):
        print("training step, %s: relative error %.2g" % (name, relative(g, w)))
    return 0


if __name__ == "__main__":
    sys.exit(main())
