"""Plain 64-bit implementations of the norms of queries and keys, of the decode
over a shared prefix and marked keys, and of eviction (torch, any device),
written from their definitions, with the error that fp32 arithmetic and
roundings may add to each value."""

import numpy as np
import torch

from _paged_reference import bias64, rows_of

BF16 = 2.0 ** -8  # half a step of bf16, relative


def turn(x, pos, base, dims, interleaved, back=False):
    """x float64 [..., T, 64] turned by positions pos [T] (or back)."""
    out = x.clone()
    pos = torch.as_tensor(pos, dtype=torch.float64, device=x.device)
    for f in range(dims // 2):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + dims // 2)
        ang = pos * base ** (-2.0 * f / dims)
        c, s = torch.cos(ang), torch.sin(ang) * (-1 if back else 1)
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., j] * c + x[..., i] * s
    return out


def _pair_size(x, dims, interleaved):
    """|x| of each value plus that of its pair's other one."""
    a = x.abs()
    if dims == 0:
        return a
    out = a.clone()
    h = dims // 2
    i = torch.arange(dims)
    j = (i ^ 1) if interleaved else (i + h) % dims
    out[..., :dims] = a[..., i] + a[..., j]
    return out


def norm_rotate(x, w, pos, eps, base, dims, interleaved):
    """(y, bound) of x float64 [h, T, 64], w float64 broadcastable, pos [T].

    fp32: the sum of 64 squares and the rsqrt err by 2^-20 relative, at most,
    sines and cosines by 2^-21, each product and sum by 2^-24; then one
    rounding to bf16."""
    n = w * x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = turn(n, pos, base, dims, interleaved)
    return y, 2.0 ** -18 * _pair_size(n, dims, interleaved) + BF16 * y.abs() + 1e-38


def norm_grads(x, g, w, pos, eps, base, dims, interleaved):
    """(dx, dx bound, terms of dw [h, T, 64]) for the output's gradient g."""
    rms = torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x / rms
    dn = turn(g, pos, base, dims, interleaved, back=True)
    size = _pair_size(g, dims, interleaved)
    u = w * dn
    dx = (u - n * (u * n).mean(-1, keepdim=True)) / rms
    mag = (w.abs() * size + n.abs() * (w.abs() * size * n.abs()).mean(-1, keepdim=True)) / rms
    return dx, 2.0 ** -17 * mag + BF16 * dx.abs() + 1e-38, dn * n, size * n.abs()


def decode(q, k_pages, v_pages, table, lens, prefix, P, key_pos, q_pos, prm, ssmax, theta, bf16_out):
    """(o, lse, weights, o_err, lse_err, w_err): o [B, H, 64]; weights and w_err a
    list of [len_b, Hkv], what this step adds to each own key's weight.

    The bounds are those of the tree's reference (_paged_reference.tree_attention):
    a logit is off by at most delta, a weight by its delta and the mean delta
    relative.  The weights enter the product with V with 24 bits (2^-22 covers the
    parts) for fp32 output, and for bf16 output with 16 bits (2^-16) or, over a
    prefix that more than 8 rows of a key head share, rounded to 8 (half a
    step: 2^-8)."""
    B, H, D = q.shape
    Hkv = k_pages.shape[1]
    G = H // Hkv
    dev = q.device
    o = torch.zeros(B, H, D, dtype=torch.float64, device=dev)
    oerr = torch.zeros_like(o)
    lse = torch.full((B, H), -float("inf"), dtype=torch.float64, device=dev)
    lerr = torch.zeros_like(lse)
    prm = [x.double().to(dev) for x in prm]
    weights, werr = [], []
    for b in range(B):
        n = int(lens[b])
        k, v = (rows_of(x, table[b], range(n)) for x in (k_pages, v_pages))
        pos = torch.arange(P, P + n, device=dev).expand(Hkv, n)
        at = P + n - 1
        if key_pos is not None:
            slots = torch.arange(n, device=dev)
            pos = key_pos[table[b].long()[slots // k_pages.shape[2]], :, slots % k_pages.shape[2]].T
            at = int(q_pos[b])
        if P:
            k, v = (torch.cat([rows_of(x, prefix, range(P)), y], 1)
                    for x, y in ((k_pages, k), (v_pages, v)))
            pos = torch.cat([torch.arange(P, device=dev).expand(Hkv, P), pos], 1)
        L = P + n
        if L == 0:
            weights.append(torch.zeros(0, Hkv, dtype=torch.float64, device=dev))
            werr.append(weights[-1])
            continue
        k, v, pos = (x.repeat_interleave(G, 0) for x in (k, v, pos))
        d = (at - pos).clamp(min=0)
        bias = torch.stack([bias64([p[h:h + 1] for p in prm[:3]], theta, d[h])[0] for h in range(H)])
        c = torch.full((H, 1), 0.125, dtype=torch.float64, device=dev)
        if ssmax:
            c = prm[3][:, None] * np.log(at + 1) * 0.125
        qt = q[b].double()
        z = c * torch.einsum("hd,hld->hl", qt, k) + bias
        delta = 2.0 ** -18 * c.abs() * torch.einsum("hd,hld->hl", qt.abs(), k.abs()) \
            + 2.0 ** -20 * bias.abs() + 2.0 ** -20
        w = torch.softmax(z, 1)
        o[b] = torch.einsum("hl,hld->hd", w, v)
        lse[b] = torch.logsumexp(z, 1)
        mag = torch.einsum("hl,hld->hd", w, v.abs())
        wd = (w * delta).sum(1)
        parts = (BF16 if P and B * G > 8 else 2.0 ** -16) if bf16_out else 2.0 ** -22
        e = torch.einsum("hl,hld->hd", w * delta, v.abs()) + wd[:, None] * mag \
            + (L * 2.0 ** -24 + parts) * mag
        oerr[b] = e + (BF16 if bf16_out else 2.0 ** -24) * (o[b].abs() + e) + 1e-38
        lerr[b] = wd + L * 2.0 ** -24 + 2.0 ** -21 * (1 + lse[b].abs())
        we = w * (delta + lerr[b][:, None] + 2.0 ** -21) + 2.0 ** -126
        weights.append(w.view(Hkv, G, L).sum(1)[:, P:].T)
        werr.append(we.view(Hkv, G, L).sum(1)[:, P:].T)
    return o, lse, weights, oerr, lerr, werr


def kept_slots(weights, budget, sink, recent):
    """Slots that stay of one sequence and key head; weights: numpy [len]."""
    n = len(weights)
    if n <= budget:
        return np.arange(n)
    middle = np.arange(sink, n - recent)
    w = weights[middle].astype(np.float64)
    w = np.where(np.isnan(w), np.inf, w)
    nan = np.isnan(weights[middle])
    order = np.lexsort((middle, -w, ~nan))[:budget - sink - recent]
    return np.sort(np.concatenate([np.arange(sink), middle[order], np.arange(n - recent, n)]))
