"""Plain 64-bit implementations of the paged-cache operators (torch, any
device), written row by row from their definitions, with the error that fp32
arithmetic and roundings may add to each value."""

import numpy as np
import torch

EPS = 1e-5


def path_to(parents, i):
    """Nodes from the root of node i's tree to node i."""
    path = []
    while i >= 0:
        path.append(int(i))
        i = int(parents[i])
    return path[::-1]


def chain(n):
    return np.arange(-1, n - 1, dtype=np.int32)


def random_tree(rng, n, forest=True):
    """parents of n nodes; several roots unless forest is False."""
    p = np.array([int(rng.integers(-1 if forest else 0, i)) if i else -1 for i in range(n)], np.int32)
    return p


def pack_trees(parents, B, N):
    out = np.full((B, N), -1, np.int32)
    for b, p in enumerate(parents):
        out[b, :len(p)] = p
    return out


def rows_of(pages, table_row, slots):
    """[h, len(slots), 64] rows of one sequence, float64."""
    page = pages.shape[2]
    slots = torch.as_tensor(slots, dtype=torch.long, device=pages.device)
    pg = table_row.to(pages.device).long()[slots // page]
    return pages[pg, :, slots % page].transpose(0, 1).double()


def bias64(prm, theta, d):
    """b_h(d) [H, *d.shape] in 64 bits; prm: alpha, beta, mu float64 [H]."""
    a, b, m = (x.view(-1, *([1] * d.dim())) for x in prm)
    d = d.double()[None]
    if theta:
        return -torch.exp(a) * ((d - 2 * torch.sinh(m)).abs() + EPS) ** b
    u = (d - m).abs()
    return -((torch.where(b <= 0, u.clamp(min=EPS), u) / a) ** b)


def tree_attention(q, k_pages, v_pages, table, lens, new, parents, prm, ssmax, theta, bf16_out):
    """(o, lse, o_err, lse_err) float64 [B, H, N, 64] / [B, H, N]; rows behind
    new[b] hold NaN.  parents: a list of arrays.

    The bounds: a logit z = c q.k + b is off by at most
      delta = 2^-18 c sum|q k| + 2^-20 |b| + 2^-20
    (64 fp32 additions of exact products at 2^-24 each of the sum of
    magnitudes; a few 1e-7 of |b|; exp2 to 2^-22 of the weight).  A relative
    change delta of the weights moves o by at most sum w delta |v| + (sum w
    delta) (sum w |v|), and the log of their sum by sum w delta.  Summing L
    weights in fp32 adds L 2^-24 relative, at most.  With bf16 output the
    weights are rounded to bf16 (half a step: 2^-8) and o is rounded once more
    (2^-8 |o|); with fp32 output they carry 24 bits (2^-22 covers the parts)."""
    B, H, N, D = q.shape
    Hkv = k_pages.shape[1]
    o = torch.full((B, H, N, D), float("nan"), dtype=torch.float64, device=q.device)
    lse, lerr, oerr = o[..., 0].clone(), o[..., 0].clone(), o.clone()
    prm = [x.double().to(q.device) for x in prm]
    for b in range(B):
        n, ln = int(new[b]), int(lens[b])
        for t in range(n):
            path = path_to(parents[b], t)
            depth = len(path) - 1
            slots = list(range(ln)) + [ln + i for i in path]
            k, v = (rows_of(x, table[b], slots).repeat_interleave(H // Hkv, 0)
                    for x in (k_pages, v_pages))
            L = len(slots)
            # the path's nodes sit at consecutive positions behind the committed keys
            bias = bias64(prm[:3], theta, L - 1 - torch.arange(L, device=q.device))
            c = torch.full((H, 1), 0.125, dtype=torch.float64, device=q.device)
            if ssmax:
                c = prm[3][:, None] * np.log(L) * 0.125
            qt = q[b, :, t].double()
            z = c * torch.einsum("hd,hld->hl", qt, k) + bias
            delta = 2.0 ** -18 * c.abs() * torch.einsum("hd,hld->hl", qt.abs(), k.abs()) \
                + 2.0 ** -20 * bias.abs() + 2.0 ** -20
            w = torch.softmax(z, 1)
            o[b, :, t] = torch.einsum("hl,hld->hd", w, v)
            lse[b, :, t] = torch.logsumexp(z, 1)
            mag = torch.einsum("hl,hld->hd", w, v.abs())
            wd = (w * delta).sum(1)
            e = torch.einsum("hl,hld->hd", w * delta, v.abs()) + wd[:, None] * mag \
                + (L * 2.0 ** -24 + 2.0 ** -22) * mag
            if bf16_out:
                e = e + 2.0 ** -8 * mag + 2.0 ** -8 * (o[b, :, t].abs() + e)
            else:
                e = e + 2.0 ** -24 * o[b, :, t].abs()
            oerr[b, :, t] = e
            lerr[b, :, t] = wd + L * 2.0 ** -24 + 2.0 ** -21 * (1 + lse[b, :, t].abs())
    return o, lse, oerr, lerr


def rotate(x, pos, base, dims, interleaved):
    """x float64 [..., 64] turned by position pos (an int)."""
    out = x.clone()
    for f in range(dims // 2):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + dims // 2)
        ang = pos * base ** (-2.0 * f / dims)
        c, s = np.cos(ang), np.sin(ang)
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., j] * c + x[..., i] * s
    return out
