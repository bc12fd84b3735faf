"""Benchmark cases of the paged-cache serving operators: the cache's writer, attention of a tree of
drafted tokens over the cache, and keeping an accepted path of the tree.

A serving step with drafted tokens runs the three in a row: the draft's keys and values are appended
behind each sequence's committed ones (``kv_append_paged``), every drafted token attends to the
committed keys and to its ancestors in the tree (``attention_decode_tree_paged``), and the keys and
values of the path that the model accepts are kept (``kv_keep_paged``).  Pages are bf16
[num_pages, Hkv, page, 64] with an int32 block table, as the paged decode reads them.

``run`` computes an operator from elementary torch operations in 32 bits, or, with ``own`` set, calls
the library.  ``exact`` is the definition in 64 bits, one sequence at a time.
"""

import math

import numpy as np
import torch

own = False

D = 64
EPS = 1e-5


def listed():
    append = dict(op="append", rot=64, pairs=False)
    tree = dict(op="tree", prior="alpha", ssmax=True, out="bf16", ragged=True)
    return [
        # One new token per sequence of a decode batch: latency is what counts.
        dict(append, name="append_token_B8_H12", B=8, H=12, Hkv=12, N=1, T=4096, page=64, tree=False),
        # The drafted trees of a large batch, written before they are verified; shared heads,
        # neighbouring dimensions rotated as pairs, half of them.
        dict(append, name="append_tree_B64_H32_Hkv8_N48", B=64, H=32, Hkv=8, N=48, T=2000, page=64,
             rot=32, pairs=True, tree=True),
        # Prompts of ragged length entering the cache after a prefill.
        dict(append, name="append_prompt_B8_H12_N8192", B=8, H=12, Hkv=12, N=8192, T=517, page=256,
             tree=False),
        # One short conversation with a few drafted tokens: the smallest call.
        dict(tree, name="tree_B1_H12_N7_T500", B=1, H=12, Hkv=12, N=7, T=500, page=64, tree=True),
        # An ordinary batch with small trees, fp32 output.
        dict(tree, name="tree_B8_H12_N16_T4096_fp32", B=8, H=12, Hkv=12, N=16, T=4096, page=64,
             tree=True, out="fp32"),
        # The long-context decode batch (32k tokens), now with a tree of 32 drafted tokens each.
        dict(tree, name="tree_B64_H12_N32_T32768", B=64, H=12, Hkv=12, N=32, T=32768, page=256,
             tree=True),
        # Heads that share keys and values, theta prior, no logit rescaling, odd sizes.
        dict(tree, name="tree_B13_H32_Hkv8_N21_T9001_theta", B=13, H=32, Hkv=8, N=21, T=9001, page=128,
             tree=True, prior="theta", ssmax=False),
        # A single very long sequence with a full tree: few heads, the key axis is all there is.
        dict(tree, name="tree_B1_H12_N64_T131072", B=1, H=12, Hkv=12, N=64, T=131072, page=256,
             tree=True),
        # Single tokens with shared heads: ordinary decoding through the same entry point.
        dict(tree, name="tree_token_B32_H32_Hkv8_N1_T16384", B=32, H=32, Hkv=8, N=1, T=16384, page=64,
             tree=False),
        # The widest call: a chain of 128 tokens (a chunk of a prompt) behind each sequence.
        dict(tree, name="tree_chain_B4_H12_N128_T20000", B=4, H=12, Hkv=12, N=128, T=20000, page=64,
             tree=False, ragged=False),
        # The accepted path of one sequence's tree, and of a batch's.
        dict(op="keep", name="keep_B1_H12_N32", B=1, H=12, Hkv=12, N=32, T=3000, page=64, tree=True),
        dict(op="keep", name="keep_B256_H32_Hkv8_N64", B=256, H=32, Hkv=8, N=64, T=1000, page=64,
             tree=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {"bytes": 0, "flops": 0}
    for c in listed():
        w = work(c)
        most = {k: max(most[k], w[k]) for k in most}
    while True:
        op = rng.choice(["append", "tree", "tree", "tree", "keep"])
        Hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
        H = Hkv * rng.choice([1, 1, 1, 2, 3, 4, 8])
        c = dict(op=op, B=_log_int(rng, 1, 256), H=H, Hkv=Hkv, page=rng.choice([64, 64, 128, 256, 320]),
                 T=_log_int(rng, 1, 131072), tree=rng.random() < 0.7)
        if op == "append":
            c["tree"] = c["tree"] and rng.random() < 0.6
            c["N"] = _log_int(rng, 1, 128 if c["tree"] else 16384)
            c["T"] = min(c["T"], 32768)
            c["rot"], c["pairs"] = rng.choice([0, 16, 32, 48, 64, 64, 64]), rng.random() < 0.4
        elif op == "tree":
            c["N"] = _log_int(rng, 1, 128)
            c["prior"] = rng.choice(["alpha", "alpha", "theta"])
            c["ssmax"], c["ragged"] = rng.random() < 0.6, rng.random() < 0.7
            c["out"] = rng.choice(["bf16", "bf16", "fp32"])
        else:
            c["N"], c["T"], c["tree"] = _log_int(rng, 1, 128), min(c["T"], 4096), True
        w = work(c)
        rows = c["B"] * H * c["N"] * (c["T"] + c["N"])  # logits that the plain form holds
        pool = c["B"] * Hkv * (c["T"] + c["N"]) * D * 4
        if (w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and rows <= 9e8
                and pool <= 4e9 and H <= 64):
            return c


# ---------------------------------------------------------------- inputs

def _numpy(case, seed):
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    key = [ord(ch) for ch in text]
    return np.random.default_rng([seed % (1 << 31)] + key)


def _lengths(case, rng):
    """Committed lengths and new tokens of each sequence: ragged, the longest length among them."""
    B, N, T = case["B"], case["N"], case["T"]
    if case["op"] == "tree" and not case["ragged"]:
        lens, new = np.full(B, T), np.full(B, N)
    else:
        lens, new = rng.integers(0, T + 1, B), rng.integers((N + 1) // 2, N + 1, B)
        lens[rng.integers(0, B)], new[rng.integers(0, B)] = T, N
    return lens.astype(np.int32), new.astype(np.int32)


def _trees(case, new, rng):
    """parents [B, N]: level by level, as a drafter that keeps its best candidates builds them; the
    first level is the widest.  Entries past a sequence's nodes are -1."""
    B, N = case["B"], case["N"]
    parents = np.full((B, N), -1, np.int32)
    for b in range(B):
        n = int(new[b])
        first, lo = max(1, min(n, int(math.ceil(math.sqrt(2 * n))))), 0
        hi = at = first
        while at < n:
            width = max(1, min(n - at, int(rng.integers(1, first + 1))))
            parents[b, at:at + width] = np.sort(rng.integers(lo, hi, width))
            lo, hi, at = at, at + width, at + width
    return parents


def _depths(parents):
    depth = np.zeros_like(parents)
    for i in range(parents.shape[1]):
        p = parents[:, i]
        depth[:, i] = np.where(p >= 0, np.take_along_axis(depth, np.maximum(p, 0)[:, None], 1)[:, 0] + 1, 0)
    return depth


def prepare(case, seed):
    rng = _numpy(case, seed)
    B, H, Hkv, N, T, page = (case[k] for k in ("B", "H", "Hkv", "N", "T", "page"))
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(rng.integers(1 << 62)))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

    lens, new = _lengths(case, rng)
    blocks = -(-(lens.astype(np.int64) + new) // page)
    max_blocks = -(-(T + N) // page)
    num_pages = B * max_blocks  # room for every sequence at its longest
    perm = rng.permutation(num_pages)[:int(blocks.sum())].astype(np.int32)
    table = np.full((B, max_blocks), -1, np.int32)
    table[np.arange(max_blocks)[None, :] < blocks[:, None]] = perm
    parents = _trees(case, new, rng) if case["tree"] else None
    st = {"case": dict(case), "k_pages": normal(num_pages, Hkv, page, D),
          "v_pages": normal(num_pages, Hkv, page, D),
          "table": torch.from_numpy(table).to(dev), "lens": torch.from_numpy(lens).to(dev),
          "new": torch.from_numpy(new).to(dev),
          "parents": None if parents is None else torch.from_numpy(parents).to(dev), "kept": {}}
    if case["op"] == "append":
        # One projection's output holds a token's queries, keys and values side by side.
        qkv = normal(B, N, H + 2 * Hkv, D)
        st["q"], st["k"], st["v"] = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
        st["q_out"] = torch.zeros(B, H, N, D, dtype=torch.bfloat16, device=dev)
    elif case["op"] == "tree":
        st["q"] = normal(B, H, N, D)
        if case["prior"] == "alpha":
            prm = [np.exp(rng.uniform(0, np.log(1e3), H)), rng.uniform(-1, 2, H),
                   rng.uniform(0, 8, H) * (rng.random(H) < 0.5)]
        else:
            prm = [rng.uniform(-3, 1, H), rng.uniform(-1, 2, H), rng.uniform(-1, 1, H)]
        prm.append(rng.uniform(0.3, 1.0, H))
        st["prm"] = [torch.from_numpy(x.astype(np.float32)).to(dev) for x in prm]
        st["o"] = torch.zeros(B, H, N, D, device=dev,
                              dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
        st["lse"] = torch.zeros(B, H, N, device=dev)
    else:
        # Where the first level holds at least as many nodes as the path, a kept slot is never the
        # source of a later one, so that a pass can be repeated on the same pages.
        depth = _depths(parents)
        accepted = np.full(B, -1, np.int32)
        for b in range(B):
            n = int(new[b])
            first = int((depth[b, :n] == 0).sum())
            good = [i for i in range(n) if depth[b, i] < first and _path(parents[b], i)[0] in
                    [0] + list(range(depth[b, i] + 1, first))]
            if rng.random() < 0.9 and good:
                accepted[b] = good[int(rng.integers(0, len(good)))]
        st["accepted"] = torch.from_numpy(accepted).to(dev)
        st["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return st


def _path(parents, i):
    path = []
    while i >= 0:
        path.append(int(i))
        i = parents[i]
    return path[::-1]


# ---------------------------------------------------------------- plain forms

def _ancestors(st):
    """(seen [B, N, N]: node j is node t or an ancestor of it; depth [B, N]), from the parents."""
    case = st["case"]
    B, N = case["B"], case["N"]
    dev = st["lens"].device
    if st["parents"] is None:
        seen = torch.ones(N, N, dtype=torch.bool, device=dev).tril().expand(B, N, N)
    else:
        step = torch.zeros(B, N, N + 1, device=dev)
        step.scatter_(2, torch.where(st["parents"] < 0, N, st["parents"]).long()[:, :, None], 1.0)
        reach = (torch.eye(N, device=dev) + step[:, :, :N]).clamp(max=1)
        # each product doubles the length of the chains that are followed: 2^7 covers 128 nodes
        for _ in range(7):
            reach = torch.matmul(reach, reach).clamp(max=1)
        seen = reach > 0
    return seen, seen.sum(2) - 1


def _slots(st, slot):
    """(page number, row in the page) of slots [B, n] of each sequence."""
    page = st["case"]["page"]
    block = torch.div(slot, page, rounding_mode="floor").clamp(max=st["table"].shape[1] - 1)
    return st["table"].long().gather(1, block), slot % page


def _rotate(x, pos, rot, pairs):
    """x [B, h, N, 64] in 32 bits, its first `rot` dimensions rotated by their positions pos [B, N]."""
    if rot == 0:
        return x
    f = torch.arange(rot // 2, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None, :, None] * torch.pow(10000.0, -2.0 * f / rot)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if pairs:
        out[..., 0:rot:2], out[..., 1:rot:2] = ra, rb
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = ra, rb
    return out


def _plain_append(st):
    case = st["case"]
    N = case["N"]
    i = torch.arange(N, device=st["lens"].device)
    depth = _ancestors(st)[1] if case["tree"] else i[None].expand(case["B"], N)
    pos = st["lens"][:, None].long() + depth
    valid = i[None] < st["new"][:, None]
    pg, row = _slots(st, st["lens"][:, None].long() + i)
    k = _rotate(st["k"].float(), pos, case["rot"], case["pairs"]).to(torch.bfloat16)
    q = _rotate(st["q"].float(), pos, case["rot"], case["pairs"]).to(torch.bfloat16)
    st["k_pages"][pg[valid], :, row[valid]] = k.transpose(1, 2)[valid]
    st["v_pages"][pg[valid], :, row[valid]] = st["v"].transpose(1, 2)[valid]
    torch.where(valid[:, None, :, None], q, st["q_out"], out=st["q_out"])
    return st["k_pages"], st["v_pages"], st["q_out"]


def _bias_table(case, prm, n, dtype):
    """b_h(d) for d = 0 .. n-1, evaluated in 64 bits."""
    a, b, m = (x.double()[:, None] for x in prm[:3])
    d = torch.arange(n, device=a.device, dtype=torch.float64)[None]
    if case["prior"] == "theta":
        bias = -torch.exp(a) * ((d - (torch.exp(m) - torch.exp(-m))).abs() + EPS) ** b
    else:
        u = (d - m).abs()
        bias = -((torch.where(b <= 0, u.clamp(min=EPS), u) / a) ** b)
    return bias.to(dtype)


def _plain_tree(st):
    case = st["case"]
    B, H, Hkv, N, page = (case[k] for k in ("B", "H", "Hkv", "N", "page"))
    dev = st["lens"].device
    G, L = H // Hkv, st["table"].shape[1] * page
    lens, new = st["lens"].long(), st["new"].long()
    seen, depth = _ancestors(st)
    j = torch.arange(L, device=dev)
    node = j[None] - lens[:, None]                                   # [B, L]: which node a key is
    at = node.clamp(0, N - 1)
    pos_k = torch.where(node < 0, j[None], lens[:, None] + depth.gather(1, at))
    dist = lens[:, None, None] + depth[:, :, None] - pos_k[:, None]    # [B, N, L]
    vis = (node < 0)[:, None] | (seen.gather(2, at[:, None].expand(B, N, L)) & (node < new[:, None])[:, None])
    pages = st["table"].long().clamp(min=0)
    # a page that no key of the sequence lies in holds other sequences' rows: masked like any other
    keys, values = (p[pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float() for p in (st["k_pages"], st["v_pages"]))
    q = st["q"].float().view(B, Hkv, G * N, D)
    z = torch.matmul(q, keys.transpose(2, 3)).view(B, H, N, L)
    if case["ssmax"]:
        c = st["prm"][3][None, :, None] * torch.log((lens[:, None] + depth + 1).float())[:, None] / 8
        z *= c[..., None]
    else:
        z *= 0.125
    bias = _bias_table(case, st["prm"], L + N, torch.float32)
    z += bias[:, dist.clamp(min=0)].transpose(0, 1)
    z.masked_fill_(~vis[:, None], -math.inf)
    m = z.amax(3, keepdim=True)
    z -= m
    p = z.exp_()
    s = p.sum(3, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * N, L), values).view(B, H, N, D) / s
    live = (torch.arange(N, device=dev)[None] < new[:, None])[:, None, :]
    torch.where(live[..., None], o.to(st["o"].dtype), st["o"], out=st["o"])
    torch.where(live, (m + s.log())[..., 0], st["lse"], out=st["lse"])
    return st["o"], st["lse"]


def _plain_keep(st):
    case = st["case"]
    N = case["N"]
    dev = st["lens"].device
    seen, depth = _ancestors(st)
    acc = st["accepted"].long()
    none = acc < 0
    at = acc.clamp(min=0)[:, None]
    on = seen.gather(1, at[..., None].expand(-1, 1, N))[:, 0] & ~none[:, None]      # [B, N]: on the path
    src_pg, src_row = _slots(st, st["lens"].long()[:, None] + torch.arange(N, device=dev))
    dst_pg, dst_row = _slots(st, st["lens"].long()[:, None] + depth)
    for pages in (st["k_pages"], st["v_pages"]):
        pages[dst_pg[on], :, dst_row[on]] = pages[src_pg[on], :, src_row[on]]
    st["new_lens"].copy_(torch.where(none, st["lens"], st["lens"] + depth.gather(1, at)[:, 0] + 1))
    return st["k_pages"], st["v_pages"], st["new_lens"]


def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        return {"append": _plain_append, "tree": _plain_tree, "keep": _plain_keep}[op](state)

    from transformer_attention_ggd_gb300 import bam_attn as ba

    kept = state["kept"]  # the workspace, rotation and parameters that a program keeps
    cache = state["k_pages"], state["v_pages"], state["table"], state["lens"]
    if op == "append":
        if not kept:
            kept.update(ws=ba.cache_workspace(), rope=ba.make_rope(10000.0, case["rot"], case["pairs"]))
        ba.bam_kv_append_paged(state["k"], state["v"], *cache, state["new"], state["parents"],
                               state["q"], state["q_out"], kept["rope"], kept["ws"])
        return state["k_pages"], state["v_pages"], state["q_out"]
    if op == "tree":
        if not kept:
            prior = ba.BAM_PRIOR_THETA if case["prior"] == "theta" else ba.BAM_PRIOR_ALPHA
            kept.update(ws=ba.tree_workspace(case["B"], case["H"], case["Hkv"], case["N"],
                                             state["table"].shape[1] * case["page"]),
                        prm=ba.make_params(*state["prm"], EPS, True, case["ssmax"], prior))
        ba.bam_attn_decode_tree_paged(state["q"], *cache, state["new"], state["parents"], state["o"],
                                      state["lse"], kept["prm"], kept["ws"])
        return state["o"], state["lse"]
    if not kept:
        kept.update(ws=ba.cache_workspace())
    ba.bam_kv_keep_paged(*cache, state["new"], state["parents"], state["accepted"], state["new_lens"],
                         kept["ws"])
    return state["k_pages"], state["v_pages"], state["new_lens"]


def work(case):
    """Expected work over the ragged lengths: one sequence has the longest length and one the most new
    tokens, the others average half and three quarters of those."""
    B, H, Hkv, N, T = (case[k] for k in ("B", "H", "Hkv", "N", "T"))
    whole = case["op"] == "tree" and not case["ragged"]
    t, n = (T, N) if whole else ((T + (B - 1) * T / 2) / B, (N + (B - 1) * (N + (N + 1) // 2) / 2) / B)
    if case["op"] == "append":
        tokens = B * n
        return {"bytes": int(tokens * 4 * D * (2 * Hkv + H)), "flops": int(tokens * 3 * case["rot"] * (Hkv + H))}
    if case["op"] == "tree":
        size = 4 if case["out"] == "fp32" else 2
        io = B * n * H * (2 * D + size * D + 4)
        return {"bytes": int(B * Hkv * (t + n) * 4 * D + io), "flops": int(4 * D * B * H * n * (t + n / 2))}
    path = max(1.0, math.log2(1 + n) / 2)
    return {"bytes": int(B * Hkv * path * 8 * D), "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    B, H, Hkv, N, page = (case[k] for k in ("B", "H", "Hkv", "N", "page"))
    if case["op"] == "tree" and B * H * N * float(case["T"]) > 1e9:
        return None
    lens, new, table = st["lens"].tolist(), st["new"].tolist(), st["table"].cpu().numpy()
    if st["parents"] is None:
        parents = np.tile(np.arange(-1, N - 1), (B, 1))
    else:
        parents = st["parents"].cpu().numpy()

    def rows(b, slots):
        """Flat rows [Hkv, len(slots)] of the pages viewed as [num_pages * Hkv * page, 64]."""
        slots = np.asarray(slots, np.int64)
        pg = table[b, slots // page].astype(np.int64)
        return torch.from_numpy((pg[None] * Hkv + np.arange(Hkv)[:, None]) * page + slots[None] % page).cuda()

    if case["op"] == "append":
        kp, vp = (st[x].double() for x in ("k_pages", "v_pages"))
        qo = st["q_out"].double()
        half = case["rot"] // 2
        first = np.arange(half) * 2 if case["pairs"] else np.arange(half)
        second = first + 1 if case["pairs"] else first + half
        for b in range(B):
            n = new[b]
            depth = _depths(parents[b:b + 1, :n])[0] if case["tree"] else np.arange(n)
            turn = torch.eye(D, dtype=torch.float64, device="cuda").repeat(n, 1, 1)
            for f in range(half):
                ang = torch.from_numpy((lens[b] + depth).astype(np.float64)).cuda() * 10000.0 ** (-f / half)
                i, k = int(first[f]), int(second[f])
                turn[:, i, i], turn[:, i, k] = ang.cos(), -ang.sin()
                turn[:, k, i], turn[:, k, k] = ang.sin(), ang.cos()
            at = rows(b, lens[b] + np.arange(n))
            kp.view(-1, D)[at] = torch.einsum("nij,hnj->hni", turn, st["k"][b, :, :n].double())
            vp.view(-1, D)[at] = st["v"][b, :, :n].double()
            qo[b, :, :n] = torch.einsum("nij,hnj->hni", turn, st["q"][b, :, :n].double())
        return kp, vp, qo

    if case["op"] == "tree":
        o, lse = st["o"].double(), st["lse"].double()
        for b in range(B):
            n, ln = new[b], lens[b]
            paths = [_path(parents[b], i) for i in range(n)]
            depth = np.array([len(p) - 1 for p in paths])
            pos_k = np.concatenate([np.arange(ln), ln + depth])
            vis = np.ones((n, ln + n), bool)
            vis[:, ln:] = False
            for t, p in enumerate(paths):
                vis[t, ln + np.array(p)] = True
            dist = torch.from_numpy(np.abs(ln + depth[:, None] - pos_k[None])).cuda()
            vis = torch.from_numpy(vis).cuda()
            at = rows(b, np.arange(ln + n))
            bias = _bias_table(case, st["prm"], ln + n + 1, torch.float64)
            scale = torch.full((H, n), 1.0, dtype=torch.float64, device="cuda")
            if case["ssmax"]:
                scale = st["prm"][3].double()[:, None] * torch.from_numpy(np.log(ln + depth + 1.0)).cuda()
            for g in range(Hkv):
                hs = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
                k, v = (st[x].view(-1, D)[at[g]].double() for x in ("k_pages", "v_pages"))
                z = st["q"][b, hs, :n].double() @ k.T * (scale[hs, :, None] / math.sqrt(D)) + bias[hs][:, dist]
                z = torch.where(vis, z, -math.inf)
                lse[b, hs, :n] = torch.logsumexp(z, 2)
                o[b, hs, :n] = torch.softmax(z, 2) @ v
        return o, lse

    kp, vp = (st[x].clone() for x in ("k_pages", "v_pages"))
    kept = []
    for b, a in enumerate(st["accepted"].tolist()):
        path = _path(parents[b], a)
        kept.append(lens[b] + len(path))
        if path:
            src, dst = rows(b, lens[b] + np.array(path)), rows(b, lens[b] + np.arange(len(path)))
            for x, old in ((kp, st["k_pages"]), (vp, st["v_pages"])):
                x.view(-1, D)[dst] = old.view(-1, D)[src]
    return kp.double(), vp.double(), torch.tensor(kept, dtype=torch.int32).cuda()
