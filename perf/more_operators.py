"""Benchmark cases of the operators around a long, bounded cache: norms of queries and keys with their
rotation, decode over a prefix that a whole batch shares and over keys that carry positions and
accumulated weights, and eviction by those weights.

Training: the queries and keys of every head are normalised and rotated in one pass before the
attention, and its gradients go back the same way (``qk_norm``).  Serving: new tokens enter the paged
cache through the same norm and rotation (``append``), each decoding step attends to the shared prefix,
read once for the whole batch, and to the sequence's own keys, adding each key's attention weight to
what it has gathered so far (``decode``), and when the cache is full the keys that gathered least leave
it (``evict``).  Pages are bf16 [num_pages, Hkv, page, 64] with an int32 block table; a key's position
and weight lie in int32 and fp32 pages [num_pages, Hkv, page] beside it.

``run`` computes an operator from elementary torch operations in 32 bits, or, with ``own`` set, calls
the library.  ``exact`` is the definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

D = 64
EPS = 1e-5        # of the prior
NORM_EPS = 1e-6   # of the norms
BASE = 10000.0


def listed():
    norm = dict(op="qk_norm", rot=64, pairs=False, per_head=False, packed=False)
    append = dict(op="append", rot=64, pairs=False, per_head=False, marked=True)
    decode = dict(op="decode", prior="alpha", ssmax=True, out="bf16", P=0, marked=False)
    return [
        # The training step's shape: 8 sequences of 512 tokens, 12 heads.
        dict(norm, name="qk_norm_train_B8_H12_T512", B=8, H=12, Hkv=12, T=512),
        # Long training sequences of odd length, shared key heads, weights of each head, half of the
        # dimensions turned as neighbouring pairs, several documents packed into a row.
        dict(norm, name="qk_norm_train_B4_H32_Hkv8_T16383", B=4, H=32, Hkv=8, T=16383, rot=32,
             pairs=True, per_head=True, packed=True),
        # One new token for each sequence of a decode batch: latency is what counts.
        dict(append, name="append_norm_token_B64_H32_Hkv8", B=64, H=32, Hkv=8, N=1, T=4096, page=64),
        # Prompts of ragged length entering the cache.
        dict(append, name="append_norm_prompt_B8_H12_N8192", B=8, H=12, Hkv=12, N=8192, T=517, page=256,
             marked=False),
        # A few users ask about a short document: the smallest decode.
        dict(decode, name="decode_shared_B4_H12_P1000_T40", B=4, H=12, Hkv=12, P=1000, T=40, page=64),
        # A batch that shares a long document of 32k tokens, with ragged conversations behind it.
        dict(decode, name="decode_shared_B64_H12_P32768_T512", B=64, H=12, Hkv=12, P=32768, T=512,
             page=256),
        # A large batch behind a system prompt of 8k tokens, shared heads, theta prior, fp32 output.
        dict(decode, name="decode_shared_B256_H32_Hkv8_P8111_T300_fp32", B=256, H=32, Hkv=8, P=8111,
             T=300, page=64, prior="theta", ssmax=False, out="fp32"),
        # Bounded caches of 8k keys that gather their weights.
        dict(decode, name="decode_weights_B64_H12_T8192", B=64, H=12, Hkv=12, T=8192, page=64, marked=True),
        # One long context with shared heads that gathers its weights: the key axis is all there is.
        dict(decode, name="decode_weights_B1_H32_Hkv8_T131072", B=1, H=32, Hkv=8, T=131072, page=256,
             marked=True),
        # A small batch of short caches loses a few keys.
        dict(op="evict", name="evict_B8_Hkv8_600_to_512", B=8, Hkv=8, T=600, budget=512, sink=4, recent=64,
             page=64),
        # A large batch after 256 tokens beyond its budget.
        dict(op="evict", name="evict_B64_Hkv12_4352_to_4096", B=64, Hkv=12, T=4352, budget=4096, sink=4,
             recent=512, page=64),
        # A long prompt cut down to half after its prefill.
        dict(op="evict", name="evict_B1_Hkv12_131072_to_65536", B=1, Hkv=12, T=131072, budget=65536,
             sink=16, recent=1024, page=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        old = most.setdefault(c["op"], w)
        most[c["op"]] = {k: max(old[k], w[k]) for k in w}
    while True:
        op = rng.choice(["qk_norm", "append", "decode", "decode", "decode", "evict"])
        Hkv = rng.choice([1, 2, 3, 4, 8, 12, 16])
        H = Hkv * rng.choice([1, 1, 1, 2, 3, 4, 8])
        page = rng.choice([64, 64, 128, 256, 320])
        if op == "qk_norm":
            c = dict(op=op, B=_log_int(rng, 1, 64), H=H, Hkv=Hkv, T=_log_int(rng, 1, 65536),
                     rot=rng.choice([0, 16, 32, 48, 64, 64, 64]), pairs=rng.random() < 0.4,
                     per_head=rng.random() < 0.5, packed=rng.random() < 0.5)
        elif op == "append":
            c = dict(op=op, B=_log_int(rng, 1, 256), H=H, Hkv=Hkv, N=_log_int(rng, 1, 16384),
                     T=_log_int(rng, 1, 16384), page=page, rot=rng.choice([0, 16, 32, 48, 64, 64, 64]),
                     pairs=rng.random() < 0.4, per_head=rng.random() < 0.5, marked=rng.random() < 0.5)
        elif op == "decode":
            c = dict(op=op, B=_log_int(rng, 1, 256), H=H, Hkv=Hkv, page=page,
                     prior=rng.choice(["alpha", "alpha", "theta"]), ssmax=rng.random() < 0.6,
                     out=rng.choice(["bf16", "bf16", "fp32"]), marked=rng.random() < 0.4,
                     P=_log_int(rng, 1, 131072) if rng.random() < 0.7 else 0, T=_log_int(rng, 1, 131072))
        else:
            T = _log_int(rng, 2, 131072)
            budget = _log_int(rng, max(1, T // 8), T)
            sink = rng.randint(0, min(16, budget))
            c = dict(op=op, B=_log_int(rng, 1, 128), Hkv=Hkv, T=T, budget=budget, sink=sink,
                     recent=rng.randint(0, (budget - sink) // 2), page=page)
        w = work(c)
        if any(w[k] > most[op][k] for k in w):
            continue
        T = c["T"]
        pool = c["B"] * Hkv * (T + c.get("N", 0) + c.get("budget", 0)) * D * 4
        logits = c["B"] * H * (T + c.get("P", 0))
        if H <= 64 and pool <= 4e9 and (op != "decode" or logits <= 2e8):
            return c


# ---------------------------------------------------------------- inputs

def _numpy(case, seed):
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return np.random.default_rng([seed % (1 << 31)] + [ord(ch) for ch in text])


def _cache(st, gen, B, Hkv, page, num_pages, table):
    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    st["k_pages"], st["v_pages"] = normal(num_pages, Hkv, page, D), normal(num_pages, Hkv, page, D)
    st["table"] = torch.from_numpy(table).cuda()


def _marks(st, gen, case, lens, start, gap):
    """Positions of the keys that are left, ascending to start + gap * T at most, each head with its own,
    and the weights that they gathered: a few large ones, many small, some never seen at all."""
    B, Hkv, page, T = case["B"], case["Hkv"], case["page"], case["T"]
    num = st["k_pages"].shape[0]
    st["key_pos"] = torch.zeros(num, Hkv, page, dtype=torch.int32, device="cuda")
    st["key_weight"] = torch.zeros(num, Hkv, page, device="cuda")
    last = start + gap * T
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        steps = torch.randint(1, gap + 1, (Hkv, n), generator=gen, device="cuda")
        pos = last - steps.flip(1).cumsum(1).flip(1) + steps[:, -1:]
        w = torch.exp(2.5 * torch.randn(Hkv, n, generator=gen, device="cuda")) * 0.05
        w *= torch.rand(Hkv, n, generator=gen, device="cuda") < 0.85
        slot = torch.arange(n, device="cuda")
        at = st["table"][b].long()[slot // page]
        st["key_pos"][at, :, slot % page] = pos.int().T
        st["key_weight"][at, :, slot % page] = w.T
    return last


def _tables(rng, blocks, max_blocks, first=0):
    """A block table [B, max_blocks] of shuffled pages (entries behind a sequence's blocks are -1), and
    the first page behind them; there is room for every sequence at its longest."""
    total = len(blocks) * max_blocks
    table = np.full((len(blocks), max_blocks), -1, np.int32)
    pages = first + rng.permutation(total).astype(np.int32)
    table[np.arange(max_blocks)[None] < blocks[:, None]] = pages[:int(blocks.sum())]
    return table, first + total


def prepare(case, seed):
    rng = _numpy(case, seed)
    op, B, Hkv, T = case["op"], case["B"], case["Hkv"], case["T"]
    gen = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 62)))
    st = {"case": dict(case), "kept": {}}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    def i32(x):
        return torch.from_numpy(np.asarray(x, np.int32)).cuda()

    def ragged(lo, hi):
        x = rng.integers(lo, hi + 1, B)
        x[rng.integers(0, B)] = hi
        return x.astype(np.int32)

    if op in ("qk_norm", "append"):
        H = case["H"]
        # weights near one, as training leaves them
        shape = lambda h: (h, D) if case["per_head"] else (D,)
        st["wq"], st["wk"] = (1 + 0.2 * torch.randn(shape(h), generator=gen, device="cuda") for h in (H, Hkv))
    if op == "qk_norm":
        # One projection's output holds a token's queries, keys and values side by side; so does its
        # gradient.
        qkv = normal(B, T, H + 2 * Hkv, D) * 3
        st["q"], st["k"], _ = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
        st["gq"], st["gk"] = normal(B, H, T, D), normal(B, Hkv, T, D)
        st["positions"] = None
        if case["packed"]:
            start = np.sort(rng.integers(0, T, (B, 3)), 1)
            start[:, 0] = 0
            t = np.arange(T)
            doc = (t[None, :, None] >= start[:, None]).sum(2) - 1
            st["positions"] = i32(t[None] - np.take_along_axis(start, doc, 1))
        st["q_out"], st["k_out"] = torch.empty(B, H, T, D, dtype=torch.bfloat16, device="cuda"), \
            torch.empty(B, Hkv, T, D, dtype=torch.bfloat16, device="cuda")
        grad = torch.zeros(B, T, H + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
        st["dq"], st["dk"], _ = (x.transpose(1, 2) for x in grad.split([H, Hkv, Hkv], 2))
        st["dwq"], st["dwk"] = torch.empty_like(st["wq"]), torch.empty_like(st["wk"])
        return st

    page = case["page"]
    if op == "append":
        N = case["N"]
        lens, new = ragged(0, T), ragged((N + 1) // 2, N)
        max_blocks = -(-(T + N) // page)
        table, num = _tables(rng, -(-(lens.astype(np.int64) + new) // page), max_blocks)
        _cache(st, gen, B, Hkv, page, num, table)
        qkv = normal(B, N, H + 2 * Hkv, D) * 3
        st["q"], st["k"], st["v"] = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
        st["q_out"] = torch.zeros(B, H, N, D, dtype=torch.bfloat16, device="cuda")
        st["lens"], st["new"], st["pos"] = i32(lens), i32(new), None
        if case["marked"]:
            st["span"] = 200000
            # the sequences have been longer than what is left of them
            st["pos"] = i32(lens + rng.integers(0, 100000, B))
            st["key_pos"] = torch.zeros(num, Hkv, page, dtype=torch.int32, device="cuda")
            st["key_weight"] = torch.ones(num, Hkv, page, device="cuda")
        return st

    if op == "decode":
        H, P = case["H"], case["P"]
        lens = ragged(0 if P else 1, T)
        prefix_blocks = -(-P // page)
        prefix, first = _tables(rng, np.array([prefix_blocks]), prefix_blocks)
        table, num = _tables(rng, -(-lens.astype(np.int64) // page), -(-T // page), first)
        _cache(st, gen, B, Hkv, page, num, table)
        st["lens"] = i32(lens)
        if P:
            st["prefix"], st["prefix_len"] = i32(prefix[0]), i32([P])
        st["q"] = normal(B, H, D)
        if case["prior"] == "alpha":
            prm = [np.exp(rng.uniform(0, np.log(1e3), H)), rng.uniform(-1, 2, H),
                   rng.uniform(0, 8, H) * (rng.random(H) < 0.5)]
        else:
            prm = [rng.uniform(-3, 1, H), rng.uniform(-1, 2, H), rng.uniform(-1, 1, H)]
        prm.append(rng.uniform(0.3, 1.0, H))
        st["prm"] = [torch.from_numpy(x.astype(np.float32)).cuda() for x in prm]
        st["q_pos"], st["span"] = None, P + T
        if case["marked"]:
            last = _marks(st, gen, case, lens, P, 3)
            st["q_pos"], st["span"] = i32(np.full(B, last)), last + 1
        st["o"] = torch.zeros(B, H, D, device="cuda",
                              dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
        st["lse"] = torch.zeros(B, H, device="cuda")
        return st

    budget = case["budget"]
    lens = rng.integers(min(budget + 1, T), T + 1, B)
    lens[rng.random(B) < 0.1] = max(1, budget // 2)  # a few sequences are still short
    lens[rng.integers(0, B)] = T
    # What is kept goes to fresh pages (the old ones belong to a fork of the sequence as well), so that a
    # pass can be repeated.
    max_blocks = -(-T // page)
    table, num = _tables(rng, -(-lens // page), max_blocks)
    out, num = _tables(rng, -(-np.minimum(lens, budget) // page), -(-min(budget, T) // page), num)
    _cache(st, gen, B, Hkv, page, num, table)
    st["lens"], st["out"], st["new_lens"] = i32(lens), i32(out), i32(np.zeros(B))
    st["span"] = _marks(st, gen, case, lens, 0, 2) + 1
    return st


# ---------------------------------------------------------------- plain forms

def _rotate(x, pos, rot, pairs, back=False):
    """x [B, h, T, 64] in 32 bits, its first `rot` dimensions turned by their positions pos [B, T]."""
    if rot == 0:
        return x
    f = torch.arange(rot // 2, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None, :, None] * torch.pow(BASE, -2.0 * f / rot)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if back:
        sin = -sin
    out = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if pairs:
        out[..., 0:rot:2], out[..., 1:rot:2] = ra, rb
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = ra, rb
    return out


def _weight(w):
    """[64] or [h, 64] -> broadcast over [B, h, T, 64]."""
    return w if w.dim() == 1 else w[:, None]


def _norm(x):
    """(x / rms, 1 / rms) in 32 bits."""
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)
    return x * r, r


def _plain_qk_norm(st):
    case = st["case"]
    B, T, rot, pairs = case["B"], case["T"], case["rot"], case["pairs"]
    pos = st["positions"]
    if pos is None:
        pos = torch.arange(T, device="cuda").expand(B, T)
    for x, w, y, g, dx, dw in (("q", "wq", "q_out", "gq", "dq", "dwq"), ("k", "wk", "k_out", "gk", "dk", "dwk")):
        n, r = _norm(st[x])
        w32 = _weight(st[w])
        st[y].copy_(_rotate(n * w32, pos, rot, pairs))
        dn = _rotate(st[g].float(), pos, rot, pairs, back=True)
        st[dw].copy_((dn * n).double().sum((0, 2) if case["per_head"] else (0, 1, 2)))
        dn = dn * w32
        st[dx].copy_(r * (dn - n * (dn * n).mean(-1, keepdim=True)))
    return tuple(st[x] for x in ("q_out", "k_out", "dq", "dk", "dwq", "dwk"))


def _slots(table, page, slot):
    block = (slot // page).clamp(max=table.shape[1] - 1)
    return table.long().gather(1, block), slot % page


def _plain_append(st):
    case = st["case"]
    N, rot, pairs = case["N"], case["rot"], case["pairs"]
    i = torch.arange(N, device="cuda")
    first = st["lens"] if st["pos"] is None else st["pos"]
    pos = first[:, None].long() + i
    valid = i[None] < st["new"][:, None]
    pg, row = _slots(st["table"], case["page"], st["lens"][:, None].long() + i)
    q, k = (_rotate(_norm(st[x])[0] * _weight(st[w]), pos, rot, pairs).to(torch.bfloat16)
            for x, w in (("q", "wq"), ("k", "wk")))
    pg, row = pg[valid], row[valid]
    st["k_pages"][pg, :, row] = k.transpose(1, 2)[valid]
    st["v_pages"][pg, :, row] = st["v"].transpose(1, 2)[valid]
    torch.where(valid[:, None, :, None], q, st["q_out"], out=st["q_out"])
    if not case["marked"]:
        return st["k_pages"], st["v_pages"], st["q_out"]
    st["key_pos"][pg, :, row] = pos[valid].int()[:, None]
    st["key_weight"][pg, :, row] = 0.0
    return st["k_pages"], st["v_pages"], st["q_out"], st["key_pos"], st["key_weight"]


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


def _plain_decode(st):
    case = st["case"]
    B, H, Hkv, P, page = (case[k] for k in ("B", "H", "Hkv", "P", "page"))
    G, L = H // Hkv, st["table"].shape[1] * page
    lens = st["lens"].long()
    j = torch.arange(L, device="cuda")
    pages = st["table"].long().clamp(min=0)
    # a page that no key of the sequence lies in holds other sequences' rows: masked like any other
    keys, values = (p[pages].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D).float()
                    for p in (st["k_pages"], st["v_pages"]))
    if case["marked"]:
        pos = st["q_pos"].long()
        key_pos = st["key_pos"][pages].permute(0, 2, 1, 3).reshape(B, Hkv, 1, L).expand(B, Hkv, G, L)
        dist = pos[:, None, None, None] - key_pos
    else:
        pos = P + lens - 1
        dist = (lens[:, None] - 1 - j)[:, None, None].expand(B, Hkv, G, L)
    q = st["q"].float().view(B, Hkv, G, D)
    if case["ssmax"]:
        c = st["prm"][3][None] * torch.log((pos + 1).float())[:, None] / 8
    else:
        c = torch.full((B, H), 0.125, device="cuda")
    bias = _bias_table(case, st["prm"], st["span"], torch.float32)
    head = torch.arange(H, device="cuda").view(1, Hkv, G, 1)
    z = torch.matmul(q, keys.transpose(2, 3)) * c.view(B, Hkv, G, 1) + bias[head, dist.clamp(0, st["span"] - 1)]
    z.masked_fill_((j[None] >= lens[:, None])[:, None, None], -math.inf)
    if P:
        at = st["prefix"].long()
        pk, pv = (p[at].transpose(0, 1).reshape(Hkv, -1, D)[:, :P].float() for p in (st["k_pages"], st["v_pages"]))
        zp = torch.matmul(q.transpose(0, 1).reshape(Hkv, B * G, D), pk.transpose(1, 2))
        zp = zp.view(Hkv, B, G, P).transpose(0, 1) * c.view(B, Hkv, G, 1)
        zp += bias[head, (pos[:, None] - torch.arange(P, device="cuda"))[:, None, None]]
        m = torch.maximum(z.amax(3, keepdim=True), zp.amax(3, keepdim=True))
        zp = (zp - m).exp_()
    else:
        m = z.amax(3, keepdim=True)
    p = (z - m).exp_()
    s = p.sum(3, keepdim=True)
    o = torch.matmul(p, values)
    if P:
        s = s + zp.sum(3, keepdim=True)
        o = o + torch.matmul(zp.transpose(0, 1).reshape(Hkv, B * G, P), pv).view(Hkv, B, G, D).transpose(0, 1)
    st["o"].copy_((o / s).view(B, H, D))
    st["lse"].copy_((m + s.log()).view(B, H))
    if not case["marked"]:
        return st["o"], st["lse"]
    valid = (j[None] < lens[:, None]).nonzero(as_tuple=True)
    pg, row = st["table"].long()[valid[0], valid[1] // page], valid[1] % page
    st["key_weight"][pg, :, row] += (p / s).sum(2)[valid[0], :, valid[1]]
    return st["o"], st["lse"], st["key_weight"]


def _plain_evict(st):
    case = st["case"]
    B, Hkv, page, budget, sink, recent = (case[k] for k in ("B", "Hkv", "page", "budget", "sink", "recent"))
    L = st["table"].shape[1] * page
    lens = st["lens"].long()
    pages = st["table"].long().clamp(min=0)
    j = torch.arange(L, device="cuda")
    w = st["key_weight"][pages].permute(0, 2, 1, 3).reshape(B, Hkv, L)
    always = (j[None] < sink) | (j[None] >= (lens - recent)[:, None]) | (lens <= budget)[:, None]
    w = torch.where(always[:, None], math.inf, w)
    w = torch.where((j[None] >= lens[:, None])[:, None], -math.inf, w)
    # the budget largest, ties to the lowest slot, back in order
    top = torch.sort(w, dim=2, descending=True, stable=True).indices[..., :budget].sort(2).values
    n = min(budget, L)
    new = lens.clamp(max=budget)
    valid = (torch.arange(n, device="cuda")[None] < new[:, None]).nonzero(as_tuple=True)
    b, m = valid
    dst, drow = st["out"].long()[b, m // page], m % page
    src = top[b, :, m]                                               # [n, Hkv]
    spg, srow = st["table"].long()[b[:, None], src // page], src % page
    head = torch.arange(Hkv, device="cuda")[None]
    for x in ("k_pages", "v_pages", "key_pos", "key_weight"):
        st[x][dst, :, drow] = st[x][spg, head, srow]
    st["new_lens"].copy_(new)
    return st["k_pages"], st["v_pages"], st["key_pos"], st["key_weight"], st["new_lens"]


def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        return {"qk_norm": _plain_qk_norm, "append": _plain_append, "decode": _plain_decode,
                "evict": _plain_evict}[op](state)

    from transformer_attention_ggd_gb300 import bam_attn as ba

    kept = state["kept"]  # the workspace, norm, rotation and parameters that a program keeps
    if op in ("qk_norm", "append") and not kept:
        kept.update(norm=ba.make_qk_norm(state["wq"], state["wk"], NORM_EPS),
                    rope=ba.make_rope(BASE, case["rot"], case["pairs"]), marks=None)
        if op == "qk_norm":
            kept.update(ws=ba.qk_norm_workspace(case["B"], case["H"], case["Hkv"], case["T"]))
        else:
            kept.update(ws=ba.cache_workspace())
    if "key_pos" in state and not kept.get("marks"):
        kept.update(marks=ba.make_marks(state["key_pos"], state["key_weight"], state["span"]))
    if op == "qk_norm":
        ba.bam_qk_norm_fwd(state["q"], state["k"], state["q_out"], state["k_out"], state["positions"],
                           kept["norm"], kept["rope"])
        ba.bam_qk_norm_bwd(state["q"], state["k"], state["gq"], state["gk"], state["dq"], state["dk"],
                           state["dwq"], state["dwk"], state["positions"], kept["norm"], kept["rope"],
                           kept["ws"])
        return tuple(state[x] for x in ("q_out", "k_out", "dq", "dk", "dwq", "dwk"))
    cache = state["k_pages"], state["v_pages"], state["table"], state["lens"]
    if op == "append":
        ba.bam_kv_append_norm_paged(state["k"], state["v"], *cache, state["new"], None, state["q"],
                                    state["q_out"], kept["norm"], kept["rope"], state["pos"],
                                    kept["marks"], kept["ws"])
        out = state["k_pages"], state["v_pages"], state["q_out"]
        return out + (state["key_pos"], state["key_weight"]) if case["marked"] else out
    Tmax = state["table"].shape[1] * case["page"]
    if op == "decode":
        if "prm" not in kept:
            prior = ba.BAM_PRIOR_THETA if case["prior"] == "theta" else ba.BAM_PRIOR_ALPHA
            Pmax = state["prefix"].numel() * case["page"] if case["P"] else 0
            kept.update(prm=ba.make_params(*state["prm"], EPS, True, case["ssmax"], prior),
                        ws=ba.shared_workspace(case["B"], case["H"], case["Hkv"], Pmax, Tmax,
                                               state["span"] if case["marked"] else 0))
        ba.bam_attn_decode_shared_paged(state["q"], *cache, state.get("prefix"), state.get("prefix_len"),
                                        state["q_pos"], kept.get("marks"), 1.0, state["o"], state["lse"],
                                        kept["prm"], kept["ws"])
        out = state["o"], state["lse"]
        return out + (state["key_weight"],) if case["marked"] else out
    if "ws" not in kept:
        kept.update(ws=ba.evict_workspace(case["B"], case["Hkv"], Tmax, case["budget"]))
    ba.bam_kv_evict_paged(*cache, kept["marks"], state["out"], state["new_lens"], case["budget"],
                          case["sink"], case["recent"], kept["ws"])
    return state["k_pages"], state["v_pages"], state["key_pos"], state["key_weight"], state["new_lens"]


def work(case):
    """Expected work over the ragged lengths: one sequence has the longest, the others average half of it
    (three quarters of the new tokens)."""
    op, B, Hkv, T = case["op"], case["B"], case["Hkv"], case["T"]
    mean = lambda lo, hi: (hi + (B - 1) * (lo + hi) / 2) / B
    if op == "qk_norm":
        rows = B * T * (case["H"] + Hkv)
        return {"bytes": int(rows * 10 * D), "flops": int(rows * (15 * D + 6 * case["rot"]))}
    if op == "append":
        tokens = B * mean((case["N"] + 1) // 2, case["N"])
        H, marks = case["H"], 8 * Hkv if case["marked"] else 0
        return {"bytes": int(tokens * (4 * D * (2 * Hkv + H) + marks)),
                "flops": int(tokens * (4 * D + 3 * case["rot"]) * (Hkv + H))}
    if op == "decode":
        H, P, t = case["H"], case["P"], mean(0 if case["P"] else 1, T)
        size = 4 if case["out"] == "fp32" else 2
        key = 4 * D + (12 if case["marked"] else 0)
        return {"bytes": int(Hkv * (P * 4 * D + B * t * key) + B * H * (2 * D + size * D + 4)),
                "flops": int(4 * D * B * H * (P + t))}
    budget = min(case["budget"], T)
    t = mean(min(case["budget"] + 1, T), T)
    return {"bytes": int(B * Hkv * (4 * t + budget * 2 * (4 * D + 8))), "flops": int(B * Hkv * t)}


# ---------------------------------------------------------------- the definition in 64 bits

def _turns(pos, rot, pairs):
    """Rotation matrices [n, 64, 64] of positions pos (numpy)."""
    half = rot // 2
    turn = torch.eye(D, dtype=torch.float64, device="cuda").repeat(len(pos), 1, 1)
    for f in range(half):
        i, k = (2 * f, 2 * f + 1) if pairs else (f, f + half)
        ang = torch.from_numpy(np.asarray(pos, np.float64)).cuda() * BASE ** (-f / half)
        turn[:, i, i], turn[:, i, k] = ang.cos(), -ang.sin()
        turn[:, k, i], turn[:, k, k] = ang.sin(), ang.cos()
    return turn


def _rms64(x):
    return torch.sqrt(torch.square(x).sum(-1, keepdim=True) / D + NORM_EPS)


def _exact_qk_norm(case, st):
    B, T = case["B"], case["T"]
    positions = np.tile(np.arange(T), (B, 1)) if st["positions"] is None else st["positions"].cpu().numpy()
    outs = []
    for x, w, g, h in (("q", "wq", "gq", case["H"]), ("k", "wk", "gk", case["Hkv"])):
        y = torch.empty(B, h, T, D, dtype=torch.float64, device="cuda")
        dx, dw = torch.empty_like(y), torch.zeros(h, D, dtype=torch.float64, device="cuda")
        wt = st[w].double().expand(h, D)[:, None]
        for b in range(B):
            for t0 in range(0, T, 2048):
                t = slice(t0, min(T, t0 + 2048))
                turn = _turns(positions[b, t], case["rot"], case["pairs"])
                v, gr = st[x][b, :, t].double(), st[g][b, :, t].double()
                rms = _rms64(v)
                y[b, :, t] = torch.einsum("nij,hnj->hni", turn, wt * v / rms)
                dn = torch.einsum("nji,hnj->hni", turn, gr)
                dw += (dn * v / rms).sum(1)
                u = dn * wt
                dx[b, :, t] = u / rms - v * (u * v).sum(-1, keepdim=True) / (D * rms ** 3)
        outs.append((y, dx, dw if case["per_head"] else dw.sum(0)))
    (q, dq, dwq), (k, dk, dwk) = outs
    return q, k, dq, dk, dwq, dwk


def _exact_append(case, st):
    Hkv, page = case["Hkv"], case["page"]
    lens, new, table = st["lens"].tolist(), st["new"].tolist(), st["table"].cpu().numpy()
    first = lens if st["pos"] is None else st["pos"].tolist()
    kp, vp, qo = (st[x].double() for x in ("k_pages", "v_pages", "q_out"))
    wq, wk = (st[w].double().expand(h, D)[:, None] for w, h in (("wq", case["H"]), ("wk", Hkv)))
    for b in range(case["B"]):
        for t0 in range(0, new[b], 2048):
            n = np.arange(t0, min(new[b], t0 + 2048))
            turn = _turns(first[b] + n, case["rot"], case["pairs"])
            at = torch.from_numpy(table[b, (lens[b] + n) // page].astype(np.int64)).cuda()
            row = torch.from_numpy((lens[b] + n) % page).cuda()
            t = slice(t0, t0 + len(n))
            k, q = st["k"][b, :, t].double(), st["q"][b, :, t].double()
            kp[at, :, row] = torch.einsum("nij,hnj->nhi", turn, wk * k / _rms64(k))
            qo[b, :, t] = torch.einsum("nij,hnj->hni", turn, wq * q / _rms64(q))
            vp[at, :, row] = st["v"][b, :, t].double().transpose(0, 1)
            if case["marked"]:
                st["key_pos"][at, :, row] = torch.from_numpy(first[b] + n).cuda().int()[:, None]
                st["key_weight"][at, :, row] = 0
    if case["marked"]:
        return kp, vp, qo, st["key_pos"], st["key_weight"].double()
    return kp, vp, qo


def _exact_decode(case, st):
    B, H, Hkv, P, page = (case[k] for k in ("B", "H", "Hkv", "P", "page"))
    G = H // Hkv
    lens, table = st["lens"].tolist(), st["table"].long()
    o, lse = st["o"].double(), st["lse"].double()
    weight = st["key_weight"].double() if case["marked"] else None
    a, be, mu, s = (x.double() for x in st["prm"])
    if P:
        j = torch.arange(P, device="cuda")
        pk, pv = (x[st["prefix"].long()[j // page], :, j % page].double() for x in (st["k_pages"], st["v_pages"]))
    for b in range(B):
        j = torch.arange(lens[b], device="cuda")
        pg, row = table[b][j // page], j % page
        k, v = (x[pg, :, row].double() for x in (st["k_pages"], st["v_pages"]))  # [L, Hkv, 64]
        if case["marked"]:
            at, kpos = int(st["q_pos"][b]), st["key_pos"][pg, :, row].double()
        else:
            at, kpos = P + lens[b] - 1, (P + j).double()[:, None].expand(-1, Hkv)
        if P:
            k, v = torch.cat([pk, k]), torch.cat([pv, v])
            kpos = torch.cat([torch.arange(P, device="cuda").double()[:, None].expand(-1, Hkv), kpos])
        for g in range(Hkv):
            hs = slice(g * G, (g + 1) * G)
            d = (at - kpos[:, g])[None]
            A, Be, Mu = (x[hs][:, None] for x in (a, be, mu))
            if case["prior"] == "theta":
                bias = -torch.exp(A) * torch.pow((d - 2 * torch.sinh(Mu)).abs() + EPS, Be)
            else:
                u = (d - Mu).abs()
                bias = -torch.pow(torch.where(Be <= 0, u.clamp(min=EPS), u) / A, Be)
            c = s[hs][:, None] * math.log(at + 1) if case["ssmax"] else 1.0
            z = st["q"][b, hs].double() @ k[:, g].T * c / math.sqrt(D) + bias
            lse[b, hs] = torch.logsumexp(z, 1)
            w = torch.exp(z - lse[b, hs][:, None])
            o[b, hs] = w @ v[:, g]
            if case["marked"]:
                weight[pg, g, row] += w[:, P:].sum(0)
    return (o, lse, weight) if case["marked"] else (o, lse)


def _exact_evict(case, st):
    page, budget, sink, recent = (case[k] for k in ("page", "budget", "sink", "recent"))
    lens, table, out = st["lens"].tolist(), st["table"].long(), st["out"].long()
    weights = st["key_weight"].cpu().numpy().astype(np.float64)
    host = table.cpu().numpy()
    pools = {x: st[x].clone() for x in ("k_pages", "v_pages", "key_pos", "key_weight")}
    new = []
    for b, n in enumerate(lens):
        m = min(n, budget)
        new.append(m)
        i = torch.arange(m, device="cuda")
        to, trow = out[b][i // page], i % page
        slot = np.arange(n)
        for g in range(case["Hkv"]):
            kept = slot
            if n > budget:
                middle = slot[sink:n - recent]
                w = weights[host[b, middle // page], g, middle % page]
                order = np.lexsort((middle, -w))[:budget - sink - recent]
                kept = np.sort(np.concatenate([slot[:sink], middle[order], slot[n - recent:]]))
            at = torch.from_numpy(kept).cuda()
            pg, row = table[b][at // page], at % page
            for x in pools:
                pools[x][to, g, trow] = st[x][pg, g, row]
    return (pools["k_pages"].double(), pools["v_pages"].double(), pools["key_pos"],
            pools["key_weight"].double(), torch.tensor(new, dtype=torch.int32).cuda())


def exact(case, seed):
    if case["op"] == "decode" and case["B"] * case["H"] * float(case["P"] + case["T"]) > 2e9:
        return None
    st = prepare(case, seed)
    return {"qk_norm": _exact_qk_norm, "append": _exact_append, "decode": _exact_decode,
            "evict": _exact_evict}[case["op"]](case, st)
