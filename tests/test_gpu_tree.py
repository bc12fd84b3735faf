"""GPU tests of the paged-cache operators for drafted tokens: append, tree
attention and keep, each against a plain 64-bit implementation, their
refusals on the device, and a serving step that runs them together."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from transformer_attention_ggd_gb300 import bam_attn as ba
from transformer_attention_ggd_gb300.inputs import random_params, random_theta_params

from _gpu_helpers import LSE_ATOL, LSE_RTOL, O_ATOL, dev_f32
from _paged_reference import (chain, pack_trees, path_to, random_tree, rotate, rows_of,
                              tree_attention)

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ba.load_library()


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


class Cache:
    """Pages of which only the rows that a sequence uses hold numbers: every
    other row (pages of nobody, rows behind a sequence) holds `junk`."""

    def __init__(self, seed, Hkv, page, used, max_blocks, junk=NAN):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B = len(used)
        blocks = [-(-int(u) // page) for u in used]
        num = sum(blocks) + 2
        perm = rng.permutation(num)
        table = np.full((B, max_blocks), -1, np.int32)
        self.k = torch.full((num, Hkv, page, 64), junk, dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        at = 0
        for b in range(B):
            table[b, :blocks[b]] = perm[at:at + blocks[b]]
            at += blocks[b]
            for i in range(blocks[b]):
                n = min(page, int(used[b]) - i * page)
                for x in (self.k, self.v):
                    x[int(table[b, i]), :, :n] = _normal(gen, Hkv, n, 64)
        self.table = _i32(table)
        self.rng, self.gen = rng, gen


def _prm(rng, H, theta):
    if theta:
        return random_theta_params(H, rng)
    p = random_params(H, rng, mu_hi=6.0)
    p["beta"][0] = -0.6
    return p


def _tree_case(seed, B, H, Hkv, N, page, lens, new, parents, ssmax, theta, out, slack=0, junk=NAN):
    """Runs one call and compares it, untouched rows included."""
    used = [int(a) + int(n) for a, n in zip(lens, new)]
    cap = -(-max(max(used), 1) // page) + slack
    c = Cache(seed, Hkv, page, used, cap, junk)
    prm = _prm(c.rng, H, theta)
    t = [dev_f32(prm[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, B, H, N, 64)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    o = torch.full((B, H, N, 64), 7.0, dtype=dt, device="cuda")
    lse = torch.full((B, H, N), 7.0, device="cuda")
    ws = ba.tree_workspace(B, H, Hkv, N, cap * page)
    ws.fill_(0xFF)  # nothing may depend on what the workspace held
    params = ba.make_params(*t, 1e-5, True, ssmax,
                            ba.BAM_PRIOR_THETA if theta else ba.BAM_PRIOR_ALPHA)
    par = None if parents is None else _i32(pack_trees(parents, B, N))
    ba.bam_attn_decode_tree_paged(q, c.k, c.v, c.table, _i32(lens), _i32(new), par, o, lse, params,
                                  ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    pl = parents if parents is not None else [chain(int(n)) for n in new]
    oref, lref, oerr, lerr = tree_attention(q, c.k, c.v, c.table, lens, new, pl, t, ssmax, theta,
                                            out == "bf16")
    for b in range(B):
        n = int(new[b])
        assert torch.all(o[b, :, n:] == 7.0) and torch.all(lse[b, :, n:] == 7.0)
        d, e = (o[b, :, :n].double() - oref[b, :, :n]).abs(), oerr[b, :, :n]
        assert torch.all(d <= e), (b, float((d / e).max()))
        d, e = (lse[b, :, :n].double() - lref[b, :, :n]).abs(), lerr[b, :, :n]
        assert torch.all(d <= e), (b, float((d / e).max()))
    return c, q, o, lse


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hkv,N", [(4, 4, 1), (3, 3, 5), (8, 2, 7), (2, 2, 16), (4, 1, 17),
                                     (6, 2, 33), (2, 2, 64), (1, 1, 65), (4, 2, 128)])
def test_tree_random_forests(H, Hkv, N, out):
    """Ragged lengths around page and tile borders, node counts from none to N."""
    rng = np.random.default_rng(100 * H + N)
    lens = [0, 1, 63, 64, 65, 200, 500]
    new = [N, max(1, N // 2), 0, N, 1, N, max(1, N - 1)]
    parents = [random_tree(rng, n) for n in new]
    _tree_case(7 + N, 7, H, Hkv, N, 64, lens, new, parents, True, False, out, slack=2)


@pytest.mark.parametrize("page", [64, 128, 320])
@pytest.mark.parametrize("theta,ssmax", [(False, False), (True, True), (True, False)])
def test_tree_priors_and_pages(page, theta, ssmax):
    rng = np.random.default_rng(page)
    lens, new = [511, 129, 62], [9, 12, 12]
    parents = [random_tree(rng, n, forest=False) for n in new]
    _tree_case(page + theta, 3, 6, 3, 12, page, lens, new, parents, ssmax, theta, "fp32")


@pytest.mark.parametrize("kind", ["chain", "star", "comb", "roots"])
@pytest.mark.parametrize("N", [2, 40, 128])
def test_tree_shapes(kind, N):
    """The deepest tree, the flattest ones, and a spine with a leaf at each node."""
    i = np.arange(N)
    parents = {"chain": None, "star": [np.where(i > 0, 0, -1)],
               "comb": [np.where(i % 2, i - 1, i - 2).clip(-1)], "roots": [np.full(N, -1)]}[kind]
    _tree_case(11, 1, 2, 1, N, 64, [75], [N], parents, True, False, "fp32")


@pytest.mark.parametrize("lens", [[5000, 3, 0, 2500], [9000], [0]])
def test_tree_long_and_split(lens):
    """One long sequence is cut into many parts; short ones are not cut."""
    B = len(lens)
    rng = np.random.default_rng(sum(lens) + 1)
    parents = [random_tree(rng, 6) for _ in lens]
    _tree_case(3, B, 4, 2, 6, 64, lens, [6] * B, parents, True, False, "fp32")


@pytest.mark.parametrize("H,Hkv,N,out", [(16, 8, 2, "bf16"), (8, 8, 3, "fp32"), (16, 8, 12, "bf16"),
                                         (8, 8, 40, "bf16"), (8, 8, 100, "fp32")])
def test_tree_many_tiles_a_cta(H, Hkv, N, out):
    """Enough tiles that every CTA goes around its ring many times, at the pace
    of several streams; repeated calls give the same bits."""
    rng = np.random.default_rng(N)
    lens, new = [16000, 9000, 15001, 12345, 7, 16100], [1, N, 2, 1, N, 1]
    parents = [random_tree(rng, n) for n in new]
    c, q, o, lse = _tree_case(N, 6, H, Hkv, N, 64, lens, new, parents, True, False, out)
    t = [dev_f32(_prm(np.random.default_rng(1), H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    par, ln, nw = _i32(pack_trees(parents, 6, N)), _i32(lens), _i32(new)
    ws = ba.tree_workspace(6, H, Hkv, N, c.k.shape[2] * c.table.shape[1])
    first = None
    for _ in range(40):
        got = ba.attention_decode_tree_paged(q, c.k, c.v, c.table, ln, *t, draft_lens=nw,
                                             parents=par, ssmax=True, ws=ws)
        first = got if first is None else first
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK


def test_tree_many_sequences():
    """More sequences than a block has threads, most of them short."""
    rng = np.random.default_rng(5)
    B = 700
    lens, new = rng.integers(0, 20, B), rng.integers(0, 4, B)
    parents = [random_tree(rng, n) for n in new]
    _tree_case(4, B, 2, 1, 3, 64, lens, new, parents, False, False, "bf16")


@pytest.mark.parametrize("B,out", [(37, "fp32"), (38, "bf16"), (39, "fp32"), (39, "bf16")])
def test_tree_about_as_many_items_as_ctas(B, out):
    """A few items less and more than CTAs, cut in different places, some of
    them empty: what was cut is recorded by item, or by CTA."""
    rng = np.random.default_rng(B)
    lens, new = rng.integers(0, 900, B), rng.integers(0, 6, B)
    lens[3], new[3], new[5], new[B - 1] = 5000, 5, 0, 0
    parents = [random_tree(rng, n) for n in new]
    _tree_case(5, B, 16, 8, 5, 64, lens, new, parents, True, False, out)


def test_tree_many_query_heads_per_key_head():
    rng = np.random.default_rng(6)
    _tree_case(8, 2, 64, 1, 5, 64, [300, 10], [5, 3], [random_tree(rng, 5), random_tree(rng, 3)],
               True, False, "fp32")


@pytest.mark.parametrize("H,N,out", [(128, 1, "bf16"), (200, 1, "fp32"), (130, 2, "bf16"),
                                     (16, 8, "bf16"), (24, 3, "fp32")])
def test_tree_one_key_head(H, N, out):
    """All query heads share one key head: row blocks that hold many heads."""
    rng = np.random.default_rng(H)
    lens, new = [700, 0, 129], [N, 1, N]
    _tree_case(H, 3, H, 1, N, 64, lens, new, [random_tree(rng, n) for n in new], True, False, out)


def test_tree_without_any_node_and_without_lse():
    """No sequence has a node: nothing is written.  A call without lse."""
    B, H, N = 5, 4, 3
    c = Cache(121, 2, 64, [70] * B, 2)
    t = [dev_f32(_prm(c.rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, B, H, N, 64)
    o, lse = torch.full((B, H, N, 64), 5.0, device="cuda"), torch.full((B, H, N), 5.0, device="cuda")
    ws = ba.tree_workspace(B, H, 2, N, 128)
    prm = ba.make_params(*t, 1e-5, True, True)
    args = (q, c.k, c.v, c.table, _i32([60] * B))
    ba.bam_attn_decode_tree_paged(*args, _i32([0] * B), None, o, lse, prm, ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    assert torch.all(o == 5.0) and torch.all(lse == 5.0)
    ba.bam_attn_decode_tree_paged(*args, None, None, o, lse, prm, ws)
    o2 = torch.full_like(o, NAN)
    ba.bam_attn_decode_tree_paged(*args, None, None, o2, None, prm, ws)
    assert torch.equal(o, o2) and torch.isfinite(o).all()


def test_tree_infinities_among_committed_keys_reach_every_node():
    """A committed value is seen by every node: an infinity in it reaches all of
    them, in its dimension alone."""
    B, H, N, ln = 1, 3, 5, 300
    for where in (3, 299):
        c = Cache(131, H, 64, [ln + N], 5)
        prm = _prm(c.rng, H, False)
        prm["beta"] = np.zeros(H, np.float32)  # every weight is of the same order
        t = [dev_f32(prm[n]) for n in ("alpha", "beta", "mu", "s")]
        q = _normal(c.gen, B, H, N, 64)
        c.v[int(c.table[0, where // 64]), :, where % 64, 7] = float("-inf")
        for dt in (torch.bfloat16, torch.float32):
            o, _ = ba.attention_decode_tree_paged(q, c.k, c.v, c.table, _i32([ln]), *t, o_dtype=dt)
            assert torch.all(o[..., 7] == float("-inf"))
            assert torch.isfinite(o[..., :7]).all() and torch.isfinite(o[..., 8:]).all()


def test_refusals_on_the_gpu_leave_the_context_usable():
    B, H, N = 2, 4, 3
    c = Cache(141, 2, 64, [40, 50], 1)
    t = [dev_f32(_prm(c.rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, B, H, N, 64)
    ln = _i32([30, 40])
    good = (q, c.k, c.v, c.table, ln)
    for i, bad in [(0, q.float()), (0, q.transpose(1, 2)), (0, q[:, :3]), (1, c.k[:, :1]),
                   (1, c.k.transpose(0, 1)), (2, c.v[..., :32]), (3, c.table.long()),
                   (3, c.table[:1]), (4, ln.float()), (4, ln[:1])]:
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, ba.BamError)):
            ba.attention_decode_tree_paged(*args, *t)
        if i:
            with pytest.raises((ValueError, ba.BamError)):
                ba.kv_append_paged(_normal(c.gen, B, 2, N, 64), _normal(c.gen, B, 2, N, 64), *args[1:])
    for kw in (dict(draft_lens=_i32([1])), dict(parents=_i32([[-1, 0]] * 2)),
               dict(parents=torch.zeros(B, N, device="cuda"))):
        with pytest.raises(ValueError):
            ba.attention_decode_tree_paged(*good, *t, **kw)
    with pytest.raises(ValueError, match="aligned rows"):
        x = _normal(c.gen, B, 2, N, 72)[..., 4:68]
        ba.kv_append_paged(x, x, *good[1:])
    with pytest.raises(ValueError, match="go together"):
        k = _normal(c.gen, B, 2, N, 64)
        ba.bam_kv_append_paged(k, k, *good[1:], None, None, q, None, None, ba.cache_workspace())
    with pytest.raises(ba.BamError, match="unsupported"):
        big = _normal(c.gen, B, H, 129, 64)
        ba.attention_decode_tree_paged(big, *good[1:], *t, ws=torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ba.BamError, match="workspace"):
        ba.attention_decode_tree_paged(*good, *t, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    o, _ = ba.attention_decode_tree_paged(*good, *t)
    assert torch.isfinite(o).all()


def test_tree_masked_nan_and_inf_have_no_effect():
    """A drafted key or value that a node does not see may hold NaN or
    infinities: only the nodes that see it get them."""
    B, H, N, page, ln = 1, 2, 12, 64, 90
    rng = np.random.default_rng(13)
    parents = [np.array([-1, 0, 0, 1, 1, 2, 2, 3, 4, 5, 6, 6])]
    c = Cache(21, H, page, [ln + N], 2, NAN)
    prm = _prm(rng, H, False)
    prm["beta"] = np.abs(prm["beta"])  # no weight of the path underflows (0 * inf would be NaN)
    t = [dev_f32(prm[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, B, H, N, 64)
    clean = [x.clone() for x in (c.k, c.v)]

    def slot(i):
        return int(c.table[0, (ln + i) // page]), (ln + i) % page

    bad = {3: NAN, 5: float("inf"), 8: float("-inf")}
    for i, value in bad.items():
        pg, r = slot(i)
        c.v[pg, :, r, 5:9] = value
        c.k[pg, :, r, 0] = NAN if i == 3 else c.k[pg, :, r, 0]
    args = (c.table, _i32([ln]), *t)
    for out in (torch.float32, torch.bfloat16):
        o, lse = ba.attention_decode_tree_paged(q, c.k, c.v, *args, parents=_i32(parents),
                                                ssmax=True, o_dtype=out)
        o2, lse2 = ba.attention_decode_tree_paged(q, *clean, *args, parents=_i32(parents),
                                                  ssmax=True, o_dtype=out)
        for n in range(N):
            seen = [i for i in path_to(parents[0], n) if i in bad]
            if not seen:
                assert torch.equal(o[:, :, n], o2[:, :, n])
                assert torch.equal(lse[:, :, n], lse2[:, :, n])
            elif 3 in seen:
                assert torch.isnan(o[:, :, n]).all() and torch.isnan(lse[:, :, n]).all()
            else:
                assert torch.equal(lse[:, :, n], lse2[:, :, n])
                assert torch.all(o[:, :, n, 5:9] == bad[seen[0]])
                assert torch.equal(o[:, :, n, 9:], o2[:, :, n, 9:])


@pytest.mark.parametrize("ln", [0, 61, 5000])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (10, 1)])
def test_tree_infinite_drafted_values_in_every_layout(H, Hkv, ln):
    """12, 48 and 120 rows a key head, on one CTA and cut: an infinite drafted
    value reaches the nodes that see it, in its dimensions, and changes no
    other bit."""
    N, page = 12, 64
    parents = [np.array([-1, 0, 0, 1, 1, 2, 2, 3, 4, 5, 6, 6])]
    c = Cache(23, Hkv, page, [ln + N], -(-(ln + N) // page), NAN)
    t = [dev_f32(_prm(np.random.default_rng(3), H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, 1, H, N, 64)
    args = (c.table, _i32([ln]), *t)
    clean = c.v.clone()
    bad = {4: (float("inf"), [0, 20, 33]), 6: (float("-inf"), [15, 47, 63])}
    for i, (value, dims) in bad.items():
        c.v[int(c.table[0, (ln + i) // page]), :, (ln + i) % page, dims] = value
    for out in (torch.float32, torch.bfloat16):
        kw = dict(parents=_i32(parents), ssmax=True, o_dtype=out)
        o, lse = ba.attention_decode_tree_paged(q, c.k, c.v, *args, **kw)
        want, lse2 = ba.attention_decode_tree_paged(q, c.k, clean, *args, **kw)
        for n in range(N):
            for i in set(path_to(parents[0], n)) & set(bad):
                want[:, :, n, bad[i][1]] = bad[i][0]
        assert torch.equal(o, want) and torch.equal(lse, lse2)


def test_tree_of_one_node_is_the_paged_decode():
    """A single node behind len keys is a decode over len + 1 keys, and the
    oracle's decode over them."""
    lens = [0, 63, 64, 700]
    B, H, page = 4, 3, 64
    c = Cache(31, H, page, [x + 1 for x in lens], 11)
    prm = _prm(c.rng, H, False)
    t = [dev_f32(prm[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, B, H, 1, 64)
    o, lse = ba.attention_decode_tree_paged(q, c.k, c.v, c.table, _i32(lens), *t, ssmax=True)
    o2, lse2 = ba.attention_decode_paged(q[:, :, 0].contiguous(), c.k, c.v, c.table,
                                         _i32([x + 1 for x in lens]), *t, ssmax=True)
    torch.testing.assert_close(o[:, :, 0], o2, rtol=0, atol=O_ATOL)
    torch.testing.assert_close(lse[:, :, 0], lse2, rtol=LSE_RTOL, atol=LSE_ATOL)
    for b, ln in enumerate(lens):
        k, v = (rows_of(x, c.table[b], range(ln + 1)).cpu().numpy()[None] for x in (c.k, c.v))
        oref, lref = oracle.decode(q[b:b + 1, :, 0].double().cpu().numpy(), k, v, prm["alpha"],
                                   prm["beta"], prm["mu"], prm["s"], ssmax=True)
        np.testing.assert_allclose(o[b, :, 0].cpu().numpy(), oref[0], rtol=0, atol=O_ATOL)
        np.testing.assert_allclose(lse[b, :, 0].cpu().numpy(), lref[0], rtol=LSE_RTOL,
                                   atol=LSE_ATOL)


def _call(c, q, lens, new, parents, t, ws=None, stream=None):
    B, H, N, _ = q.shape
    if ws is None:
        ws = ba.tree_workspace(B, H, c.k.shape[1], N, c.k.shape[2] * c.table.shape[1])
    o, lse = ba.attention_decode_tree_paged(q, c.k, c.v, c.table, lens, *t, draft_lens=new,
                                            parents=parents, ssmax=True, ws=ws, stream=stream)
    return o, lse, ba.bam_attn_check_status(ws, stream)


def test_tree_out_of_range_arguments_are_reported():
    """Lengths, parents and pages that only the device reads are clamped and
    reported; nothing is read outside the cache."""
    B, H, N, page = 2, 2, 4, 64
    c = Cache(41, H, page, [100 + N, 128], 2, 0.5)
    t = [dev_f32(_prm(c.rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, B, H, N, 64)
    par = _i32([[-1, 0, 0, 1], [-1, 0, 1, 2]])
    good = _call(c, q, _i32([100, 120]), _i32([4, 4]), par, t)
    assert good[2] == ba.BAM_OK
    for lens, new, p, same in [
            ([-3, 120], [4, 4], [[-1, 0, 0, 1], [-1, 0, 1, 2]], 1),     # committed length below 0
            ([4000, 120], [4, 4], [[-1, 0, 0, 1], [-1, 0, 1, 2]], 1),   # behind the block table
            ([100, 120], [9, 4], [[-1, 0, 0, 1], [-1, 0, 1, 2]], 1),    # more nodes than N
            ([100, 120], [-1, 4], [[-1, 0, 0, 1], [-1, 0, 1, 2]], 1),
            ([127, 120], [4, 4], [[-1, 0, 0, 1], [-1, 0, 1, 2]], 1),    # nodes behind the table
            ([100, 120], [4, 4], [[-1, 1, 0, 1], [-1, 0, 1, 2]], 1),    # its own parent
            ([100, 120], [4, 4], [[-2, 0, 0, 900], [-1, 0, 1, 2]], 1)]:
        o, lse, st = _call(c, q, _i32(lens), _i32(new), _i32(p), t)
        assert st == ba.BAM_ERR_INVALID_ARG, (lens, new, p)
        assert torch.equal(o[same], good[0][same]) and torch.equal(lse[same], good[1][same])
    for page_no in (-1, c.k.shape[0], 1 << 30):
        table = c.table.clone()
        table[0, 0] = page_no
        saved, c.table = c.table, table
        o, lse, st = _call(c, q, _i32([100, 120]), _i32([4, 4]), par, t)
        c.table = saved
        assert st == ba.BAM_ERR_INVALID_ARG
        assert torch.equal(o[1], good[0][1])
    # what lies behind a sequence's nodes is not looked at
    o, lse, st = _call(c, q, _i32([100, 120]), _i32([2, 4]), _i32([[-1, 0, 77, -9], [-1, 0, 1, 2]]), t)
    assert st == ba.BAM_OK
    assert torch.equal(o[0, :, :2], good[0][0, :, :2])


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dims,interleaved", [(64, False), (64, True), (32, False), (48, True),
                                              (16, False), (48, False), (0, False)])
@pytest.mark.parametrize("N,tree", [(1, False), (7, True), (70, False), (128, True)])
def test_append(dims, interleaved, N, tree):
    """Slices of one projection's output, ragged token counts, far positions,
    a page border inside the tokens; every other row of the pages stays."""
    B, H, Hkv, page = 4, 6, 2, 64
    rng = np.random.default_rng(N + dims)
    lens, new = [0, 61, 1000, 130], [N, max(0, N - 3), N, (N + 1) // 2]
    c = Cache(N + dims, Hkv, page, [a + n for a, n in zip(lens, new)], 18, 3.0)
    parents = [random_tree(rng, n) for n in new] if tree else None
    qkv = _normal(c.gen, B, N, H + 2 * Hkv, 64)
    q, k, v = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
    before = c.k.clone(), c.v.clone()
    q_out = torch.full((B, H, N, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = ba.cache_workspace()
    base = 10000.0
    ba.bam_kv_append_paged(k, v, c.k, c.v, c.table, _i32(lens), _i32(new),
                           None if parents is None else _i32(pack_trees(parents, B, N)), q, q_out,
                           ba.make_rope(base, dims, interleaved), ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    want_k, want_v = before[0].clone(), before[1].clone()
    for b in range(B):
        for i in range(new[b]):
            depth = len(path_to(parents[b], i)) - 1 if tree else i
            pg, r = int(c.table[b, (lens[b] + i) // page]), (lens[b] + i) % page
            for x, got in ((k[b, :, i], c.k[pg, :, r]), (q[b, :, i], q_out[b, :, i])):
                ref = rotate(x.double(), lens[b] + depth, base, dims, interleaved)
                # half a bf16 step of the result, and fp32 angles (2^-22) of the pair's magnitude
                tol = 2.0 ** -8 * ref.abs() + 2.0 ** -21 * x.double().norm(dim=-1, keepdim=True)
                assert torch.all((got.double() - ref).abs() <= tol), (b, i)
                assert torch.equal(got[:, dims:], x[:, dims:])
            want_k[pg, :, r] = c.k[pg, :, r]
            want_v[pg, :, r] = v[b, :, i]
        assert torch.all(q_out[b, :, new[b]:] == 9.0)
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)


def test_append_far_positions_and_dense_inputs():
    """Positions near 2^27 against 64-bit angles; dense inputs, all N tokens,
    no queries."""
    page, cap, ln = 1 << 16, 1 << 11, (1 << 27) - 300
    B, Hkv, N = 1, 1, 40
    gen = torch.Generator(device="cuda").manual_seed(1)
    pages = torch.zeros(2, Hkv, page, 64, dtype=torch.bfloat16, device="cuda")
    vp = pages.clone()
    table = torch.full((1, cap), -1, dtype=torch.int32, device="cuda")
    table[0, ln // page] = 1
    k, v = _normal(gen, B, Hkv, N, 64), _normal(gen, B, Hkv, N, 64)
    assert ba.kv_append_paged(k, v, pages, vp, table, _i32([ln]), rope=ba.make_rope()) is None
    for i in range(N):
        ref = rotate(k[0, :, i].double(), ln + i, 10000.0, 64, False)
        got = pages[1, :, (ln + i) % page].double()
        # 64-bit angles at 2^27 positions are good to 2^-25 themselves
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * k[0, :, i].double().norm(dim=-1, keepdim=True)
        assert torch.all((got - ref).abs() <= tol)
        assert torch.equal(vp[1, :, (ln + i) % page], v[0, :, i])


def test_append_in_place_queries_and_many_heads():
    B, H, Hkv, N, page = 3, 40, 20, 33, 64
    c = Cache(51, Hkv, page, [N + 10] * B, 1, 0.0)
    q, k, v = _normal(c.gen, B, H, N, 64), _normal(c.gen, B, Hkv, N, 64), _normal(c.gen, B, Hkv, N, 64)
    rope, ws = ba.make_rope(500.0, 64, True), ba.cache_workspace()
    out = ba.kv_append_paged(k, v, c.k.clone(), c.v.clone(), c.table, _i32([10] * B), q=q, rope=rope)
    q2 = q.clone()
    ba.bam_kv_append_paged(k, v, c.k, c.v, c.table, _i32([10] * B), None, None, q2, q2, rope, ws)
    assert torch.equal(out, q2) and not torch.equal(q, q2)


def test_append_bad_slots_are_skipped_and_reported():
    B, Hkv, N, page = 2, 2, 8, 64
    c = Cache(61, Hkv, page, [64, 128], 2, 0.0)
    k, v = _normal(c.gen, B, Hkv, N, 64), _normal(c.gen, B, Hkv, N, 64)
    ws = ba.cache_workspace()

    def call(lens, new, parents=None, table=None):
        kp, vp = c.k.clone(), c.v.clone()
        ba.bam_kv_append_paged(k, v, kp, vp, c.table if table is None else table, _i32(lens),
                               _i32(new), parents, None, None, None, ws)
        return kp, vp, ba.bam_attn_check_status(ws)

    kp, vp, st = call([10, 100], [8, 8])
    assert st == ba.BAM_OK and ba.bam_attn_check_status(ws) == ba.BAM_OK
    # the second sequence's last four tokens lie behind its block table
    kp, vp, st = call([10, 124], [8, 8])
    assert st == ba.BAM_ERR_INVALID_ARG
    want = c.k.clone()
    want[int(c.table[0, 0]), :, 10:18] = k[0]
    want[int(c.table[1, 1]), :, 60:64] = k[1, :, :4]
    assert torch.equal(kp, want)
    for bad in (-1, c.k.shape[0], -(1 << 31)):
        table = c.table.clone()
        table[1, 1] = bad
        kp, vp, st = call([10, 100], [8, 8], table=table)
        assert st == ba.BAM_ERR_INVALID_ARG
        want = c.v.clone()
        want[int(c.table[0, 0]), :, 10:18] = v[0]
        assert torch.equal(vp, want)
    for lens, new, par in [([-1, 100], [8, 8], None), ([10, 1 << 30], [8, 8], None),
                           ([10, 100], [8, 9], None), ([10, 100], [8, -1], None),
                           ([10, 100], [8, 8], _i32([[-1] * 8, [-1, 0, 2, 0, 0, 0, 0, 0]]))]:
        assert call(lens, new, par)[2] == ba.BAM_ERR_INVALID_ARG, (lens, new)


# ---------------------------------------------------------------- keep

@pytest.mark.parametrize("Hkv,N", [(1, 1), (3, 9), (12, 40), (40, 128)])
@pytest.mark.parametrize("alias", [False, True])
def test_keep(Hkv, N, alias):
    """The rows of each path, in order; everything else in the pages stays;
    lengths in place or not."""
    rng = np.random.default_rng(N + Hkv)
    B, page = 6, 64
    lens, new = [0, 60, 63, 64, 300, 5], [N, N, max(1, N - 2), N, 1, 0]
    # deep trees: each node follows one of the three nodes before it
    parents = [np.array([-1 if i == 0 else max(0, i - int(rng.integers(1, 4))) for i in range(n)])
               for n in new]
    accepted = [new[0] - 1, new[1] - 1, new[2] // 2, -1, 0, -1]
    c = Cache(71, Hkv, page, [a + n for a, n in zip(lens, new)], 8)
    want = c.k.clone(), c.v.clone()
    lens_out = list(lens)
    for b in range(B):
        path = path_to(parents[b], accepted[b])
        lens_out[b] += len(path)
        for x, old in zip(want, (c.k, c.v)):
            for m, i in enumerate(path):
                d, s = lens[b] + m, lens[b] + i
                x[int(c.table[b, d // page]), :, d % page] = old[int(c.table[b, s // page]), :, s % page]
    ln = _i32(lens)
    ws = ba.cache_workspace()
    got = ba.kv_keep_paged(c.k, c.v, c.table, ln, _i32(accepted), _i32(pack_trees(parents, B, N)),
                           _i32(new), ln if alias else None, ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    assert got.tolist() == lens_out
    assert alias or ln.tolist() == lens
    for x, y in zip((c.k, c.v), want):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_keep_of_a_chain_moves_nothing():
    c = Cache(81, 2, 64, [30, 90], 2)
    before = c.k.clone()
    ln = _i32([20, 80])
    ws = ba.cache_workspace()
    ba.bam_kv_keep_paged(c.k, c.v, c.table, ln, _i32([10, 10]), None, _i32([4, -1]), ln, ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK and ln.tolist() == [25, 80]
    assert torch.equal(c.k.view(torch.int16), before.view(torch.int16))


def test_keep_bad_arguments_are_reported():
    B, N = 2, 5
    c = Cache(91, 2, 64, [65, 65], 2, 0.0)
    par = _i32([[-1, 0, 0, 1, 2]] * 2)
    ws = ba.cache_workspace()

    def call(accepted, table=None, parents=par, lens=(60, 60)):
        kp, vp = c.k.clone(), c.v.clone()
        n = ba.kv_keep_paged(kp, vp, c.table if table is None else table, _i32(lens),
                             _i32(accepted), parents, None, None, ws)
        return kp, n.tolist(), ba.bam_attn_check_status(ws)

    good = call([4, 4])
    assert good[1:] == ([63, 63], ba.BAM_OK)
    for acc in (5, -2, 1 << 30):
        kp, n, st = call([acc, 4])
        assert st == ba.BAM_ERR_INVALID_ARG and n == [60, 63]
        p = int(c.table[0, 0])
        assert torch.equal(kp[p], c.k[p])
    table = c.table.clone()
    table[0, 1] = 99
    kp, n, st = call([4, 4], table)
    assert st == ba.BAM_ERR_INVALID_ARG and n == [60, 63] and torch.equal(kp[int(c.table[0, 0])], c.k[int(c.table[0, 0])])
    assert call([4, 4], parents=_i32([[-1, 0, 2, 1, 2], [-1, 0, 0, 1, 2]]))[2] == ba.BAM_ERR_INVALID_ARG
    assert call([4, 4], lens=(126, 60))[2] == ba.BAM_ERR_INVALID_ARG


# ---------------------------------------------------------------- together

def _serve(seed, stream=None):
    """Append a draft, attend, keep a path, append one more token and decode
    it with the paged decode; compared with contiguous sequences."""
    B, H, Hkv, N, page, mb = 3, 4, 4, 10, 64, 3
    rng = np.random.default_rng(seed)
    lens = np.array([62, 5, 0])
    c = Cache(seed, Hkv, page, [mb * page] * B, mb)
    t = [dev_f32(_prm(rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    rope = ba.make_rope(10000.0, 64)
    parents = [random_tree(rng, N) for _ in range(B)]
    par = _i32(pack_trees(parents, B, N))
    q, k, v = (_normal(c.gen, B, H, N, 64) for _ in range(3))
    q1, k1, v1 = (_normal(c.gen, B, H, 1, 64) for _ in range(3))
    hist = [(rows_of(c.k, c.table[b], range(lens[b])), rows_of(c.v, c.table[b], range(lens[b])))
            for b in range(B)]
    ln = _i32(lens)
    acc = np.array([N - 1, 4, 0])
    torch.cuda.synchronize()
    qr = ba.kv_append_paged(k, v, c.k, c.v, c.table, ln, None, par, q, rope, stream=stream)
    o, _ = ba.attention_decode_tree_paged(qr, c.k, c.v, c.table, ln, *t, parents=par, ssmax=True,
                                          stream=stream)
    ba.kv_keep_paged(c.k, c.v, c.table, ln, _i32(acc), par, None, ln, stream=stream)
    q1r = ba.kv_append_paged(k1, v1, c.k, c.v, c.table, ln, q=q1, rope=rope, stream=stream)
    o1, _ = ba.attention_decode_paged(q1r[:, :, 0].contiguous(), c.k, c.v, c.table, ln + 1, *t,
                                      ssmax=True)
    torch.cuda.synchronize()
    prm = [x.cpu().numpy().astype(np.float64) for x in t]
    for b in range(B):
        for n in range(N + 1):
            path = path_to(parents[b], int(acc[b]) if n == N else n)
            ks = torch.cat([hist[b][0]] + [rotate(k[b, :, i].double(), lens[b] + m, 1e4, 64, False)[:, None]
                                           for m, i in enumerate(path)], 1)
            vs = torch.cat([hist[b][1]] + [v[b, :, i].double()[:, None] for i in path], 1)
            qq, got = q[b, :, n % N].double(), o[b, :, n % N]
            if n == N:
                ks = torch.cat([ks, rotate(k1[b, :, 0].double(), ks.shape[1], 1e4, 64, False)[:, None]], 1)
                vs = torch.cat([vs, v1[b].double()], 1)
                qq, got = q1[b, :, 0].double(), o1[b]
            qq = rotate(qq, ks.shape[1] - 1, 1e4, 64, False)
            ref, _ = oracle.decode(qq.cpu().numpy()[None], ks.cpu().numpy()[None],
                                   vs.cpu().numpy()[None], *prm, ssmax=True)
            # rotated rows are rounded to bf16: 2^-8 of q and of k moves a logit by up to
            # 2 * 2^-8 c |q| |k| (about 64 * 0.125 * 0.66 s ln n), a weight by as much
            np.testing.assert_allclose(got.float().cpu().numpy(), ref[0], rtol=0, atol=0.15)


def test_serving_step():
    _serve(1)


def test_serving_step_on_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _serve(2, s)


@pytest.mark.parametrize("raw", [False, True])
def test_helpers_clear_their_outputs_on_the_stream_they_are_given(raw):
    """The current stream is busy for some milliseconds: what the helpers clear
    before the kernels write it must not wait behind that."""
    B, H, N = 2, 3, 4
    c = Cache(161, H, 64, [70 + N] * B, 2)
    t = [dev_f32(_prm(c.rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    q, k, v = (_normal(c.gen, B, H, N, 64) for _ in range(3))
    lens, new = _i32([70] * B), _i32([N, N - 1])
    par, acc = _i32([[-1, 0, 0, 2]] * B), _i32([3, 2])

    def step(stream):
        q2 = ba.kv_append_paged(k, v, c.k, c.v, c.table, lens, new, par, q, ba.make_rope(),
                                stream=stream)
        o, lse = ba.attention_decode_tree_paged(q2, c.k, c.v, c.table, lens, *t, draft_lens=new,
                                                parents=par, stream=stream)
        return q2, o, lse, ba.kv_keep_paged(c.k, c.v, c.table, lens, acc, par, new, stream=stream)

    want = step(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = step(s.cuda_stream if raw else s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_captured_step_replays_with_new_lengths():
    """One graph of append, attention and keep, replayed for several steps with
    lengths, drafts and accepted nodes that change on the device, equals the
    same calls made one by one; a second graph shares the workspaces."""
    B, H, Hkv, N, page, mb = 4, 4, 2, 6, 64, 4
    rng = np.random.default_rng(17)

    def fresh():
        c = Cache(101, Hkv, page, [mb * page] * B, mb, 0.0)
        t = [dev_f32(_prm(np.random.default_rng(3), H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
        st = dict(c=c, t=t, ln=_i32([0, 60, 130, 7]), new=_i32([N] * B), par=_i32([[-1] * N] * B),
                  acc=_i32([-1] * B), q=_normal(c.gen, B, H, N, 64), k=_normal(c.gen, B, Hkv, N, 64),
                  v=_normal(c.gen, B, Hkv, N, 64), qo=torch.zeros(B, H, N, 64, dtype=torch.bfloat16, device="cuda"),
                  o=torch.zeros(B, H, N, 64, device="cuda"), lse=torch.zeros(B, H, N, device="cuda"),
                  ws=ba.tree_workspace(B, H, Hkv, N, mb * page))
        st["prm"] = ba.make_params(*t, 1e-5, True, True)
        return st

    rope = ba.make_rope()

    def attend(s):
        ba.bam_kv_append_paged(s["k"], s["v"], s["c"].k, s["c"].v, s["c"].table, s["ln"], s["new"],
                               s["par"], s["q"], s["qo"], rope, s["ws"])
        ba.bam_attn_decode_tree_paged(s["qo"], s["c"].k, s["c"].v, s["c"].table, s["ln"], s["new"],
                                      s["par"], s["o"], s["lse"], s["prm"], s["ws"])

    def keep(s):
        ba.bam_kv_keep_paged(s["c"].k, s["c"].v, s["c"].table, s["ln"], s["new"], s["par"], s["acc"],
                             s["ln"], s["ws"])

    a, g = fresh(), fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for f in (attend, keep):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                f(g)
            graphs.append(graph)
    torch.cuda.synchronize()
    for step in range(5):
        new = rng.integers(0, N + 1, B)
        parents = [random_tree(rng, n) for n in new]
        acc = [int(rng.integers(-1, n)) if n else -1 for n in new]
        x = [_normal(a["c"].gen, *a[n].shape) for n in ("q", "k", "v")]
        for s in (a, g):
            s["new"].copy_(_i32(new))
            s["par"].copy_(_i32(pack_trees(parents, B, N)))
            s["acc"].copy_(_i32(acc))
            for n, val in zip(("q", "k", "v"), x):
                s[n].copy_(val)
        attend(a)
        keep(a)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(a["o"], g["o"]) and torch.equal(a["lse"], g["lse"])
        assert torch.equal(a["ln"], g["ln"]) and torch.equal(a["c"].k, g["c"].k)
    assert ba.bam_attn_check_status(g["ws"]) == ba.BAM_OK


def test_two_calls_at_once():
    """Two streams, two workspaces, the same cache."""
    B, H, N = 2, 4, 9
    c = Cache(111, 2, 64, [4000, 700], 64)
    t = [dev_f32(_prm(c.rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    qs = [_normal(c.gen, B, H, N, 64) for _ in range(2)]
    lens = _i32([3990, 690])
    alone = [_call(c, q, lens, None, None, t)[:2] for q in qs]
    wss = [ba.tree_workspace(B, H, 2, N, 64 * 64) for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for q, ws, s in zip(qs, wss, streams):
            with torch.cuda.stream(s):
                got.append(ba.attention_decode_tree_paged(q, c.k, c.v, c.table, lens, *t, ssmax=True,
                                                          ws=ws))
        torch.cuda.synchronize()
        for x, y in zip(got, alone):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
