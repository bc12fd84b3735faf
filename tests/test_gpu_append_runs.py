"""GPU tests of the append with norms where it walks over long or many prompts, in each
of its turns, with and without queries, norms and marks; and of keys alone."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from _bounded_reference import norm_rotate, turn

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ba.load_library()


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _check(seed, H, Hkv, N, lens, new, dims=64, pairs=False, per_head=True, marked=True, norm=True, queries=True,
           page=64):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = len(lens)
    blocks = [max(1, -(-(n + m) // page)) for n, m in zip(lens, new)]
    num = sum(blocks) + 2
    perm = rng.permutation(num)
    table = np.full((B, max(blocks)), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    kp, vp = _normal(gen, num, Hkv, page, 64), _normal(gen, num, Hkv, page, 64)
    kpos = torch.full((num, Hkv, page), -7, dtype=torch.int32, device="cuda")
    kw = torch.full((num, Hkv, page), 5.0, device="cuda")
    k0, v0 = kp.clone(), vp.clone()
    qkv = _normal(gen, B, N, H + 2 * Hkv, 64) * 2
    q, k, v = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
    wq, wk = (1 + 0.3 * torch.randn((h, 64) if per_head else (64,), generator=gen, device="cuda") for h in (H, Hkv))
    first = rng.integers(0, 1 << 20, B)
    qo = torch.full((B, H, N, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    ws = ba.cache_workspace()
    ba.bam_kv_append_norm_paged(
        k, v, kp, vp, _i32(table), _i32(lens), _i32(new), None, q if queries else None, qo if queries else None,
        ba.make_qk_norm(wq, wk, EPS) if norm else None, ba.make_rope(10000.0, dims, pairs), _i32(first),
        ba.make_marks(kpos, kw, 1 << 21) if marked else None, ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    # every token at once: its place, its position, its row in the pages
    b = np.repeat(np.arange(B), new)
    t = np.concatenate([np.arange(n) for n in new]).astype(np.int64)
    slot = np.asarray(lens)[b] + t
    pg, row = torch.from_numpy(table[b, slot // page].astype(np.int64)).cuda(), torch.from_numpy(slot % page).cuda()
    pos = torch.from_numpy(first[b] + t).cuda()
    b, t = torch.from_numpy(b).cuda(), torch.from_numpy(t).cuda()
    got = {"k": kp[pg, :, row].transpose(0, 1), "q": qo[b, :, t].transpose(0, 1)}
    for name, x, w in (("k", k, wk), ("q", q, wq)):
        if name == "q" and not queries:
            continue
        x = x[b, :, t].transpose(0, 1).double()
        w = w.double()[:, None] if per_head else w.double()
        if norm:
            y, bound = norm_rotate(x, w, pos, EPS, 10000.0, dims, pairs)
        else:  # the angles' 2^-21 of a pair, products and sums, one rounding
            y = turn(x, pos, 10000.0, dims, pairs)
            bound = 2.0 ** -18 * 2 * x.abs().amax(-1, keepdim=True) + 2.0 ** -8 * y.abs()
        d = (got[name].double() - y).abs()
        assert torch.all(d <= bound), (name, float((d / bound).max()))
    assert torch.equal(vp[pg, :, row], v[b, :, t])
    if marked:
        assert torch.equal(kpos[pg, :, row], pos.int()[:, None].expand(-1, Hkv))
        assert torch.all(kw[pg, :, row] == 0)
        kpos[pg, :, row], kw[pg, :, row] = -7, 5.0
    assert torch.all(kpos == -7) and torch.all(kw == 5.0)
    kp[pg, :, row], vp[pg, :, row] = k0[pg, :, row], v0[pg, :, row]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)
    if queries:
        qo[b, :, t] = 3.0
    assert torch.all(qo == 3.0)


# Lengths whose token tiles are many more than the SMs; none at all first, last and in a row.
LENS, NEW = [5, 130, 0, 77, 1, 64, 9, 0], [0, 2000, 1, 0, 0, 1500, 1999, 0]


@pytest.mark.parametrize("dims,pairs", [(0, False), (32, False), (64, False), (48, True), (64, True)])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 5), (42, 3)])
def test_long_prompts(H, Hkv, dims, pairs):
    _check(H + dims, H, Hkv, 2000, LENS, NEW, dims, pairs)


@pytest.mark.parametrize("queries", [True, False])
@pytest.mark.parametrize("norm,per_head", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("marked", [True, False])
def test_long_prompts_without_some_of_it(queries, norm, per_head, marked):
    for H, Hkv, dims, pairs in ((1, 1, 64, False), (8, 2, 32, True), (6, 6, 0, False)):
        _check(H, H, Hkv, 2000, LENS, NEW, dims, pairs, per_head, marked, norm, queries)


@pytest.mark.parametrize("B", [153, 400, 2000])
@pytest.mark.parametrize("N", [1, 3, 9])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (4, 4), (39, 3)])
def test_few_tokens_of_many_sequences(H, Hkv, N, B):
    rng = np.random.default_rng(B + N)
    lens, new = rng.integers(0, 130, B), rng.integers(0, N + 1, B)
    new[0], new[-1], new[B // 2] = N, 0, N
    _check(B + N, H, Hkv, N, lens.tolist(), new.tolist(), 64, N == 3, N != 3)


@pytest.mark.parametrize("N", [1, 200])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (3, 3), (32, 1)])
def test_keys_alone_with_weights_of_each_head(H, Hkv, N):
    """A shared document's keys: a model's weights fit its query heads, which the call
    does not see."""
    _check(H + N, H, Hkv, N, [0, 64, 70], [N, N - 1, N], queries=False)


def test_weights_that_do_not_fit_the_keys_are_refused():
    x = torch.zeros(1, 2, 3, 64, device="cuda", dtype=torch.bfloat16)
    pages = torch.zeros(2, 2, 64, 64, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 3, 64, device="cuda", dtype=torch.bfloat16)
    table, lens = _i32([[0, 1]]), _i32([0])
    w = lambda h: torch.ones(h, 64, device="cuda")
    for wq, wk, qs in ((w(4), w(4), None), (w(2), w(2), q), (w(4), w(1), q)):
        with pytest.raises(ValueError, match="weights"):
            ba.kv_append_norm_paged(x, x, pages, pages, table, lens, q=qs, norm=ba.make_qk_norm(wq, wk))
    ba.kv_append_norm_paged(x, x, pages, pages, table, lens, norm=ba.make_qk_norm(w(4), w(2)))
    ba.kv_append_norm_paged(x, x, pages, pages, table, lens, q=q, norm=ba.make_qk_norm(w(4), w(2)))
    torch.cuda.synchronize()
