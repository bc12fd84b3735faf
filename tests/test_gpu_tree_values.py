"""Tree attention where values are extreme: what a node does not see, or weighs
with nothing, leaves no trace; an infinity that it sees reaches it however the
work was dealt."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from _gpu_helpers import dev_f32
from _paged_reference import path_to
from test_gpu_tree import NAN, Cache, _i32, _lib, _normal, _prm  # noqa: F401

pytestmark = pytest.mark.gpu

LARGEST = torch.finfo(torch.bfloat16).max
TREE = np.array([-1, 0, 0, 1, 1, 2, 2, 3, 4, 5, 6, 6])
# rows a key head: 12, 48 and 120 (four copies, two and one of a row)
LAYOUTS = [(2, 2), (8, 2), (10, 1)]


def _flat(H):
    """A prior that is -1 at every distance, and s = 1."""
    return [dev_f32(np.full(H, x, np.float32)) for x in (1.0, 0.0, 0.0, 1.0)]


@pytest.mark.parametrize("ln", [0, 61, 5000])
@pytest.mark.parametrize("H,Hkv", LAYOUTS)
def test_large_values_out_of_sight(H, Hkv, ln):
    """The largest finite values, of both signs, in drafted nodes: the nodes
    that do not see them keep every bit, with both output types."""
    N, page = len(TREE), 64
    c = Cache(31, Hkv, page, [ln + N], -(-(ln + N) // page), NAN)
    t = [dev_f32(_prm(np.random.default_rng(4), H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, 1, H, N, 64)
    args = (c.table, _i32([ln]), *t)
    clean = c.v.clone()
    bad = {4: LARGEST, 6: -LARGEST}
    for i, value in bad.items():
        c.v[int(c.table[0, (ln + i) // page]), :, (ln + i) % page] = value
    unseen = [n for n in range(N) if not set(path_to(TREE, n)) & set(bad)]
    assert len(unseen) == 7
    for out in (torch.float32, torch.bfloat16):
        kw = dict(parents=_i32(TREE[None]), ssmax=True, o_dtype=out)
        o, lse = ba.attention_decode_tree_paged(q, c.k, c.v, *args, **kw)
        want, lse2 = ba.attention_decode_tree_paged(q, c.k, clean, *args, **kw)
        assert torch.equal(lse, lse2)
        assert torch.equal(o[:, :, unseen], want[:, :, unseen])


@pytest.mark.parametrize("ln", [61, 5000])
@pytest.mark.parametrize("H,Hkv", LAYOUTS)
def test_large_values_of_vanishing_weight(H, Hkv, ln):
    """Every seventh committed key lies 128 below the others (log2 e 128 = 184:
    its weight is 0 in 32 bits) and holds the largest value: no bit changes."""
    N, page = len(TREE), 64
    c = Cache(32, Hkv, page, [ln + N], -(-(ln + N) // page), NAN)
    q = torch.full((1, H, N, 64), 4.0, dtype=torch.bfloat16, device="cuda")
    clean = c.v.clone()
    for j in range(3, ln, 7):
        pg, r = int(c.table[0, j // page]), j % page
        c.k[pg, :, r] = -4.0
        clean[pg, :, r] = 1.0
        c.v[pg, :, r] = LARGEST if j % 2 else -LARGEST
    args = (c.table, _i32([ln]), *_flat(H))
    for out in (torch.float32, torch.bfloat16):
        kw = dict(parents=_i32(TREE[None]), o_dtype=out)
        o, lse = ba.attention_decode_tree_paged(q, c.k, c.v, *args, **kw)
        want, lse2 = ba.attention_decode_tree_paged(q, c.k, clean, *args, **kw)
        assert torch.equal(o, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B", [1, 400])
@pytest.mark.parametrize("ln", [100, 5000])
@pytest.mark.parametrize("H,Hkv", LAYOUTS)
def test_drafted_infinities_of_vanishing_weight(H, Hkv, ln, B):
    """The first 100 committed keys lie 128 above all others, so the weights of
    the drafted ones are 0 beside them.  An infinite drafted value reaches the
    nodes that see it all the same, whether the sequence is cut (alone, its
    tiles go to many CTAs) or not (among 400 that share its pages)."""
    N, page = len(TREE), 64
    c = Cache(33, Hkv, page, [ln + N], -(-(ln + N) // page), NAN)
    for j in range(ln + N):
        c.k[int(c.table[0, j // page]), :, j % page] = 4.0 if j < 100 else 0.0
    table, lens = c.table.expand(B, -1).contiguous(), _i32([ln] * B)
    q = torch.full((B, H, N, 64), 4.0, dtype=torch.bfloat16, device="cuda")
    args = (table, lens, *_flat(H))
    clean = c.v.clone()
    bad = {4: (float("inf"), [0, 20, 33]), 6: (float("-inf"), [15, 47, 63])}
    for i, (value, dims) in bad.items():
        c.v[int(c.table[0, (ln + i) // page]), :, (ln + i) % page, dims] = value
    for out in (torch.float32, torch.bfloat16):
        kw = dict(parents=_i32(np.tile(TREE, (B, 1))), o_dtype=out)
        o, lse = ba.attention_decode_tree_paged(q, c.k, c.v, *args, **kw)
        want, lse2 = ba.attention_decode_tree_paged(q, c.k, clean, *args, **kw)
        assert torch.isfinite(want).all()
        for n in range(N):
            for i in set(path_to(TREE, n)) & set(bad):
                want[:, :, n, bad[i][1]] = bad[i][0]
        assert torch.equal(o, want) and torch.equal(lse, lse2)
