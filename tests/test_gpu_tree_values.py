"""Tree attention where values are extreme or the key axis is long: what a node
does not see, or weighs with nothing, leaves no trace; an infinity that it sees
reaches it however the work was dealt; sums keep their bits over a long run."""

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


@pytest.mark.parametrize("N", [1, 40, 100])
def test_fp32_output_over_a_long_run(N):
    """304 sequences share 32768 keys of about the same weight, so that every
    CTA sums one item of 512 tiles; positive values, so that roundings which
    lean to one side add up.

    The bound, in units of sum w |v|.  Weights: as in tree_attention, a logit
    is off by delta, and o by twice its mean.  Sums of products: at most 96
    steps (16 keys, one of three parts) run on in the tensor core, each of which
    may cut off a last place: 96 * 2^-23; 64 such runs, the parts of a cut item
    (3) and copies (4) add at half a place (2^-24), the latter with factors good to
    2^-22.  Sum of weights: 18 additions in a tile, 32 tiles a run, 64 runs, 7
    parts and copies at 2^-24."""
    B, T, page = 304, 32768, 256
    ln = T - N
    gen = torch.Generator(device="cuda").manual_seed(N)
    k, v = _normal(gen, T // page, 1, page, 64), _normal(gen, T // page, 1, page, 64).abs()
    q = _normal(gen, B, 1, N, 64) * 0.05
    table = _i32(np.tile(np.arange(T // page), (B, 1)))
    o, lse = ba.attention_decode_tree_paged(q, k, v, table, _i32([ln] * B), *_flat(1))
    kd, vd = k.view(T, 64).double(), v.view(T, 64).double()
    for b in (0, 151, 303):
        for t in sorted({0, N // 2, N - 1}):
            n = ln + t + 1
            z = kd[:n] @ q[b, 0, t].double() * 0.125 - 1.0
            w = torch.softmax(z, 0)
            ref = w @ vd[:n]
            delta = 2.0 ** -18 * 0.125 * (kd[:n].abs() @ q[b, 0, t].double().abs()) + 2.0 ** -19
            err = (w * delta) @ vd[:n] + (w @ delta) * ref
            err += (96 * 2 + 64 + 7 + 7 * 4 + 18 + 32 + 64 + 7) * 2.0 ** -24 * ref
            d = (o[b, 0, t].double() - ref).abs()
            assert torch.all(d <= err), (b, t, float((d / ref).max()), float((err / ref).max()))


def test_bf16_output_over_a_very_long_run():
    """76 sequences of 4 key heads share 2^20 keys of about the same weight; 100
    rows a key head: every CTA sums one item of 16384 tiles, in four steps each.

    The mean of the relative errors.  It leans to one side by what the sums
    lose, at most: a run of 64 tiles in the tensor core at 4 * 2^-23 a tile, 256
    runs at 2^-24, three parts of a cut item at 7 * 2^-24, and 18 additions in a
    tile, 64 tiles, 256 runs and 3 parts of the sum of weights at 2^-24; 2^-18
    for the logits, as above.  Rounding the 256 outputs, spread over an octave, to
    bf16 leans to no side: at most 2^-8 each, six standard deviations of their
    mean are 6 * 2^-8 / sqrt(3 * 256).  The weights' own rounding averages out
    over 2^20 keys: 6 * 2^-8 * 2^-10."""
    B, Hkv, N, T, page = 76, 4, 100, 1 << 20, 256
    ln = T - N
    gen = torch.Generator(device="cuda").manual_seed(5)
    k = _normal(gen, T // page, Hkv, page, 64)
    v = (_normal(gen, T // page, Hkv, page, 64).abs()
         * (1 + torch.rand(1, Hkv, 1, 64, generator=gen, device="cuda"))).to(torch.bfloat16)
    q = _normal(gen, B, Hkv, N, 64) * 0.05
    table = _i32(np.tile(np.arange(T // page), (B, 1)))
    o, lse = ba.attention_decode_tree_paged(q, k, v, table, _i32([ln] * B), *_flat(Hkv),
                                            o_dtype=torch.bfloat16)
    lean = (64 * 4 * 2 + 256 + 21 + 18 + 64 + 256 + 3) * 2.0 ** -24 + 2.0 ** -18
    bound = lean + 6 * 2.0 ** -8 / np.sqrt(3 * Hkv * 64) + 6 * 2.0 ** -18
    for b, t in ((0, 0), (40, 57), (75, 99)):
        n, rel = ln + t + 1, []
        for h in range(Hkv):
            kd, vd = (x[:, h].reshape(T, 64)[:n].double() for x in (k, v))
            w = torch.softmax(kd @ q[b, h, t].double() * 0.125, 0)
            ref = w @ vd
            rel.append((o[b, h, t].double() - ref) / ref)
        rel = torch.cat(rel)
        assert abs(float(rel.mean())) <= bound, (b, t, float(rel.mean()), bound)
        assert float(rel.abs().max()) <= 2.0 ** -8 + bound
