"""Appends of so many tokens that a CTA takes several token tiles one after the
other, across heads, tiles and sequences, against 64-bit rotations."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from _paged_reference import pack_trees, random_tree
from test_gpu_tree import Cache, _i32, _lib, _normal  # noqa: F401

pytestmark = pytest.mark.gpu


def _rotate(x, pos, base, dims, interleaved):
    """x float64 [B, h, N, 64] turned by positions pos [B, N]."""
    out = x.clone()
    for f in range(dims // 2):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + dims // 2)
        ang = pos.double()[:, None] * base ** (-2.0 * f / dims)
        out[..., i] = x[..., i] * ang.cos() - x[..., j] * ang.sin()
        out[..., j] = x[..., j] * ang.cos() + x[..., i] * ang.sin()
    return out


def _depths(parents):
    d = np.zeros(len(parents), np.int64)
    for i, p in enumerate(parents):
        d[i] = d[p] + 1 if p >= 0 else 0
    return d


def _case(seed, H, Hkv, N, page, lens, new, parents, dims, interleaved, in_place=False):
    B = len(lens)
    # token tiles of 16: more of them than 304 resident CTAs take at once
    assert B * -(-N // 16) > 2 * 304
    used = [a + n for a, n in zip(lens, new)]
    c = Cache(seed, Hkv, page, used, -(-max(used) // page), 3.0)
    if in_place:
        q, k, v = (_normal(c.gen, B, h, N, 64) for h in (H, Hkv, Hkv))
        q_in = q.clone()
        q_out = q
    else:
        qkv = _normal(c.gen, B, N, H + 2 * Hkv, 64)
        q, k, v = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
        q_in = q
        q_out = torch.full((B, H, N, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    rest = q_out.clone()
    before = c.k.clone(), c.v.clone()
    ws = ba.cache_workspace()
    base = 10000.0
    ba.bam_kv_append_paged(k, v, c.k, c.v, c.table, _i32(lens), _i32(new),
                           None if parents is None else _i32(pack_trees(parents, B, N)), q, q_out,
                           ba.make_rope(base, dims, interleaved), ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK

    i = torch.arange(N, device="cuda")
    live = i[None] < _i32(new)[:, None]
    depth = i.expand(B, N).clone()
    if parents is not None:
        for b, p in enumerate(parents):
            depth[b, :len(p)] = torch.from_numpy(_depths(p)).cuda()
    start = _i32(lens)[:, None].long()
    slot = (start + i).clamp(max=c.table.shape[1] * page - 1)
    pg, row = c.table.long().gather(1, slot // page), slot % page
    want_k, want_v = before
    got_k = c.k[pg[live], :, row[live]]            # [tokens, Hkv, 64]
    want_k[pg[live], :, row[live]] = got_k
    want_v[pg[live], :, row[live]] = v.transpose(1, 2)[live]
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)
    off = (~live)[:, None, :].expand(B, H, N)
    assert torch.equal(q_out[off], rest[off])
    for x, got in ((k, got_k), (q_in, q_out.transpose(1, 2)[live])):
        ref = _rotate(x.double(), start + depth, base, dims, interleaved).transpose(1, 2)[live]
        x = x.transpose(1, 2)[live]
        # half a bf16 step of the result, and fp32 angles (2^-22) of the pair's magnitude
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -21 * x.double().norm(dim=-1, keepdim=True)
        assert torch.all((got.double() - ref).abs() <= tol)
        assert torch.equal(got[..., dims:], x[..., dims:])


@pytest.mark.parametrize("dims,interleaved,page", [(64, False, 64), (32, True, 320), (0, False, 64)])
def test_ragged_prompts(dims, interleaved, page):
    """Prompts of thousands of tokens among some of few and of none."""
    rng = np.random.default_rng(dims)
    new = [3000, 0, 1, 2999, 17, 0, 0, 3000, 16, 1500, 15, 2048]
    lens = rng.integers(0, 700, len(new)).tolist()
    _case(1, 6, 2, 3000, page, lens, new, None, dims, interleaved)


@pytest.mark.parametrize("H,Hkv,N,interleaved", [(4, 2, 128, False), (40, 8, 48, True)])
def test_drafts_of_a_large_batch(H, Hkv, N, interleaved):
    """Trees of more sequences than CTAs, so that one CTA crosses sequences; 40
    heads take several units of a tile."""
    rng = np.random.default_rng(N)
    B = 340
    new = rng.integers(0, N + 1, B)
    new[:3] = N, 0, 1
    lens = rng.integers(0, 300, B).tolist()
    _case(2, H, Hkv, N, 64, lens, new.tolist(), [random_tree(rng, int(n)) for n in new], 48, interleaved)


def test_queries_in_place():
    rng = np.random.default_rng(7)
    new = rng.integers(0, 41, 330)
    _case(3, 20, 20, 40, 64, rng.integers(0, 200, 330).tolist(), new.tolist(),
          [random_tree(rng, int(n)) for n in new], 64, False, in_place=True)


def test_prompts_with_queries_in_place():
    _case(4, 3, 3, 2500, 64, [5, 0, 64, 1000], [2500, 2400, 33, 2500], None, 64, True, in_place=True)
