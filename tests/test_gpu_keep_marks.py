"""GPU tests of a kept draft in a cache with marks: positions and weights move with their
keys, and the next marked decode and eviction see them."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from _bounded_reference import decode, kept_slots
from _gpu_helpers import dev_f32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ba.load_library()


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _draft(rng, B, N):
    """Random trees, and the path from a root to a node of each (-1: none)."""
    parents = np.stack([[rng.integers(-1, i) for i in range(N)] for _ in range(B)])
    accepted = rng.integers(-1, N, B)
    accepted[0] = N - 1
    paths = []
    for b in range(B):
        path, i = [], int(accepted[b])
        while i >= 0:
            path.append(i)
            i = int(parents[b][i])
        paths.append(path[::-1])
    return parents, accepted, paths


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("Hkv,N,page", [(1, 6, 64), (2, 40, 64), (12, 128, 128), (40, 17, 64)])
def test_marks_move_with_their_keys(Hkv, N, page, alias):
    rng = np.random.default_rng(Hkv + N)
    gen = torch.Generator(device="cuda").manual_seed(N)
    B, lens = 4, [60, 0, 200, 63]
    parents, accepted, paths = _draft(rng, B, N)
    mb = -(-(max(lens) + N) // page)
    table = rng.permutation(B * mb + 1)[:B * mb].reshape(B, mb)
    kp, vp = _normal(gen, B * mb + 1, Hkv, page, 64), _normal(gen, B * mb + 1, Hkv, page, 64)
    kpos = torch.randint(0, 1 << 20, kp.shape[:3], generator=gen, device="cuda", dtype=torch.int32)
    kw = torch.rand(kp.shape[:3], generator=gen, device="cuda")
    marks, ws = ba.make_marks(kpos, kw, 1 << 20), ba.cache_workspace()
    want = [x.cpu().clone() for x in (kp.view(torch.int16), vp.view(torch.int16), kpos, kw)]
    free = torch.zeros(want[2].shape, dtype=torch.bool)  # what is left of the draft
    for b in range(B):
        old = [x.clone() for x in want]
        for m, node in enumerate(paths[b]):
            s, d = lens[b] + node, lens[b] + m
            for x, y in zip(want, old):
                x[table[b, d // page], :, d % page] = y[table[b, s // page], :, s % page]
        for s in range(lens[b] + len(paths[b]), lens[b] + N):
            free[table[b, s // page], :, s % page] = True
    ln = _i32(lens)
    new = ba.kv_keep_paged(kp, vp, _i32(table), ln, _i32(accepted), _i32(parents), new_lens=ln if alias else None,
                           ws=ws, marks=marks)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    assert new.tolist() == [n + len(p) for n, p in zip(lens, paths)]
    for x, y in zip((kp.view(torch.int16), vp.view(torch.int16), kpos, kw), want):
        assert torch.equal(x.cpu()[~free], y[~free])


def test_marks_stay_where_a_path_cannot_be_kept():
    gen = torch.Generator(device="cuda").manual_seed(1)
    kp, vp = _normal(gen, 3, 2, 64, 64), _normal(gen, 3, 2, 64, 64)
    kpos = torch.arange(3 * 2 * 64, device="cuda", dtype=torch.int32).view(3, 2, 64)
    kw = torch.rand(3, 2, 64, generator=gen, device="cuda")
    saved = [x.clone() for x in (kp, vp, kpos, kw)]
    ws = ba.cache_workspace()
    new = ba.kv_keep_paged(kp, vp, _i32([[0, 9]]), _i32([62]), _i32([3]), _i32([[-1, 0, 0, 2]]), ws=ws,
                           marks=ba.make_marks(kpos, kw, 1000))
    assert ba.bam_attn_check_status(ws) == ba.BAM_ERR_INVALID_ARG and new.tolist() == [62]
    assert all(torch.equal(x, y) for x, y in zip((kp, vp, kpos, kw), saved))


def test_a_draft_in_a_marked_cache_and_the_steps_after_it():
    """Append a branching draft with marks, keep a path, decode, evict; the keep and the
    decode captured and replayed."""
    rng, gen = np.random.default_rng(5), torch.Generator(device="cuda").manual_seed(5)
    B, H, Hkv, page, N = 2, 4, 2, 64, 8
    lens, first = [61, 30], [500, 900]
    table = _i32([[3, 0], [1, 4]])
    kp, vp = _normal(gen, 5, Hkv, page, 64), _normal(gen, 5, Hkv, page, 64)
    kpos = torch.randint(0, 400, (5, Hkv, page), generator=gen, device="cuda", dtype=torch.int32)
    kw = torch.rand(5, Hkv, page, generator=gen, device="cuda")
    marks = ba.make_marks(kpos, kw, 1 << 16)
    parents, path = [[-1, -1, 0, 1, 1, 4, 4, 6]] * B, [1, 4, 6, 7]
    t = [dev_f32(x) for x in ([30.0] * H, [0.8] * H, [1.0] * H, [0.7] * H)]
    k, v = _normal(gen, B, Hkv, N, 64), _normal(gen, B, Hkv, N, 64)
    ln, q = _i32(lens), _normal(gen, B, H, 64)
    ba.kv_append_norm_paged(k, v, kp, vp, table, ln, parents=_i32(parents), first_pos=_i32(first), marks=marks)
    acc, par, at = _i32([7, 6]), _i32(parents), _i32([600, 950])
    params = ba.make_params(*t, 1e-5, True, True)
    cws, sws = ba.cache_workspace(), ba.shared_workspace(B, H, Hkv, 0, 2 * page, 1 << 16)
    o, lse = torch.zeros(B, H, 64, device="cuda"), torch.zeros(B, H, device="cuda")

    def steps():
        ba.bam_kv_keep_paged(kp, vp, table, ln, None, par, acc, ln, cws, marks=marks)
        ba.bam_attn_decode_shared_paged(q, kp, vp, table, ln, None, None, at, marks, 1.0, o, lse, params, sws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    graph.replay()
    torch.cuda.synchronize()
    kept = [path, path[:3]]
    assert ln.tolist() == [65, 33]
    for b in range(B):
        for m, node in enumerate(kept[b]):
            s = lens[b] + m
            pg = int(table[b, s // page])
            assert torch.equal(kp[pg, :, s % page], k[b, :, node]) and torch.equal(vp[pg, :, s % page], v[b, :, node])
            assert torch.all(kpos[pg, :, s % page] == first[b] + m)  # depth m
    n = ln.tolist()
    oref, lref, wref, oerr, lerr, werr = decode(q, kp, vp, table, n, None, 0, kpos, at, t, True, False, False)
    assert torch.all((o.double() - oref).abs() <= oerr) and torch.all((lse.double() - lref).abs() <= lerr)
    for b in range(B):  # the kept keys' weights began at 0
        for m in range(len(kept[b])):
            s = lens[b] + m
            d = (kw[int(table[b, s // page]), :, s % page].double() - wref[b][s]).abs()
            assert torch.all(d <= werr[b][s] + 2.0 ** -23 * wref[b][s])
    before = [x.clone() for x in (kpos, kw)]
    ba.kv_evict_paged(kp, vp, table, ln, marks, 32, 2, 4, new_lens=ln)
    assert ln.tolist() == [32, 32]
    for b in range(B):
        for h in range(Hkv):
            s, m, rows = np.arange(n[b]), np.arange(32), table[b].cpu().numpy()
            keep = kept_slots(before[1].cpu().numpy()[rows[s // page], h, s % page], 32, 2, 4)
            for x, y in zip((kpos, kw), before):
                assert torch.equal(x[rows[m // page], h, m % page], y[rows[keep // page], h, keep % page])


def test_keep_refuses_marks_of_another_pool():
    kp = torch.zeros(2, 2, 64, 64, device="cuda", dtype=torch.bfloat16)
    marks = ba.make_marks(torch.zeros(1, 2, 64, device="cuda", dtype=torch.int32), torch.zeros(1, 2, 64, device="cuda"), 9)
    with pytest.raises(ValueError, match="marks"):
        ba.kv_keep_paged(kp, kp.clone(), _i32([[0, 1]]), _i32([3]), _i32([0]), _i32([[-1, 0]]), marks=marks)
