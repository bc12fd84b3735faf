"""Every kind of wait of the tree attention kernel gives up once, in the
debug build: the call then reports it, writes NaN to the rows of every node and
to no other, and leaves the context and the workspace usable.

The waits are counted over the whole grid, so which one an ordinal hits depends
on how the CTAs run; ordinals are drawn until each kind has been hit.  The call
makes more waits than the largest of them: each of its 1402 items is waited for,
and its S, keys, values and last product, by 128 threads.  As the debug library is a
build of its own, `test_in_the_debug_build` runs this module in a child
process."""

import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from _gpu_helpers import dev_f32
from _paged_reference import pack_trees, random_tree
from test_gpu_tree import Cache, _i32, _normal, _prm

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
IN_DEBUG = ba.DEBUG
# the sites of csrc/tree.cu
KINDS = {"producer": {60, 61}, "product": {63, 64, 65, 66}, "item": {67}, "S": {68},
         "keys and values": {69}, "P V": {70}, "item's end": {71}, "copies": {72}}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.skipif(IN_DEBUG, reason="this is the child process")
def test_in_the_debug_build():
    from transformer_attention_ggd_gb300 import build
    build.build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p",
                        "no:cacheprovider", os.path.abspath(__file__)],
                       cwd=ROOT, env=dict(os.environ, BAM_ATTN_DEBUG="1"), capture_output=True,
                       text=True, timeout=600)
    tail = r.stdout[-6000:] + r.stderr[-3000:]
    assert r.returncode == 0 and "1 passed" in r.stdout, tail


@pytest.mark.skipif(not IN_DEBUG, reason="runs in the debug-library child process")
def test_every_kind_of_wait_gives_up():
    B, H, Hkv, N, page = 701, 4, 2, 5, 64
    rng = np.random.default_rng(3)
    lens, new = rng.integers(1, 30, B), rng.integers(1, N + 1, B)
    lens[350] = 6000
    c = Cache(7, Hkv, page, lens + new, 95)
    parents = _i32(pack_trees([random_tree(rng, n) for n in new], B, N))
    t = [dev_f32(_prm(rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    prm = ba.make_params(*t, 1e-5, True, True)
    q = _normal(c.gen, B, H, N, 64)
    ws = ba.tree_workspace(B, H, Hkv, N, 95 * page)
    lens, new = _i32(lens), _i32(new)
    live = (torch.arange(N, device="cuda")[None] < new[:, None])[:, None].expand(B, H, N)
    o, lse = torch.empty(B, H, N, 64, device="cuda"), torch.empty(B, H, N, device="cuda")

    def call():
        o.fill_(3.0)
        lse.fill_(3.0)
        ba.bam_attn_decode_tree_paged(q, c.k, c.v, c.table, lens, new, parents, o, lse, prm, ws)

    call()
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    good = o.clone(), lse.clone()
    missing = dict(KINDS)
    for _ in range(6000):
        assert ba.bam_attn_debug_arm_giveup(ws, int(rng.integers(1, 500_000))) == ba.BAM_OK
        call()
        site = int(ws[:16].cpu().numpy().view(np.int32)[2])
        assert ba.bam_attn_check_status(ws) == ba.BAM_ERR_TIMEOUT
        kind = next(k for k, sites in KINDS.items() if site in sites)
        if kind in missing:
            del missing[kind]
            assert torch.isnan(o[live]).all() and torch.isnan(lse[live]).all()
            assert torch.all(o[~live] == 3.0) and torch.all(lse[~live] == 3.0)
        if not missing:
            break
    assert not missing, missing
    ba.bam_attn_debug_arm_giveup(ws, 0)
    call()
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
