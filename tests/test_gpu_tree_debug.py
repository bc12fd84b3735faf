"""The tree attention in the bounds-checking build: its bulk copies stay in
bounds, and its give-up paths are driven without a fault or a hang.

The n-th bounded wait of a call gives up as if its time limit had passed
(bam_attn_debug_arm_giveup): the call must report BAM_ERR_TIMEOUT and write
NaN to the rows of every node (and to no other), the context must stay usable,
and the next call on the same workspace must be right.  The debug library is a
build of its own and a process loads one library, so
`test_in_the_debug_build` runs this module again in a child process."""

import os
import re
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from _gpu_helpers import dev_f32
from _paged_reference import pack_trees, random_tree
from test_gpu_tree import Cache, _i32, _normal, _prm, _tree_case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
IN_DEBUG = ba.DEBUG
debug_only = pytest.mark.skipif(not IN_DEBUG, reason="runs in the debug-library child process")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.skipif(IN_DEBUG, reason="this is the child process")
def test_in_the_debug_build():
    from transformer_attention_ggd_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, BAM_ATTN_DEBUG="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p",
                        "no:cacheprovider", os.path.abspath(__file__)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = r.stdout[-6000:] + r.stderr[-3000:]
    assert r.returncode == 0, tail
    assert int(re.search(r"(\d+) passed", r.stdout).group(1)) >= 20, tail


@debug_only
@pytest.mark.parametrize("H,Hkv,N,page,out", [(4, 4, 7, 64, "bf16"), (8, 1, 9, 128, "fp32"),
                                              (2, 2, 60, 64, "bf16"), (2, 1, 128, 320, "bf16"),
                                              (40, 1, 3, 64, "bf16"), (128, 1, 1, 64, "fp32")])
def test_copies_stay_in_bounds(H, Hkv, N, page, out):
    assert ba.bam_attn_debug_build()
    rng = np.random.default_rng(N)
    lens, new = [0, 1, 700, 63, 1500], [N, 1, N, 0, max(1, N - 1)]
    _tree_case(N, 5, H, Hkv, N, page, lens, new, [random_tree(rng, n) for n in new], True, False,
               out, slack=1)


@debug_only
@pytest.mark.parametrize("N", [5, 50, 100])
@pytest.mark.parametrize("at", [1, 2, 7, 30, 200, 1500])
def test_giveup(N, at):
    B, H, Hkv, page = 3, 4, 2, 64
    rng = np.random.default_rng(N)
    lens, new = [3000, 20, 900], [N, max(1, N - 2), 0]
    c = Cache(N, Hkv, page, [a + n for a, n in zip(lens, new)], 50)
    parents = pack_trees([random_tree(rng, n) for n in new], B, N)
    t = [dev_f32(_prm(rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    prm = ba.make_params(*t, 1e-5, True, True)
    q = _normal(c.gen, B, H, N, 64)
    ws = ba.tree_workspace(B, H, Hkv, N, 50 * page)

    def call():
        o = torch.full((B, H, N, 64), 3.0, device="cuda")
        lse = torch.full((B, H, N), 3.0, device="cuda")
        ba.bam_attn_decode_tree_paged(q, c.k, c.v, c.table, _i32(lens), _i32(new), _i32(parents), o,
                                      lse, prm, ws)
        return o, lse, ba.bam_attn_check_status(ws)

    good = call()
    assert good[2] == ba.BAM_OK
    assert ba.bam_attn_debug_arm_giveup(ws, at) == ba.BAM_OK
    o, lse, st = call()
    ba.bam_attn_debug_arm_giveup(ws, 0)
    assert st in (ba.BAM_ERR_TIMEOUT, ba.BAM_OK)
    assert st == ba.BAM_ERR_TIMEOUT or at > 200  # a call may have fewer waits than that
    for b in range(B):
        if st == ba.BAM_ERR_TIMEOUT:
            assert torch.isnan(o[b, :, :new[b]]).all() and torch.isnan(lse[b, :, :new[b]]).all()
        assert torch.all(o[b, :, new[b]:] == 3.0) and torch.all(lse[b, :, new[b]:] == 3.0)
    again = call()
    assert again[2] == ba.BAM_OK
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
