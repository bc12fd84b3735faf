"""The shared decode in the bounds-checking build: its copies stay in bounds, and
its give-up paths are driven without a fault or a hang.

The n-th bounded wait of a call gives up as if its time limit had passed: the
call must report BAM_ERR_TIMEOUT, write NaN to every row and leave the weights as
they were, and the next call on the same workspace must be right.  A process
loads one library, so `test_in_the_debug_build` runs this module again in a
child process."""

import os
import re
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from _gpu_helpers import dev_f32
from test_gpu_shared import Cache, _case, _i32, _normal, _prm

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
@pytest.mark.parametrize("marked", [False, True])
@pytest.mark.parametrize("H,Hkv,page,P,out", [(4, 4, 64, 0, "bf16"), (8, 1, 128, 1000, "fp32"),
                                              (2, 2, 320, 64, "bf16"), (40, 2, 64, 129, "fp32")])
def test_copies_stay_in_bounds(H, Hkv, page, P, out, marked):
    assert ba.bam_attn_debug_build()
    _case(P + H, H, Hkv, page, [0, 1, 700, 63, 1500], P, marked, out=out, slack=1, prefix_slack=1)
    _case(P + H, H, Hkv, page, [7] * 90, P, marked, out=out)


@debug_only
@pytest.mark.parametrize("marked", [False, True])
@pytest.mark.parametrize("at", [1, 2, 7, 30, 200, 1500, 5000])
def test_giveup(at, marked):
    B, H, Hkv, P = 40, 4, 2, 5000
    rng = np.random.default_rng(at)
    lens = [3000, 20] + [60] * (B - 2)
    c = Cache(3, Hkv, 64, lens, P)
    t = [dev_f32(_prm(rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    prm = ba.make_params(*t, 1e-5, True, True)
    q = _normal(c.gen, B, H, 64)
    ws = ba.shared_workspace(B, H, Hkv, c.prefix.numel() * 64, c.table.shape[1] * 64, c.max_pos if marked else 0)
    marks = ba.make_marks(c.pos, c.w, c.max_pos) if marked else None
    w0 = c.w.clone()

    def call():
        c.w.copy_(w0)
        o, lse = torch.full((B, H, 64), 3.0, device="cuda"), torch.full((B, H), 3.0, device="cuda")
        ba.bam_attn_decode_shared_paged(q, c.k, c.v, c.table, _i32(lens), c.prefix, _i32([P]),
                                        c.q_pos if marked else None, marks, 1.0, o, lse, prm, ws)
        return o, lse, c.w.view(torch.int32).clone(), ba.bam_attn_check_status(ws)

    good = call()
    assert good[3] == ba.BAM_OK
    assert ba.bam_attn_debug_arm_giveup(ws, at) == ba.BAM_OK
    o, lse, w, st = call()
    ba.bam_attn_debug_arm_giveup(ws, 0)
    assert st == ba.BAM_ERR_TIMEOUT
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    assert torch.equal(w, w0.view(torch.int32))
    again = call()
    assert again[3] == ba.BAM_OK
    assert all(torch.equal(x, y) for x, y in zip(again[:3], good[:3]))


@debug_only
@pytest.mark.parametrize("B,out", [(20, "bf16"), (50, "fp32"), (130, "bf16")])
@pytest.mark.parametrize("at", [1, 40, 700, 4000])
def test_giveup_of_every_prefix_variant(at, B, out):
    H, P = 2, 9000
    rng = np.random.default_rng(at)
    lens = [b % 3 for b in range(B)]
    c = Cache(4, H, 64, lens, P)
    t = [dev_f32(_prm(rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    prm = ba.make_params(*t, 1e-5, True, True)
    q = _normal(c.gen, B, H, 64)
    ws = ba.shared_workspace(B, H, H, c.prefix.numel() * 64, c.table.shape[1] * 64)

    def call():
        o = torch.full((B, H, 64), 3.0, device="cuda", dtype=torch.bfloat16 if out == "bf16" else torch.float32)
        ba.bam_attn_decode_shared_paged(q, c.k, c.v, c.table, _i32(lens), c.prefix, _i32([P]), None, None, 1.0, o,
                                        None, prm, ws)
        return o, ba.bam_attn_check_status(ws)

    good, st = call()
    assert st == ba.BAM_OK
    assert ba.bam_attn_debug_arm_giveup(ws, at) == ba.BAM_OK
    o, st = call()
    ba.bam_attn_debug_arm_giveup(ws, 0)
    assert st == ba.BAM_ERR_TIMEOUT and torch.isnan(o).all()
    o, st = call()
    assert st == ba.BAM_OK and torch.equal(o, good)
