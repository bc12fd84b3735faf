"""Host-side refusals of the paged-cache operators (append, tree attention,
keep): every call here returns before anything is launched, so no GPU is
needed.  Also pins the tests' 64-bit tree attention on the oracle."""

import ctypes
import struct

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from transformer_attention_ggd_gb300 import bam_attn as ba
from transformer_attention_ggd_gb300 import build as lib_build

from _paged_reference import path_to, random_tree, rows_of, tree_attention

FAKE = 0x7F0000000000  # 256-aligned, never dereferenced
OK_SIZES = dict(B=2, H=4, Hkv=2, N=8, page=64, mb=4, pages=8, D=64)


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return ba.load_library()


def vp(x):
    return ctypes.c_void_p(x)


def _sizes(kw):
    z = dict(OK_SIZES)
    z.update({k: kw[k] for k in z if k in kw})
    return z


def _append(lib, **kw):
    z = _sizes(kw)
    p = {n: kw.get(n, FAKE) for n in ("k", "v", "q", "qo", "kp", "vp", "bt", "lens", "new", "par", "ws")}
    rope = kw.get("rope", ba.BamRope(10000.0, 64, 0))
    st = kw.get("strides", [64 * 8 * 2, 64 * 8, 64] * 3)
    return lib.bam_kv_append_paged(
        vp(p["k"]), vp(p["v"]), vp(p["q"]), vp(p["qo"]), (ctypes.c_int64 * 9)(*st) if st else None,
        vp(p["kp"]), vp(p["vp"]), vp(p["bt"]), vp(p["lens"]), vp(p["new"]), vp(p["par"]), z["B"],
        z["H"], z["Hkv"], z["N"], z["page"], z["mb"], z["pages"], z["D"],
        ctypes.byref(rope) if rope else None, vp(p["ws"]), kw.get("ws_bytes", 1 << 30), None)


def _tree(lib, **kw):
    z = _sizes(kw)
    p = {n: kw.get(n, FAKE) for n in ("q", "kp", "vp", "bt", "lens", "new", "par", "o", "lse", "ws")}
    prm = kw.get("prm", ba.BamParams(FAKE, FAKE, FAKE, FAKE, 1e-5, 1, 1, ba.BAM_PRIOR_ALPHA))
    return lib.bam_attn_decode_tree_paged(
        vp(p["q"]), vp(p["kp"]), vp(p["vp"]), vp(p["bt"]), vp(p["lens"]), vp(p["new"]), vp(p["par"]),
        vp(p["o"]), 1, vp(p["lse"]), z["B"], z["H"], z["Hkv"], z["N"], z["page"], z["mb"], z["pages"],
        z["D"], ctypes.byref(prm) if prm else None, vp(p["ws"]), kw.get("ws_bytes", 1 << 30), None)


def _keep(lib, **kw):
    z = _sizes(kw)
    p = {n: kw.get(n, FAKE) for n in ("kp", "vp", "bt", "lens", "new", "par", "acc", "nl", "ws")}
    return lib.bam_kv_keep_paged(
        vp(p["kp"]), vp(p["vp"]), vp(p["bt"]), vp(p["lens"]), vp(p["new"]), vp(p["par"]), vp(p["acc"]),
        vp(p["nl"]), z["B"], z["Hkv"], z["N"], z["page"], z["mb"], z["pages"], z["D"], vp(p["ws"]),
        kw.get("ws_bytes", 1 << 30), None)


@pytest.mark.parametrize("call", [_append, _tree, _keep])
@pytest.mark.parametrize("kw,want", [
    (dict(B=0), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"), (dict(N=0), "INVALID_ARG"),
    (dict(mb=0), "INVALID_ARG"), (dict(pages=0), "INVALID_ARG"), (dict(page=32), "INVALID_ARG"),
    (dict(page=96), "INVALID_ARG"), (dict(D=128), "UNSUPPORTED"), (dict(B=65536), "UNSUPPORTED"),
    (dict(N=129), "UNSUPPORTED"), (dict(page=1 << 20, mb=1 << 10), "UNSUPPORTED"),
    (dict(pages=1 << 30, Hkv=4), "UNSUPPORTED"), (dict(bt=0), "INVALID_ARG"),
    (dict(lens=0), "INVALID_ARG"), (dict(bt=FAKE + 2), "INVALID_ARG"),
    (dict(new=FAKE + 2), "INVALID_ARG"), (dict(par=FAKE + 1), "INVALID_ARG"),
    (dict(kp=0), "INVALID_ARG"), (dict(vp=FAKE + 8), "INVALID_ARG"), (dict(ws=0), "WORKSPACE"),
    (dict(ws=FAKE + 16), "WORKSPACE"), (dict(ws_bytes=100), "WORKSPACE")])
def test_refusals_of_every_operator(lib, call, kw, want):
    assert call(lib, **kw) == getattr(ba, "BAM_ERR_" + want)


@pytest.mark.parametrize("kw,want", [
    (dict(k=0), "INVALID_ARG"), (dict(v=FAKE + 8), "INVALID_ARG"), (dict(q=0), "INVALID_ARG"),
    (dict(qo=0), "INVALID_ARG"), (dict(H=3), "INVALID_ARG"),
    (dict(rope=ba.BamRope(10000.0, 8, 0)), "INVALID_ARG"),
    (dict(rope=ba.BamRope(10000.0, 80, 0)), "INVALID_ARG"),
    (dict(rope=ba.BamRope(10000.0, -16, 0)), "INVALID_ARG"),
    (dict(rope=ba.BamRope(0.0, 64, 0)), "INVALID_ARG"),
    (dict(rope=ba.BamRope(float("inf"), 64, 0)), "INVALID_ARG"),
    (dict(rope=ba.BamRope(float("nan"), 64, 0)), "INVALID_ARG"),
    (dict(rope=ba.BamRope(10000.0, 64, 2)), "INVALID_ARG"),
    (dict(strides=[512, 64, 60] * 3), "INVALID_ARG"),
    (dict(strides=[512, -64, 64] * 3), "INVALID_ARG")])
def test_append_refusals(lib, kw, want):
    assert _append(lib, **kw) == getattr(ba, "BAM_ERR_" + want)


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), "INVALID_ARG"), (dict(o=0), "INVALID_ARG"), (dict(o=FAKE + 8), "INVALID_ARG"),
    (dict(lse=FAKE + 2), "INVALID_ARG"), (dict(H=3), "INVALID_ARG"), (dict(prm=None), "INVALID_ARG"),
    (dict(prm=ba.BamParams(FAKE, FAKE, FAKE, 0, 1e-5, 1, 1, 0)), "INVALID_ARG"),
    (dict(prm=ba.BamParams(FAKE, FAKE, FAKE, 0, 0.0, 1, 0, 0)), "INVALID_ARG"),
    (dict(prm=ba.BamParams(FAKE, FAKE, FAKE, 0, 1e-5, 1, 0, 7)), "INVALID_ARG")])
def test_tree_refusals(lib, kw, want):
    assert _tree(lib, **kw) == getattr(ba, "BAM_ERR_" + want)


@pytest.mark.parametrize("kw", [dict(acc=0), dict(acc=FAKE + 2), dict(nl=0), dict(nl=FAKE + 1)])
def test_keep_refusals(lib, kw):
    assert _keep(lib, **kw) == ba.BAM_ERR_INVALID_ARG


def test_tree_workspace_sizes(lib):
    n = ba.bam_attn_tree_workspace_size(4, 8, 2, 16, 4096)
    assert n > 0 and n % 256 == 0
    for bad in [(0, 8, 2, 16, 4096), (4, 7, 2, 16, 4096), (4, 8, 2, 129, 4096), (4, 8, 2, 16, 0),
                (4, 8, 2, 0, 4096), (4, 8, 2, 16, 1 << 29), (65536, 8, 2, 16, 64)]:
        assert ba.bam_attn_tree_workspace_size(*bad) == 0
    assert ba.bam_attn_tree_workspace_size(4, 8, 2, 16, 4096, 128) == 0


def test_make_rope_checks_its_arguments():
    assert ba.make_rope(500.0, 32, True).interleaved == 1
    for bad in (dict(dims=8), dict(dims=80), dict(dims=-16), dict(base=0.0), dict(base=float("inf")),
                dict(base=float("nan"))):
        with pytest.raises(ValueError):
            ba.make_rope(**bad)


def test_binding_refuses_host_tensors_before_the_library():
    x = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    table, par = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 8, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    prm = ba.make_params(*(torch.ones(2) for _ in range(4)))
    for f in (lambda: ba.bam_kv_append_paged(x, x, pages, pages, table, i, i, par, None, None, None, ws),
              lambda: ba.bam_attn_decode_tree_paged(x, pages, pages, table, i, i, par, x, None, prm, ws),
              lambda: ba.bam_kv_keep_paged(pages, pages, table, i, i, par, i, i, ws)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()


@pytest.mark.parametrize("theta,ssmax", [(False, True), (True, False)])
def test_reference_tree_attention_is_a_decode_over_each_path(theta, ssmax):
    """Every node's row is the oracle's decode over the committed keys followed
    by the node's path."""
    rng = np.random.default_rng(3)
    g = torch.Generator().manual_seed(3)
    B, H, Hkv, N, page = 2, 4, 2, 6, 64
    lens, new = [70, 0], [6, 4]
    kp, vpg = (torch.randn(5, Hkv, page, 64, generator=g).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[3, 1], [4, -1]], dtype=torch.int32)
    parents = [random_tree(rng, n) for n in new]
    q = torch.randn(B, H, N, 64, generator=g).to(torch.bfloat16)
    prm = [rng.uniform(0.5, 2, H), rng.uniform(-0.5, 1.5, H), rng.uniform(0, 1, H), rng.uniform(0.3, 1, H)]
    o, lse, oerr, lerr = tree_attention(q, kp, vpg, table, lens, new, parents,
                                        [torch.from_numpy(x) for x in prm], ssmax, theta, False)
    for b in range(B):
        for t in range(new[b]):
            slots = list(range(lens[b])) + [lens[b] + i for i in path_to(parents[b], t)]
            k, v = (rows_of(x, table[b], slots).repeat_interleave(2, 0).numpy()[None] for x in (kp, vpg))
            oref, lref = oracle.decode(q[b:b + 1, :, t].double().numpy(), k, v, *prm, ssmax=ssmax,
                                       **({"prior": ba.BAM_PRIOR_THETA} if theta else {}))
            np.testing.assert_allclose(o[b, :, t].numpy(), oref[0], rtol=0, atol=1e-10)
            np.testing.assert_allclose(lse[b, :, t].numpy(), lref[0], rtol=0, atol=1e-10)
    assert float(oerr[:, :, 0].max()) < 1e-3


WORDS = {"append": [FAKE, FAKE, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                    2, 4, 2, 3, 64, 4, 8, 64, 0, FAKE, 1 << 30, 0],
         "tree": [FAKE] * 8 + [0, FAKE, 2, 4, 2, 3, 64, 4, 8, 64, 0, FAKE, 1 << 30, 0],
         "keep": [FAKE] * 8 + [2, 2, 3, 64, 4, 8, 64, FAKE, 1 << 30, 0]}


@pytest.mark.parametrize("op,at,value,want", [
    ("append", 11, 0, "INVALID_ARG"), ("append", 12, 3, "INVALID_ARG"), ("append", 14, 129, "UNSUPPORTED"),
    ("append", 15, 32, "INVALID_ARG"), ("append", 18, 128, "UNSUPPORTED"), ("append", 2, 0, "INVALID_ARG"),
    ("append", 0, FAKE + 8, "INVALID_ARG"), ("append", 21, 100, "WORKSPACE"), ("append", 4, 2, "INVALID_ARG"),
    ("append", 11, (1 << 32) + 2, "INVALID_ARG"), ("append", 10, FAKE + 1, "INVALID_ARG"),
    ("tree", 10, 0, "INVALID_ARG"), ("tree", 12, 3, "INVALID_ARG"), ("tree", 17, 128, "UNSUPPORTED"),
    ("tree", 18, 0, "INVALID_ARG"), ("tree", 13, 129, "UNSUPPORTED"), ("tree", 8, 1 << 32, "INVALID_ARG"),
    ("tree", 16, 1 << 33, "INVALID_ARG"), ("tree", 3, 0, "INVALID_ARG"),
    ("keep", 8, 0, "INVALID_ARG"), ("keep", 10, 129, "UNSUPPORTED"), ("keep", 11, 96, "INVALID_ARG"),
    ("keep", 6, 0, "INVALID_ARG"), ("keep", 7, FAKE + 2, "INVALID_ARG"), ("keep", 16, 100, "WORKSPACE"),
    ("keep", 15, 0, "WORKSPACE"), ("keep", 13, -(1 << 32) + 8, "INVALID_ARG")])
def test_refusals_of_calls_by_words(lib, op, at, value, want):
    words = list(WORDS[op])
    words[at] = value
    number = list(WORDS).index(op)
    assert lib.bam_paged_call(number, struct.pack(f"{len(words)}q", *words)) == getattr(ba, "BAM_ERR_" + want)


def test_calls_by_words_need_an_operator_and_words(lib):
    words = struct.pack("32q", *([0] * 32))
    for op in (-1, 3, 1 << 20):
        assert lib.bam_paged_call(op, words) == ba.BAM_ERR_INVALID_ARG
    assert lib.bam_paged_call(0, None) == ba.BAM_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        ba._struct_address(object(), ba.BamRope)


@pytest.mark.parametrize("base", [1.0 - 2.0 ** -53, 0.5, 1e-12, 1e-300, -1.0])
def test_a_rotation_needs_a_base_of_at_least_one(lib, base):
    """Below it a position is many turns, of which 64 bits hold no fraction that
    is right at far positions (none at all for 1e-300)."""
    assert _append(lib, rope=ba.BamRope(base, 64, 0)) == ba.BAM_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="at least 1"):
        ba.make_rope(base)
