"""Host-side refusals of the norms, the appends with norms, the shared decode and
the eviction: every call here returns before anything is launched, so no GPU is
needed.  Also pins the tests' references on the oracle and on differences."""

import ctypes
import struct

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from transformer_attention_ggd_gb300 import bam_attn as ba
from transformer_attention_ggd_gb300 import build as lib_build

from _bounded_reference import decode, kept_slots, norm_grads, norm_rotate

FAKE = 0x7F0000000000  # 256-aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return ba.load_library()


NORM = ba.BamQkNorm(FAKE, FAKE, 1e-6, 0)
MARKS = ba.BamMarks(FAKE, FAKE, 1 << 20)
PRM = ba.BamParams(FAKE, FAKE, FAKE, FAKE, 1e-5, 1, 1, ba.BAM_PRIOR_ALPHA)


def _addr(x):
    return ctypes.addressof(x) if isinstance(x, ctypes.Structure) else x


def _bits(x):
    return struct.unpack("<i", struct.pack("<f", x))[0]


# Arguments of each operator in order, by name; strides follow where the flag is 1.
CALLS = {
    "append": (3, dict(k=FAKE, v=FAKE, q=FAKE, q_out=FAKE, flag=0, kp=FAKE, vp=FAKE, bt=FAKE, lens=FAKE,
                       new=FAKE, par=FAKE, B=2, H=4, Hkv=2, N=8, page=64, mb=4, pages=8, D=64, norm=NORM,
                       rope=0, first=FAKE, marks=MARKS, ws=FAKE, ws_bytes=1 << 30, stream=0)),
    "fwd": (4, dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, flag=0, pos=FAKE, B=2, H=4, Hkv=2, T=8, D=64,
                    norm=NORM, rope=0, stream=0)),
    "bwd": (5, dict(q=FAKE, k=FAKE, gq=FAKE, gk=FAKE, dq=FAKE, dk=FAKE, flag=0, dwq=FAKE, dwk=FAKE, pos=FAKE,
                    B=2, H=4, Hkv=2, T=8, D=64, norm=NORM, rope=0, ws=FAKE, ws_bytes=1 << 30, stream=0)),
    "decode": (6, dict(q=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, lens=FAKE, pt=FAKE, plen=FAKE, qpos=FAKE,
                       marks=MARKS, decay=_bits(1.0), o=FAKE, o_fp32=1, lse=FAKE, B=2, H=4, Hkv=2, page=64,
                       mb=4, pb=2, pages=8, D=64, prm=PRM, ws=FAKE, ws_bytes=1 << 30, stream=0)),
    "evict": (7, dict(kp=FAKE, vp=FAKE, bt=FAKE, lens=FAKE, marks=MARKS, out=FAKE, new=FAKE, B=2, Hkv=2,
                      page=64, mb=4, ob=2, pages=8, D=64, budget=100, sink=4, recent=20, ws=FAKE,
                      ws_bytes=1 << 30, stream=0)),
}
SIZES = {"append": 26, "fwd": 14, "bwd": 20, "decode": 25, "evict": 20}


def _call(lib, name, steps=(), **kw):
    number, args = CALLS[name]
    args = {**args, **kw}
    assert len(args) == SIZES[name]
    words = [_addr(x) for x in args.values()] + list(steps)
    return lib.bam_paged_call(number, struct.pack(f"{len(words)}q", *words))


CACHED = [(dict(B=0), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"), (dict(page=96), "INVALID_ARG"),
          (dict(mb=0), "INVALID_ARG"), (dict(pages=0), "INVALID_ARG"), (dict(D=128), "UNSUPPORTED"),
          (dict(B=65536), "UNSUPPORTED"), (dict(page=1 << 20, mb=1 << 10), "UNSUPPORTED"),
          (dict(bt=0), "INVALID_ARG"), (dict(lens=FAKE + 2), "INVALID_ARG"), (dict(kp=0), "INVALID_ARG"),
          (dict(vp=FAKE + 8), "INVALID_ARG"), (dict(ws=0), "WORKSPACE"), (dict(ws=FAKE + 16), "WORKSPACE"),
          (dict(ws_bytes=100), "WORKSPACE"), (dict(B=1 << 32), "INVALID_ARG"),
          (dict(marks=ba.BamMarks(0, FAKE, 5)), "INVALID_ARG"),
          (dict(marks=ba.BamMarks(FAKE, 0, 5)), "INVALID_ARG"),
          (dict(marks=ba.BamMarks(FAKE + 8, FAKE, 5)), "INVALID_ARG"),
          (dict(marks=ba.BamMarks(FAKE, FAKE, 0)), "INVALID_ARG"),
          (dict(marks=ba.BamMarks(FAKE, FAKE, (1 << 28) + 1)), "INVALID_ARG")]


@pytest.mark.parametrize("name", ["append", "decode", "evict"])
@pytest.mark.parametrize("kw,want", CACHED)
def test_refusals_of_the_cache_operators(lib, name, kw, want):
    assert _call(lib, name, **kw) == getattr(ba, "BAM_ERR_" + want)


BAD_NORMS = [ba.BamQkNorm(0, FAKE, 1e-6, 0), ba.BamQkNorm(FAKE, 0, 1e-6, 0),
             ba.BamQkNorm(FAKE + 4, FAKE, 1e-6, 0), ba.BamQkNorm(FAKE, FAKE, 0.0, 0),
             ba.BamQkNorm(FAKE, FAKE, 1e-32, 0), ba.BamQkNorm(FAKE, FAKE, float("nan"), 0),
             ba.BamQkNorm(FAKE, FAKE, float("inf"), 0), ba.BamQkNorm(FAKE, FAKE, 1e-6, 2)]
BAD_ROPES = [ba.BamRope(10000.0, 8, 0), ba.BamRope(0.5, 64, 0), ba.BamRope(10000.0, 64, 2)]


@pytest.mark.parametrize("name", ["append", "fwd", "bwd"])
@pytest.mark.parametrize("which", range(len(BAD_NORMS) + len(BAD_ROPES)))
def test_refusals_of_norms_and_rotations(lib, name, which):
    bad = (BAD_NORMS + BAD_ROPES)[which]
    kw = dict(norm=bad) if which < len(BAD_NORMS) else dict(rope=bad)
    assert _call(lib, name, **kw) == ba.BAM_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,want", [
    (dict(B=0), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"), (dict(Hkv=0), "INVALID_ARG"),
    (dict(T=0), "INVALID_ARG"), (dict(D=32), "UNSUPPORTED"), (dict(H=65536), "UNSUPPORTED"),
    (dict(B=1 << 16, T=1 << 16), "UNSUPPORTED"), (dict(q=0), "INVALID_ARG"), (dict(k=FAKE + 8), "INVALID_ARG"),
    (dict(norm=0), "INVALID_ARG"), (dict(pos=FAKE + 2), "INVALID_ARG"), (dict(flag=2), "INVALID_ARG"),
    (dict(T=1 << 32), "INVALID_ARG")])
def test_norm_refusals(lib, name, kw, want):
    assert _call(lib, name, **kw) == getattr(ba, "BAM_ERR_" + want)


@pytest.mark.parametrize("kw", [dict(dwq=0), dict(dwk=FAKE + 2), dict(gq=0), dict(dk=FAKE + 4)])
def test_norm_gradient_refusals(lib, kw):
    assert _call(lib, "bwd", **kw) == ba.BAM_ERR_INVALID_ARG
    assert _call(lib, "bwd", ws_bytes=100) == ba.BAM_ERR_WORKSPACE


@pytest.mark.parametrize("name,tensors", [("fwd", 4), ("bwd", 6)])
@pytest.mark.parametrize("at,steps", [
    (0, [2048, 512, 60]), (1, [-8, 512, 64]), (-1, [2048, 0, 64]), (-1, [512, 512, 64]),
    (-1, [1024, 512, 32]), (-2, [0, 512, 64]), (-2, [64, 128, 64])])
def test_norm_strides(lib, name, tensors, at, steps):
    """Steps that are negative, not of 16 bytes, or make rows of an output overlap (a
    batch of 2, 4 and 2 heads, 8 tokens)."""
    good = [[2048, 512, 64], [1024, 512, 64]] * (tensors // 2)
    good[at] = steps
    assert _call(lib, name, steps=sum(good, []), flag=1) == ba.BAM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,want", [
    (dict(q=0), "INVALID_ARG"), (dict(o=FAKE + 8), "INVALID_ARG"), (dict(lse=FAKE + 2), "INVALID_ARG"),
    (dict(H=3), "INVALID_ARG"), (dict(prm=0), "INVALID_ARG"), (dict(pt=0), "INVALID_ARG"),
    (dict(plen=0), "INVALID_ARG"), (dict(pb=0), "INVALID_ARG"), (dict(pb=-1), "INVALID_ARG"),
    (dict(pt=0, plen=0), "INVALID_ARG"), (dict(marks=0), "INVALID_ARG"), (dict(qpos=0), "INVALID_ARG"),
    (dict(qpos=FAKE + 1), "INVALID_ARG"), (dict(pt=FAKE + 2), "INVALID_ARG"),
    (dict(decay=_bits(-0.5)), "INVALID_ARG"), (dict(decay=_bits(1.01)), "INVALID_ARG"),
    (dict(decay=_bits(float("nan"))), "INVALID_ARG"), (dict(pb=1 << 22), "UNSUPPORTED"),
    (dict(B=60000, H=400), "UNSUPPORTED"), (dict(o_fp32=1 << 40), "INVALID_ARG")])
def test_decode_refusals(lib, kw, want):
    assert _call(lib, "decode", **kw) == getattr(ba, "BAM_ERR_" + want)


@pytest.mark.parametrize("kw", [
    dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=81), dict(new=0), dict(new=FAKE + 1), dict(marks=0),
    dict(out=0), dict(ob=0), dict(ob=1), dict(ob=-2), dict(out=FAKE + 2),
    dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1, budget=100)])
def test_evict_refusals(lib, kw):
    assert _call(lib, "evict", **kw) == ba.BAM_ERR_INVALID_ARG


def test_workspace_sizes(lib):
    n = ba.bam_qk_norm_workspace_size(8, 12, 12, 512)
    assert n > 0 and n % 256 == 0
    for bad in [(0, 4, 2, 8), (2, 0, 2, 8), (2, 4, 0, 8), (2, 4, 2, 0), (2, 65536, 2, 8), (1 << 16, 4, 2, 1 << 16)]:
        assert ba.bam_qk_norm_workspace_size(*bad) == 0
    assert ba.bam_qk_norm_workspace_size(2, 4, 2, 8, 128) == 0
    plain = ba.bam_attn_shared_workspace_size(2, 4, 2, 128, 256)
    marked = ba.bam_attn_shared_workspace_size(2, 4, 2, 128, 256, 1000)
    assert 0 < plain < marked and plain % 256 == 0 and marked % 256 == 0
    for bad in [(0, 4, 2, 128, 256), (2, 3, 2, 128, 256), (2, 4, 2, -1, 256), (2, 4, 2, 128, 0),
                (2, 4, 2, 1 << 28, 64), (2, 4, 2, 128, 256, -1), (2, 4, 2, 128, 256, (1 << 28) + 1),
                (60000, 400, 2, 0, 64), (2, 4, 2, 128, 256, 0, 128)]:
        assert ba.bam_attn_shared_workspace_size(*bad) == 0
    n = ba.bam_kv_evict_workspace_size(2, 2, 256, 100)
    assert n > 0 and n % 256 == 0
    assert ba.bam_kv_evict_workspace_size(2, 2, 256, 1 << 30) == ba.bam_kv_evict_workspace_size(2, 2, 256, 256)
    for bad in [(0, 2, 256, 100), (2, 0, 256, 100), (2, 2, 0, 100), (2, 2, 256, 0), (2, 2, 1 << 29, 5)]:
        assert ba.bam_kv_evict_workspace_size(*bad) == 0


def test_binding_refuses_host_tensors_before_the_library():
    x = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    i, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    norm = ba.make_qk_norm(torch.ones(64), torch.ones(64))
    marks = ba.make_marks(torch.zeros(4, 2, 64, dtype=torch.int32), torch.zeros(4, 2, 64), 10)
    prm = ba.make_params(*(torch.ones(2) for _ in range(4)))
    w, q = torch.ones(64), x[:, :, 0].contiguous()
    for f in (lambda: ba.bam_qk_norm_fwd(x, x, x, x, None, norm),
              lambda: ba.bam_qk_norm_bwd(x, x, x, x, x, x, w, w, None, norm, None, ws),
              lambda: ba.bam_kv_append_norm_paged(x, x, pages, pages, table, i, i, None, None, None, norm, None, i,
                                                  marks, ws),
              lambda: ba.bam_attn_decode_shared_paged(q, pages, pages, table, i, None, None, i, marks, 1.0, q, None,
                                                      prm, ws),
              lambda: ba.bam_kv_evict_paged(pages, pages, table, i, marks, None, i, 5, 1, 1, ws)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()


@pytest.mark.parametrize("theta,ssmax,P", [(False, True, 70), (True, False, 0), (True, True, 130)])
def test_reference_decode_is_the_oracle_over_prefix_and_own_keys(theta, ssmax, P):
    rng = np.random.default_rng(P)
    g = torch.Generator().manual_seed(3)
    B, H, Hkv, page, lens = 3, 4, 2, 64, [5, 64, 90]
    kp, vp = (torch.randn(8, Hkv, page, 64, generator=g).to(torch.bfloat16) for _ in range(2))
    prefix, table = torch.tensor([6, 1, 0], dtype=torch.int32), torch.tensor([[2, -1], [3, -1], [4, 5]], dtype=torch.int32)
    q = torch.randn(B, H, 64, generator=g).to(torch.bfloat16)
    prm = [rng.uniform(0.5, 2, H), rng.uniform(-0.5, 1.5, H), rng.uniform(0, 1, H), rng.uniform(0.3, 1, H)]
    t = [torch.from_numpy(x) for x in prm]
    o, lse, w, *_ = decode(q, kp, vp, table, lens, prefix, P, None, None, t, ssmax, theta, False)
    for b in range(B):
        rows = [(int(prefix[j // page]), j % page) for j in range(P)]
        rows += [(int(table[b, j // page]), j % page) for j in range(lens[b])]
        pg, row = (torch.tensor(x) for x in zip(*rows))
        k, v = (x[pg, :, row].transpose(0, 1).double().repeat_interleave(2, 0).numpy()[None] for x in (kp, vp))
        oref, lref = oracle.decode(q[b:b + 1].double().numpy(), k, v, *prm, ssmax=ssmax,
                                   **({"prior": ba.BAM_PRIOR_THETA} if theta else {}))
        np.testing.assert_allclose(o[b].numpy(), oref[0], rtol=0, atol=1e-10)
        np.testing.assert_allclose(lse[b].numpy(), lref[0], rtol=0, atol=1e-10)
        if P == 0:
            np.testing.assert_allclose(w[b].sum(0).numpy(), 2.0, atol=1e-12)


def test_reference_of_marked_keys_is_the_plain_one_when_none_has_left():
    g = torch.Generator().manual_seed(4)
    kp, vp = (torch.randn(4, 1, 64, 64, generator=g).to(torch.bfloat16) for _ in range(2))
    table, prefix = torch.tensor([[2, 1]], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    q = torch.randn(1, 2, 64, generator=g).to(torch.bfloat16)
    t = [torch.tensor([3.0, 9.0]), torch.tensor([1.0, -0.5]), torch.tensor([0.5, 2.0]), torch.tensor([1.0, 0.6])]
    pos = torch.zeros(4, 1, 64, dtype=torch.int32)
    pos[2, 0], pos[1, 0] = 40 + torch.arange(64), 104 + torch.arange(64)
    a = decode(q, kp, vp, table, [100], prefix, 40, None, None, t, True, False, False)
    b = decode(q, kp, vp, table, [100], prefix, 40, pos, torch.tensor([139]), t, True, False, False)
    for x, y in zip(a, b):
        for u, v in zip(x, y):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dims,pairs", [(0, False), (32, True), (64, False)])
def test_reference_norm_gradients_are_differences(dims, pairs):
    g = torch.Generator().manual_seed(dims)
    x, gy, w = (torch.randn(2, 3, 64, generator=g).double() for _ in range(3))
    w = w[:, :1]
    pos = torch.tensor([0, 7, 100000])
    args = (pos, 1e-3, 10000.0, dims, pairs)
    dx, _, terms, _ = norm_grads(x, gy, w, *args)
    f = lambda a, b: float((norm_rotate(a, b, *args)[0] * gy).sum())
    u, v, h = torch.randn(x.shape, generator=g).double(), torch.randn(w.shape, generator=g).double(), 1e-6
    assert abs((f(x + h * u, w) - f(x - h * u, w)) / (2 * h) - float((dx * u).sum())) < 1e-7
    assert abs((f(x, w + h * v) - f(x, w - h * v)) / (2 * h) - float((terms.sum(1, keepdim=True) * v).sum())) < 1e-7


def test_reference_of_kept_slots():
    nan, inf = float("nan"), float("inf")
    w = np.array([0.0, 5.0, 1.0, 5.0, -0.0, 0.0, nan, -1.0, inf, 2.0], np.float32)
    assert kept_slots(w, 20, 0, 0).tolist() == list(range(10))
    assert kept_slots(w, 1, 0, 0).tolist() == [6]
    assert kept_slots(w, 3, 0, 0).tolist() == [1, 6, 8]
    assert kept_slots(w, 7, 0, 1).tolist() == [0, 1, 2, 3, 6, 8, 9]
    assert kept_slots(w, 8, 0, 1).tolist() == [0, 1, 2, 3, 4, 6, 8, 9]
    assert kept_slots(w, 4, 2, 2).tolist() == [0, 1, 8, 9]


KEEP = dict(kp=FAKE, vp=FAKE, bt=FAKE, lens=FAKE, draft=FAKE, par=FAKE, acc=FAKE, new=FAKE, marks=MARKS, B=2, Hkv=2,
            N=8, page=64, mb=4, pages=8, D=64, ws=FAKE, ws_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("kw,want", CACHED + [
    (dict(N=129), "UNSUPPORTED"), (dict(N=0), "INVALID_ARG"), (dict(acc=0), "INVALID_ARG"),
    (dict(new=FAKE + 2), "INVALID_ARG"), (dict(marks=0), "INVALID_ARG"),
    (dict(N=1 << 32), "INVALID_ARG")])
def test_refusals_of_the_keep_with_marks(lib, kw, want):
    args = {**KEEP, **kw}
    assert len(args) == 19
    words = [_addr(x) for x in args.values()]
    assert lib.bam_paged_call(8, struct.pack("19q", *words)) == getattr(ba, "BAM_ERR_" + want)


def test_binding_refuses_marks_on_the_host():
    pages = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    i, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32)
    marks = ba.make_marks(torch.zeros(4, 2, 64, dtype=torch.int32), torch.zeros(4, 2, 64), 10)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ba.bam_kv_keep_paged(pages, pages, table, i, i, None, i, i, torch.zeros(256, dtype=torch.uint8), marks=marks)
    with pytest.raises(TypeError, match="BamMarks"):
        ba._struct_address(object(), ba.BamMarks)
