"""GPU tests of the decode over a shared prefix and over keys with positions and
accumulated weights, against a plain 64-bit implementation; and of a serving
loop that runs append, decode and eviction together."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba
from transformer_attention_ggd_gb300.inputs import random_params, random_theta_params

from _bounded_reference import decode, kept_slots, norm_rotate
from _gpu_helpers import dev_f32

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ba.load_library()


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _prm(rng, H, theta):
    if theta:
        return random_theta_params(H, rng)
    p = random_params(H, rng, mu_hi=6.0)
    p["beta"][0] = -0.6
    return p


class Cache:
    """Pages of which only the rows that a sequence or the prefix uses hold
    numbers: every other row holds `junk`, its position -9 and its weight NaN."""

    def __init__(self, seed, Hkv, page, lens, P, slack=0, prefix_slack=0, gap=3, junk=NAN):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B = len(lens)
        blocks = [-(-int(n) // page) for n in lens]
        pb = -(-P // page)
        num = sum(blocks) + pb + 2
        perm = rng.permutation(num)
        self.k = torch.full((num, Hkv, page, 64), junk, dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.pos = torch.full((num, Hkv, page), -9, dtype=torch.int32, device="cuda")
        self.w = torch.full((num, Hkv, page), NAN, device="cuda")
        table = np.full((B, max(1, max(blocks) + slack)), -1, np.int32)
        prefix = np.full(pb + prefix_slack, -1, np.int32)
        prefix[:pb] = perm[:pb]
        at = pb
        for b in range(B):
            table[b, :blocks[b]] = perm[at:at + blocks[b]]
            at += blocks[b]
        top = P + gap * max(max(lens), 1)
        for row, n in [(prefix, P)] + [(table[b], int(lens[b])) for b in range(B)]:
            pos = top - np.cumsum(rng.integers(1, gap + 1, (n, Hkv)), 0)[::-1] + 1
            for i in range(-(-n // page)):
                m = min(page, n - i * page)
                for x in (self.k, self.v):
                    x[int(row[i]), :, :m] = _normal(gen, Hkv, m, 64)
                if row is not prefix:
                    self.pos[int(row[i]), :, :m] = _i32(pos[i * page:i * page + m].T)
                    self.w[int(row[i]), :, :m] = torch.rand(Hkv, m, generator=gen, device="cuda")
        self.q_pos = _i32([top + b for b in range(B)])
        self.max_pos = top + B
        self.table, self.prefix = _i32(table), _i32(prefix) if len(prefix) else None
        self.rng, self.gen, self.lens, self.P, self.page = rng, gen, lens, P, page


def _case(seed, H, Hkv, page, lens, P, marked, ssmax=True, theta=False, out="fp32", decay=1.0, slack=0,
          prefix_slack=0, junk=NAN, cache=None):
    """One call against the reference, bit-repeated on a dirty workspace."""
    B = len(lens)
    c = cache or Cache(seed, Hkv, page, lens, P, slack, prefix_slack, junk=junk)
    prm = _prm(c.rng, H, theta)
    t = [dev_f32(prm[n]) for n in ("alpha", "beta", "mu", "s")]
    q = _normal(c.gen, B, H, 64)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    prior = ba.BAM_PRIOR_THETA if theta else ba.BAM_PRIOR_ALPHA
    marks = ba.make_marks(c.pos, c.w, c.max_pos) if marked else None
    w0, p0 = c.w.clone(), c.pos.clone()
    pmax = 0 if c.prefix is None else c.prefix.numel() * page
    ws = ba.shared_workspace(B, H, Hkv, pmax, c.table.shape[1] * page, c.max_pos if marked else 0)
    ws.fill_(0xFF)
    plen = None if c.prefix is None else _i32([P])
    params = ba.make_params(*t, 1e-5, True, ssmax, prior)
    o, lse = torch.full((B, H, 64), 7.0, dtype=dt, device="cuda"), torch.full((B, H), 7.0, device="cuda")
    args = (q, c.k, c.v, c.table, _i32(lens), c.prefix, plen, c.q_pos if marked else None, marks)
    ba.bam_attn_decode_shared_paged(*args, decay, o, lse, params, ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    oref, lref, wref, oerr, lerr, werr = decode(
        q, c.k, c.v, c.table, lens, c.prefix, P, c.pos if marked else None, c.q_pos, t, ssmax, theta,
        out == "bf16")
    empty = torch.tensor([P + int(n) == 0 for n in lens], device="cuda")
    assert torch.all(o[empty] == 0) and torch.all(lse[empty] == -float("inf"))
    for got, want, bound in ((o, oref, oerr), (lse, lref, lerr)):
        d, e = (got[~empty].double() - want[~empty]).abs(), bound[~empty]
        assert torch.all(d <= e), float((d / e).max())
    if marked:
        assert torch.equal(c.pos, p0)
        seen = torch.zeros_like(c.w, dtype=torch.bool)
        for b, n in enumerate(lens):
            s = torch.arange(int(n), device="cuda")
            pg, row = c.table[b].long()[s // page], s % page
            seen[pg, :, row] = True
            want = decay * w0[pg, :, row].double() + wref[b]
            d = (c.w[pg, :, row].double() - want).abs()
            assert torch.all(d <= werr[b] + 2.0 ** -23 * want), b
        assert torch.isnan(c.w[~seen]).all()
    else:
        assert torch.equal(c.w.isnan(), w0.isnan())
    again, lagain, w1 = torch.empty_like(o), torch.empty_like(lse), c.w.clone()
    if marked:
        c.w.copy_(w0)
    ba.bam_attn_decode_shared_paged(*args, decay, again, lagain, params, ws)
    assert torch.equal(o, again) and torch.equal(lse, lagain)
    assert torch.equal(c.w.view(torch.int32), w1.view(torch.int32))
    return c, q, t, o, lse


LENS = [0, 1, 63, 64, 65, 129, 300]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("marked", [False, True])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (6, 3), (8, 2), (7, 1), (16, 2), (9, 1), (34, 2)])
def test_shared_heads(H, Hkv, marked, out):
    _case(H + 10 * Hkv, H, Hkv, 64, LENS, 200, marked, out=out, slack=1)


@pytest.mark.parametrize("marked", [False, True])
@pytest.mark.parametrize("P", [0, 1, 63, 64, 65, 127, 128, 129, 500, 3001])
def test_shared_prefix_lengths(P, marked):
    _case(P, 4, 2, 64, LENS, P, marked, prefix_slack=P % 3, out="bf16" if P % 2 else "fp32")


@pytest.mark.parametrize("page", [64, 128, 320])
@pytest.mark.parametrize("theta,ssmax,decay", [(False, False, 1.0), (True, True, 0.5), (True, False, 0.0)])
def test_shared_priors_pages_and_decay(page, theta, ssmax, decay):
    for marked in (False, True):
        _case(page + theta, 6, 3, page, [511, 129, 62, 0], 333, marked, ssmax, theta, decay=decay)


@pytest.mark.parametrize("B", [1, 2, 15, 16, 17, 33, 65, 129, 300])
def test_shared_batch_sizes(B):
    """Rows of the prefix around the tiles that hold them."""
    rng = np.random.default_rng(B)
    _case(B, 2, 1, 64, rng.integers(0, 70, B).tolist(), 777, B % 2 == 0, out="bf16" if B % 3 else "fp32")
    _case(B, 3, 3, 64, rng.integers(0, 70, B).tolist(), 150, B % 2 == 1)


@pytest.mark.parametrize("B", [8, 9, 32, 64, 128])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_shared_rows_that_fill_a_variant(B, out):
    _case(B, 3, 3, 64, [i % 5 for i in range(B)], 777, False, out=out, prefix_slack=40)


@pytest.mark.parametrize("out,P", [("fp32", 14000), ("bf16", 140000)])
@pytest.mark.parametrize("flat", [False, True])
def test_shared_sums_that_leave_tensor_memory(out, P, flat):
    """75 blocks of rows, each in two parts that are longer than an accumulator takes
    on (of three chains of 8 tiles, four of 128), more than once; with equal keys and
    positive values every step rounds to the same side.  Against some of the
    sequences."""
    B, H = 600, 16
    c = Cache(P, 1, 64, [1] * B, P)
    if flat:
        c.k[c.prefix.long()] = 0
        c.v.copy_(c.v.abs())
    t = [dev_f32(x) for x in ([5.0] * H, [0.3] * H, [1.0] * H, [1.0] * H)]
    q = _normal(c.gen, B, H, 64)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    lens = _i32([1] * B)
    ws = ba.shared_workspace(B, H, 1, c.prefix.numel() * 64, 64)
    ws.fill_(0xFF)
    o, lse = ba.attention_decode_shared_paged(q, c.k, c.v, c.table, lens, *t, prefix_table=c.prefix,
                                              prefix_len=_i32([P]), o_dtype=dt, ws=ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    some = [0, 7, 8, 300, 599]
    oref, lref, _, oerr, lerr, _ = decode(q[some], c.k, c.v, c.table[some], [1] * len(some), c.prefix, P, None,
                                          None, t, False, False, out == "bf16")
    for got, want, bound in ((o, oref, oerr), (lse, lref, lerr)):
        d = (got[some].double() - want).abs()
        assert torch.all(d <= bound), float((d / bound).max())
    again, lagain = ba.attention_decode_shared_paged(q, c.k, c.v, c.table, lens, *t, prefix_table=c.prefix,
                                                     prefix_len=_i32([P]), o_dtype=dt, ws=ws)
    assert torch.equal(o, again) and torch.equal(lse, lagain)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hkv", [(4, 2, 1), (5, 2, 1), (20, 3, 1), (50, 1, 1), (150, 2, 2)])
def test_shared_weights_have_as_many_bits_whoever_shares_the_prefix(B, H, Hkv, out):
    """Values +1 and -1 of neighbouring keys nearly cancel, so that the output's own
    rounding is small beside a weight's: 2^-16 of the sum of the weights (1) with bf16
    output, over a prefix of few rows and of many."""
    P, n = 70, 2
    c = Cache(B, Hkv, 64, [n] * B, P)
    sign = torch.randint(0, 2, (c.v.shape[0], Hkv, 32, 1, 64), generator=c.gen, device="cuda") * 2 - 1
    sign = torch.cat([sign, -sign], 3).reshape(c.v.shape).to(torch.bfloat16)
    c.v.copy_(torch.where(torch.isnan(c.v), c.v, sign))
    for row in (c.prefix.long(), c.table.long().clamp(min=0)):
        c.k[row] = 0
    t = [dev_f32(x) for x in ([40.0] * H, [0.6] * H, [1.0] * H, [1.0] * H)]
    q, lens = _normal(c.gen, B, H, 64), [n] * B
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    o, _ = ba.attention_decode_shared_paged(q, c.k, c.v, c.table, _i32(lens), *t, prefix_table=c.prefix,
                                            prefix_len=_i32([P]), o_dtype=dt)
    oref, _, _, oerr, _, _ = decode(q, c.k, c.v, c.table, lens, c.prefix, P, None, None, t, False, False, False)
    bound = oerr  # with fp32 output: a weight's delta and 2^-22, and 2^-24 for each key's sum
    if out == "bf16":
        bound = oerr + 2.0 ** -16
        bound = bound + 2.0 ** -8 * (oref.abs() + bound)
    d = (o.double() - oref).abs()
    assert torch.all(d <= bound), float((d / bound).max())


@pytest.mark.parametrize("lens,P,H,Hkv,marked", [([9000], 0, 8, 2, True), ([0], 9000, 4, 4, False),
                                                 ([20000, 5], 70, 4, 2, True), ([1] * 40, 20001, 8, 2, False),
                                                 ([0, 1], 40000, 2, 1, True)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_shared_long_keys(lens, P, H, Hkv, marked, out):
    _case(P + len(lens), H, Hkv, 64, lens, P, marked, out=out)


def test_shared_without_a_prefix_is_the_paged_decode():
    """Against the decode that is there already, within both operators' errors."""
    lens = [1, 64, 300, 1000]
    c, q, t, o, lse = _case(3, 4, 4, 64, lens, 0, False)
    o2, lse2 = ba.attention_decode_paged(q, c.k, c.v, c.table, _i32(lens), *t, ssmax=True)
    torch.testing.assert_close(o, o2, rtol=0, atol=1e-4)
    torch.testing.assert_close(lse, lse2, rtol=1e-5, atol=1e-4)


def test_shared_prefix_equals_the_same_keys_as_own():
    """A prefix of whole pages, or the same pages at the head of each own table."""
    P, lens = 256, [5, 70, 130]
    c, q, t, o, lse = _case(4, 4, 2, 64, lens, P, False)
    joint = torch.cat([c.prefix.expand(3, -1), c.table], 1).contiguous()
    o2, lse2 = ba.attention_decode_shared_paged(q, c.k, c.v, joint, _i32([P + n for n in lens]), *t, ssmax=True)
    torch.testing.assert_close(o, o2, rtol=0, atol=2e-5)
    torch.testing.assert_close(lse, lse2, rtol=1e-6, atol=1e-5)


@pytest.mark.parametrize("junk", [float("inf"), -3e38])
def test_shared_keys_out_of_sight_have_no_effect(junk):
    _case(5, 4, 2, 64, LENS, 100, True, junk=junk, slack=2)
    _case(6, 4, 2, 128, LENS, 130, False, junk=junk, prefix_slack=1)


@pytest.mark.parametrize("where", ["prefix", "own"])
def test_shared_infinities_and_nan_reach_the_rows_that_see_them(where):
    H = 3
    c = Cache(7, H, 64, [70, 40], 150)
    row = int((c.prefix if where == "prefix" else c.table[0])[1])
    t = [dev_f32(x) for x in ([5.0] * H, [0.0] * H, [0.0] * H, [1.0] * H)]  # equal biases
    q = _normal(c.gen, 2, H, 64)
    c.v[row, 1, 3, 9] = float("-inf")
    args = (c.table, _i32([70, 40]), *t)
    for dt in (torch.bfloat16, torch.float32):
        o, lse = ba.attention_decode_shared_paged(q, c.k, c.v, *args, prefix_table=c.prefix,
                                                  prefix_len=_i32([150]), o_dtype=dt)
        hit = [0, 1] if where == "prefix" else [0]
        assert torch.all(o[hit, 1, 9] == float("-inf")) and torch.isfinite(lse).all()
        o[hit, 1, 9] = 0
        assert torch.isfinite(o).all()
        c.k[row, 2, 3, 0] = NAN
        o, lse = ba.attention_decode_shared_paged(q, c.k, c.v, *args, prefix_table=c.prefix,
                                                  prefix_len=_i32([150]), o_dtype=dt)
        assert torch.isnan(o[hit, 2]).all() and torch.isnan(lse[hit, 2]).all()
        assert torch.isfinite(lse[:, :2]).all()
        c.k[row, 2, 3, 0] = 0.5


def test_shared_sharp_and_flat_rows():
    """One key takes all the weight, or all have the same: sums over long runs of
    equal positive values."""
    P, n = 20000, 500
    for out, marked in (("fp32", False), ("bf16", True)):
        c = Cache(8, 1, 64, [n, n], P)
        c.k[c.prefix.long()] = 0
        c.k[c.table.long().clamp(min=0)] = 0
        c.v.copy_(torch.where(torch.isnan(c.v), c.v, c.v.abs()))
        _case(8, 2, 1, 64, [n, n], P, marked, ssmax=False, out=out, cache=c)
        c = Cache(9, 1, 64, [n, n], P)
        c.k[c.prefix.long()[100]] *= 40
        _case(9, 2, 1, 64, [n, n], P, marked, ssmax=True, out=out, cache=c)


def test_shared_far_positions():
    """Positions near 2^28 with few keys: distances keep their value, and the
    prefix is that far away."""
    c = Cache(10, 2, 64, [100, 30], 0)
    far = (1 << 24) - 10000
    c.pos += far
    c.q_pos += far
    c.max_pos += far
    _case(10, 4, 2, 64, [100, 30], 0, True, cache=c)
    c = Cache(11, 2, 64, [100, 30], 90)
    c.q_pos += 100000
    c.max_pos += 100000
    _case(11, 4, 2, 64, [100, 30], 90, True, cache=c)


def test_shared_reports_what_is_out_of_range():
    c = Cache(12, 2, 64, [100, 30], 90)
    t = [dev_f32(x) for x in ([5.0] * 4, [1.0] * 4, [0.0] * 4, [1.0] * 4)]
    q = _normal(c.gen, 2, 4, 64)
    ws = ba.shared_workspace(2, 4, 2, 128, 128, c.max_pos)
    base = dict(lens=[100, 30], plen=90, table=c.table, prefix=c.prefix, q_pos=c.q_pos, marks=True)

    def call(**kw):
        a = {**base, **kw}
        marks = ba.make_marks(c.pos, c.w, c.max_pos) if a["marks"] else None
        o, lse = ba.attention_decode_shared_paged(
            q, c.k, c.v, a["table"], _i32(a["lens"]), *t, prefix_table=a["prefix"],
            prefix_len=_i32([a["plen"]]), q_pos=a["q_pos"] if marks else None, marks=marks, ws=ws)
        return ba.bam_attn_check_status(ws)

    bad_table, bad_prefix = c.table.clone(), c.prefix.clone()
    bad_table[1, 0] = c.k.shape[0]
    bad_prefix[1] = -1
    assert call() == ba.BAM_OK
    for kw in (dict(lens=[129, 30]), dict(lens=[100, -1]), dict(plen=129), dict(plen=-5),
               dict(table=bad_table), dict(prefix=bad_prefix), dict(q_pos=_i32([-1, 5000])),
               dict(q_pos=_i32([400, c.max_pos])), dict(q_pos=_i32([50, 400]))):
        assert call(**kw) == ba.BAM_ERR_INVALID_ARG, kw
        assert call() == ba.BAM_OK
    for kw in (dict(lens=[129, 30]), dict(plen=129), dict(prefix=bad_prefix)):
        assert call(marks=False, **kw) == ba.BAM_ERR_INVALID_ARG, kw
    assert call() == ba.BAM_OK


def test_shared_refusals():
    c = Cache(13, 2, 64, [100, 30], 90)
    t = [dev_f32([1.0] * 4) for _ in range(4)]
    q = _normal(c.gen, 2, 4, 64)
    ln, plen = _i32([100, 30]), _i32([90])
    marks = ba.make_marks(c.pos, c.w, c.max_pos)
    good = (q, c.k, c.v, c.table, ln)
    call = lambda *a, **kw: ba.attention_decode_shared_paged(*(a or good), *t, **kw)
    for i, bad in [(0, q.float()), (0, q[:, :3]), (0, q[:1]), (1, c.k[:, :1]), (2, c.v[..., :32]),
                   (3, c.table.long()), (3, c.table[:1]), (4, ln.float()), (4, ln[:1])]:
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, ba.BamError)):
            call(*args)
    for kw in (dict(prefix_table=c.prefix), dict(prefix_len=plen), dict(marks=marks), dict(q_pos=c.q_pos),
               dict(prefix_table=c.prefix.long(), prefix_len=plen),
               dict(prefix_table=c.prefix[:0], prefix_len=plen),
               dict(prefix_table=c.prefix, prefix_len=_i32([90, 90])),
               dict(marks=marks, q_pos=c.q_pos[:1]), dict(marks=marks, q_pos=c.q_pos.long()),
               dict(marks=ba.make_marks(c.pos[:1], c.w[:1], 99), q_pos=c.q_pos)):
        with pytest.raises(ValueError):
            call(**kw)
    for decay in (-0.1, 1.5, NAN):
        with pytest.raises(ba.BamError):
            call(marks=marks, q_pos=c.q_pos, decay=decay)
    with pytest.raises(ba.BamError):
        call(ws=torch.zeros(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="float16"):
        call(o_dtype=torch.float16)
    o, _ = call()
    assert torch.isfinite(o).all()


def test_shared_without_lse():
    c, q, t, o, _ = _case(14, 4, 2, 64, [100, 30], 90, False)
    ws = ba.shared_workspace(2, 4, 2, 128, 128)
    o2 = torch.empty_like(o)
    ba.bam_attn_decode_shared_paged(q, c.k, c.v, c.table, _i32([100, 30]), c.prefix, _i32([90]), None, None,
                                    1.0, o2, None, ba.make_params(*t, 1e-5, True, True), ws)
    assert torch.equal(o, o2)


def test_shared_two_streams_and_two_graphs():
    """Calls at once with a workspace each; graphs that were captured on one
    workspace, replayed in turn with other lengths."""
    lens = [700, 64, 0, 1500]
    c = Cache(15, 2, 64, lens, 5000)
    t = [dev_f32(x) for x in ([50.0] * 8, [0.7] * 8, [1.0] * 8, [0.5] * 8)]
    prm = ba.make_params(*t, 1e-5, True, True)
    sizes = (4, 8, 2, c.prefix.numel() * 64, c.table.shape[1] * 64)
    ln, plen = _i32(lens), _i32([5000])
    qs = [_normal(c.gen, 4, 8, 64) for _ in range(2)]
    want = [ba.attention_decode_shared_paged(q, c.k, c.v, c.table, ln, *t, prefix_table=c.prefix,
                                             prefix_len=plen, ssmax=True) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [ba.shared_workspace(*sizes) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs = [ba.attention_decode_shared_paged(q, c.k, c.v, c.table, ln, *t, prefix_table=c.prefix,
                                                 prefix_len=plen, ssmax=True, ws=ws, stream=st)
                for q, ws, st in zip(qs, wss, streams)]
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graphs, results = [], []
    for q in qs:
        o, lse = torch.zeros(4, 8, 64, device="cuda"), torch.zeros(4, 8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ba.bam_attn_decode_shared_paged(q, c.k, c.v, c.table, ln, c.prefix, plen, None, None, 1.0, o, lse,
                                            prm, wss[0])
        graphs.append(g)
        results.append((o, lse))
    for n, p in ((lens, 5000), ([700, 10, 0, 1], 4000)):
        ln.copy_(_i32(n))
        plen.copy_(_i32([p]))
        want = [ba.attention_decode_shared_paged(q, c.k, c.v, c.table, ln, *t, prefix_table=c.prefix,
                                                 prefix_len=plen, ssmax=True) for q in qs]
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(results, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_beyond_32_bits():
    """Pages behind the first 5 GB of a pool, and logits behind the first 8 GB of a
    workspace: appends, decoding and evictions equal those of a small pool and table."""
    B, H, Hkv, page, P = 64, 32, 2, 64, 100
    lens, extra = [70 + b % 50 for b in range(B)], 300000
    c = Cache(23, Hkv, page, lens, P)
    t = [dev_f32(_prm(c.rng, H, False)[n]) for n in ("alpha", "beta", "mu", "s")]
    q, k, v = _normal(c.gen, B, H, 64), _normal(c.gen, B, Hkv, 1, 64), _normal(c.gen, B, Hkv, 1, 64)
    room = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    n = c.k.shape[0]
    outs = []
    for far in (False, True):
        pools = [c.k, c.v, c.pos, c.w]
        table, prefix = c.table, c.prefix
        if far:
            pools = [torch.empty((extra + n,) + x.shape[1:], dtype=x.dtype, device="cuda") for x in pools]
            for x, y in zip(pools, (c.k, c.v, c.pos, c.w)):
                x[extra:].copy_(y)
            table = torch.where(table < 0, table, table + extra)
            table = torch.cat([table, room.expand(B, 16384)], 1).contiguous()
            prefix = prefix + extra
        else:
            pools = [x.clone() for x in pools]
        kp, vp, pos, w = pools
        assert not far or kp.numel() * 2 > 4 << 30
        marks = ba.make_marks(pos, w, c.max_pos)
        at = _i32([m - 1 for m in lens])  # the last key again
        ba.kv_append_norm_paged(k, v, kp, vp, table, at, first_pos=c.q_pos, marks=marks)
        ws = ba.shared_workspace(B, H, Hkv, prefix.numel() * page, table.shape[1] * page, c.max_pos)
        o, lse = ba.attention_decode_shared_paged(q, kp, vp, table, _i32(lens), *t, prefix_table=prefix,
                                                  prefix_len=_i32([P]), q_pos=c.q_pos, marks=marks, ws=ws)
        assert ba.bam_attn_check_status(ws) == ba.BAM_OK
        assert not far or ws.numel() > 8 << 30
        del ws
        new = ba.kv_evict_paged(kp, vp, table, _i32(lens), marks, 64, 3, 20)
        outs.append([o, lse, new] + [x[-n:].clone() for x in pools])
    for x, y in zip(*outs):
        if x.dtype == torch.bfloat16:
            x, y = x.view(torch.int16), y.view(torch.int16)
        torch.testing.assert_close(x, y, rtol=1e-4, atol=1e-4, equal_nan=True)


def test_serving_with_a_bounded_cache():
    """A shared document, prompts that enter the cache through norms and rotation,
    decoding steps that gather weights, evictions whenever the caches are full,
    all of it captured step by step and replayed; every step against the
    reference on a mirror of the cache."""
    g = torch.Generator(device="cuda").manual_seed(21)
    rng = np.random.default_rng(21)
    B, H, Hkv, page, P, budget, sink, recent, full = 3, 4, 2, 64, 150, 80, 4, 20, 96
    mb, pb, steps = 2, 3, 40
    num = pb + B * mb
    kp, vp = (torch.full((num, Hkv, page, 64), NAN, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kpos = torch.full((num, Hkv, page), -1, dtype=torch.int32, device="cuda")
    kw = torch.full((num, Hkv, page), NAN, device="cuda")
    marks = ba.make_marks(kpos, kw, 1 << 16)
    prefix, table = _i32(np.arange(pb)), _i32(pb + np.arange(B * mb).reshape(B, mb))
    wq, wk = (1 + 0.2 * torch.randn(64, generator=g, device="cuda") for _ in range(2))
    norm, rope = ba.make_qk_norm(wq, wk, 1e-6), ba.make_rope(10000.0, 32)
    prm = _prm(rng, H, False)
    t = [dev_f32(prm[n]) for n in ("alpha", "beta", "mu", "s")]
    params = ba.make_params(*t, 1e-5, True, True)
    cws, ews = ba.cache_workspace(), ba.evict_workspace(B, Hkv, mb * page, budget)
    sws = ba.shared_workspace(B, H, Hkv, pb * page, mb * page, 1 << 16)
    # the document: one sequence of P tokens in the prefix' pages
    doc = _normal(g, 1, Hkv, P, 64)
    ba.bam_kv_append_norm_paged(doc, doc, kp, vp, prefix[None], _i32([0]), None, None, None, None, norm, rope,
                                None, None, cws)
    plen = _i32([P])
    lens, pos = _i32([0] * B), _i32([P] * B)
    # prompts of different lengths
    new = [30, 80, 7]
    x = _normal(g, B, Hkv, 80, 64)
    ba.bam_kv_append_norm_paged(x, x, kp, vp, table, lens, _i32(new), None, None, None, norm, rope, pos, marks, cws)
    lens += _i32(new)
    pos += _i32(new)
    # one decoding step over fixed buffers
    k, v, q = _normal(g, B, Hkv, 1, 64), _normal(g, B, Hkv, 1, 64), _normal(g, B, H, 1, 64)
    qn, o, lse = torch.zeros_like(q), torch.zeros(B, H, 64, device="cuda"), torch.zeros(B, H, device="cuda")

    def step():
        ba.bam_kv_append_norm_paged(k, v, kp, vp, table, lens, None, None, q, qn, norm, rope, pos, marks, cws)
        lens.add_(1)
        ba.bam_attn_decode_shared_paged(qn.view(B, H, 64), kp, vp, table, lens, prefix, plen, pos, marks, 0.9, o,
                                        lse, params, sws)
        pos.add_(1)

    def evict():
        ba.bam_kv_evict_paged(kp, vp, table, lens, marks, None, lens, budget, sink, recent, ews)

    torch.cuda.synchronize()
    saved = [y.clone() for y in (kp, vp, kpos, kw, lens, pos)]
    graphs = []
    for f in (step, evict):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f()
        graphs.append(gr)
    for y, z in zip((kp, vp, kpos, kw, lens, pos), saved):
        y.copy_(z)
    evictions = 0
    for i in range(steps):
        for y in (k, v, q):
            y.copy_(_normal(g, *y.shape))
        before = [y.clone() for y in (kw, lens, pos)]
        graphs[0].replay()
        torch.cuda.synchronize()
        n = lens.tolist()
        assert n == (before[1] + 1).tolist() and pos.tolist() == (before[2] + 1).tolist()
        for b in range(B):
            y, bound = norm_rotate(q[b].double(), wq.double(), before[2][b:b + 1].double(), 1e-6, 10000.0, 32, False)
            assert torch.all((qn[b].double() - y).abs() <= bound)
        at = before[2]
        oref, lref, wref, oerr, lerr, werr = decode(qn.view(B, H, 64), kp, vp, table, n, prefix, P, kpos, at, t,
                                                    True, False, False)
        assert torch.all((o.double() - oref).abs() <= oerr) and torch.all((lse.double() - lref).abs() <= lerr)
        for b in range(B):
            s = torch.arange(n[b], device="cuda")
            pg, row = table[b].long()[s // page], s % page
            old = before[0][pg, :, row].double()
            old[-1] = 0  # the new key's
            want = 0.9 * old + wref[b]
            assert torch.all((kw[pg, :, row].double() - want).abs() <= werr[b] + 2.0 ** -23 * want)
            assert torch.all(kpos[pg[-1:], :, row[-1:]] == at[b])
        if max(n) >= full:
            evictions += 1
            before = [y.clone() for y in (kp.view(torch.int16), vp.view(torch.int16), kpos, kw)]
            graphs[1].replay()
            torch.cuda.synchronize()
            assert lens.tolist() == [min(m, budget) for m in n]
            for b in range(B):
                for h in range(Hkv):
                    s = np.arange(n[b])
                    rows = table[b].cpu().numpy()
                    w = before[3].cpu().numpy()[rows[s // page], h, s % page]
                    kept = kept_slots(w, budget, sink, recent)
                    m = np.arange(len(kept))
                    for y, z in zip((kp.view(torch.int16), vp.view(torch.int16), kpos, kw), before):
                        assert torch.equal(y[rows[m // page], h, m % page], z[rows[kept // page], h, kept % page])
    assert evictions >= 2
    for ws in (cws, sws, ews):
        assert ba.bam_attn_check_status(ws) == ba.BAM_OK


def test_shared_decay_is_read_at_each_call():
    """A number of any kind, of a tensor too, that changed between two calls."""
    c = Cache(33, 2, 64, [70, 5], 0)
    t = [dev_f32(x) for x in ([5.0] * 4, [1.0] * 4, [0.0] * 4, [1.0] * 4)]
    q, lens, w0 = _normal(c.gen, 2, 4, 64), _i32([70, 5]), c.w.clone()
    marks, box = ba.make_marks(c.pos, c.w, c.max_pos), torch.tensor(1.0)

    def step(decay):
        c.w.copy_(w0)
        ba.attention_decode_shared_paged(q, c.k, c.v, c.table, lens, *t, q_pos=c.q_pos, marks=marks, decay=decay)
        return c.w.view(torch.int32).clone()

    for value in (1.0, 0.25, 0.0):
        box.fill_(value)
        assert torch.equal(step(box), step(value))


def test_shared_weights_of_far_keys_add_up():
    """Far from every key the logits are large (10^6, and the least that a bias may be):
    what a step adds to a sequence's weights is 1 for each query head all the same.  A
    weight and the sum that divides it have the same logits, so that only the
    exponentials' 2^-22 each and the sums of n terms count."""
    lens, H, Hkv = [70, 300, 1], 4, 2
    for P in (0, 40):
        c = Cache(31 + P, Hkv, 64, lens, P)
        c.q_pos += 1000000
        c.max_pos += 1000000
        c.k[c.table.long().clamp(min=0)] = 0
        prm = [dev_f32(x) for x in ([1.0] * H, [1.0, 1.0, 40.0, 40.0], [0.0] * H, [1.0] * H)]
        marks = ba.make_marks(c.pos, c.w, c.max_pos)
        for decay, old in ((0.0, 0.0), (1.0, 1.0)):
            w0 = c.w.clone()
            ba.attention_decode_shared_paged(_normal(c.gen, 3, H, 64), c.k, c.v, c.table, _i32(lens), *prm,
                                             q_pos=c.q_pos, marks=marks, decay=decay)
            for b, n in enumerate(lens):
                s = torch.arange(n, device="cuda")
                pg, row = c.table[b].long()[s // 64], s % 64
                got, was = c.w[pg, :, row].double(), w0[pg, :, row].double()
                added = got.sum(0) - old * was.sum(0)
                bound = 2 * (n * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -24 * got.sum(0)
                assert torch.all((added - H // Hkv).abs() <= bound), (decay, b, added.tolist())
