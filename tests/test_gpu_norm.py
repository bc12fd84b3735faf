"""GPU tests of the norms of queries and keys with their rotation: forward,
gradients (against the formula and against differences), strides, values,
refusals, streams and graphs, and the append that normalises."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba
from transformer_attention_ggd_gb300.autograd import bam_attention, qk_norm

from _bounded_reference import norm_grads, norm_rotate
from _gpu_helpers import GRAD_RTOL

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ba.load_library()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _weights(gen, H, Hkv, per_head):
    return tuple(1 + 0.3 * torch.randn((h, 64) if per_head else (64,), generator=gen, device="cuda")
                 for h in (H, Hkv))


def _w64(w):
    return w.double()[:, None] if w.dim() == 2 else w.double()


def _check(got, want, bound):
    d = (got.double() - want).abs()
    assert torch.all(d <= bound), float((d / bound).max())


def _run(seed, B, H, Hkv, T, dims, pairs, per_head, packed, scale=1.0, fused=True):
    """Forward and backward of one shape against the reference."""
    g = _gen(seed)
    if fused:  # slices of one projection's output, and of its gradient
        qkv = _normal(g, B, T, H + 2 * Hkv, 64) * scale
        q, k, _ = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
        grad = torch.full((B, T, H + 2 * Hkv, 64), 7.0, device="cuda", dtype=torch.bfloat16)
        dq, dk, dv = (x.transpose(1, 2) for x in grad.split([H, Hkv, Hkv], 2))
    else:
        q, k = _normal(g, B, H, T, 64) * scale, _normal(g, B, Hkv, T, 64) * scale
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), None
    wq, wk = _weights(g, H, Hkv, per_head)
    gq, gk = _normal(g, B, H, T, 64), _normal(g, B, Hkv, T, 64)
    pos = None
    if packed:
        pos = torch.randint(-3, 200000, (B, T), generator=g, device="cuda").int()
    rope = ba.make_rope(10000.0, dims, pairs)
    norm = ba.make_qk_norm(wq, wk, EPS)
    qo, ko = (torch.full((B, h, T, 64), 9.0, device="cuda", dtype=torch.bfloat16) for h in (H, Hkv))
    ba.bam_qk_norm_fwd(q, k, qo, ko, pos, norm, rope)
    ws = ba.qk_norm_workspace(B, H, Hkv, T)
    ws.fill_(0xFF)
    dwq, dwk = torch.full_like(wq, 3.0), torch.full_like(wk, 3.0)
    ba.bam_qk_norm_bwd(q, k, gq, gk, dq, dk, dwq, dwk, pos, norm, rope, ws)
    for x, w, y, gy, dx, dw in ((q, wq, qo, gq, dq, dwq), (k, wk, ko, gk, dk, dwk)):
        terms, sizes = 0, 0
        for b in range(B):
            p = torch.arange(T, device="cuda") if pos is None else pos[b]
            args = (_w64(w), p, EPS, 10000.0, dims, pairs)
            _check(y[b], *norm_rotate(x[b].double(), *args))
            want, bound, t, s = norm_grads(x[b].double(), gy[b].double(), *args)
            _check(dx[b], want, bound)
            terms, sizes = terms + t.sum(1), sizes + s.sum(1)
        if not per_head:
            terms, sizes = terms.sum(0), sizes.sum(0)
        # the terms to 2^-18; a CTA's fp32 sums of at most some 60 values in a row: 2^-18
        _check(dw, terms, 2.0 ** -17 * sizes + 1e-30)
    if dv is not None:
        assert torch.all(dv == 7.0)
    return q, k, wq, wk, gq, gk, pos, rope, (qo, ko, dq, dk, dwq, dwk)


@pytest.mark.parametrize("dims,pairs", [(0, False), (16, True), (32, False), (48, True), (64, False),
                                        (64, True)])
@pytest.mark.parametrize("per_head,packed", [(False, False), (True, True)])
def test_norm_rotations_and_weights(dims, pairs, per_head, packed):
    _run(dims, 2, 5, 3, 37, dims, pairs, per_head, packed)


@pytest.mark.parametrize("B,H,Hkv,T", [(1, 1, 1, 1), (1, 1, 1, 15), (3, 2, 1, 16), (2, 4, 4, 17),
                                       (70, 12, 12, 1), (1, 12, 12, 512), (2, 40, 8, 129),
                                       (1, 3, 2, 5000), (1, 130, 1, 33)])
@pytest.mark.parametrize("per_head", [False, True])
def test_norm_shapes(B, H, Hkv, T, per_head):
    _run(B + T, B, H, Hkv, T, 64, False, per_head, False, fused=T % 2 == 1)


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e4, 1e19, 1e30, 2.0 ** 120])
def test_norm_of_large_and_small_values(scale):
    """Squares far outside of fp32: rows above 1e18 are scaled before they are
    squared, rows of tiny values are governed by eps."""
    _run(5, 1, 2, 2, 19, 64, False, False, False, scale=scale)


def test_norm_of_zero_rows_and_infinities():
    g = _gen(1)
    q, k = _normal(g, 1, 2, 20, 64), _normal(g, 1, 2, 20, 64)
    q[0, 0, 3] = 0
    q[0, 1, 4, 5] = float("inf")
    k[0, 0, 7, 9] = float("nan")
    wq, wk = _weights(g, 2, 2, False)
    qo, ko = ba.qk_norm_forward(q, k, wq, wk)
    assert torch.all(qo[0, 0, 3] == 0)
    assert torch.isnan(qo[0, 1, 4, 5]) and torch.all(qo[0, 1, 4, :5] == 0) and torch.isnan(ko[0, 0, 7]).all()
    for x, rows in ((qo, [(1, 4)]), (ko, [(0, 7)])):
        fine = x.clone()
        for h, t in rows:
            fine[0, h, t] = 0
        assert torch.isfinite(fine).all()


def test_norm_in_place_equals_out_of_place():
    g = _gen(2)
    q, k = _normal(g, 2, 3, 50, 64), _normal(g, 2, 3, 50, 64)
    wq, wk = _weights(g, 3, 3, False)
    rope, norm = ba.make_rope(), ba.make_qk_norm(wq, wk)
    want = ba.qk_norm_forward(q, k, wq, wk, rope=rope)
    gq, gk = _normal(g, 2, 3, 50, 64), _normal(g, 2, 3, 50, 64)
    grads = ba.qk_norm_backward(q, k, gq, gk, wq, wk, rope=rope)
    ws = ba.qk_norm_workspace(2, 3, 3, 50)
    dwq, dwk = torch.empty_like(wq), torch.empty_like(wk)
    ba.bam_qk_norm_bwd(q, k, gq, gk, gq, gk, dwq, dwk, None, norm, rope, ws)
    for a, b in zip((gq, gk, dwq, dwk), grads):
        assert torch.equal(a, b)
    ba.bam_qk_norm_fwd(q, k, q, k, None, norm, rope)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_norm_gradients_against_differences():
    """d/dt of sum(y g) along random directions, from the reference's forward
    in 64 bits; the gradients are those of the kernels."""
    q, k, wq, wk, gq, gk, pos, rope, out = _run(11, 1, 2, 2, 24, 32, True, True, True)
    g = _gen(12)
    for x, w, gy, dx, dw in ((q, wq, gq, out[2], out[4]), (k, wk, gk, out[3], out[5])):
        x64, w64, g64 = x[0].double(), _w64(w), gy[0].double()
        f = lambda a, b: float((norm_rotate(a, b, pos[0], EPS, 10000.0, 32, True)[0] * g64).sum())
        u, v = torch.randn(x64.shape, generator=g, device="cuda").double(), torch.randn(
            w64.shape, generator=g, device="cuda").double()
        h = 1e-5
        want = (f(x64 + h * u, w64) - f(x64 - h * u, w64)) / (2 * h)
        # dx is rounded to bf16: at most 2^-8 of each term
        assert abs(float((dx[0].double() * u).sum()) - want) <= 1e-6 * abs(want) + 1.1 * BF * float(
            (dx[0].double() * u).abs().sum())
        want = (f(x64, w64 + h * v) - f(x64, w64 - h * v)) / (2 * h)
        got = float((dw.double()[:, None] * v).sum())
        assert abs(got - want) <= 1e-5 * float((dw.double()[:, None] * v).abs().sum()) + 1e-5 * abs(want)


BF = 2.0 ** -8


def test_norm_is_repeatable_and_runs_on_streams_and_in_graphs():
    g = _gen(3)
    B, H, Hkv, T = 2, 12, 4, 700
    q, k, gq, gk = (_normal(g, B, h, T, 64) for h in (H, Hkv, H, Hkv))
    wq, wk = _weights(g, H, Hkv, True)
    rope, norm = ba.make_rope(), ba.make_qk_norm(wq, wk)
    first = ba.qk_norm_backward(q, k, gq, gk, wq, wk, rope=rope)
    fwd = ba.qk_norm_forward(q, k, wq, wk, rope=rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = ba.qk_norm_backward(q, k, gq, gk, wq, wk, rope=rope, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    outs = [torch.zeros_like(x) for x in fwd + first]
    ws = ba.qk_norm_workspace(B, H, Hkv, T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ba.bam_qk_norm_fwd(q, k, outs[0], outs[1], None, norm, rope)
        ba.bam_qk_norm_bwd(q, k, gq, gk, *outs[2:], None, norm, rope, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, fwd + first))
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    want = ba.qk_norm_forward(q, k, wq, wk, rope=rope) + ba.qk_norm_backward(q, k, gq, gk, wq, wk, rope=rope)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_norm_gradients_in_a_graph():
    """Forward and gradients by autograd, captured after the eager graphs are gone."""
    g = _gen(6)
    q, k, gq, gk = (_normal(g, 2, h, 90, 64) for h in (3, 1, 3, 1))
    wq, wk = _weights(g, 3, 1, True)
    leaves = [x.requires_grad_() for x in (q, k, wq, wk)]

    def step():
        return torch.autograd.grad(qk_norm(*leaves, rope=ba.make_rope()), leaves, (gq, gk))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_norm_has_gradients_of_the_first_order_only():
    g = _gen(7)
    leaves = [x.requires_grad_() for x in (*(_normal(g, 1, 2, 5, 64) for _ in range(2)), *_weights(g, 2, 2, False))]
    grads = torch.autograd.grad(sum(x.float().pow(2).sum() for x in qk_norm(*leaves)), leaves, create_graph=True)
    with pytest.raises(RuntimeError):
        grads[0].float().sum().backward()


def test_gradients_that_begin_anywhere():
    """Outputs joined behind three other numbers: their gradients are slices whose rows lie
    on no 16 bytes."""
    g = _gen(11)
    q, k = (_normal(g, 1, 2, 40, 64).requires_grad_() for _ in range(2))
    wq, wk = (x.requires_grad_() for x in _weights(g, 2, 2, False))
    prm = [torch.tensor(x, device="cuda").requires_grad_() for x in ([5.0, 20.0], [1.0, 0.5], [0.3, 2.5])]
    v = _normal(g, 1, 2, 40, 64).requires_grad_()
    up = _normal(g, 3 * 5120 + 3)
    parts = [x.flatten() for x in (*qk_norm(q, k, wq, wk), bam_attention(v, v, v, *prm))]
    leaves = (q, k, wq, wk, v, *prm)
    got = torch.autograd.grad(torch.cat([torch.zeros_like(up[:3])] + parts), leaves, up, retain_graph=True)
    want = torch.autograd.grad(parts, leaves, [up[3 + 5120 * i:][:5120].clone() for i in range(3)])
    assert all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))
    for a, b in zip(got[4:], want[4:]):  # dQ and the scalars' sums have no order of their own
        torch.testing.assert_close(a.float(), b.float(), rtol=2.0 ** -6, atol=2.0 ** -6 * float(b.abs().max()))


@pytest.mark.parametrize("per_head", [False, True])
def test_infinite_gradients_reach_the_weights_as_themselves(per_head):
    """dw is the sum of dn n: infinite where one of its terms is, NaN where two cancel, and
    finite in every other place."""
    g = _gen(12)
    q, k = _normal(g, 2, 3, 700, 64), _normal(g, 2, 3, 700, 64)
    wq, wk = _weights(g, 3, 3, per_head)
    gq, gk = _normal(g, 2, 3, 700, 64), _normal(g, 2, 3, 700, 64)
    q[1, 2, 650, 5], q[0, 1, 3, 9], q[1, 1, 600, 9], q[0, 2, 1, 20] = 1.0, 1.0, 1.0, -2.0
    gq[1, 2, 650, 5] = gq[0, 1, 3, 9] = gq[0, 2, 1, 20] = float("inf")
    gq[1, 1, 600, 9] = float("-inf")
    _, _, dwq, dwk = ba.qk_norm_backward(q, k, gq, gk, wq, wk)
    assert torch.isfinite(dwk).all()
    want = torch.zeros(3, 64, device="cuda")
    want[2, 5], want[1, 9], want[2, 20] = float("inf"), float("nan"), float("-inf")
    want = want if per_head else want.sum(0)
    bad = ~torch.isfinite(want)
    torch.testing.assert_close(dwq[bad], want[bad], rtol=0, atol=0, equal_nan=True)
    assert torch.isfinite(dwq[~bad]).all()


def test_norm_of_a_broadcast_input():
    """A batch of one, expanded: each copy's gradient, summed by autograd."""
    g = _gen(8)
    q, k = (_normal(g, 1, 2, 40, 64).requires_grad_() for _ in range(2))
    wq, wk = (x.requires_grad_() for x in _weights(g, 2, 2, False))
    gq, gk = _normal(g, 3, 2, 40, 64), _normal(g, 3, 2, 40, 64)
    wide = [x.expand(3, -1, -1, -1) for x in (q, k)]
    got = torch.autograd.grad(qk_norm(*wide, wq, wk), (wide[0], wide[1], wq, wk), (gq, gk))
    dense = [x.detach().expand(3, -1, -1, -1).contiguous() for x in (q, k)]
    want = ba.qk_norm_backward(*dense, gq, gk, wq.detach(), wk.detach())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dq, = torch.autograd.grad(qk_norm(*(x.expand(3, -1, -1, -1) for x in (q, k)), wq, wk)[0], q, gq)
    assert dq.shape == q.shape and torch.isfinite(dq).all()


@pytest.mark.parametrize("per_head", [False, True])
def test_norm_of_places_beyond_32_bits(per_head):
    """The stride of a batch of one may be anything: its places then take 64 bits."""
    g = _gen(9)
    H, Hkv, T = 9, 2, 130
    q, k, gq, gk = (_normal(g, 1, h, T, 64) for h in (H, Hkv, H, Hkv))
    far = [x.as_strided(x.shape, (1 << 40,) + x.stride()[1:]) for x in (q, k, gq, gk)]
    wq, wk = _weights(g, H, Hkv, per_head)
    rope = ba.make_rope(10000.0, 32)
    pos = torch.arange(T, 0, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    want = ba.qk_norm_forward(q, k, wq, wk, pos, rope) + ba.qk_norm_backward(q, k, gq, gk, wq, wk, pos, rope)
    got = ba.qk_norm_forward(*far[:2], wq, wk, pos, rope) + ba.qk_norm_backward(*far, wq, wk, pos, rope)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_norm_then_attention_trains_all_parameters():
    """The training path: norms, attention and their gradients, against the same
    step in 64 bits."""
    g = _gen(4)
    B, H, T = 2, 3, 70
    qkv = (_normal(g, B, T, 3 * H, 64)).requires_grad_()
    wq, wk = (x.requires_grad_() for x in _weights(g, H, H, False))
    prm = [torch.tensor(x, device="cuda").requires_grad_() for x in
           ([5.0, 20.0, 3.0], [1.0, 0.5, 1.5], [0.3, 2.5, 1.2], [0.5, 0.7, 0.9])]
    dO = _normal(g, B, H, T, 64)
    q, k, v = (x.transpose(1, 2) for x in qkv.split(H, 2))
    rope = ba.make_rope(10000.0, 64)
    qn, kn = qk_norm(q, k, wq, wk, rope=rope)
    o = bam_attention(qn, kn, v.contiguous(), *prm, ssmax=True)
    o.backward(dO)

    leaves = [x.detach().double().requires_grad_() for x in (qkv, wq, wk, *prm)]
    q64, k64, v64 = (x.transpose(1, 2) for x in leaves[0].split(H, 2))
    pos = torch.arange(T, device="cuda")

    def rot(x, w):
        n = w * x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        f = torch.arange(32, device="cuda").double()
        ang = pos.double()[:, None] * 10000.0 ** (-f / 32)
        a, b = n[..., :32], n[..., 32:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    al, be, mu, s = (x[:, None, None] for x in leaves[3:])
    d = (pos[:, None] - pos[None]).double()
    c = s * torch.log(pos.double() + 1)[:, None] / 8
    z = c * (rot(q64, leaves[1]) @ rot(k64, leaves[2]).transpose(2, 3)) - ((d - mu).abs() / al) ** be
    z = z.masked_fill(d < 0, -float("inf"))
    (torch.softmax(z, -1) @ v64).backward(dO.double())
    # q' and k' are rounded to bf16 once more than in the definition, as are the
    # gradients between the two operators: the relative bound of the attention's gradients
    for got, want in zip((qkv, wq, wk, *prm), leaves):
        e = (got.grad.double() - want.grad).abs().max() / want.grad.abs().max()
        assert float(e) < GRAD_RTOL, float(e)


@pytest.mark.parametrize("dims,pairs", [(0, False), (64, False), (32, True)])
@pytest.mark.parametrize("B,H,Hkv,T", [(8, 32, 32, 512), (8, 64, 8, 512), (8, 48, 8, 512), (1, 64, 8, 1300),
                                       (1, 40, 10, 2500), (1, 48, 4, 2500), (1, 70, 70, 2500)])
def test_norm_of_many_heads_with_weights_of_their_own(B, H, Hkv, T, dims, pairs):
    """So many tokens that a CTA takes 13 to 16 passes of heads, whose sums it holds all at once."""
    _run(H + Hkv + dims, B, H, Hkv, T, dims, pairs, True, False)


def test_norm_refusals():
    g = _gen(6)
    q, k = _normal(g, 2, 4, 8, 64), _normal(g, 2, 2, 8, 64)
    wq, wk = _weights(g, 4, 2, True)
    good = ba.make_qk_norm(wq, wk)
    out = torch.empty_like(q), torch.empty_like(k)
    for args in ((q.float(), k, *out), (q, k[:1], *out), (q, k, out[0][:, :2], out[1]),
                 (q, k, out[0], out[1].cpu())):
        with pytest.raises((ValueError, ba.BamError)):
            ba.bam_qk_norm_fwd(*args, None, good)
    with pytest.raises(ValueError, match="positions"):
        ba.bam_qk_norm_fwd(q, k, *out, torch.zeros(2, 9, dtype=torch.int32, device="cuda"), good)
    with pytest.raises(ValueError, match="weights"):
        ba.bam_qk_norm_fwd(q, k, *out, None, ba.make_qk_norm(wk, wk))
    with pytest.raises(ba.BamError):  # rows of the output lie on one another
        ba.bam_qk_norm_fwd(q, k, out[0][:, :1].expand(2, 4, 8, 64), out[1], None, good)
    with pytest.raises(ValueError, match="both"):
        ba.make_qk_norm(wq, wk[0])
    with pytest.raises(ValueError, match="eps"):
        ba.make_qk_norm(wq, wk, 0.0)
    with pytest.raises(ValueError, match="aligned"):
        ba.make_qk_norm(torch.ones(65, device="cuda")[1:], torch.ones(64, device="cuda"))
    x = _normal(g, 2, 4, 8, 72)[..., 4:68]
    with pytest.raises(ValueError, match="aligned rows"):
        ba.bam_qk_norm_fwd(x, k, *out, None, good)
    ba.bam_qk_norm_fwd(q, k, *out, None, good)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- append

def _append(seed, B, H, Hkv, N, page, lens, new, dims, pairs, per_head, marked, parents=None, norm=True):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    blocks = [-(-(l + N) // page) for l in lens]
    num = sum(blocks) + 1
    perm = rng.permutation(num)
    table = np.full((B, max(blocks)), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    kp, vp = _normal(g, num, Hkv, page, 64), _normal(g, num, Hkv, page, 64)
    kpos = torch.full((num, Hkv, page), -7, dtype=torch.int32, device="cuda")
    kw = torch.full((num, Hkv, page), 5.0, device="cuda")
    k0, v0 = kp.clone(), vp.clone()
    qkv = _normal(g, B, N, H + 2 * Hkv, 64) * 2
    q, k, v = (x.transpose(1, 2) for x in qkv.split([H, Hkv, Hkv], 2))
    wq, wk = _weights(g, H, Hkv, per_head)
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
    first = [int(l) + 1000 * (b + 1) for b, l in enumerate(lens)] if marked else None
    qo = torch.full((B, H, N, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    ws = ba.cache_workspace()
    par = None if parents is None else i32(parents)
    ba.bam_kv_append_norm_paged(
        k, v, kp, vp, i32(table), i32(lens), i32(new), par, q, qo,
        ba.make_qk_norm(wq, wk, EPS) if norm else None, ba.make_rope(10000.0, dims, pairs),
        None if first is None else i32(first), ba.make_marks(kpos, kw, 1 << 20) if marked else None, ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    used = torch.zeros(num, page, dtype=torch.bool, device="cuda")
    for b in range(B):
        n = int(new[b])
        depth = np.arange(n)
        if parents is not None:
            depth = np.zeros(n, int)
            for i in range(n):
                depth[i] = depth[parents[b][i]] + 1 if parents[b][i] >= 0 else 0
        pos = (lens[b] if first is None else first[b]) + depth
        slot = np.arange(lens[b], lens[b] + n)
        pg, row = torch.from_numpy(table[b, slot // page].astype(np.int64)).cuda(), torch.from_numpy(slot % page).cuda()
        used[pg, row] = True
        ps = torch.from_numpy(pos).cuda()
        for x, w, y in ((q, wq, qo[b, :, :n]), (k, wk, kp[pg, :, row].transpose(0, 1))):
            if norm:
                _check(y, *norm_rotate(x[b, :, :n].double(), _w64(w), ps, EPS, 10000.0, dims, pairs))
        assert torch.equal(vp[pg, :, row].transpose(0, 1), v[b, :, :n])
        assert torch.all(qo[b, :, n:] == 3.0)
        if marked:
            assert torch.equal(kpos[pg, :, row], ps.int()[:, None].expand(n, Hkv))
            assert torch.all(kw[pg, :, row] == 0)
    away = ~used[:, None].expand(num, Hkv, page)
    assert torch.equal(kp[away], k0[away]) and torch.equal(vp[away], v0[away])
    assert torch.all(kpos[away] == -7) and torch.all(kw[away] == 5.0)
    if not norm:  # the plain append's results, bit for bit
        k1, v1, q1 = k0.clone(), v0.clone(), torch.full_like(qo, 3.0)
        if first is None:
            ba.bam_kv_append_paged(k, v, k1, v1, i32(table), i32(lens), i32(new), par, q, q1,
                                   ba.make_rope(10000.0, dims, pairs), ws)
            assert torch.equal(kp, k1) and torch.equal(vp, v1) and torch.equal(qo, q1)


@pytest.mark.parametrize("dims,pairs", [(0, False), (32, True), (64, False), (48, False)])
@pytest.mark.parametrize("marked,per_head", [(True, False), (False, True)])
@pytest.mark.parametrize("H,Hkv,N", [(1, 1, 1), (8, 2, 1), (5, 5, 7), (12, 12, 100), (42, 3, 3)])
def test_append_norm(H, Hkv, N, dims, pairs, marked, per_head):
    lens, new = [0, 63, 64, 200], [N, max(0, N - 1), 0, (N + 1) // 2]
    _append(N + H, 4, H, Hkv, N, 64, lens, new, dims, pairs, per_head, marked)


def test_append_norm_of_many_tiles():
    """More token tiles than CTAs: they are dealt out."""
    lens = [5, 130, 0, 77, 1, 64]
    _append(9, 6, 4, 2, 2000, 128, lens, [2000, 1999, 1, 0, 1500, 2000], 64, False, True, True)


def test_append_norm_positions_follow_a_tree():
    parents = [[-1, -1, 0, 2, 1, 4], [-1, 0, 1, 2, 3, 4]]
    _append(10, 2, 4, 2, 6, 64, [60, 0], [6, 5], 64, False, False, True, parents=parents)


@pytest.mark.parametrize("N", [1, 30])
def test_append_without_norm_is_the_plain_append(N):
    _append(13, 3, 4, 2, N, 64, [0, 63, 100], [N, N, N - 1], 64, True, False, False, norm=False)


def test_append_reports_positions_out_of_range():
    g = _gen(14)
    kp, vp = _normal(g, 2, 1, 64, 64), _normal(g, 2, 1, 64, 64)
    kpos, kw = torch.zeros(2, 1, 64, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, 64, device="cuda")
    x = _normal(g, 1, 1, 4, 64)
    table, ln = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    ws = ba.cache_workspace()
    for first, max_pos, want in ((10, 14, ba.BAM_OK), (10, 13, ba.BAM_ERR_INVALID_ARG),
                                 (-1, 100, ba.BAM_ERR_INVALID_ARG),
                                 ((1 << 28) + 1, 1 << 28, ba.BAM_ERR_INVALID_ARG)):
        f = torch.tensor([first], dtype=torch.int32, device="cuda")
        ba.kv_append_norm_paged(x, x, kp, vp, table, ln, first_pos=f, marks=ba.make_marks(kpos, kw, max_pos), ws=ws)
        assert ba.bam_attn_check_status(ws) == want
