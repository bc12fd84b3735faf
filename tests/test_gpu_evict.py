"""GPU tests of eviction from a paged cache by accumulated weight, in place and
to other pages, against a plain implementation."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from _bounded_reference import kept_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ba.load_library()


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


class Cache:
    """Pages whose rows, positions and weights are all different bits."""

    def __init__(self, seed, Hkv, page, lens, weights, spare=0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        blocks = [-(-int(n) // page) for n in lens]
        cap = max(1, max(blocks))
        num = sum(blocks) + 2 + spare
        perm = rng.permutation(num)
        table = np.full((len(lens), cap), -1, np.int32)
        at = 0
        for b, n in enumerate(blocks):
            table[b, :n] = perm[at:at + n]
            at += n
        self.spare = perm[at:]
        self.k, self.v = (torch.randint(-30000, 30000, (num, Hkv, page, 64), generator=gen, device="cuda",
                                        dtype=torch.int16).view(torch.bfloat16) for _ in range(2))
        self.pos = torch.randint(0, 1 << 20, (num, Hkv, page), generator=gen, device="cuda", dtype=torch.int32)
        self.w = torch.from_numpy(weights(rng, (num, Hkv, page)).astype(np.float32)).cuda()
        self.table, self.rng = table, rng

    def host(self):
        return [x.cpu() for x in (self.k.view(torch.int16), self.v.view(torch.int16), self.pos,
                                  self.w.view(torch.int32))]


def random_weights(rng, shape):
    return np.exp(2 * rng.standard_normal(shape))


def few_values(rng, shape):
    return rng.integers(0, 3, shape).astype(np.float64)


def odd_values(rng, shape):
    w = rng.standard_normal(shape)
    w[rng.random(shape) < 0.2] = np.nan
    w[rng.random(shape) < 0.1] = np.inf
    w[rng.random(shape) < 0.1] = -np.inf
    w[rng.random(shape) < 0.2] = 0.0
    w[rng.random(shape) < 0.2] = -0.0
    return w


def equal_weights(rng, shape):
    return np.full(shape, 0.25)


def _evict(seed, Hkv, page, lens, budget, sink, recent, weights, out=False, alias=False):
    B = len(lens)
    need = [-(-min(int(n), budget) // page) for n in lens]
    c = Cache(seed, Hkv, page, lens, weights, spare=sum(need) if out else 0)
    before = c.host()
    cap = c.table.shape[1]
    out_table, dst = None, c.table
    if out:
        blocks = -(-min(budget, cap * page) // page)
        dst = np.full((B, blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            dst[b, :n] = c.spare[at:at + n]
            at += n
        out_table = _i32(dst)
    ln = _i32(lens)
    new = ln if alias else torch.full((B,), -5, dtype=torch.int32, device="cuda")
    ws = ba.evict_workspace(B, Hkv, cap * page, budget)
    ws.fill_(0xFF)
    marks = ba.make_marks(c.pos, c.w, 1 << 20)
    ba.bam_kv_evict_paged(c.k, c.v, _i32(c.table), ln, marks, out_table, new, budget, sink, recent, ws)
    assert ba.bam_attn_check_status(ws) == ba.BAM_OK
    after = c.host()
    assert new.tolist() == [min(int(n), budget) for n in lens]
    want = [x.clone() for x in before]
    free = torch.zeros(before[2].shape, dtype=torch.bool)  # in place: slots behind the kept ones
    w = before[3].view(torch.float32).numpy()
    for b, n in enumerate(lens):
        n = int(n)
        s = np.arange(n)
        for h in range(Hkv):
            kept = kept_slots(w[c.table[b, s // page], h, s % page], budget, sink, recent)
            m = np.arange(len(kept))
            src = c.table[b, kept // page], h, kept % page
            to = dst[b, m // page], h, m % page
            for x, y in zip(want, before):
                x[to] = y[src]
            if not out and n > budget:
                t = np.arange(len(kept), n)
                free[c.table[b, t // page], h, t % page] = True
    for x, y in zip(after, want):
        assert torch.equal(x[~free], y[~free])
    return c


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("weights", [random_weights, few_values, odd_values, equal_weights])
@pytest.mark.parametrize("page,budget,sink,recent", [(64, 100, 4, 20), (64, 64, 0, 0), (128, 130, 0, 130),
                                                     (320, 200, 200, 0), (64, 1, 0, 0), (64, 1, 0, 1),
                                                     (64, 300, 5, 100)])
def test_evict(page, budget, sink, recent, weights, out):
    _evict(budget + out, 3, page, [0, 1, 63, 64, 65, 99, 100, 101, 200, 300, 301, 640], budget, sink, recent,
           weights, out)


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("n,budget", [(5000, 4000), (5000, 4999), (5000, 2), (20011, 9000), (70001, 65003)])
def test_evict_long_sequences(n, budget, out):
    """Many waves of a cluster of CTAs, in place and not."""
    _evict(n, 2, 64, [n, n // 3], budget, 1, min(budget // 3, 500), random_weights, out)
    _evict(n + 1, 1, 256, [n], budget, 0, 0, few_values, out)


def test_evict_many_sequences():
    rng = np.random.default_rng(1)
    _evict(2, 8, 64, rng.integers(0, 400, 100), 150, 4, 30, random_weights)


def test_evict_new_lens_may_be_cache_lens():
    _evict(3, 2, 64, [100, 500, 301], 300, 4, 50, few_values, alias=True)
    _evict(4, 2, 64, [100, 500, 301], 300, 4, 50, few_values, out=True, alias=True)


def test_evict_moves_nothing_when_the_last_keys_are_the_lightest():
    def falling(rng, shape):
        return np.zeros(shape)  # ties: the lowest slots stay
    c = _evict(5, 2, 64, [500], 400, 0, 0, falling)
    del c


def test_evict_a_budget_beyond_the_table_keeps_all():
    _evict(6, 2, 64, [100, 64], 10000, 9000, 500, random_weights)


def test_evict_is_repeatable_and_runs_on_streams_and_in_graphs():
    lens, budget = [900, 1300, 40], 500
    results = []
    for mode in ("eager", "stream", "graph"):
        c = Cache(7, 4, 64, lens, few_values)
        marks, ln, table = ba.make_marks(c.pos, c.w, 1 << 20), _i32(lens), _i32(c.table)
        ws = ba.evict_workspace(3, 4, c.table.shape[1] * 64, budget)
        new = torch.zeros_like(ln)
        call = lambda stream=None: ba.bam_kv_evict_paged(c.k, c.v, table, ln, marks, None, new, budget, 4, 64,
                                                         ws, stream)
        torch.cuda.synchronize()
        if mode == "eager":
            call()
        elif mode == "stream":
            side = torch.cuda.Stream()
            call(side)
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            graph.replay()
        torch.cuda.synchronize()
        results.append([x.clone() for x in c.host()] + [new.cpu()])
    for r in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, results[0]))


def test_evict_reports_bad_lengths_and_pages():
    """A sequence with a page out of range keeps its pages and its length; the
    others are evicted."""
    for bad in ("page", "out", "long", "negative"):
        lens, budget, page = [200, 300], 100, 64
        c = Cache(8, 2, page, lens, random_weights, spare=4)
        before = c.host()
        table, ln, out = c.table.copy(), list(lens), None
        if bad == "page":
            table[1, 2] = c.k.shape[0]
        elif bad == "out":
            out = np.stack([c.spare[:2], [c.spare[2], -3]])
        elif bad == "long":
            ln[1] = table.shape[1] * page + 7
        else:
            ln[1] = -1
        ws = ba.evict_workspace(2, 2, table.shape[1] * page, budget)
        marks = ba.make_marks(c.pos, c.w, 1 << 20)
        new = ba.kv_evict_paged(c.k, c.v, _i32(table), _i32(ln), marks, budget, 4, 20,
                                None if out is None else _i32(out), ws=ws)
        assert ba.bam_attn_check_status(ws) == ba.BAM_ERR_INVALID_ARG
        assert ba.bam_attn_check_status(ws) == ba.BAM_OK
        assert new.tolist() == [100, {"page": 300, "out": 300, "long": 100, "negative": 0}[bad]]
        after = c.host()
        if bad != "long":
            pages = c.table[1][c.table[1] >= 0]
            for x, y in zip(after, before):
                assert torch.equal(x[pages], y[pages])


def test_evict_refusals():
    c = Cache(9, 2, 64, [200, 300], random_weights)
    marks, ln, table = ba.make_marks(c.pos, c.w, 1 << 20), _i32([200, 300]), _i32(c.table)
    good = dict(budget=100, sink=4, recent=20)
    for kw in (dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=50, recent=51)):
        with pytest.raises(ba.BamError):
            ba.kv_evict_paged(c.k, c.v, table, ln, marks, **{**good, **kw})
    with pytest.raises(ba.BamError):  # room for 64 of 100 keys
        ba.kv_evict_paged(c.k, c.v, table, ln, marks, **good, out_table=_i32([[0], [1]]))
    for args in ((c.k.float(), c.v, table, ln), (c.k, c.v[:, :1], table, ln), (c.k, c.v, table.long(), ln),
                 (c.k, c.v, table, ln[:1])):
        with pytest.raises((ValueError, ba.BamError)):
            ba.kv_evict_paged(*args, marks, **good)
    with pytest.raises(ValueError, match="marks"):
        ba.kv_evict_paged(c.k, c.v, table, ln, ba.make_marks(c.pos[:1], c.w[:1], 9), **good)
    with pytest.raises(ba.BamError):
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        ba.kv_evict_paged(c.k, c.v, table, ln, marks, **good, ws=ws)
    with pytest.raises(ValueError):
        ba.make_marks(c.pos, c.w, 0)
    with pytest.raises(ValueError):
        ba.make_marks(c.pos, c.w.double(), 10)


@pytest.mark.parametrize("bad", ["page", "out", "long", "negative"])
def test_evict_goes_on_beside_a_bad_sequence(bad):
    """The good sequence's keys are evicted as if it stood alone, and one whose length is
    too long as if it filled its table."""
    lens, budget, page, sink, recent = [200, 300], 100, 64, 4, 20
    c = Cache(8, 2, page, lens, random_weights, spare=4)
    before = c.host()
    table, ln, out = c.table.copy(), list(lens), None
    if bad == "page":
        table[1, 2] = c.k.shape[0]
    elif bad == "out":
        out = np.stack([c.spare[:2], [c.spare[2], -3]])
    elif bad == "long":
        ln[1] = table.shape[1] * page + 7
    else:
        ln[1] = -1
    new = ba.kv_evict_paged(c.k, c.v, _i32(table), _i32(ln), ba.make_marks(c.pos, c.w, 1 << 20), budget, sink, recent,
                            None if out is None else _i32(out))
    after, w = c.host(), before[3].view(torch.float32).numpy()
    assert new[0] == budget
    for b, n in [(0, 200)] + ([(1, table.shape[1] * page)] if bad == "long" else []):
        dst = table[b] if out is None else out[b]
        for h in range(2):
            s, m = np.arange(n), np.arange(budget)
            kept = kept_slots(w[table[b, s // page], h, s % page], budget, sink, recent)
            for x, y in zip(after, before):
                assert torch.equal(x[dst[m // page], h, m % page], y[table[b, kept // page], h, kept % page])


@pytest.mark.parametrize("out", [False, True])
def test_evict_of_more_slots_than_shared_memory_holds(out):
    """8 CTAs hold 327680 weights; what lies behind is read from the pages each time."""
    _evict(10 + out, 1, 256, [400003, 1000], 250001, 5, 1000, random_weights, out)
    _evict(12 + out, 1, 64, [330001], 329000, 0, 0, few_values, out)
