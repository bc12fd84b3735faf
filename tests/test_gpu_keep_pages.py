"""Keeping a path whose pages are not all there."""

import pytest

torch = pytest.importorskip("torch")

from transformer_attention_ggd_gb300 import bam_attn as ba

from test_gpu_tree import Cache, _i32, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [lambda pages: -1, lambda pages: pages, lambda pages: 1 << 30])
def test_a_chain_on_a_page_out_of_range_is_not_kept(bad):
    """As with a tree: the sequence keeps its length and the call reports it.  A
    path that ends before the page, or that is empty, does not look at it."""
    c = Cache(83, 2, 64, [128, 128], 2, 0.0)
    before = c.k.clone(), c.v.clone()
    table = c.table.clone()
    table[0, 1] = bad(c.k.shape[0])
    ws = ba.cache_workspace()

    def keep(lens, accepted):
        new = ba.kv_keep_paged(c.k, c.v, table, _i32(lens), _i32(accepted), None, _i32([10, 10]),
                               None, ws)
        return new.tolist(), ba.bam_attn_check_status(ws)

    assert keep([60, 60], [4, 4]) == ([60, 65], ba.BAM_ERR_INVALID_ARG)
    assert keep([60, 60], [3, 4]) == ([64, 65], ba.BAM_OK)
    assert keep([64, 60], [-1, 4]) == ([64, 65], ba.BAM_OK)
    assert keep([64, 60], [0, 4]) == ([64, 65], ba.BAM_ERR_INVALID_ARG)
    assert torch.equal(c.k, before[0]) and torch.equal(c.v, before[1])
