"""Tree attention of rows that max_ctx cuts inside their context (GPU): tokens at
max_ctx and past it are not attended, whatever the cache holds there."""
import math

import pytest
import torch

from tests.spec_helpers import chain, fill_cache, random_tree
from tests.tree_bounds import assert_within, bounded_reference

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")

CODECS = [("gaussian", False), ("gaussian", True), ("affine", False), ("affine", True)]


def _poison(cache, b, at):
    """Norms that reach the output of whoever attends them, from slot `at` on."""
    cache.v_norm[b, :, at:] = math.nan
    cache.k_norm[b, :, at:] = math.inf
    if cache.k_rnorm is not None:
        cache.k_rnorm[b, :, at:] = math.nan


@pytest.mark.parametrize("codebook,qjl", CODECS)
@pytest.mark.parametrize("lens,cut", [([310, 64], 200), ([310, 290], 129), ([310, 303], 127), ([700, 128], 1),
                                      ([640, 500], 384), ([2000, 130], 1000)])
@pytest.mark.parametrize("dtype,n,G", [(torch.bfloat16, 8, 2), (torch.float16, 3, 1)])
def test_a_cut_inside_the_context(codebook, qjl, lens, cut, dtype, n, G):
    cb = tq.Codebook(128, 3, 4, codebook=codebook, qjl=qjl)
    cache = fill_cache(tq, cb, 2, 2, 2000, lens, seed=cut)
    for b, L in enumerate(lens):
        _poison(cache, b, cut)
    q = (torch.randn(2, n, 2 * G, 128, generator=torch.Generator().manual_seed(cut)) * 2).to(dtype)
    sees = random_tree(n, cut)
    got = tq.tq_tree_attention(cb, cache, q.cuda(), mask=tq.pack_tree_mask(sees).cuda(), max_ctx=cut)
    assert torch.isfinite(got).all()
    assert int(cache.status.item()) == tq.TQ_FLAG_MAXCTX
    assert_within(got, *bounded_reference(cb, cache, q, sees, lens, max_ctx=cut))
    again = tq.tq_tree_attention(cb, cache, q.cuda(), mask=tq.pack_tree_mask(sees).cuda(), max_ctx=cut)
    assert torch.equal(got, again)


@pytest.mark.parametrize("cut", [1000, 20000, 20001])
def test_a_cut_of_a_long_row(cut):
    """Every block's share ends inside the context; the last tile is cut."""
    L, n = 40005, 5
    cb = tq.Codebook(128, 3, 4)
    cache = fill_cache(tq, cb, 1, 1, 40016, [L], seed=3)
    _poison(cache, 0, cut)
    q = torch.randn(1, n, 2, 128, generator=torch.Generator().manual_seed(4)).half()
    got = tq.tq_tree_attention(cb, cache, q.cuda(), max_ctx=cut)
    assert_within(got, *bounded_reference(cb, cache, q, chain(n), [L], max_ctx=cut))


@pytest.mark.parametrize("d,rows", [(64, (40, 8)), (256, (9, 4)), (128, (1, 1)), (128, (60, 2))])
def test_a_cut_at_every_column_count(d, rows):
    n, G = rows
    cb = tq.Codebook(d, 3, 4, qjl=d == 256)
    cache = fill_cache(tq, cb, 1, 1, 512, [500], seed=3)
    _poison(cache, 0, 170)
    q = torch.randn(1, n, G, d, generator=torch.Generator().manual_seed(4)).bfloat16()
    got = tq.tq_tree_attention(cb, cache, q.cuda(), max_ctx=170)
    assert_within(got, *bounded_reference(cb, cache, q, chain(n), [500], max_ctx=170))
