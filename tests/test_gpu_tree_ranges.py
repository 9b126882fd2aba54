"""Queries of very different sizes in one call (GPU): a padded draft that holds whatever
its memory held, as long as it is finite, leaves the other drafts' answers as they are,
and has its own."""
import math

import pytest
import torch

from tests.spec_helpers import chain, fill_cache
from tests.tree_bounds import assert_within, bounded_reference

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")


def _small_cache(cb, L, seed):
    """Keys of norm about 1."""
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(1, 1, L, cb.head_dim, generator=g) / math.sqrt(cb.head_dim)
    v = torch.randn(1, 1, L, cb.head_dim, generator=g)
    cache = tq.Cache(cb, 1, 1, (L + 15) // 16 * 16)
    tq.tq_quantize_append(cb, cache, k.cuda(), v.cuda())
    return cache


@pytest.mark.parametrize("d,qjl,codebook", [(64, False, "gaussian"), (128, False, "gaussian"), (128, True, "gaussian"),
                                            (256, True, "sphere"), (128, False, "affine"), (64, True, "affine")])
@pytest.mark.parametrize("rows", [(6, 2), (40, 2), (25, 8)])
@pytest.mark.parametrize("size", [1e6, 1e30, 3e37])
def test_a_huge_row_among_ordinary_ones(d, qjl, codebook, rows, size):
    n, G = rows
    cb = tq.Codebook(d, 3, 4, qjl=qjl, codebook=codebook)
    L = n + 260
    cache = _small_cache(cb, L, seed=n)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(1, n, G, d, generator=g).mul(4 * math.sqrt(d)).bfloat16()
    wild = [(1, 0), (n - 1, G - 1)]
    for i, h in wild:
        q[0, i, h] = (torch.randn(d, generator=g) * size / 4).clamp(-size, size).bfloat16()
    got = tq.tq_tree_attention(cb, cache, q.cuda())
    out, tol, acc = bounded_reference(cb, cache, q, chain(n), [L])
    assert torch.isfinite(got).all()
    # (the huge rows attend one token: their scores differ by more than any rounding)
    assert_within(got, out, tol, acc)
    for i, h in wild:
        q[0, i, h] = 0
    tame = tq.tq_tree_attention(cb, cache, q.cuda())
    out, tol, acc = bounded_reference(cb, cache, q, chain(n), [L])
    assert_within(tame, out, tol, acc)


@pytest.mark.parametrize("rows", [(5, 1), (30, 4)])
def test_small_rows_under_a_large_scale(rows):
    """fp16 rows from 60000 down to 1e-3, with a softmax scale that makes the small ones count."""
    n, G = rows
    cb = tq.Codebook(128, 3, 4)
    L = n + 200
    cache = _small_cache(cb, L, seed=n)
    g = torch.Generator().manual_seed(6)
    sizes = torch.logspace(math.log10(1e-3), math.log10(1.4e4), n)
    q = (torch.randn(1, n, G, 128, generator=g).clamp(-4, 4) * sizes[None, :, None, None]).half()
    got = tq.tq_tree_attention(cb, cache, q.cuda(), softmax_scale=700.0)
    assert_within(got, *bounded_reference(cb, cache, q, chain(n), [L], scale=700.0))


def test_scores_far_below_zero():
    """Every token opposes the query: the largest score is about -1e33."""
    cb = tq.Codebook(128, 4, 4)
    L, d = 150, 128
    g = torch.Generator().manual_seed(7)
    base = torch.randn(d, generator=g)
    k = base + 0.05 * torch.randn(1, 1, L, d, generator=g)
    v = torch.randn(1, 1, L, d, generator=g)
    cache = tq.Cache(cb, 1, 1, 160)
    tq.tq_quantize_append(cb, cache, k.cuda(), v.cuda())
    q = (base * -1e32).expand(1, 3, 2, d).bfloat16().contiguous()
    got = tq.tq_tree_attention(cb, cache, q.cuda())
    assert_within(got, *bounded_reference(cb, cache, q, chain(3), [L]))


def test_sizes_within_a_call_do_not_move_ordinary_rows():
    """Rows up to 2^16 apart share a scale; a row of zeros counts for nothing."""
    cb = tq.Codebook(128, 3, 4)
    cache = fill_cache(tq, cb, 1, 1, 320, [300], seed=4)
    q = torch.randn(1, 8, 2, 128, generator=torch.Generator().manual_seed(8)).bfloat16()
    q[0, 3] *= 2.0 ** 10
    q[0, 5] = 0
    out = tq.tq_tree_attention(cb, cache, q.cuda())
    assert_within(out, *bounded_reference(cb, cache, q, chain(8), [300]))


@pytest.mark.parametrize("codebook", ["gaussian", "affine"])
@pytest.mark.parametrize("rows", [(4, 1), (30, 8)])
@pytest.mark.parametrize("dtype,size", [(torch.float16, 2e4), (torch.bfloat16, 1e25), (torch.float16, 900.0)])
def test_scores_whose_steps_are_larger_than_one(dtype, size, rows, codebook):
    """Every query and key is large: scores of 2^27 and more, whose fp32 steps exceed the
    room of a weight.  The largest score still decides, and nothing overflows."""
    n, G = rows
    cb = tq.Codebook(128, 3, 4, codebook=codebook)
    L = n + 300
    g = torch.Generator().manual_seed(9)
    k = torch.randn(1, 1, L, 128, generator=g) * (4e3 if codebook == "gaussian" else 1e4)
    v = torch.randn(1, 1, L, 128, generator=g) * torch.logspace(-3, 2, L)[:, None]
    cache = tq.Cache(cb, 1, 1, (L + 15) // 16 * 16)
    tq.tq_quantize_append(cb, cache, k.cuda(), v.cuda())
    q = (torch.randn(1, n, G, 128, generator=g).clamp(-3, 3) * size).to(dtype)
    got = tq.tq_tree_attention(cb, cache, q.cuda())
    assert torch.isfinite(got).all()
    assert_within(got, *bounded_reference(cb, cache, q, chain(n), [L]))
