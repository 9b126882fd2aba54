"""Tree attention (GPU) against its formula in float64, held to a bound that wrong
answers do not meet (test_tree_bounds.py): every codec, type and row class, long rows
over many blocks, queries that are stored keys', ragged batches of more units than
blocks."""
import pytest
import torch

from tests.spec_helpers import chain, fill_cache, random_tree, rotation
from tests.tree_bounds import _stored, assert_within, bounded_reference, found, passes

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")

DTYPES = [torch.bfloat16, torch.float16]


def _q(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _check(cb, cache, q, sees, lens, drafts=None, **kw):
    got = tq.tq_tree_attention(cb, cache, q.cuda(), mask=tq.pack_tree_mask(sees).cuda())
    ref = bounded_reference(cb, cache, q, sees, lens, drafts=drafts, **kw)
    assert_within(got if drafts is None else got[:, drafts], *ref)
    return got, ref


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kb,vb,qjl,codebook", [
    (3, 4, False, "gaussian"), (3, 4, True, "sphere"), (2, 2, True, "gaussian"), (2, 2, False, "gaussian"),
    (2, 3, False, "gaussian"), (3, 3, True, "gaussian"), (4, 4, False, "gaussian"), (2, 3, True, "sphere"),
    (4, 4, True, "affine"), (2, 3, False, "affine"), (3, 4, False, "affine"), (2, 2, True, "affine"),
    (3, 3, False, "affine")])
def test_codecs(d, kb, vb, qjl, codebook, dtype):
    cb = tq.Codebook(d, kb, vb, qjl=qjl, seed=kb * 8 + vb, codebook=codebook)
    lens, H = [301, 133], 2
    cache = fill_cache(tq, cb, 2, H, 320, lens, seed=d + kb)
    for n, G in ((5, 2), (13, 4)):
        sees = random_tree(n, seed=n)
        _check(cb, cache, _q((2, n, H * G, d), dtype, 7), sees, lens, drafts=[0, n // 2, n - 1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 256])
def test_row_counts(G, n, dtype):
    cb = tq.Codebook(128, 3, 4, seed=n)
    lens = [n + 140]
    cache = fill_cache(tq, cb, 1, 1, 400, lens, seed=G)
    drafts = sorted({0, n // 3, 15 % n, 16 % n, 31 % n, 32 % n, 64 % n, n - 1})
    got, ref = _check(cb, cache, _q((1, n, G, 128), dtype, n), random_tree(n, seed=n + G), lens, drafts=drafts)
    if n > 4:
        assert not passes(ref[0].roll(1, 1), *ref, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [(3, 4), (40, 4), (9, 1)])
@pytest.mark.parametrize("qjl,codebook", [(False, "gaussian"), (True, "gaussian"), (False, "affine")])
def test_long_rows_over_many_blocks(rows, qjl, codebook, dtype):
    """40005 tokens in about 148 shares; some queries are keys that the row stores, in its
    first, an inner and its last tile."""
    n, G = rows
    d, L = 128, 40005
    cb = tq.Codebook(d, 3, 4, qjl=qjl, codebook=codebook)
    cache = fill_cache(tq, cb, 1, 1, 40016, [L], seed=5)
    keys = _stored(cb, cache, "k", 0, 0, L)[0].cpu()
    q = _q((1, n, G, d), torch.float32, 3)
    for j, (i, g, at) in enumerate([(0, 0, 7), (1, G - 1, 23456), (2, 0, L - n - 2), (n - 1, G - 1, L - n)]):
        q[0, i, g] = (keys[at] @ rotation(cb)).float() * (0.5 + 0.25 * j)
    q = q.to(dtype)
    drafts = sorted({0, 1, 2, n // 2, n - 1})
    got, ref = _check(cb, cache, q, random_tree(n, 4), [L], drafts=drafts)
    assert not passes(torch.zeros_like(ref[0]), *ref, dtype)
    # and what a lost block would leave
    kept = _stored(cb, cache, "v", 0, 0, L)[0]
    assert found(ref[0] - (kept[23400:23670].sum(0) / L).expand_as(ref[0]), *ref, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_ragged_batches(d, dtype):
    """More units than blocks, of rows from none to some tiles: shares that begin and end
    inside rows."""
    cb = tq.Codebook(d, 3, 4, qjl=d == 64)
    B, H, G, n = 45, 4, 2, 7
    lens = [(b * 137) % 1500 for b in range(B)]
    cache = fill_cache(tq, cb, B, H, 1504, lens, seed=d)
    q = _q((B, n, H * G, d), dtype, 2)
    got, ref = _check(cb, cache, q, random_tree(n, 6), lens, drafts=[0, n - 1])
    for b, length in enumerate(lens):
        if length < n:
            assert torch.all(got[b] == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.02, 0.3, 1.0])
def test_flat_and_peaked_scores(scale, dtype):
    cb = tq.Codebook(128, 4, 4)
    lens = [700]
    cache = fill_cache(tq, cb, 1, 2, 704, lens, seed=9)
    q = _q((1, 11, 8, 128), dtype, 5)
    sees = random_tree(11, 2)
    got = tq.tq_tree_attention(cb, cache, q.cuda(), mask=tq.pack_tree_mask(sees).cuda(), softmax_scale=scale)
    ref = bounded_reference(cb, cache, q, sees, lens, scale=scale)
    assert_within(got, *ref)
    wrong = tq.tq_tree_attention(cb, cache, q.cuda(), softmax_scale=scale)
    assert found(wrong.double(), *ref, dtype)             # a chain instead of the tree
