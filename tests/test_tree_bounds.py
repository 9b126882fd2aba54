"""The bound that the tree attention is held to finds wrong answers (CPU only): zeros, a
share of a long row that was left out, another query's row do not pass for the formula's
result in any row; a mask that was not read, or drafts that were hidden, not in all."""
import math

import pytest
import torch

from tests.spec_helpers import chain, decoded, random_tree, rotation
from tests.tree_bounds import BLOCKS, assert_within, bounded_reference, found, passes
from turboquant_kv_cache_rht_b200 import tq


def _cache(cb, L, seed, kv_heads=1):
    """Codes and norms as the codec leaves them: every level about as often as it is met."""
    c = tq.Cache(cb, 1, kv_heads, (L + 15) // 16 * 16, device="cpu")
    g = torch.Generator().manual_seed(seed)
    for name in ("k_codes", "v_codes"):
        t = getattr(c, name)
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for name in ("k_norm", "v_norm"):
        t = getattr(c, name)
        if cb.affine:
            t[..., 0::2] = 0.3 + 0.02 * torch.rand(t[..., 0::2].shape, generator=g)
            t[..., 1::2] = -2.2 + 0.1 * torch.rand(t[..., 1::2].shape, generator=g)
        else:
            t.copy_(math.sqrt(cb.head_dim) * (1 + 0.1 * torch.randn(t.shape, generator=g)))
    if cb.qjl:
        c.k_signs.copy_(torch.randint(0, 256, c.k_signs.shape, generator=g, dtype=torch.uint8))
        c.k_rnorm.fill_(0.19 * math.sqrt(cb.head_dim))
    return c


def _rounded(out, dtype):
    return out.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("qjl,codebook", [(False, "gaussian"), (True, "gaussian"), (False, "affine")])
def test_a_long_row(dtype, qjl, codebook):
    cb = tq.Codebook(128, 3, 4, qjl=qjl, codebook=codebook)
    L, n = 40005, 2
    c = _cache(cb, L, 1)
    q = torch.randn(1, n, 2, 128, generator=torch.Generator().manual_seed(2)).to(dtype)
    out, tol, acc = bounded_reference(cb, c, q, chain(n), [L])
    assert_within(_rounded(out, dtype), out, tol, acc)
    assert not passes(torch.zeros_like(out), out, tol, acc, dtype)
    # one block's share of the row left out: the formula of what is left
    lost = _cache(cb, L, 1)
    at, some = 20000, L // BLOCKS
    for name in ("k_codes", "v_codes", "k_norm", "v_norm", "k_signs", "k_rnorm"):
        t = getattr(lost, name)
        if t is not None:
            t[:, :, at:L - some] = t[:, :, at + some:L].clone()
    assert not passes(bounded_reference(cb, lost, q, chain(n), [L - some])[0], out, tol, acc, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("qjl,codebook", [(False, "gaussian"), (True, "gaussian"), (False, "affine")])
def test_masks_and_rows(dtype, qjl, codebook):
    cb = tq.Codebook(128, 3, 4, qjl=qjl, codebook=codebook)
    L, n, G = 1024, 6, 2
    c = _cache(cb, L, 3)
    q = torch.randn(1, n, G, 128, generator=torch.Generator().manual_seed(4)).to(dtype)
    sees = random_tree(n, 5)
    out, tol, acc = bounded_reference(cb, c, q, sees, [L])
    other = lambda s: bounded_reference(cb, c, q, s, [L])[0]
    # one draft of a thousand tokens may weigh less than the roundings: not every row shows it
    assert found(other(torch.ones(n, n, dtype=torch.bool)), out, tol, acc, dtype)        # the mask ignored
    assert found(other(torch.zeros(n, n, dtype=torch.bool)), out, tol, acc, dtype)       # every draft hidden
    assert found(other(sees & ~torch.eye(n, dtype=torch.bool)), out, tol, acc, dtype)    # from itself alone
    assert not passes(out.roll(1, 1), out, tol, acc, dtype)                              # another draft's row
    assert not passes(out.roll(1, 2), out, tol, acc, dtype)                              # another head's
    assert not passes(out * (1 + 2.0 ** -4), out, tol, acc, dtype)


def test_a_peaked_row():
    """A query that is a stored key's: the answer is that token's value, and no other."""
    cb = tq.Codebook(128, 3, 4)
    L, n = 5000, 1
    c = _cache(cb, L, 6)
    q = (decoded(cb, c, "k", 0, 0, L)[[1234]] @ rotation(cb) * 1.5)[None, None].half()
    out, tol, acc = bounded_reference(cb, c, q, chain(n), [L])
    v = decoded(cb, c, "v", 0, 0, L) @ rotation(cb)
    assert float((out[0, 0, 0] - v[1234]).abs().max()) < 0.3
    for wrong in (v[1233], v.mean(0), torch.zeros(128, dtype=torch.float64)):
        assert not passes(wrong.expand_as(out), out, tol, acc, torch.float16)
