"""One token that outweighs the others by far, over a long flat tail (GPU): the tail's
weights are small, but there are many, and a unit's row is one block's alone."""
import math

import pytest
import torch

from tests.spec_helpers import chain, rotation
from tests.tree_bounds import assert_within, bounded_reference, passes, _stored

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")


@pytest.mark.parametrize("codebook", ["gaussian", "affine"])
@pytest.mark.parametrize("ctx,at", [(131072, 0), (131072, 70001), (131072, 131000), (20000, 3)])
@pytest.mark.parametrize("bits", [18.0, 22.0, 25.5])
def test_a_peak_over_a_flat_tail(codebook, ctx, at, bits):
    """`bits`: by how many powers of two the peak outweighs one token of the tail.  As
    many units as blocks, so that no share is shorter than a row."""
    d, n, H = 64, 2, 2
    B = 74
    cb = tq.Codebook(d, 2, 2, codebook=codebook)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(2, 1, 1, 2, d, generator=g)                       # key and value of the peak and of the tail
    x[1] *= (x[1, ..., :1, :].norm() / x[1].norm(dim=-1, keepdim=True))
    small = tq.Cache(cb, 1, 1, 16)
    tq.tq_quantize_append(cb, small, x[0].cuda(), x[1].cuda())
    cap = (ctx + n + 15) // 16 * 16
    cache = tq.Cache(cb, B, H, cap)
    for name in ("k_codes", "v_codes", "k_norm", "v_norm"):
        t, s = getattr(cache, name), getattr(small, name)
        t[:] = s[:, :, 1:2]
        t[:, :, at:at + 1] = s[:, :, :1]
    cache.seq_lens.fill_(ctx + n)
    key = _stored(cb, small, "k", 0, 0, 2)[0].cpu()                  # [2, d], rotated
    q = ((key[0] - key[1]) @ rotation(cb)).half()
    apart = float((rotation(cb) @ q.double()) @ (key[0] - key[1]))
    scale = bits * math.log(2) / apart
    q = q.expand(B, n, H, d).contiguous()
    got = tq.tq_tree_attention(cb, cache, q.cuda(), softmax_scale=scale)
    assert torch.equal(got, got[:1, :, :1].expand_as(got))
    out, tol, acc = bounded_reference(cb, _row(cache), q[:1, :, :1], chain(n), [ctx + n], scale=scale, share=ctx + n)
    assert_within(got[:1, :, :1], out, tol, acc)
    # a tail that vanished would not pass where it weighs more than the peak's own rounding
    if ctx * 2.0 ** -bits > 2.0 ** -9:
        v = _stored(cb, small, "v", 0, 0, 2)[0].cuda()
        if codebook != "affine":
            v = v @ rotation(cb).cuda()
        lost = (v[0] / (1 + (ctx + n - 1) * 2.0 ** -bits)).expand_as(out)
        found = not passes(lost, out, tol, acc, torch.float16)
        assert found


def _row(cache):
    """The first row and head as a cache of their own."""
    one = tq.Cache.__new__(tq.Cache)
    one.__dict__.update(cache.__dict__)
    one.batch = one.kv_heads = 1
    for name in ("k_codes", "v_codes", "k_norm", "v_norm"):
        setattr(one, name, getattr(cache, name)[:1, :1])
    return one
