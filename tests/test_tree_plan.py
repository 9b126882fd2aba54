"""Every shape the tree attention accepts has a plan (CPU): the host lays out
shared and tensor memory for it, and says how large its workspace is."""
import pytest

from turboquant_kv_cache_rht_b200 import tq


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kb,vb", [(2, 2), (2, 3), (3, 3), (3, 4), (4, 4)])
@pytest.mark.parametrize("qjl", [False, True])
@pytest.mark.parametrize("codebook", ["gaussian", "affine"])
def test_every_shape_has_a_plan(d, kb, vb, qjl, codebook):
    cb = tq.Codebook(d, kb, vb, qjl=qjl, codebook=codebook)
    last = 0
    for n in (1, 2, 4, 5, 8, 16, 33, 64, 128, 256):
        for g in (1, 2, 4, 8):
            size = tq.tq_tree_workspace_bytes(cb, 2, 2 * g, 2, n, 512)
            # every row's sum, maximum and output, in fp32
            assert size >= 4 * 2 * 2 * n * g * (d + 2)
        assert size >= last
        last = size
        # a longer context takes more blocks' partials, up to one wave of blocks
        assert tq.tq_tree_workspace_bytes(cb, 2, 2, 2, n, 1 << 20) >= tq.tq_tree_workspace_bytes(cb, 2, 2, 2, n, 128)
        assert tq.tq_tree_workspace_bytes(cb, 2, 2, 2, n, 1 << 20) == tq.tq_tree_workspace_bytes(cb, 2, 2, 2, n, 1 << 24)
