"""The speculative-decoding calls together, as a program makes them: a prompt is
appended, forked into samples, drafts are appended and verified against plain
float64 attention, the accepted path is kept, and the next step goes on from it."""
import pytest
import torch

from tests.spec_helpers import arrays, assert_tree_close, random_tree, tree_reference

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")


@pytest.mark.parametrize("d,qjl,codebook", [(128, False, "gaussian"), (64, True, "gaussian"), (128, True, "affine")])
def test_draft_verify_keep(d, qjl, codebook):
    cb = tq.Codebook(d, 3, 4, qjl=qjl, codebook=codebook)
    B, H, G, cap, n = 3, 2, 2, 256, 9
    rope = tq.Rope(d, cap)
    cache = tq.Cache(cb, B, H, cap)
    g = torch.Generator().manual_seed(1)

    def qkv(tokens):
        x = torch.randn(B, tokens, H * G + 2 * H, d, generator=g).bfloat16().cuda().transpose(1, 2)
        return x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]

    # the prompt, a chunk of which every token attends what is before it
    q, k, v = qkv(50)
    qr, _ = tq.tq_rope_append(cb, cache, rope, k, v, q=q)
    lens = [50] * B
    chain = torch.ones(50, 50, dtype=torch.bool).tril()
    assert_tree_close(tq.tq_tree_attention(cb, cache, qr), *tree_reference(cb, cache, qr, chain, lens))
    # the first sample's prompt is every sample's
    tq.tq_cache_copy(cb, cache, cache, torch.tensor([1, 2], dtype=torch.int32).cuda(),
                     torch.zeros(2, dtype=torch.int32).cuda())
    kept = [arrays(cache)] * B
    for step in range(3):
        sees = random_tree(n, step)
        depth = (sees.sum(-1) - 1).to(torch.int32).expand(B, n).contiguous().cuda()
        q, k, v = qkv(n)
        start = cache.seq_lens.clone()
        qr, _ = tq.tq_rope_append(cb, cache, rope, k, v, q=q, positions=depth, relative=True)
        lens = [x + n for x in lens]
        out = tq.tq_tree_attention(cb, cache, qr, mask=tq.pack_tree_mask(sees).cuda())
        assert_tree_close(out, *tree_reference(cb, cache, qr, sees, lens))
        # accept the path to one leaf in each row
        before = arrays(cache)
        paths = [sees[(4 + 2 * b + step) % n].nonzero().flatten().tolist() for b in range(B)]
        index = torch.zeros(B, n, dtype=torch.int32)
        for b, p in enumerate(paths):
            index[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        tq.tq_cache_compact(cb, cache, index.cuda(), torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda(),
                            start=start)
        lens = [x - n + len(p) for x, p in zip(lens, paths)]
        assert cache.seq_lens.tolist() == lens
        after = arrays(cache)
        for b, p in enumerate(paths):
            s = lens[b] - len(p)
            for name in after:
                assert torch.equal(after[name][b, :, :s], before[name][b, :, :s])
                assert torch.equal(after[name][b, :, s:lens[b]], before[name][b, :, [s + i for i in p]])
    # and a plain decode step reads the same cache
    q, k, v = qkv(1)
    qr, _ = tq.tq_rope_append(cb, cache, rope, k, v, q=q)
    lens = [x + 1 for x in lens]
    ref, tol = tree_reference(cb, cache, qr, torch.ones(1, 1, dtype=torch.bool), lens)
    assert_tree_close(tq.tq_tree_attention(cb, cache, qr), ref, tol)
    dec = tq.tq_decode_attention(cb, cache, qr[:, 0].contiguous()).cpu().double()
    assert ((dec - ref[:, 0]).abs().amax(-1) <= 2e-3 * ref[:, 0].abs().amax(-1) + tol[:, 0].amax(-1)).all()
    assert int(cache.status.item()) == 0
