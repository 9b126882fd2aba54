"""The speculative-decoding calls together, as a program makes them: a prompt is
appended, forked into samples, drafts are appended and verified against plain
float64 attention, the accepted path is kept, and the next step goes on from it."""
import pytest
import torch

from tests.spec_helpers import arrays, assert_tree_close, decoded, random_tree, rotation, tree_reference

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


def test_offsets_past_32_bits():
    """A row whose codes pass 4 GB: drafts are appended at its end, attended, and
    thinned.  The context's keys and values are zeros, so each of its tokens weighs
    exp(0) and adds nothing."""
    d, ctx, n = 256, 34_000_000, 5
    cb = tq.Codebook(d, 4, 4)
    cache = tq.Cache(cb, 1, 1, ctx + 16)
    assert cache.k_codes.numel() > 1 << 32
    cache.seq_lens.fill_(ctx)
    rope = tq.Rope(d, 64)
    x = torch.randn(1, n, 4, d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda().transpose(1, 2)
    x[:, 2:3] *= 3.0
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous()
    qr, _ = tq.tq_rope_append(cb, cache, rope, x[:, 2:3], x[:, 3:], q=x[:, :2], positions=pos)
    out = tq.tq_tree_attention(cb, cache, qr).cpu().double()
    # the drafts alone, as a row of their own: scores and values of the same bytes
    small = tq.Cache(cb, 1, 1, 16)
    for name in ("k_codes", "v_codes", "k_norm", "v_norm"):
        getattr(small, name)[:, :, :n] = getattr(cache, name)[:, :, ctx:ctx + n]
    small.seq_lens.fill_(n)
    R = rotation(cb)
    k, v = (decoded(cb, small, w, 0, 0, n) for w in "kv")
    for h in range(2):
        s = (qr[0, :, h].cpu().double() @ R.T) @ k.T / d ** 0.5
        w = torch.where(torch.ones(n, n, dtype=torch.bool).tril(), s.exp(), torch.zeros_like(s))
        want = (w @ v) @ R / (ctx + w.sum(-1, keepdim=True))
        # the bound of tree_reference, on the weighted values; and half a bf16 step
        u = 2.0 ** -11
        delta = ((qr[0, :, h].cpu().double() @ R.T).abs() @ k.abs().T / d ** 0.5).amax(-1, keepdim=True)
        tol = ((w @ v.abs()) * (3 * u + 4 * u * delta)).norm(dim=-1, keepdim=True) / ctx
        assert ((out[0, :, h] - want).abs() <= tol + want.abs() * 2.0 ** -8).all()
    kept = {name: getattr(cache, name)[:, :, [ctx, ctx + 3]].clone() for name in ("k_codes", "v_codes", "k_norm", "v_norm")}
    tq.tq_cache_compact(cb, cache, torch.tensor([[0, 3]], dtype=torch.int32).cuda(), torch.tensor([2], dtype=torch.int32).cuda(),
                        start=torch.tensor([ctx], dtype=torch.int32).cuda())
    assert cache.seq_lens.tolist() == [ctx + 2] and int(cache.status.item()) == 0
    for name, t in kept.items():
        assert torch.equal(getattr(cache, name)[:, :, ctx:ctx + 2], t), name
    # and a row copied from past 4 GB of the arrays
    two = tq.Cache(cb, 2, 1, 17_000_016)
    two.k_codes[1, 0, :48] = torch.arange(48, dtype=torch.uint8, device="cuda")[:, None]
    two.seq_lens.copy_(torch.tensor([0, 17_000_001], dtype=torch.int32))
    one = tq.Cache(cb, 1, 1, 17_000_016)
    tq.tq_cache_copy(cb, one, two, torch.tensor([0], dtype=torch.int32).cuda(), torch.tensor([1], dtype=torch.int32).cuda())
    assert one.seq_lens.tolist() == [17_000_001]
    assert torch.equal(one.k_codes[0, 0, :64], two.k_codes[1, 0, :64])


def test_a_stream_of_its_own_and_whole_rows():
    """A call on a stream of its own orders what it allocates there; drafts rejected
    whole (a count of zero) and accepted whole leave a row as it should be."""
    cb = tq.Codebook(64, 2, 2)
    cache = tq.Cache(cb, 2, 1, 64)
    rope = tq.Rope(64, 64)
    x = torch.randn(2, 4, 3, 64, generator=torch.Generator().manual_seed(3)).half().cuda().transpose(1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for step in range(3):
        qr, _ = tq.tq_rope_append(cb, cache, rope, x[:, 1:2], x[:, 2:], q=x[:, :1], stream=s)
        out = tq.tq_tree_attention(cb, cache, qr, stream=s)
        tq.tq_cache_compact(cb, cache, torch.arange(4, dtype=torch.int32).expand(2, 4).contiguous().cuda(),
                            torch.tensor([4, 0], dtype=torch.int32).cuda(),
                            start=torch.tensor([4 * step, 0], dtype=torch.int32).cuda(), stream=s)
    s.synchronize()
    assert cache.seq_lens.tolist() == [12, 0] and int(cache.status.item()) == 0
    assert torch.isfinite(out).all()
