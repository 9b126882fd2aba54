"""Tree attention of drafted tokens (GPU) against its formula in float64 on the
same packed bytes, at every head_dim, code width, codec, group size and row
count class, with masks that leave rows empty, ragged and too short rows, and
the calls that the header allows: captured, on another stream, twice at once."""
import math

import pytest
import torch

from tests.spec_helpers import (assert_tree_close, chain, fill_cache, random_tree, tree_reference)

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")


def _q(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _check(cb, cache, q, sees, lens, mask, **kw):
    got = tq.tq_tree_attention(cb, cache, q.cuda(), mask=mask, **{k: v for k, v in kw.items() if k != "scale"},
                               softmax_scale=kw.get("scale") or 0.0)
    torch.cuda.synchronize()
    out, tol = tree_reference(cb, cache, q, sees, lens, kw.get("scale"), kw.get("max_ctx"))
    assert_tree_close(got, out, tol)
    return got


# every width and codec of every head_dim, few and many rows
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kb,vb,qjl,codebook", [
    (3, 4, False, "gaussian"), (3, 4, True, "sphere"), (2, 2, True, "gaussian"), (2, 2, False, "gaussian"),
    (2, 3, False, "gaussian"), (3, 3, True, "gaussian"), (4, 4, False, "gaussian"),
    (4, 4, True, "affine"), (2, 3, False, "affine"), (3, 4, False, "affine"), (2, 2, True, "affine")])
def test_codecs(d, kb, vb, qjl, codebook):
    cb = tq.Codebook(d, kb, vb, qjl=qjl, seed=kb * 8 + vb, codebook=codebook)
    lens, H = [301, 133], 2
    cache = fill_cache(tq, cb, 2, H, 320, lens, seed=d + kb)
    for n, G, dtype in ((5, 2, torch.bfloat16), (13, 4, torch.float16)):
        sees = random_tree(n, seed=n)
        _check(cb, cache, _q((2, n, H * G, d), dtype, 7), sees, lens, tq.pack_tree_mask(sees).cuda())


# row counts around the column counts that the kernel works with
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 256])
def test_row_counts(G, n):
    cb = tq.Codebook(128, 3, 4, seed=n)
    lens = [n + 140]
    cache = fill_cache(tq, cb, 1, 1, 400, lens, seed=G)
    sees = random_tree(n, seed=n + G)
    _check(cb, cache, _q((1, n, G, 128), torch.bfloat16, n), sees, lens, tq.pack_tree_mask(sees).cuda())


@pytest.mark.parametrize("d,qjl", [(64, False), (256, False), (256, True), (128, True), (64, True)])
@pytest.mark.parametrize("rows", [(40, 8), (9, 8), (33, 2), (100, 2)])
def test_row_counts_of_other_shapes(d, qjl, rows):
    n, G = rows
    cb = tq.Codebook(d, 3, 4, qjl=qjl, seed=n)
    lens = [n + 150]
    cache = fill_cache(tq, cb, 1, 2, 272, lens, seed=G)
    for dtype in (torch.bfloat16, torch.float16):
        _check(cb, cache, _q((1, n, 2 * G, d), dtype, n), chain(n), lens, None)


# contexts around the tile and split borders; ragged, empty and too short rows
@pytest.mark.parametrize("qjl", [False, True])
def test_lengths(qjl):
    n, H, G, d = 6, 2, 4, 128
    lens = [0, 5, 6, 7, 127, 128, 129, 134, 255, 256, 257, 640, 1000, 1024, 3, 12]
    cb = tq.Codebook(d, 3, 4, qjl=qjl)
    cache = fill_cache(tq, cb, len(lens), H, 1024, lens, seed=1)
    q = _q((len(lens), n, H * G, d), torch.float16, 2)
    got = _check(cb, cache, q, chain(n), lens, None)
    for b, L in enumerate(lens):
        if L < n:
            assert torch.all(got[b] == 0)
    assert int(cache.status.item()) == 0


@pytest.mark.parametrize("rows", [(3, 4), (40, 4)])
def test_long_context_over_many_splits(rows):
    n, G = rows
    d, L = 128, 40005
    cb = tq.Codebook(d, 3, 4)
    cache = fill_cache(tq, cb, 1, 1, 40016, [L], seed=5)
    q = _q((1, n, G, d), torch.float16, 3)
    q[0, 0, 0] = fill_key(cb, 9) * 1.2          # one peaked row
    sees = random_tree(n, 4)
    _check(cb, cache, q, sees, [L], tq.pack_tree_mask(sees).cuda())


def fill_key(cb, seed):
    return torch.randn(cb.head_dim, generator=torch.Generator().manual_seed(seed)).half()


def test_rising_scores_move_the_running_maximum():
    """Keys that grow along the row: every tile raises the maximum."""
    cb = tq.Codebook(128, 4, 4)
    L, n = 1500, 4
    g = torch.Generator().manual_seed(3)
    base = torch.randn(128, generator=g)
    grow = torch.linspace(0.1, 6.0, L)[:, None]
    k = (base[None] * grow + 0.1 * torch.randn(L, 128, generator=g))[None, None]
    v = torch.randn(1, 1, L, 128, generator=g)
    cache = tq.Cache(cb, 1, 1, 1504)
    tq.tq_quantize_append(cb, cache, k.cuda(), v.cuda())
    q = (base[None, None, None] * torch.tensor([1.0, -1.0, 0.3, 2.0])[None, :, None, None]).to(torch.float16)
    _check(cb, cache, q.contiguous(), chain(n), [L], None)


# masks: empty rows, a mask per batch row, bits past n_q are not read
def test_masks():
    cb = tq.Codebook(128, 3, 4)
    B, n, H, G, d = 3, 37, 1, 2, 128
    lens = [n, n + 3, 300]          # the first row has no context: an empty mask row attends nothing
    cache = fill_cache(tq, cb, B, H, 304, lens, seed=8)
    sees = torch.stack([random_tree(n, s) for s in range(B)])
    sees[:, 5] = False
    sees[:, 20] = True              # a draft may attend any other, later ones too
    mask = tq.pack_tree_mask(sees)
    mask[..., 1] |= -32             # bits 5.. of the second word: drafts 37 and past
    q = _q((B, n, G, d), torch.float16, 9)
    got = _check(cb, cache, q, sees, lens, mask.cuda())
    assert torch.all(got[0, 5] == 0)
    none = torch.zeros(n, 2, dtype=torch.int32).cuda()
    out = tq.tq_tree_attention(cb, cache, q.cuda(), mask=none)
    assert torch.all(out[0] == 0)
    ref, tol = tree_reference(cb, cache, q, torch.zeros(n, n, dtype=torch.bool), lens)
    assert_tree_close(out, ref, tol)


def test_what_a_draft_does_not_attend_cannot_reach_it():
    """Norms of infinity and NaN at drafts that the mask hides, and past the row's end."""
    for codebook in ("gaussian", "affine"):
        cb = tq.Codebook(128, 3, 4, codebook=codebook, qjl=True)
        n, L = 6, 150
        cache = fill_cache(tq, cb, 1, 1, 176, [L], seed=2)
        for name, val in (("k_norm", math.nan), ("v_norm", math.inf), ("v_norm", math.nan)):
            getattr(cache, name)[0, 0, L - n + 2] = val
            getattr(cache, name)[0, 0, L:] = val
        cache.k_rnorm[0, 0, L:] = math.inf
        sees = chain(n)
        sees[:, 2] = False
        q = _q((1, n, 4, 128), torch.bfloat16, 1)
        got = _check(cb, cache, q, sees, [L], tq.pack_tree_mask(sees).cuda())
        assert torch.isfinite(got).all()
        sees[4, 2] = True           # and who attends it gets what it holds
        got = tq.tq_tree_attention(cb, cache, q.cuda(), mask=tq.pack_tree_mask(sees).cuda())
        assert not torch.isfinite(got[0, 4]).any() and torch.isfinite(got[0, [0, 1, 2, 3, 5]]).all()


@pytest.mark.parametrize("qs,vs", [(1e4, 1e-4), (1e-5, 3e2), (300.0, 1.0)])
def test_magnitudes(qs, vs):
    # the largest norm, 300 * 10 * sqrt(128) = 34e3 and a few percent, is an fp16 number (65504)
    cb = tq.Codebook(128, 3, 4)
    g = torch.Generator().manual_seed(4)
    k = torch.randn(1, 1, 200, 128, generator=g) * (0.01 if qs > 1 else 50)
    v = torch.randn(1, 1, 200, 128, generator=g) * vs * torch.logspace(-2, 1, 200)[:, None]
    cache = tq.Cache(cb, 1, 1, 208)
    tq.tq_quantize_append(cb, cache, k.cuda(), v.cuda())
    q = _q((1, 3, 2, 128), torch.bfloat16, 5, qs)
    q[0, 1] *= 1e-3                 # rows of one call differ in size
    _check(cb, cache, q, chain(3), [200], None, scale=0.02)


def test_softmax_scale_and_max_ctx():
    cb = tq.Codebook(128, 3, 4)
    lens = [310, 64]
    cache = fill_cache(tq, cb, 2, 2, 320, lens, seed=6)
    q = _q((2, 8, 4, 128), torch.float16, 3)
    _check(cb, cache, q, chain(8), lens, None, scale=0.31)
    assert int(cache.status.item()) == 0
    _check(cb, cache, q, chain(8), lens, None, max_ctx=305)     # cuts into the first row's drafts
    assert int(cache.status.item()) == tq.TQ_FLAG_MAXCTX
    out = tq.tq_tree_attention(cb, cache, q.cuda(), max_ctx=0)
    assert torch.all(out == 0)


def test_one_draft_is_the_decode():
    """n_q = 1 answers what the single-token decode answers, within both bounds."""
    cb = tq.Codebook(128, 3, 4)
    cache = fill_cache(tq, cb, 2, 2, 512, [500, 77], seed=6)
    q = _q((2, 1, 8, 128), torch.float16, 3)
    tree = tq.tq_tree_attention(cb, cache, q.cuda()).float()[:, 0]
    dec = tq.tq_decode_attention(cb, cache, q.cuda()[:, 0].contiguous())
    assert (tree - dec).abs().max() <= 4e-3 * dec.abs().max()


def test_repeats_captures_streams_and_two_calls_at_once():
    cb = tq.Codebook(128, 3, 4)
    n, lens = 17, [900, 333]
    cache = fill_cache(tq, cb, 2, 2, 912, lens, seed=1)
    q = _q((2, n, 8, 128), torch.bfloat16, 2).cuda()
    mask = tq.pack_tree_mask(random_tree(n, 3)).cuda()
    ref = tq.tq_tree_attention(cb, cache, q, mask=mask)
    for _ in range(5):
        assert torch.equal(tq.tq_tree_attention(cb, cache, q, mask=mask), ref)
    torch.cuda.synchronize()
    # two streams at once, each with its own workspace
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [tq.tq_tree_attention(cb, cache, q, mask=mask, stream=s) for _ in range(8) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    # two graphs that share a workspace, replayed one after the other on changed inputs
    need = tq.tq_tree_workspace_bytes(cb, 2, 8, 2, n, cache.capacity)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    o1, o2 = torch.empty_like(q), torch.empty_like(q)
    graphs = []
    for o in (o1, o2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.tq_tree_attention(cb, cache, q, mask=mask, out=o, workspace=ws)
        graphs.append(g)
    ws.fill_(255)                     # the workspace needs no clearing
    for L in ([900, 333], [20, 0], [700, 912]):
        cache.seq_lens.copy_(torch.tensor(L, dtype=torch.int32))
        o1.fill_(7.0), o2.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = tq.tq_tree_attention(cb, cache, q, mask=mask)
        assert torch.equal(o1, want) and torch.equal(o2, want)


def test_nothing_is_written_past_the_buffers():
    cb = tq.Codebook(128, 3, 4, qjl=True)
    n = 9
    cache = fill_cache(tq, cb, 1, 2, 160, [150], seed=1)
    before = {k: getattr(cache, k).clone() for k in ("k_codes", "v_codes", "k_norm", "v_norm", "k_signs", "seq_lens")}
    need = tq.tq_tree_workspace_bytes(cb, 1, 8, 2, n, 160)
    buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    q = _q((1, n, 8, 128), torch.bfloat16, 2).cuda()
    obuf = torch.full((q.numel() + 2048,), 3.0, dtype=q.dtype, device="cuda")
    out = obuf[1024:1024 + q.numel()].view(q.shape)
    tq.tq_tree_attention(cb, cache, q, out=out, workspace=buf[4096:4096 + max(need, 16)])
    torch.cuda.synchronize()
    assert torch.all(buf[:4096] == 0xA5) and torch.all(buf[4096 + max(need, 16):] == 0xA5)
    assert torch.all(obuf[:1024] == 3) and torch.all(obuf[1024 + q.numel():] == 3)
    assert all(torch.equal(getattr(cache, k), t) for k, t in before.items())


def test_many_rows():
    """More batch rows than the kernel has threads, most of them empty."""
    cb = tq.Codebook(64, 2, 2)
    B, n = 700, 2
    lens = [(b * 7) % 33 if b % 5 == 0 else 0 for b in range(B)]
    cache = fill_cache(tq, cb, B, 1, 48, lens, seed=1)
    _check(cb, cache, _q((B, n, 2, 64), torch.float16, 2), chain(n), lens, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [(6, 2), (50, 8)])
def test_a_bad_query_stays_in_its_row(dtype, rows):
    """Infinities and NaN in one draft's query; the scale that the rows share is the others'."""
    n, G = rows
    cb = tq.Codebook(128, 3, 4, qjl=True)
    lens = [n + 100]
    cache = fill_cache(tq, cb, 1, 1, 176, lens, seed=2)
    q = _q((1, n, G, 128), dtype, 1)
    q[0, 1, 0, 5], q[0, 2, 1, 9] = math.inf, math.nan
    got = tq.tq_tree_attention(cb, cache, q.cuda())
    ok = torch.ones(n, G, dtype=torch.bool)
    ok[1, 0] = ok[2, 1] = False
    assert not torch.isfinite(got[0].cpu()[~ok]).any()
    clean = q.clone()
    clean[0, 1, 0] = clean[0, 2, 1] = 0
    ref, tol = tree_reference(cb, cache, clean, chain(n), lens)
    got = got.cpu()
    got[0][~ok], ref[0][~ok] = 0, 0
    assert_tree_close(got, ref, tol)
