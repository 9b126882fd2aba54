"""Compaction and copies of cache rows (GPU): bytes against indexing on the host."""
import pytest
import torch

from tests.spec_helpers import ARRAYS, arrays

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")

SHAPES = [(128, 3, 4, False, "gaussian"), (64, 3, 3, True, "gaussian"), (256, 2, 2, True, "sphere"),
          (128, 4, 4, True, "affine"), (64, 2, 3, False, "affine"), (256, 4, 4, True, "affine")]


def _cache(shape, B, H, cap, lens, seed):
    d, kb, vb, qjl, codebook = shape
    cb = tq.Codebook(d, kb, vb, qjl=qjl, codebook=codebook)
    c = tq.Cache(cb, B, H, cap)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for name in ARRAYS:
        t = getattr(c, name)
        if t is not None:
            w = t.view(torch.uint8) if t.dtype != torch.uint8 else t
            w.copy_(torch.randint(0, 256, w.shape, generator=g, device="cuda", dtype=torch.uint8))
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    return cb, c


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("per_head", [False, True])
def test_compact(shape, per_head):
    B, H, cap = 4, 3, 3008
    lens, start = [3000, 2049, 70, 0], [10, 0, 65, 0]
    cb, c = _cache(shape, B, H, cap, lens, 1)
    g = torch.Generator().manual_seed(2)
    counts = [2500, 1, 0, 0]
    index = torch.full((B, H, 2990), -7, dtype=torch.int32)
    for b in range(B):
        for h in range(H):
            order = torch.randperm(max(lens[b] - start[b], 1), generator=g)[:counts[b]].sort().values
            index[b, h, :counts[b]] = order.to(torch.int32)
    if not per_head:
        index = index[:, 0].contiguous()
    want = arrays(c)
    for b in range(B):
        for h in range(H):
            src = start[b] + (index[b, h] if per_head else index[b])[:counts[b]].long()
            for t in want.values():
                t[b, h, start[b]:start[b] + counts[b]] = t[b, h, src]
    tq.tq_cache_compact(cb, c, index.cuda(), _i32(counts), start=_i32(start))
    torch.cuda.synchronize()
    got = arrays(c)
    assert c.seq_lens.tolist() == [s + n for s, n in zip(start, counts)]
    assert int(c.status.item()) == 0 and torch.all(c.append_sync == 0)
    for name in want:
        for b in range(B):
            n = start[b] + counts[b]
            assert torch.equal(got[name][b, :, :n], want[name][b, :, :n]), name
            assert torch.equal(got[name][b, :, lens[b]:], want[name][b, :, lens[b]:]), name


@pytest.mark.parametrize("count", [1, 16, 255, 256, 257, 2047, 2048, 2049, 5000])
def test_compact_counts_around_the_chunks(count):
    cb, c = _cache(SHAPES[0], 1, 2, 5008, [5000], 3)
    index = torch.randperm(5000, generator=torch.Generator().manual_seed(count))[:count].sort().values.to(torch.int32)
    want = {k: t[:, :, index.long()] for k, t in arrays(c).items()}
    tq.tq_cache_compact(cb, c, index[None].cuda(), _i32([count]))
    got = arrays(c)
    assert c.seq_lens.tolist() == [count]
    for name in want:
        assert torch.equal(got[name][:, :, :count], want[name]), name


def test_compact_bad_lists():
    """A list that is out of range or does not ascend leaves the length; a bad start
    or count leaves the row."""
    cb, c = _cache(SHAPES[0], 7, 1, 64, [40] * 7, 3)
    before = arrays(c)
    index = _i32([[0, 1, 5], [0, 1, 40], [2, 2, 3], [-1, 0, 1], [0, 1, 2], [0, 1, 2], [5, 4, 6]])
    counts, start = _i32([3, 3, 3, 3, 4, 3, 3]), _i32([0, 0, 0, 0, 0, 41, 30])
    tq.tq_cache_compact(cb, c, index, counts, start=start)
    torch.cuda.synchronize()
    assert int(c.status.item()) == tq.TQ_FLAG_INDEX
    assert c.seq_lens.tolist() == [3, 40, 40, 40, 40, 40, 40] and torch.all(c.append_sync == 0)
    got = arrays(c)
    for name, t in before.items():
        assert torch.equal(got[name][4:6], t[4:6]), name
        assert torch.equal(got[name][6, :, :30], t[6, :, :30]), name
        assert torch.equal(got[name][:, :, 40:], t[:, :, 40:]), name
    c.status.zero_()
    tq.tq_cache_compact(cb, c, _i32([[0]] * 7), _i32([1] * 7))      # and the next call is clean
    assert c.seq_lens.tolist() == [1] * 7 and int(c.status.item()) == 0


def test_compact_nothing_listed():
    cb, c = _cache(SHAPES[0], 2, 1, 32, [20, 30], 3)
    tq.tq_cache_compact(cb, c, torch.zeros(2, 0, dtype=torch.int32).cuda(), _i32([0, 0]), start=_i32([7, 0]))
    assert c.seq_lens.tolist() == [7, 0]


@pytest.mark.parametrize("shape", SHAPES)
def test_copy_between_caches(shape):
    H, lens = 3, [500, 33, 0, 1, 517]
    cb, src = _cache(shape, 5, H, 528, lens, 1)
    _, dst = _cache(shape, 7, H, 800, [9] * 7, 2)
    want, s = arrays(dst), arrays(src)
    pairs = [(0, 4, 999), (6, 0, 499), (1, 1, 33), (2, 2, 5), (3, 0, -3), (5, 3, 1)]
    new = [9] * 7
    for to, frm, n in pairs:
        n = max(0, min(n, lens[frm]))
        new[to] = n
        for name in want:
            want[name][to, :, :n] = s[name][frm, :, :n]
    tq.tq_cache_copy(cb, dst, src, _i32([p[0] for p in pairs]), _i32([p[1] for p in pairs]),
                     lengths=_i32([p[2] for p in pairs]))
    got = arrays(dst)
    assert dst.seq_lens.tolist() == new and int(dst.status.item()) == 0
    for name in want:
        assert torch.equal(got[name], want[name]), name
        assert torch.equal(arrays(src)[name], s[name]), name


@pytest.mark.parametrize("n", [0, 1, 7, 8, 15, 16, 17, 47, 48, 500, 2049])
def test_fork_lengths(n):
    cb, c = _cache(SHAPES[1], 4, 2, 2064, [n, 3, 3, 3], 1)
    want = arrays(c)
    for t in want.values():
        t[1:, :, :n] = t[:1, :, :n]
    tq.tq_cache_copy(cb, c, c, _i32([1, 2, 3]), _i32([0, 0, 0]), max_len=n)
    got = arrays(c)
    assert c.seq_lens.tolist() == [n] * 4 and int(c.status.item()) == 0
    for name in want:
        assert torch.equal(got[name], want[name]), name


def test_copy_refused_pairs():
    """Each bad pair is skipped, sets its flag, and leaves the others."""
    cb, c = _cache(SHAPES[0], 6, 1, 64, [10, 20, 30, 40, 50, 60], 1)
    before = arrays(c)
    # row 1 twice, and read by the second pair; rows out of range; a row to itself (silent)
    dst, src = [1, 0, 6, -1, 2, 1, 5], [3, 1, 2, 2, -1, 4, 5]
    tq.tq_cache_copy(cb, c, c, _i32(dst), _i32(src))
    got = arrays(c)
    # row 1 is a dst and another pair's src, so that pair is skipped; pair (0, 1) reads it unharmed
    assert c.seq_lens.tolist() == [20, 20, 30, 40, 50, 60]
    assert int(c.status.item()) == tq.TQ_FLAG_INDEX
    for name, t in before.items():
        assert torch.equal(got[name][0, :, :20], t[1, :, :20]) and torch.equal(got[name][1:], t[1:]), name
    _, small = _cache(SHAPES[0], 2, 1, 32, [5, 5], 1)
    tq.tq_cache_copy(cb, small, c, _i32([0, 1]), _i32([2, 3]))
    assert small.seq_lens.tolist() == [30, 5] and int(small.status.item()) == tq.TQ_FLAG_CAPACITY
    small.status.zero_()
    tq.tq_cache_copy(cb, small, c, _i32([0, 1]), _i32([2, 3]), max_len=12)
    assert small.seq_lens.tolist() == [12, 12] and int(small.status.item()) == tq.TQ_FLAG_MAXCTX


def test_captured():
    cb, c = _cache(SHAPES[0], 2, 1, 64, [40, 0], 3)
    want = arrays(c)
    idx, cnt = _i32([[0, 3, 4, 9], [0, 0, 0, 0]]), _i32([4, 0])
    to, frm = _i32([1]), _i32([0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_cache_compact(cb, c, idx, cnt)
        tq.tq_cache_copy(cb, c, c, to, frm)
    assert c.seq_lens.tolist() == [40, 0]
    g.replay()
    got = arrays(c)
    assert c.seq_lens.tolist() == [4, 4]
    for name, t in want.items():
        for r in (0, 1):
            assert torch.equal(got[name][r, :, :4], t[0, :, [0, 3, 4, 9]]), name
