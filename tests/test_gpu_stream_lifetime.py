"""Tensors of one stream used by a call on another (GPU): the caller may drop them as
soon as the call returns, though the other stream has not reached it yet."""
import pytest
import torch

from tests.spec_helpers import arrays, fill_cache, random_tree

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")


class Busy:
    """A stream that is occupied for a while, behind everything of the default one."""

    def __enter__(self):
        self.s = torch.cuda.Stream()
        self.s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.s):
            torch.cuda._sleep(100_000_000)
        return self.s

    def __exit__(self, *exc):
        torch.cuda.synchronize()


def _overwrite(shape, dtype, n=8):
    """Takes what the allocator has to give of this size, and fills it."""
    return [torch.empty(shape, dtype=dtype, device="cuda").fill_(3) for _ in range(n)]


@pytest.mark.parametrize("as_address", [False, True])
def test_tree_attention(as_address):
    cb = tq.Codebook(128, 3, 4)
    n = 9
    cache = fill_cache(tq, cb, 2, 2, 512, [500, 77], seed=6)
    src = torch.randn(2, n, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    bits = tq.pack_tree_mask(random_tree(n, 2)).cuda()
    want = tq.tq_tree_attention(cb, cache, src, mask=bits)
    torch.cuda.synchronize()
    q, mask = src.clone(), bits.clone()
    with Busy() as s:
        got = tq.tq_tree_attention(cb, cache, q, mask=mask, stream=s.cuda_stream if as_address else s)
        del q, mask
        other = _overwrite(src.shape, src.dtype) + _overwrite(bits.shape, bits.dtype)
    assert torch.equal(got, want) and len(other) == 16


def test_rope_append_compact_and_copy():
    cb = tq.Codebook(128, 3, 4, qjl=True)
    B, H, n = 2, 2, 5
    rope = tq.Rope(128, 256)
    x = torch.randn(B, 4 + 2 * H, n, 128, generator=torch.Generator().manual_seed(3)).half().cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    depth, start = i32(*([[0, 1, 1, 2, 3]] * B)), i32(40, 0)
    index, counts, to, frm = i32(*([[0, 2, 4]] * B)), i32(3, 2), i32(1), i32(0)

    def calls(cache, q, k, v, depth, start, index, counts, to, frm, length, stream=None):
        out, _ = tq.tq_rope_append(cb, cache, rope, k, v, q=q, positions=depth, relative=True, start=start, stream=stream)
        tq.tq_cache_compact(cb, cache, index, counts, start=start, stream=stream)
        tq.tq_cache_copy(cb, cache, cache, to, frm, lengths=length, stream=stream)
        return out

    args = [x[:, :4], x[:, 4:4 + H], x[:, 4 + H:], depth, start, index, counts, to, frm, i32(42)]
    one, two = (fill_cache(tq, cb, B, H, 64, [40, 7], seed=6) for _ in range(2))
    want = calls(one, *args)
    torch.cuda.synchronize()
    copies = [a.clone() for a in args]
    with Busy() as s:
        got = calls(two, *copies, stream=s)
        del copies
        for a in args:
            _overwrite(a.shape, a.dtype)
    assert torch.equal(got, want)
    assert torch.equal(one.seq_lens, two.seq_lens) and int(two.status.item()) == 0
    for b, length in enumerate(one.seq_lens.tolist()):
        for name, t in arrays(one).items():
            assert torch.equal(arrays(two)[name][b, :, :length], t[b, :, :length]), name
