"""Rotary positions fused with the append (GPU): the table against float64, the
rotated queries and keys against the formula, the stored bytes against the
append of the same rotated fp32 keys (which the codec tests pin to the oracle)."""
import math

import numpy as np
import pytest
import torch

from tests.spec_helpers import arrays

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("turboquant_kv_cache_rht_b200.tq")


def frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=0, beta=(32.0, 1.0), bands=(1.0, 4.0)):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        pair = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(beta[0])), 0), min(math.ceil(pair(beta[1])), rot - 1)
        r = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / factor * r + f * (1 - r), (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)
    if scaling == "bands":
        turns = original * f / (2 * math.pi)
        s = np.clip((turns - bands[0]) / (bands[1] - bands[0]), 0, 1)
        return (1 - s) * f / factor + s * f, 1.0
    return f, 1.0


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=4.0, original_max=4096),
            dict(scaling="bands", factor=8.0, original_max=8192)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot", [2, 6, 64, 128, 256])
def test_table(kw, rot):
    rope = tq.Rope(rot, 40000, **kw)
    f, m = frequencies(rot, scaling=kw.get("scaling"), factor=kw.get("factor", 1.0), original=kw.get("original_max", 0))
    pos = np.array([0, 1, 2, 77, 4095, 16384, 39999], np.float64)
    a = pos[:, None] * f[None]
    want = np.stack([np.cos(a) * m, np.sin(a) * m], -1)
    got = rope.table[torch.tensor(pos.astype(np.int64)).cuda()].cpu().numpy().astype(np.float64)
    # fp32 half a step, and the frequency's own rounding over 40000 positions in float64
    assert np.abs(got - want).max() <= 2.0 ** -24 * abs(m) * 1.01 + 40000 * 2.0 ** -50


def rotated(x, rope, pos):
    """fp32, every product and sum rounded by itself: x [B, h, n, d], pos [B, n]."""
    rot = rope.rot_dim
    t = rope.table[pos.long()][:, None]                      # [B, 1, n, rot / 2, 2]
    c, s = t[..., 0], t[..., 1]
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if rope.interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * c - b * s, b * c + a * s
    y = torch.stack((ra, rb), -1).flatten(-2) if rope.interleaved else torch.cat((ra, rb), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _inputs(B, Hq, H, n, d, dtype, seed, layout):
    x = torch.randn((B, n, Hq + 2 * H, d), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    x = x.transpose(1, 2)
    if layout == "heads":
        x = x.contiguous()
    return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]


CASES = [  # d, kb, vb, qjl, codebook, rot, interleaved, dtype, B, Hq, H, n, layout
    (128, 3, 4, False, "gaussian", 128, False, torch.bfloat16, 3, 8, 2, 1, "fused"),
    (128, 3, 4, True, "sphere", 128, True, torch.float16, 2, 4, 4, 7, "heads"),
    (128, 4, 4, True, "affine", 64, False, torch.float32, 1, 2, 1, 33, "fused"),
    (64, 2, 3, False, "gaussian", 64, False, torch.float32, 2, 3, 1, 5, "fused"),
    (64, 3, 4, True, "gaussian", 26, True, torch.bfloat16, 1, 4, 2, 300, "heads"),
    (256, 2, 2, True, "gaussian", 100, False, torch.bfloat16, 2, 2, 2, 9, "fused"),
    (256, 3, 3, False, "affine", 256, True, torch.float16, 1, 4, 1, 129, "fused"),
    (128, 3, 4, False, "gaussian", 128, False, torch.bfloat16, 1, 8, 2, 2000, "fused"),     # bulk form
    (64, 4, 4, True, "gaussian", 22, False, torch.float16, 3, 4, 4, 1500, "heads"),
    (256, 2, 3, True, "affine", 10, True, torch.float32, 1, 2, 2, 1700, "fused"),
    (128, 2, 2, False, "gaussian", 2, False, torch.bfloat16, 2, 16, 8, 400, "heads"),
    (128, 3, 3, True, "gaussian", 8, True, torch.float32, 5, 1, 1, 1100, "fused"),
    # bulk queries whose rotated channels are whole blocks of 16
    (128, 3, 4, False, "gaussian", 64, True, torch.bfloat16, 2, 12, 2, 517, "fused"),
    (128, 3, 4, False, "gaussian", 16, False, torch.float16, 1, 3, 1, 1501, "heads"),
    (64, 2, 3, False, "gaussian", 64, True, torch.float32, 3, 5, 1, 701, "fused"),
    (64, 2, 2, True, "affine", 48, False, torch.bfloat16, 1, 1, 1, 2049, "heads"),
    (256, 4, 4, False, "gaussian", 256, False, torch.float16, 1, 8, 1, 600, "fused"),
    (256, 2, 2, True, "gaussian", 160, True, torch.float32, 2, 2, 2, 900, "heads"),
]


@pytest.mark.parametrize("case", CASES)
def test_matches_rotation_then_append(case):
    d, kb, vb, qjl, codebook, rot, inter, dtype, B, Hq, H, n, layout = case
    cb = tq.Codebook(d, kb, vb, qjl=qjl, seed=3, codebook=codebook)
    cap = (n + 60 + 15) // 16 * 16
    rope = tq.Rope(rot, cap, interleaved=inter, scaling="linear", factor=2.0)
    q, k, v = _inputs(B, Hq, H, n, d, dtype, n, layout)
    start = torch.tensor([(13 * b) % 41 for b in range(B)], dtype=torch.int32).cuda()
    one, two = (tq.Cache(cb, B, H, cap) for _ in range(2))
    one.seq_lens.copy_(start), two.seq_lens.copy_(start)
    pos = start[:, None] + torch.arange(n, device="cuda")
    qr, kr = tq.tq_rope_append(cb, one, rope, k, v, q=q, keys_out=True)
    keys = rotated(k, rope, pos)
    tq.tq_quantize_append(cb, two, keys.contiguous(), v.float().contiguous())
    torch.cuda.synchronize()
    assert torch.equal(one.seq_lens, start + n) and int(one.status.item()) == 0
    assert torch.equal(one.append_sync, torch.zeros_like(one.append_sync))
    for name, t in arrays(two).items():
        assert torch.equal(arrays(one)[name], t), name
    assert torch.equal(qr, rotated(q, rope, pos).to(dtype).transpose(1, 2))
    assert torch.equal(kr, keys.to(dtype).transpose(1, 2))


def test_queries_against_float64():
    rope = tq.Rope(128, 32768)
    cb = tq.Codebook(128, 3, 4)
    cache = tq.Cache(cb, 1, 1, 32768)
    cache.seq_lens.fill_(32000)
    q, k, v = _inputs(1, 2, 1, 700, 128, torch.float32, 1, "fused")
    qr, _ = tq.tq_rope_append(cb, cache, rope, k, v, q=q)
    f, _ = frequencies(128)
    a = torch.tensor((32000 + np.arange(700))[:, None] * f[None])
    x = q.cpu().double()
    z = torch.complex(x[..., :64], x[..., 64:]) * torch.polar(torch.ones_like(a), a)
    want = torch.cat((z.real, z.imag), -1).transpose(1, 2)
    # three roundings of fp32: the table entry, the product, the sum
    size = (z.abs() * math.sqrt(2)).repeat(1, 1, 1, 2).transpose(1, 2)
    assert ((qr.cpu().double() - want).abs() <= 3 * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("n", [3, 1300])
def test_positions_and_start(n):
    """Tree positions (relative and absolute); a start below the length discards drafts."""
    cb = tq.Codebook(128, 3, 4, qjl=True)
    B, H, Hq = 3, 2, 4
    rope = tq.Rope(128, 4096)
    q, k, v = _inputs(B, Hq, H, n, 128, torch.bfloat16, 5, "fused")
    start = torch.tensor([0, 17, 30], dtype=torch.int32).cuda()
    off = torch.randint(0, 50, (B, n), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    got = []
    for rel in (True, False):
        c = tq.Cache(cb, B, H, 1344)
        c.seq_lens.fill_(30)
        p = off if rel else off + start[:, None]
        qr, _ = tq.tq_rope_append(cb, c, rope, k, v, q=q, positions=p, relative=rel, start=start)
        assert torch.equal(c.seq_lens, start + n) and int(c.status.item()) == 0
        assert torch.equal(qr, rotated(q, rope, start[:, None] + off).to(q.dtype).transpose(1, 2))
        got.append(arrays(c))
    for name in got[0]:
        assert torch.equal(got[0][name], got[1][name]), name


@pytest.mark.parametrize("n", [2, 1000])
def test_rows_that_do_not_fit(n):
    cb = tq.Codebook(128, 3, 4)
    B, H = 4, 1
    cap = (n + 15) // 16 * 16 + 16
    rope = tq.Rope(128, 8)                       # positions past the table are clamped
    q, k, v = _inputs(B, 2, H, n, 128, torch.float16, 5, "fused")
    c = tq.Cache(cb, B, H, cap)
    before = arrays(c)
    lens = torch.tensor([cap - n, cap - n + 1, 4, 4], dtype=torch.int32).cuda()
    c.seq_lens.copy_(lens)
    start = torch.tensor([cap - n, cap - n + 1, 5, -1], dtype=torch.int32).cuda()
    qr, _ = tq.tq_rope_append(cb, c, rope, k, v, q=q, start=start)
    assert c.seq_lens.tolist() == [cap, cap - n + 1, 4, 4]
    assert int(c.status.item()) == tq.TQ_FLAG_CAPACITY | tq.TQ_FLAG_INDEX
    after = arrays(c)
    for name in before:
        assert torch.equal(after[name][1:], before[name][1:]), name
    pos = (start[:, None] + torch.arange(n, device="cuda")).clamp(0, 7)
    assert torch.equal(qr, rotated(q, rope, pos).to(q.dtype).transpose(1, 2))
    assert torch.all(c.append_sync == 0)


def test_without_queries_empty_and_outputs_given():
    cb = tq.Codebook(128, 3, 4)
    rope = tq.Rope(128, 64)
    q, k, v = _inputs(1, 2, 1, 4, 128, torch.bfloat16, 5, "fused")
    c = tq.Cache(cb, 1, 1, 32)
    assert tq.tq_rope_append(cb, c, rope, k, v) == (None, None)
    tq.tq_rope_append(cb, c, rope, k[:, :, :0], v[:, :, :0])
    assert c.seq_lens.tolist() == [4]
    qo, ko = torch.empty(1, 4, 2, 128, dtype=q.dtype, device="cuda"), torch.empty(1, 4, 1, 128, dtype=q.dtype, device="cuda")
    a, b = tq.tq_rope_append(cb, c, rope, k, v, q=q, q_out=qo, keys_out=ko, start=torch.zeros(1, dtype=torch.int32).cuda())
    assert a is qo and b is ko and c.seq_lens.tolist() == [4]


def test_captured_and_on_another_stream():
    cb = tq.Codebook(128, 3, 4)
    rope = tq.Rope(128, 512)
    q, k, v = _inputs(2, 8, 2, 3, 128, torch.bfloat16, 5, "fused")
    c, ref = tq.Cache(cb, 2, 2, 64), tq.Cache(cb, 2, 2, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qr, _ = tq.tq_rope_append(cb, ref, rope, k, v, q=q, stream=s)
    torch.cuda.synchronize()
    out = torch.empty_like(qr)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_rope_append(cb, c, rope, k, v, q=q, q_out=out)
    assert c.seq_lens.tolist() == [0, 0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, qr) and c.seq_lens.tolist() == [3, 3]
    for name, t in arrays(ref).items():
        assert torch.equal(arrays(c)[name], t)
    g.replay()
    assert c.seq_lens.tolist() == [6, 6]
