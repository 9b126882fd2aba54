"""A plain float64 form of the speculative-decoding operators, for their tests:
the cache's arrays are unpacked bit by bit and the formulas written out."""
from __future__ import annotations

import math

import torch


def hadamard(d):
    i = torch.arange(d)
    par = torch.zeros(d, d, dtype=torch.int64)
    for b in range(9):
        par ^= ((i[:, None] & i[None, :]) >> b) & 1
    return 1.0 - 2.0 * par.double()


def rotation(cb, second=False):
    """R (rows of the orthonormal rotation), float64 [d, d]."""
    s = cb.tables()["signs2" if second else "signs1"].double()
    return hadamard(cb.head_dim) * s / math.sqrt(cb.head_dim)


def unpack(packed, bits):
    """uint8 [..., n] -> codes [..., 8 n / bits], a little-endian bit stream."""
    b = ((packed[..., None].to(torch.int64) >> torch.arange(8)) & 1).flatten(-2)
    return (b.unflatten(-1, (-1, bits)) << torch.arange(bits)).sum(-1)


def decoded(cb, cache, which, b, h, n):
    """float64 [n, d]: keys or values of a row in their stored frame (rotated, but
    for the affine codec's values)."""
    bits = cb.k_bits if which == "k" else cb.v_bits
    code = unpack(getattr(cache, which + "_codes")[b, h, :n].cpu(), bits)
    norm = getattr(cache, which + "_norm")[b, h, :n].cpu().double()
    if cb.affine:
        m = norm.unflatten(-1, (-1, 2))
        return (m[..., :1] * code.double().unflatten(-1, (-1, 64)) + m[..., 1:]).flatten(-2)
    cent = cb.tables()["k_centroids" if which == "k" else "v_centroids"].double()
    return cent[code] * (norm / math.sqrt(cb.head_dim))[:, None]


def chain(n):
    return torch.ones(n, n, dtype=torch.bool).tril()


def random_tree(n, seed):
    """bool [n, n]: draft i attends its ancestors and itself."""
    g = torch.Generator().manual_seed(seed)
    sees = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        if p >= 0:
            sees[i] = sees[p]
        sees[i, i] = True
    return sees


def tree_reference(cb, cache, q, sees, lens, scale=None, max_ctx=None):
    """(out, tol) float64 [B, n, Hq, d].  `tol` bounds the kernel's error from its
    documented roundings; u is half a step of fp16, 2^-11:
      the weights p are rounded to fp16 (u each; the running maximum is taken with
        the value's magnitude, so they stay in fp16's normal range or are below
        2^-22 of the largest: 2^-22 more), values of the affine codec too (u),
        centroids times a fitted factor (below u);
      the rotated query is rounded to fp16 (u of each channel; a bf16 call's only,
        an fp16 call's is held in two parts, 2^-22), keys like values: a score is
        off by at most 2 u sum_c |q_c k_c| scale, its weight by that relatively and
        the softmax by twice that.  The same for the sketch, whose factor is
        rounded too.
    Weighted, |o - o'| <= eta sum_t p_t |v_t| in the values' frame, and the rotation
    back keeps the 2-norm.  Half a step of the output type is added by the caller."""
    B, n, Hq, d = q.shape
    H = cache.kv_heads
    G = Hq // H
    u = 2.0 ** -11
    R1, R2 = rotation(cb), rotation(cb, True) if cb.qjl else None
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(B, n, Hq, d, dtype=torch.float64)
    tol = torch.zeros(B, n, Hq, d, dtype=torch.float64)
    for b in range(B):
        L = lens[b]
        if L < n:
            continue
        ctx, end = L - n, min(L, cache.capacity if max_ctx is None else max_ctx)
        s = sees[b] if sees.dim() == 3 else sees
        vis = torch.ones(n, L, dtype=torch.bool)
        vis[:, ctx:] = s
        vis = vis[:, :end]
        for h in range(H):
            k, v = (decoded(cb, cache, w, b, h, end) for w in "kv")
            for gh in range(G):
                x = q[b, :, h * G + gh].cpu().double() @ R1.T                 # [n, d]
                score = x @ k.T * scale
                size = x.abs() @ k.nan_to_num().abs().T * scale
                if cb.qjl:
                    sign = 2.0 * unpack(cache.k_signs[b, h, :end].cpu(), 1).double() - 1.0
                    c = math.sqrt(math.pi / (2 * d)) * scale
                    rn = cache.k_rnorm[b, h, :end].cpu().double()
                    w = x @ R2.T
                    score = score + c * rn * (w @ sign.T)
                    size = size + c * rn.nan_to_num() * w.abs().sum(-1, keepdim=True)
                score = score.masked_fill(~vis, -math.inf)
                top = score.amax(-1, keepdim=True) if end > 0 else torch.zeros(n, 1).double()
                p = (score - torch.where(top.isinf(), torch.zeros_like(top), top)).exp()
                p = torch.where(vis, p, torch.zeros_like(p))
                l = p.sum(-1, keepdim=True)
                p = torch.where(l > 0, p / l, torch.zeros_like(p))
                used = vis.any(0)   # what no draft attends may hold anything
                vv = torch.where(used[:, None], v, torch.zeros_like(v))
                o = p @ vv
                delta = torch.where(vis, size, torch.zeros_like(size)).amax(-1, keepdim=True) if end else 0
                eta = 3 * u + 2 * 2 * u * delta
                t = (p @ vv.abs() * eta).norm(dim=-1, keepdim=True)
                out[b, :, h * G + gh] = o if cb.affine else o @ R1
                tol[b, :, h * G + gh] = t + 1e-30
    return out, tol


def assert_tree_close(got, out, tol):
    """Every element within half a step of its type and `tol`."""
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * half
    err = (got.cpu().double() - out).abs()
    lim = half * out.abs() * 1.0001 + tol * (1 + half) + tiny
    worst = (err / lim).max()
    assert bool((err <= lim).all()), f"worst error is {float(worst):.3g} of its bound"


def fill_cache(tq, cb, batch, kv_heads, capacity, lens, seed):
    """A cache filled through the append, with a few outlier channels."""
    g = torch.Generator().manual_seed(seed)
    n = max(max(lens), 1)
    k = torch.randn(batch, kv_heads, n, cb.head_dim, generator=g)
    v = torch.randn(batch, kv_heads, n, cb.head_dim, generator=g)
    k[..., 3] *= 6.0
    v[..., 9] *= 6.0
    cache = tq.Cache(cb, batch, kv_heads, capacity)
    tq.tq_quantize_append(cb, cache, k.cuda(), v.cuda())
    cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    return cache


ARRAYS = ("k_codes", "v_codes", "k_signs", "k_norm", "v_norm", "k_rnorm")


def arrays(cache):
    """The cache's arrays as raw bytes on the host, [B, H, capacity, bytes]."""
    out = {}
    for name in ARRAYS:
        t = getattr(cache, name)
        if t is not None:
            t = t.cpu()
            out[name] = (t if t.dtype == torch.uint8 else t.view(torch.int16)).reshape(*t.shape[:3], -1).clone()
    return out
