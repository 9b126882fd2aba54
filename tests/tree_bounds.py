"""The tree attention's formula in float64, with a bound of its roundings that a
wrong answer does not pass.

Which operands the kernel rounds is documented; what a rounding is, is not known,
only that it is at most half a step: u = 2^-11 of the value for fp16, and half of
2^-24 below 2^-14.  The roundings of different weights, channels and tokens are taken
as independent and centred, so a sum of a_i times such errors is below
K sqrt(sum a_i^2) u with a probability of 1 - 2 exp(-K^2 / 2) (Hoeffding): 1 - 3e-14
for K = 8.  The first-order effects on output channel e of a row, with its weights p,
values v (in the output's frame), output o, rotated query x and keys k:
  weights        K u |p_t v_te|_t, or u sum_t p_t |v_te| where that is less (few tokens)
  queries        K u_q |x_c J_ce|_c,  J_ce = scale sum_t p_t k_tc (v_te - o_e),
                 u_q = u for bf16, 2^-22 for fp16 (held in two parts)
  sketch         its queries as above with u for either type; its factor, per token:
                 K u |p_t s_t (v_te - o_e)|_t, s_t the sketch's part of the score
  affine codec   values as weights; keys, per token: K u |p_t g_t (v_te - o_e)|_t,
                 g_t = scale |x_c k_tc|_c
  tables         the centroids' own rounding is the same for every token: the
                 formula is evaluated with the rounded tables too, and the difference added
  fp32           the score's sums, the exponential and the sum of weights, counted at
                 their worst; the output's accumulation at its worst too: up to 2^-23
                 of each stored channel for every 16 tokens (a product may truncate),
                 as a 2-norm, which the rotation back keeps
  small weights  a weight below 2^-14 is rounded to a multiple of 2^-24, where the
                 row's largest is at least 2^4: 2^-29 of it per token, at its worst
  beyond         the above is of first order.  Where a score may be off by e > 0.1, a
                 weight is off by a factor of exp(2 e) at most, so the output by (exp(2 e)
                 - 1) sum_t p_t |v_te - o_e|; and it is still a mean of the values of tokens
                 whose scores are within 2 e of the largest (others' weights, e^-28 or less,
                 aside): off by no more than the farthest of these values
Elements are held to the sum of these, rows to their 2-norm, where the accumulation
counts once.
"""
from __future__ import annotations

import math

import torch

from tests.spec_helpers import rotation

K = 8.0
U = 2.0 ** -11


def _codes(packed, bits):
    b = ((packed[..., None].to(torch.int16) >> torch.arange(8, device=packed.device)) & 1).flatten(-2)
    return (b.unflatten(-1, (-1, bits)).long() << torch.arange(bits, device=packed.device)).sum(-1)


def _rounded_table(cent):
    """fp16(lam c) / lam, lam on a grid of [1, 2) with the smallest largest error."""
    pos = cent[cent > 0].float()
    lam = 1 + torch.arange(1 << 16, dtype=torch.float32) / (1 << 16)
    x = lam[:, None] * pos
    err = ((x.half().double() - x.double()).abs() / x.double()).amax(1)
    best = lam[err.argmin()]
    return (cent.float() * best).half().double() / best.double()


def _stored(cb, cache, which, b, h, n):
    """(values, values with the rounded table, the norm or exponent that is factored
    out), float64 [n, d], [n, d], [n], in the stored frame."""
    bits = cb.k_bits if which == "k" else cb.v_bits
    packed = getattr(cache, which + "_codes")[b, h, :n]
    code = _codes(packed, bits)
    norm = getattr(cache, which + "_norm")[b, h, :n].double()
    if cb.affine:
        m = norm.unflatten(-1, (-1, 2))
        x = (m[..., :1] * code.double().unflatten(-1, (-1, 64)) + m[..., 1:]).flatten(-2)
        return x, x, m.abs().amax((-1, -2))
    cent = cb.tables()["k_centroids" if which == "k" else "v_centroids"].double()
    by = (norm / math.sqrt(cb.head_dim))[:, None]
    dev = packed.device
    return cent.to(dev)[code] * by, _rounded_table(cent).to(dev)[code] * by, norm


def visible(sees, n, length, end):
    """bool [n, end]: which of a row's first `end` tokens each draft attends."""
    vis = torch.ones(n, length, dtype=torch.bool)
    vis[:, length - n:] = sees.cpu()
    return vis[:, :end]


BLOCKS = 148  # that the tokens of all units are shared out to


def bounded_reference(cb, cache, q, sees, lens, scale=None, max_ctx=None, drafts=None, share=None):
    """(out, tol, acc) on the cache's device: float64 [B, n, Hq, d] twice, and the
    accumulation's 2-norm [B, n, Hq, 1].  `drafts`: only these, in this order.  `share`:
    the most tokens of a row that one block may take (default: a 148th of all rows', and
    a few tiles)."""
    B, n, Hq, d = q.shape
    H, dev = cache.kv_heads, cache.k_codes.device
    G = Hq // H
    R1 = rotation(cb).to(dev)
    R2 = rotation(cb, True).to(dev) if cb.qjl else None
    scale = 1 / math.sqrt(d) if scale is None else scale
    uq = U if q.dtype == torch.bfloat16 else 2.0 ** -22
    drafts = list(range(n)) if drafts is None else drafts
    if share is None:  # (a unit has at most ceil(rows / 64) blocks of query rows)
        share = sum(lens) * H * -(-n * G // 64) // BLOCKS + 512
    out = torch.zeros(B, len(drafts), Hq, d, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    acc = torch.zeros(B, len(drafts), Hq, 1, dtype=torch.float64, device=dev)
    q = q.to(dev).double()
    for b in range(B):
        L = lens[b]
        end = min(L, cache.capacity if max_ctx is None else max_ctx)
        if L < n or end == 0:
            continue
        vis = visible(sees[b] if sees.dim() == 3 else sees, n, L, end).to(dev)
        used = vis.any(0)[:, None]
        for h in range(H):
            k, kt, _ = _stored(cb, cache, "k", b, h, end)
            v, vt, vn = _stored(cb, cache, "v", b, h, end)
            zero = torch.zeros((), dtype=torch.float64, device=dev)
            k, kt, v, vt = (torch.where(used, t, zero) for t in (k, kt, v, vt))
            vn = torch.where(used[:, 0], vn, zero)
            stored = v
            if not cb.affine:
                v, vt = v @ R1, vt @ R1
            if cb.qjl:
                sign = 2.0 * _codes(cache.k_signs[b, h, :end], 1).double() - 1.0
                rn = torch.where(used[:, 0], cache.k_rnorm[b, h, :end].double(), zero) * math.sqrt(math.pi / (2 * d))
            unit = q[b, :, h * G:(h + 1) * G]
            # below 2^-14 a query's half step is 2^-25, where d max|q| (which bounds sqrt(d) |x|) is
            # brought to 2^13 .. 2^14 (2^9 .. 2^10 with the sketch), that of the unit's largest row
            # or, where rows differ by more than 2^16, of its own: 2^-25 2^-13 sqrt(d) max|q| of x
            tiny = math.sqrt(d) * 2.0 ** (-34 if cb.qjl else -38)
            for at, i in enumerate(drafts):
                for g in range(G):
                    x = R1 @ unit[i, g]
                    floor = torch.minimum(unit.abs().max(), 2.0 ** 17 * unit[i, g].abs().max()) * tiny
                    sk = scale * rn * (sign @ (R2 @ x)) if cb.qjl else torch.zeros(end, dtype=torch.float64, device=dev)

                    def weights(keys):
                        s = (scale * (keys @ x) + sk).masked_fill(~vis[i], -math.inf)
                        top = s.max()
                        if not bool(torch.isfinite(top)):
                            return s, torch.zeros_like(s)
                        e = (s - top).exp()
                        return s, e / e.sum()

                    s, p = weights(k)
                    o = p @ v
                    out[b, at, h * G + g] = o
                    o_table = weights(kt)[1] @ vt
                    away = v - o
                    xx = (x * x + floor * floor * (2.0 ** 22 if uq == U else 2.0 ** 44))
                    t = U * torch.minimum(K * ((p * p) @ (v * v)).sqrt(), p @ v.abs())
                    J = scale * (k * p[:, None]).T @ away
                    first = K * uq * (xx @ (J * J)).sqrt()
                    g2 = (k * k) @ xx * scale * scale
                    any_seen = bool(vis[i].any())
                    worst = K * uq * g2[vis[i]].max().sqrt() if any_seen else zero
                    if cb.qjl:
                        w = R2 @ x
                        J2 = scale * (sign * (rn * p)[:, None]).T @ away
                        ww = w * w + floor * floor * 2.0 ** 22
                        first = first + K * U * (ww @ (J2 * J2)).sqrt()
                        first = first + K * U * ((p * p * sk * sk) @ (away * away)).sqrt()
                        worst = worst + K * U * ((rn * scale).max() * ww.sum().sqrt() + sk.abs().max())
                    if cb.affine:
                        vv = v * v + (vn * 2.0 ** -14)[:, None] ** 2
                        t = t + U * torch.minimum(K * ((p * p) @ vv).sqrt(), p @ vv.sqrt())
                        g2 = (k * k + 2.0 ** -28) @ xx * scale * scale
                        first = first + K * U * ((p * p * g2) @ (away * away)).sqrt()
                        worst = worst + K * U * g2[vis[i]].max().sqrt() if any_seen else worst
                    lin = 2.0 ** -20 * (scale * (k.abs() @ x.abs()) + 2 * sk.abs() + 2 * torch.where(vis[i], s, zero).abs().max() + 4)
                    t = t + first * (1 + 2 * worst) + (p * lin) @ away.abs()
                    e = worst + lin[vis[i]].max() if any_seen else zero
                    if float(e) > 0.1:
                        far = away[s >= s.max() - 2 * e - 28].abs().amax(0)
                        # (past e = 10 the smaller weights are not held exactly enough for the first)
                        t = t + (far if float(e) > 10 else torch.minimum(far, torch.expm1(2 * e) * (p @ away.abs())))
                    acc[b, at, h * G + g] = (min(end, share) / 16 + 64) * 2.0 ** -23 * (p @ stored.abs()).norm()
                    small = (p * vn).max() * 2.0 ** -29
                    t = t + small * (v.abs() / vn.clamp_min(1e-300)[:, None]).masked_fill(~vis[i][:, None], 0.0).sum(0)
                    tol[b, at, h * G + g] = t + (o_table - o).abs()
    return out, tol, acc


def limits(got_dtype, out, tol):
    """`tol` and half a step of the output's type."""
    half = torch.finfo(got_dtype).eps / 2
    tiny = torch.finfo(got_dtype).smallest_normal * half
    return half * out.abs() * 1.0001 + tol * (1 + half) + tiny


def _worst(err, out, tol, acc, dtype):
    """The largest error of each row over what it may be: of its elements, and of its 2-norm."""
    lim = limits(dtype, out, tol)
    return torch.maximum((err / (lim + acc)).amax(-1), err.norm(dim=-1) / (lim.norm(dim=-1) + acc[..., 0]))


def assert_within(got, out, tol, acc):
    worst = _worst((got.to(out.device).double() - out).abs(), out, tol, acc, got.dtype).max()
    assert bool(worst <= 1), f"worst error is {float(worst):.3g} of its bound"


def passes(wrong, out, tol, acc, dtype):
    """Whether a wrong answer would pass for the right one in some row that it changes."""
    worst = _worst((wrong.to(dtype).double() - out).abs(), out, tol, acc, dtype)
    return bool((worst <= 1)[(wrong != out).any(-1)].any())


def found(wrong, out, tol, acc, dtype):
    """Whether assert_within would refuse a wrong answer: some row of it is out of bounds."""
    return bool((_worst((wrong.to(dtype).double() - out).abs(), out, tol, acc, dtype) > 1).any())
