"""Speculative decoding over the packed KV cache: what its operators are measured on.

Four operators that a program calls around each verification step:

  append   rotary positions of the queries and keys, fused with quantize-and-append
           (tq.tq_rope_append)
  tree     attention of a tree (or chain) of drafted tokens over the packed cache
           (tq.tq_tree_attention)
  compact  keep the accepted slots of every row and free the rest (tq.tq_cache_compact)
  copy     copy or fork rows of a cache (tq.tq_cache_copy)

``run`` computes a case with elementary torch operations in 32 bits (angles in
64), or, with ``own`` set, through the framework's calls.  Codes, sign bits and
copied bytes are whole numbers and compared as such: the codec is one correctly
rounded fp32 operation at a time in a fixed order, in both forms.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

SEED = 20  # seeds the rotation signs of every case
AFFINE_GROUP = 64  # channels per group of the affine codec
ARRAYS = ("k_codes", "v_codes", "k_signs", "k_norm", "v_norm", "k_rnorm")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _tree(name, batch, heads, d, bits, ctx, n_q, mask="tree", dtype="bf16", qjl=False, codebook="gaussian"):
    c = {"op": "tree", "batch": batch, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": d,
         "k_bits": bits[0], "v_bits": bits[1], "qjl": qjl, "codebook": codebook, "ctx_min": ctx[0],
         "ctx_max": ctx[1], "n_q": n_q, "mask": mask, "dtype": dtype}
    return {**c, "name": name} if name else c


def _append(name, batch, heads, d, bits, n_new, start, rot, interleaved, scaling, fused, keys_out,
            dtype="bf16", qjl=False, codebook="gaussian"):
    c = {"op": "append", "batch": batch, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": d,
         "k_bits": bits[0], "v_bits": bits[1], "qjl": qjl, "codebook": codebook, "n_new": n_new,
         "start": start, "rot_dim": rot, "interleaved": interleaved, "scaling": scaling,
         "fused_qkv": fused, "keys_out": keys_out, "dtype": dtype}
    return {**c, "name": name} if name else c


def _compact(name, batch, kv_heads, d, bits, start, window, keep, per_head, qjl=False, codebook="gaussian"):
    c = {"op": "compact", "batch": batch, "kv_heads": kv_heads, "head_dim": d, "k_bits": bits[0],
         "v_bits": bits[1], "qjl": qjl, "codebook": codebook, "start": start, "window": window,
         "keep": keep, "per_head": per_head}
    return {**c, "name": name} if name else c


def _copy(name, rows, pairs, kv_heads, d, bits, length, fork, qjl=False, codebook="gaussian"):
    c = {"op": "copy", "rows": rows, "pairs": pairs, "kv_heads": kv_heads, "head_dim": d, "k_bits": bits[0],
         "v_bits": bits[1], "qjl": qjl, "codebook": codebook, "length": length, "fork": fork}
    return {**c, "name": name} if name else c


def listed():
    return [
        # one user, short context, a chain of drafts from a small draft model: latency
        _tree("tree chain 5, 4k", 1, (32, 8), 128, (3, 4), (4096, 4096), 5, mask="chain"),
        # one user at the gqa workload's context, a wide static tree of drafts
        _tree("tree 63, gqa 32k", 1, (32, 8), 128, (3, 4), (32705, 32705), 63),
        # a serving batch of ragged contexts, one row still empty, a modest tree each
        _tree("tree 16, ragged 16 rows", 16, (32, 8), 128, (3, 4), (0, 32768), 16),
        # few long rows whose keys carry the residual sketch (the qjl workload): the largest
        _tree("tree 25, qjl 4 x 128k", 4, (32, 8), 128, (3, 4), (98304, 131001), 25, qjl=True),
        # the long workload's shape: wide heads, 2-bit codes with the sketch
        _tree("tree 8, long d256", 1, (16, 4), 256, (2, 2), (200003, 200003), 8, qjl=True, dtype="fp16"),
        # the affine comparison codec
        _tree("tree 33, affine 32k", 1, (32, 8), 128, (4, 4), (32768, 32768), 33, codebook="affine"),
        # one decode step of a serving batch: latency
        _append("append 1, 32 rows", 32, (32, 8), 128, (3, 4), 1, 4001, 128, False, "yarn", True, False),
        # a prefill chunk of one row, whose rotated keys the dense prefill attention also reads
        _append("append 8192 prefill", 1, (32, 8), 128, (3, 4), 8192, 24576, 128, False, "linear", True, True),
        # a verification step keeps the accepted path of a 64-token tree: latency
        _compact("compact 64 -> 6, 32 rows", 32, 8, 128, (3, 4), 4000, 64, 6, False),
        # eviction: every head keeps its own half of a long row
        _compact("compact 64k -> 32k", 2, 8, 128, (3, 4), 0, 65536, 32768, True, qjl=True),
        # one prompt forked into several samples
        _copy("fork 1 -> 7, 2k", 8, 7, 8, 128, (3, 4), 2049, True),
        # beams reordered into a second cache
        _copy("copy 16 rows, 32k", 16, 16, 8, 128, (3, 4), 32768, False),
    ]


_BITS = ((2, 2), (2, 3), (3, 3), (3, 4), (4, 4))


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "append", "compact", "copy"))
    d = rng.choice((64, 128, 128, 256))
    bits = rng.choice(_BITS)
    codebook = rng.choice(("gaussian", "gaussian", "sphere", "affine"))
    qjl = rng.random() < 0.3
    kv = rng.choice((1, 2, 4, 8))
    heads = (kv * rng.choice((1, 2, 4, 8)), kv)
    batch = _log(rng, 1, 16)
    if op == "tree":
        n_q = _log(rng, 1, 64)
        ctx = _log(rng, 16, 131072)
        rows = n_q * heads[0]
        # no more tokens, and no more products, than the largest listed case has
        while batch * kv * ctx * d > 4 * 8 * 98304 * 128 or batch * rows * ctx * d > 4 * 32 * 25 * 98304 * 128:
            ctx //= 2
        low = ctx if batch == 1 else rng.randrange(0, ctx + 1)
        return _tree(None, batch, heads, d, bits, (low, ctx), n_q, mask=rng.choice(("tree", "chain")),
                     dtype=rng.choice(("bf16", "fp16")), qjl=qjl, codebook=codebook)
    if op == "append":
        n = _log(rng, 1, 8192)
        while batch * n * (heads[0] + 2 * kv) * d > 8192 * 48 * 128:
            n = (n + 1) // 2
        rot = 2 * rng.randrange(4, d // 2 + 1) if rng.random() < 0.4 else d
        return _append(None, batch, heads, d, bits, n, rng.randrange(0, 16384), rot, rng.random() < 0.5,
                       rng.choice(("none", "linear", "ntk", "yarn", "bands")), rng.random() < 0.5,
                       rng.random() < 0.5, dtype=rng.choice(("bf16", "fp16", "fp32")), qjl=qjl, codebook=codebook)
    if op == "compact":
        window = _log(rng, 2, 65536)
        while batch * kv * window * d > 2 * 8 * 65536 * 128:
            window = (window + 1) // 2
        keep = max(1, int(window * rng.uniform(0.05, 0.9)))
        return _compact(None, batch, kv, d, bits, rng.randrange(0, 2048), window, keep, rng.random() < 0.5,
                        qjl=qjl, codebook=codebook)
    fork = rng.random() < 0.5
    rows = rng.randrange(2, 17)
    pairs = rows - 1 if fork else rows
    length = _log(rng, 1, 32768)
    while pairs * kv * length * d > 16 * 8 * 32768 * 128:
        length = (length + 1) // 2
    return _copy(None, rows, pairs, kv, d, bits, length, fork, qjl=qjl, codebook=codebook)


# ---------------------------------------------------------------------------
# sizes that follow from a case
# ---------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n lengths from hi down to lo, in an order that is not sorted."""
    if n == 1:
        return [hi]
    v = [hi - (hi - lo) * i // (n - 1) for i in range(n)]
    return v[::2] + v[1::2]


def _contexts(case):
    return _spread(case["ctx_min"], case["ctx_max"], case["batch"])


def _keeps(case):
    """Slots kept of each row: the full count, and a few fewer in the other rows."""
    return [max(0, case["keep"] - (b % 3) * (1 + case["keep"] // 8)) for b in range(case["batch"])]


def _lengths(case):
    return [max(0, case["length"] - (i % 4) * (case["length"] // 8)) for i in range(case["pairs"])]


def _up16(n):
    return max(16, (n + 15) // 16 * 16)


def _row_bytes(case):
    """Bytes of one token's slot of one KV head, over all arrays."""
    d, meta = case["head_dim"], 2
    if case["codebook"] == "affine":
        meta = 4 * case["head_dim"] // AFFINE_GROUP
    return (case["k_bits"] + case["v_bits"]) * d // 8 + 2 * meta + ((d // 8 + 2) if case["qjl"] else 0)


def work(case):
    if case["op"] == "tree":
        n, d, group = case["n_q"], case["head_dim"], case["q_heads"] // case["kv_heads"]
        tokens = sum(c + n for c in _contexts(case)) * case["kv_heads"]
        io = 2 * 2 * case["batch"] * n * case["q_heads"] * d
        products = 3 if case["qjl"] else 2
        return {"bytes": tokens * _row_bytes(case) + io, "flops": 2.0 * products * n * group * d * tokens}
    if case["op"] == "append":
        size = 4 if case["dtype"] == "fp32" else 2
        b, n, d = case["batch"], case["n_new"], case["head_dim"]
        vec = b * n * d * size
        moved = vec * (2 * case["q_heads"] + 2 * case["kv_heads"] + (case["kv_heads"] if case["keys_out"] else 0))
        stored = b * n * case["kv_heads"] * _row_bytes(case)
        flops = b * n * d * (3 * (case["q_heads"] + case["kv_heads"]) + 2 * case["kv_heads"] * (math.log2(d) + 4))
        return {"bytes": moved + stored + 4 * b * n, "flops": flops}
    if case["op"] == "compact":
        kept = sum(_keeps(case))
        lists = 4 * kept * (case["kv_heads"] if case["per_head"] else 1)
        return {"bytes": 2 * kept * case["kv_heads"] * _row_bytes(case) + lists, "flops": 0}
    return {"bytes": 2 * sum(_lengths(case)) * case["kv_heads"] * _row_bytes(case), "flops": 0}


# ---------------------------------------------------------------------------
# the codec's host tables
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _levels(bits, codebook, d):
    """Lloyd-Max levels (float32, odd-symmetric) of N(0, 1), or of a coordinate of
    a random vector of length sqrt(d); the integer levels for the affine codec."""
    n = 1 << bits
    if codebook == "affine":
        return [float(j) for j in range(n)]

    def normal_mean(a, b):
        pdf = lambda x: 0.0 if math.isinf(x) else math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
        tail = lambda x: 0.5 * math.erfc(x / math.sqrt(2))
        mass = tail(a) - tail(b) if a >= 0 else tail(-b) - tail(-a) if b <= 0 else 1 - tail(-a) - tail(b)
        return (pdf(a) - pdf(b)) / mass

    def sphere_mean(a, b):
        import numpy as np
        r = math.sqrt(d)
        a, b = max(a, -r), min(b, r)
        x, w = np.polynomial.legendre.leggauss(48)
        edges = np.linspace(a, b, 1 + max(1, math.ceil(4 * (b - a))))
        z = 0.5 * (edges[1:, None] + edges[:-1, None]) + 0.5 * (edges[1:, None] - edges[:-1, None]) * x
        f = 0.5 * (edges[1:, None] - edges[:-1, None]) * w * np.exp((d - 3) / 2 * np.log1p(-z * z / d))
        return float((f * z).sum() / f.sum())

    c = [-2 + 4 * (j + 0.5) / n for j in range(n)]
    for mean in (normal_mean, sphere_mean) if codebook == "sphere" else (normal_mean,):
        for _ in range(100000):
            edge = [-math.inf] + [(c[j] + c[j + 1]) / 2 for j in range(n - 1)] + [math.inf]
            new = [mean(edge[j], edge[j + 1]) for j in range(n)]
            moved = max(abs(x - y) for x, y in zip(new, c))
            c = new
            if moved < 1e-14:
                break
    f32 = lambda x: float(torch.tensor(x, dtype=torch.float64).float())
    half = [f32((c[n // 2 + j] - c[n // 2 - 1 - j]) / 2) for j in range(n // 2)]
    return [-x for x in reversed(half)] + half


@functools.lru_cache(maxsize=None)
def _signs(second, d):
    """The +-1 diagonal of the rotation: top bits of SplitMix64 from the seed."""
    mask, golden = (1 << 64) - 1, 0x9E3779B97F4A7C15
    state, out = SEED ^ (golden if second else 0), []
    for _ in range(d):
        state = (state + golden) & mask
        z = ((state ^ (state >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return out


def _tables(case, bits):
    """(centroids, boundaries) on the GPU."""
    c = torch.tensor(_levels(bits, case["codebook"], case["head_dim"]), device="cuda")
    return c, (c[:-1] + c[1:]) * 0.5


def _sign_tensor(case, second=False):
    return torch.tensor(_signs(second, case["head_dim"]), device="cuda")


ROPE_BASE = 10000.0
ROPE_ORIGINAL = 8192
ROPE_FACTOR = 4.0


def _inverse_frequencies(case):
    """Rotation per position of each pair, and the factor on cosine and sine."""
    rot, scaling, f = case["rot_dim"], case["scaling"], ROPE_FACTOR
    base = ROPE_BASE
    if scaling == "ntk" and rot > 2:
        base = ROPE_BASE * math.pow(f, rot / (rot - 2.0))
    inv = [math.pow(base, -(2.0 * i) / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / f for x in inv], 1.0
    if scaling == "yarn":  # pairs that turn often keep their rate, slow ones are divided by the factor
        at = lambda turns: rot * math.log(ROPE_ORIGINAL / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        low, high = max(math.floor(at(32.0)), 0.0), min(math.ceil(at(1.0)), rot - 1.0)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        return [x / f * r + x * (1.0 - r) for x, r in zip(inv, ramp)], 0.1 * math.log(f) + 1.0
    if scaling == "bands":  # the same by wavelength, with a linear band between
        out = []
        for x in inv:
            turns = ROPE_ORIGINAL * x / (2.0 * math.pi)
            s = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            out.append((1.0 - s) * (x / f) + s * x)
        return out, 1.0
    return inv, 1.0


# ---------------------------------------------------------------------------
# the codec in elementary operations
# ---------------------------------------------------------------------------
def _fwht(u):
    """Unnormalized Walsh-Hadamard transform of the last axis: (a + b, a - b) at distance 1, 2, 4, ..."""
    d, h = u.shape[-1], 1
    while h < d:
        w = u.reshape(*u.shape[:-1], d // (2 * h), 2, h)
        a, b = w[..., 0, :], w[..., 1, :]
        u = torch.stack((a + b, a - b), dim=-2).reshape(u.shape)
        h *= 2
    return u


def _tree_sum(x):
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x[..., 0]


def _pack(codes, bits):
    """[..., n] codes -> uint8 [..., n * bits / 8], a little-endian bit stream."""
    g = codes.reshape(*codes.shape[:-1], -1, 8).to(torch.int64)
    word = (g << (bits * torch.arange(8, device=g.device))).sum(-1)
    out = (word[..., None] >> (8 * torch.arange(bits, device=g.device))) & 255
    return out.to(torch.uint8).flatten(-2)


def _unpack(packed, bits):
    g = packed.reshape(*packed.shape[:-1], -1, bits).to(torch.int64)
    word = (g << (8 * torch.arange(bits, device=g.device))).sum(-1)
    out = (word[..., None] >> (bits * torch.arange(8, device=g.device))) & ((1 << bits) - 1)
    return out.flatten(-2)


def _encode(case, x, keys):
    """float32 [..., d] -> the arrays of a slot: codes, norm and, for keys, signs and rnorm."""
    d, bits = case["head_dim"], case["k_bits"] if keys else case["v_bits"]
    cent, bnd = _tables(case, bits)
    root = torch.tensor(float(d), device="cuda").sqrt()
    u = _fwht(x * _sign_tensor(case))
    out = {}
    if case["codebook"] == "affine":
        y = u * torch.reciprocal(root) if keys else x
        g = y.reshape(*y.shape[:-1], -1, AFFINE_GROUP)
        low, high = g.amin(-1) + 0.0, g.amax(-1) + 0.0
        scale = ((high - low) / torch.tensor(float((1 << bits) - 1), device="cuda")).half()
        bias = low.half()
        s, b = scale.float()[..., None], bias.float()[..., None]
        code = torch.where(s == 0, torch.zeros_like(g), torch.round((g - b) / s)).clamp(0, (1 << bits) - 1)
        residual, divisor = (g - (s * code + b)).reshape(y.shape), torch.ones_like(root)
        code = code.reshape(y.shape).to(torch.int64)
        out["norm"] = torch.stack((scale, bias), -1).flatten(-2)
    else:
        n = _tree_sum(x * x).sqrt()
        inv = torch.where(n == 0, torch.zeros_like(n), torch.reciprocal(n))
        code = torch.bucketize(u * inv[..., None], bnd)
        out["norm"] = n.half()
        residual, divisor = u - out["norm"].float()[..., None] * cent[code], root
    out["codes"] = _pack(code, bits)
    if keys and case["qjl"]:
        out["rnorm"] = (_tree_sum(residual * residual).sqrt() / divisor).half()
        out["signs"] = _pack((_fwht(residual * _sign_tensor(case, True)) >= 0).to(torch.int64), 1)
    return out


def _decoded(case, cache, which, rows=slice(None), dtype=torch.float32):
    """Dequantized keys (rotated frame) or values (rotated frame; affine: as they are)."""
    d, bits = case["head_dim"], case["k_bits"] if which == "k" else case["v_bits"]
    code = _unpack(cache[which + "_codes"][rows], bits)
    norm = cache[which + "_norm"][rows].to(dtype)
    if case["codebook"] == "affine":
        n = norm.reshape(*norm.shape[:-1], -1, 2)
        g = code.to(dtype).reshape(*code.shape[:-1], -1, AFFINE_GROUP)
        return (n[..., 0:1] * g + n[..., 1:2]).reshape(code.shape)
    cent = _tables(case, bits)[0].to(dtype)
    return cent[code] * (norm / math.sqrt(d))[..., None]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _shapes(case, capacity, rows):
    d, h = case["head_dim"], case["kv_heads"]
    meta = (2 * d // AFFINE_GROUP,) if case["codebook"] == "affine" else ()
    s = {"k_codes": (torch.uint8, (case["k_bits"] * d // 8,)), "v_codes": (torch.uint8, (case["v_bits"] * d // 8,)),
         "k_norm": (torch.float16, meta), "v_norm": (torch.float16, meta)}
    if case["qjl"]:
        s |= {"k_signs": (torch.uint8, (d // 8,)), "k_rnorm": (torch.float16, ())}
    return {k: (t, (rows, h, capacity, *tail)) for k, (t, tail) in s.items()}


def _random_cache(case, gen, capacity, rows):
    """A cache of random bytes and plausible norms: what is moved, not decoded."""
    cache = {}
    for name, (dtype, shape) in _shapes(case, capacity, rows).items():
        if dtype == torch.uint8:
            cache[name] = torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=dtype)
        else:
            cache[name] = torch.randn(shape, generator=gen, device="cuda").abs().add_(1).half()
    return cache


def _drawn_cache(case, gen, lens, q):
    """A cache as the codec leaves it: rotated coordinates are near N(0, 1), and one
    token in 61 resembles a drafted query, so that the softmax has peaks."""
    b, h, d, n = case["batch"], case["kv_heads"], case["head_dim"], case["n_q"]
    group, capacity = case["q_heads"] // h, _up16(max(lens))
    cache = {k: torch.zeros(s, dtype=t, device="cuda") for k, (t, s) in _shapes(case, capacity, b).items()}
    rotated = _fwht(q.float() * _sign_tensor(case))            # [B, n, Hq, d]
    unit = rotated / rotated.square().mean(-1, keepdim=True).sqrt()
    at = torch.arange(17 % capacity, capacity, 61, device="cuda")
    which = at // 61
    for r in range(b):
        for name, bits in (("k", case["k_bits"]), ("v", case["v_bits"])):
            z = torch.randn((h, capacity, d), generator=gen, device="cuda")
            if name == "k" and case["ctx_max"] > 61:
                u = unit[r].reshape(n, h, group, d)[which % n, :, which % group]   # [tokens, H, d]
                z[:, at] = 0.6 * z[:, at] + 0.8 * u.transpose(0, 1)
            length = math.sqrt(d) * (1 + 0.1 * torch.randn((h, capacity), generator=gen, device="cuda")).abs()
            if case["codebook"] == "affine":
                g = z.reshape(h, capacity, -1, AFFINE_GROUP)
                low, high = g.amin(-1), g.amax(-1)
                scale = ((high - low) / ((1 << bits) - 1)).half()
                code = ((g - low[..., None]) / scale.float()[..., None]).round().clamp(0, (1 << bits) - 1)
                code = code.reshape(z.shape).to(torch.int64)
                cache[name + "_norm"][r] = torch.stack((scale, low.half()), -1).flatten(-2)
            else:
                cent, bnd = _tables(case, bits)
                code = torch.bucketize(z, bnd)
                cache[name + "_norm"][r] = length.half()
            cache[name + "_codes"][r] = _pack(code, bits)
            if name == "k" and case["qjl"]:
                cache["k_signs"][r] = torch.randint(0, 256, cache["k_signs"][r].shape, generator=gen, device="cuda",
                                                    dtype=torch.uint8)
                cache["k_rnorm"][r] = (length * 0.19).half()
    return cache


def _mask(case, gen):
    """Ancestor bits of a random tree, int32 [n, ceil(n / 32)]; None for a chain."""
    n = case["n_q"]
    if case["mask"] == "chain":
        return None
    pick = torch.rand(n, generator=gen, device="cuda").tolist()
    rows = []
    for i in range(n):  # a drafted token's parent is among the four before it, or the context
        parent = i - 1 - int(4 * pick[i] * pick[i])
        rows.append((rows[parent] if parent >= 0 else 0) | (1 << i))
    words = [[(r >> (32 * w)) & 0xFFFFFFFF for w in range((n + 31) // 32)] for r in rows]
    return torch.tensor(words, dtype=torch.int64).to(torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": case}
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "tree":
        n, d = case["n_q"], case["head_dim"]
        lens = [c + n for c in _contexts(case)]
        q = torch.randn((case["batch"], n, case["q_heads"], d), generator=gen, device="cuda").to(_DTYPES[case["dtype"]])
        s["cache"] = _drawn_cache(case, gen, lens, q)
        s["cache"]["seq_lens"] = torch.tensor(lens, **i32)
        s |= {"q": q, "mask": _mask(case, gen), "max_ctx": max(lens)}
        rows, capacity = case["batch"], s["cache"]["k_codes"].shape[2]
    elif case["op"] == "append":
        b, n, d, hq, hk = case["batch"], case["n_new"], case["head_dim"], case["q_heads"], case["kv_heads"]
        rows, capacity = b, _up16(case["start"] + n + 31)
        x = torch.randn((b, n, hq + 2 * hk, d), generator=gen, device="cuda")
        x[:, :, hq:hq + hk, :: d // 4] *= 20.0  # keys have a few outlier channels
        if not case["fused_qkv"]:
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        x = x.to(_DTYPES[case["dtype"]]).transpose(1, 2)  # [B, heads, n, d] views of one projection's output
        s |= {"q": x[:, :hq], "k": x[:, hq:hq + hk], "v": x[:, hq + hk:]}
        s["cache"] = {k: torch.zeros(z, dtype=t, device="cuda") for k, (t, z) in _shapes(case, capacity, b).items()}
        s["start"] = torch.tensor([case["start"] + (11 * i) % 31 for i in range(b)], **i32)
        s["cache"]["seq_lens"] = s["start"].clone()
        # tokens of a drafted tree lie at their depths; a prompt's at consecutive positions
        depth = torch.arange(n) if n > 64 else torch.div(torch.arange(n) + 1, 2, rounding_mode="floor")
        s["offsets"] = depth.to(**i32).expand(b, n).contiguous()
        s["positions"] = _up16(case["start"] + n + 31)
    elif case["op"] == "compact":
        b, w, hk = case["batch"], case["window"], case["kv_heads"]
        rows, capacity, keeps = b, _up16(case["start"] + w), _keeps(case)
        s["cache"] = _random_cache(case, gen, capacity, b)
        s["cache"]["seq_lens"] = torch.full((b,), case["start"] + w, **i32)
        order = torch.rand((b, hk if case["per_head"] else 1, w), generator=gen, device="cuda").argsort(-1)
        index = order[..., :case["keep"]].sort(-1).values.to(torch.int32)
        for r, k in enumerate(keeps):  # the kept slots of a row ascend; the list's tail is not read
            index[r, :, :k] = order[r, :, :k].sort(-1).values.to(torch.int32)
            index[r, :, k:] = -1
        s["index"] = index if case["per_head"] else index[:, 0].contiguous()
        s["counts"] = torch.tensor(keeps, **i32)
        s["start"] = torch.full((b,), case["start"], **i32)
    else:
        rows, capacity = case["rows"], _up16(case["length"])
        s["cache"] = _random_cache(case, gen, capacity, rows)
        s["cache"]["seq_lens"] = torch.full((rows,), case["length"], **i32)
        n = case["pairs"]
        if case["fork"]:  # row 0 to every other row of the same cache
            s["to"] = s["cache"]
            s["src"], s["dst"] = torch.zeros(n, **i32), torch.arange(1, n + 1, **i32)
        else:  # beams: any row of the old cache, each row of the new one once
            s["to"] = {k: torch.zeros_like(v) for k, v in s["cache"].items()}
            s["src"] = torch.randint(0, rows, (n,), generator=gen, device="cuda").to(torch.int32)
            s["dst"] = torch.randperm(rows, generator=gen, device="cuda")[:n].to(torch.int32)
        s["lengths"] = torch.tensor(_lengths(case), **i32)
        s["max_len"] = case["length"]
    if own:  # the handles that a program keeps
        from turboquant_kv_cache_rht_b200 import tq
        s["tq"] = tq
        s["cb"] = tq.Codebook(case["head_dim"], case["k_bits"], case["v_bits"], qjl=case["qjl"], seed=SEED,
                              codebook=case["codebook"])
        s["handle"] = _handle(tq, s["cb"], s["cache"], rows, case["kv_heads"], capacity)
        if case["op"] == "tree":
            need = tq.tq_tree_workspace_bytes(s["cb"], case["batch"], case["q_heads"], case["kv_heads"], case["n_q"],
                                              s["max_ctx"])
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        if case["op"] == "append":
            s["rope"] = tq.Rope(case["rot_dim"], s["positions"], base=ROPE_BASE, interleaved=case["interleaved"],
                                scaling=None if case["scaling"] == "none" else case["scaling"], factor=ROPE_FACTOR,
                                original_max=ROPE_ORIGINAL)
        if case["op"] == "compact":
            s["full"] = s["cache"]["seq_lens"].clone()
        if case["op"] == "copy":
            s["to_handle"] = s["handle"] if case["fork"] else _handle(tq, s["cb"], s["to"], rows, case["kv_heads"],
                                                                      capacity)
    return s


def _handle(tq, cb, cache, rows, kv_heads, capacity):
    """The framework's cache over these tensors (its own are a few slots, and replaced)."""
    handle = tq.Cache(cb, rows, kv_heads, 16)
    handle.capacity = capacity
    for name, tensor in cache.items():
        setattr(handle, name, tensor)
    return handle


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(state):
    return {"tree": _run_tree, "append": _run_append, "compact": _run_compact, "copy": _run_copy}[state["case"]["op"]](state)


def _bits_of(mask, n):
    """bool [n, n] of the packed ancestor bits (a chain without a mask)."""
    at = torch.arange(n, device="cuda")
    if mask is None:
        return at[None, :] <= at[:, None]
    return ((mask[:, at // 32] >> (at % 32)) & 1).bool()


def _run_tree(s):
    if own:
        return s["tq"].tq_tree_attention(s["cb"], s["handle"], s["q"], mask=s["mask"], max_ctx=s["max_ctx"],
                                         workspace=s["workspace"])
    c, cache, q = s["case"], s["cache"], s["q"].float()
    b, n, hq, d = q.shape
    h = c["kv_heads"]
    rows = (hq // h) * n
    u = _fwht(q * _sign_tensor(c)) / math.sqrt(d)                                  # R q
    grouped = lambda x: x.reshape(b, n, h, hq // h, d).permute(0, 2, 1, 3, 4).reshape(b, h, rows, d)
    score = grouped(u) @ _decoded(c, cache, "k").transpose(-1, -2)                 # [B, H, rows, tokens]
    if c["qjl"]:
        w = _fwht(u * _sign_tensor(c, True)) / math.sqrt(d)
        sign = 2.0 * _unpack(cache["k_signs"], 1).float() - 1.0
        sketch = grouped(w) @ sign.transpose(-1, -2)
        score += math.sqrt(math.pi / (2 * d)) * cache["k_rnorm"].float()[:, :, None, :] * sketch
    score *= 1.0 / math.sqrt(d)
    # token t of a row: context below len - n, drafted token t - (len - n) after it
    t = torch.arange(score.shape[-1], device="cuda") - (cache["seq_lens"][:, None] - n)    # [B, tokens]
    tree = _bits_of(s["mask"], n)[:, t.clamp(0, n - 1)].transpose(0, 1)                    # [B, n, tokens]
    seen = torch.where((t >= 0)[:, None], tree & (t < n)[:, None], torch.ones_like(tree))
    seen = seen[:, None, :, None, :].expand(b, 1, n, hq // h, t.shape[-1]).reshape(b, 1, rows, -1)
    score = torch.where(seen, score, torch.full((), -math.inf, device="cuda"))
    p = (score - score.amax(-1, keepdim=True)).exp()
    o = (p @ _decoded(c, cache, "v")) / p.sum(-1, keepdim=True)
    if c["codebook"] != "affine":
        o = _fwht(o) / math.sqrt(d) * _sign_tensor(c)                              # R^T o
    return o.reshape(b, h, n, hq // h, d).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d).to(s["q"].dtype)


def _rotary(x, cos, sin, case):
    """[B, heads, n, d] turned by the angles of [B, n, rot / 2]."""
    rot = case["rot_dim"]
    cos, sin = cos[:, None], sin[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., rot:]), -1)
    a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), -1)


def _run_append(s):
    c, cache = s["case"], s["cache"]
    if own:
        q, k = s["tq"].tq_rope_append(s["cb"], s["handle"], s["rope"], s["k"], s["v"], q=s["q"], positions=s["offsets"],
                                      relative=True, start=s["start"], keys_out=c["keys_out"])
    else:
        n = c["n_new"]
        inv, factor = _inverse_frequencies(c)
        at = s["start"][:, None].double() + s["offsets"].double()
        angle = at[..., None] * torch.tensor(inv, dtype=torch.float64, device="cuda")
        cos, sin = (angle.cos() * factor).float(), (angle.sin() * factor).float()
        q = _rotary(s["q"].float(), cos, sin, c).to(s["q"].dtype).transpose(1, 2).contiguous()
        keys = _rotary(s["k"].float(), cos, sin, c)
        k = keys.to(s["k"].dtype).transpose(1, 2).contiguous() if c["keys_out"] else None
        slot = (s["start"][:, None] + torch.arange(n, device="cuda")).long()
        row = torch.arange(c["batch"], device="cuda")[:, None]
        for which, x in (("k", keys), ("v", s["v"].float())):
            for name, v in _encode(c, x, which == "k").items():
                cache[which + "_" + name][row, :, slot] = v.transpose(1, 2)
        cache["seq_lens"].copy_(s["start"] + n)
    return {"q": q, **({"k": k} if c["keys_out"] else {}), **cache}


def _run_compact(s):
    c, cache = s["case"], s["cache"]
    if own:
        cache["seq_lens"].copy_(s["full"])  # a pass before this one has left the kept slots' lengths
        s["tq"].tq_cache_compact(s["cb"], s["handle"], s["index"], s["counts"], start=s["start"])
        return dict(cache)
    b, h = c["batch"], c["kv_heads"]
    index = s["index"] if s["index"].dim() == 3 else s["index"][:, None]
    index = index.expand(b, h, index.shape[-1]).long()
    i = torch.arange(index.shape[-1], device="cuda").expand(index.shape)
    kept = i < s["counts"][:, None, None]
    start = s["start"].long()[:, None, None]
    to = start + i
    source = torch.where(kept, start + index, to)  # past the kept slots nothing moves
    row, head = torch.arange(b, device="cuda")[:, None, None], torch.arange(h, device="cuda")[None, :, None]
    for name in ARRAYS:
        if name in cache:
            cache[name][row, head, to] = cache[name][row, head, source]
    cache["seq_lens"].copy_(s["start"] + s["counts"])
    return dict(cache)


def _run_copy(s):
    c, cache, to = s["case"], s["cache"], s["to"]
    if own:
        s["tq"].tq_cache_copy(s["cb"], s["to_handle"], s["handle"], s["dst"], s["src"], lengths=s["lengths"],
                              max_len=s["max_len"])
        return dict(to)
    src, dst = s["src"].long(), s["dst"].long()
    length = torch.minimum(s["lengths"], cache["seq_lens"][src])
    n = c["length"]
    kept = torch.arange(n, device="cuda") < length[:, None]
    for name in ARRAYS:
        if name in cache:
            tail = (1,) * (cache[name].dim() - 3)
            new, old = cache[name][src, :, :n], to[name][dst, :, :n]
            to[name][dst, :, :n] = torch.where(kept.reshape(len(src), 1, n, *tail), new, old)
    to["seq_lens"][dst] = length
    return dict(to)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _hadamard(d):
    """Sylvester's matrix: the sign of entry (i, j) is the parity of i & j."""
    i = torch.arange(d, device="cuda")
    both, parity = i[:, None] & i[None, :], torch.zeros((d, d), dtype=torch.int64, device="cuda")
    for bit in range(9):
        parity ^= (both >> bit) & 1
    return 1.0 - 2.0 * parity.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    return None  # bytes are moved: nothing is computed


def _exact_tree(case, s):
    cache, n, d, h = s["cache"], case["n_q"], case["head_dim"], case["kv_heads"]
    group = case["q_heads"] // h
    r1 = _hadamard(d) * _sign_tensor(case).double() / math.sqrt(d)                 # rows of R
    r2 = _hadamard(d) * _sign_tensor(case, True).double() / math.sqrt(d)
    sees = _bits_of(s["mask"], n).tolist()
    out = torch.zeros((case["batch"], n, case["q_heads"], d), dtype=torch.float64, device="cuda")
    for b, length in enumerate(cache["seq_lens"].tolist()):
        hidden = torch.zeros((n, length), dtype=torch.bool)
        for i in range(n):
            for j in range(n):
                hidden[i, length - n + j] = not sees[i][j]
        hidden = hidden.cuda().repeat_interleave(group, 0)
        for head in range(h):
            at = (b, head, slice(0, length))
            q = s["q"][b, :, head * group:(head + 1) * group].double().reshape(n * group, d)
            k = _decoded(case, cache, "k", at, torch.float64) @ r1                 # keys in their own frame
            v = _decoded(case, cache, "v", at, torch.float64)
            v = v if case["codebook"] == "affine" else v @ r1
            score = q @ k.T
            if case["qjl"]:
                sign = 2.0 * _unpack(cache["k_signs"][at], 1).double() - 1.0
                score += math.sqrt(math.pi / (2 * d)) * cache["k_rnorm"][at].double() * (q @ r1.T @ r2.T @ sign.T)
            weight = torch.softmax((score / math.sqrt(d)).masked_fill(hidden, -math.inf), -1)
            out[b, :, head * group:(head + 1) * group] = (weight @ v).reshape(n, group, d)
    return out


def _exact_append(case, s):
    rot, n, d = case["rot_dim"], case["n_new"], case["head_dim"]
    inv, factor = _inverse_frequencies(case)
    at = (s["start"][:, None] + s["offsets"]).double()
    turn = torch.polar(torch.full((), factor, dtype=torch.float64, device="cuda").expand(*at.shape, rot // 2),
                       at[..., None] * torch.tensor(inv, dtype=torch.float64, device="cuda"))[:, None]

    def rotated(x):
        x = x.double()
        pair = (lambda y: y.reshape(*y.shape[:-1], rot // 2, 2)) if case["interleaved"] else (
            lambda y: y.reshape(*y.shape[:-1], 2, rot // 2).transpose(-1, -2))
        z = torch.view_as_real(torch.view_as_complex(pair(x[..., :rot]).contiguous()) * turn)
        z = z if case["interleaved"] else z.transpose(-1, -2)
        return torch.cat((z.flatten(-2), x[..., rot:]), -1)

    keys, values = rotated(s["k"]), s["v"].double()
    out = {"q": rotated(s["q"]).transpose(1, 2), "seq_lens": None}
    if case["keys_out"]:
        out["k"] = keys.transpose(1, 2)
    r1 = _hadamard(d) * _sign_tensor(case).double()
    slot = (s["start"][:, None] + torch.arange(n, device="cuda")).long()
    row = torch.arange(case["batch"], device="cuda")[:, None]
    for which, x, bits in (("k", keys, case["k_bits"]), ("v", values, case["v_bits"])):
        u = x @ r1.T                                                                # unnormalized
        if case["codebook"] == "affine":
            y = (u / math.sqrt(d) if which == "k" else x).unflatten(-1, (-1, AFFINE_GROUP))
            low, high = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
            scale = (high - low) / ((1 << bits) - 1)
            norm = torch.cat((scale, low), -1).flatten(-2)
            scale, low = scale.half().double(), low.half().double()
            code = ((y - low) / scale.clamp_min(1e-300)).round().clamp(0, (1 << bits) - 1)
            left = (y - (scale * code + low)).flatten(-2).norm(dim=-1)
        else:
            norm = x.norm(dim=-1)
            cent, bnd = (t.double() for t in _tables(case, bits))
            code = torch.bucketize(u / norm.clamp_min(1e-300)[..., None], bnd)
            left = (u - norm.half().double()[..., None] * cent[code]).norm(dim=-1) / math.sqrt(d)
        whole = s["cache"][which + "_norm"].double()
        whole[row, :, slot] = norm.transpose(1, 2)
        out[which + "_norm"], out[which + "_codes"] = whole, None
        if which == "k" and case["qjl"]:
            whole = s["cache"]["k_rnorm"].double()
            whole[row, :, slot] = left.transpose(1, 2)
            out["k_rnorm"], out["k_signs"] = whole, None
    return out
