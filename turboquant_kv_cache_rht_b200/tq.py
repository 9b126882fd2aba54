"""Python binding of libtq (ctypes).  Argument marshalling only.

Every call below forwards to the C entry point of the same name in
``include/tq.h``; all codec and attention work runs in the CUDA kernels of
``libtq.so``.  PyTorch supplies device memory (the cache, inputs, outputs and
workspace are torch tensors owned by the caller) and the current CUDA stream.

Importing this module loads ``libtq.so`` from the package directory and raises
ImportError if it has not been built (``python -m
turboquant_kv_cache_rht_b200.build``); there is no fallback implementation.
"""
from __future__ import annotations

import ctypes as C
import math
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtq.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libtq.so is not built ({_LIB_PATH}); run "
                      "`python -m turboquant_kv_cache_rht_b200.build`")
lib = C.CDLL(_LIB_PATH)

TQ_OK, TQ_ERR_INVALID, TQ_ERR_UNSUPPORTED, TQ_ERR_CUDA, TQ_ERR_CAPACITY, TQ_ERR_NOMEM = range(6)
TQ_FLAG_CAPACITY = 1
TQ_FLAG_MAXCTX = 2
TQ_FLAG_LAYOUT = 4
TQ_FLAG_INDEX = 8
TQ_FLAG_TIMEOUT = 16
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
EXPORTS = ("tq_codebook_init", "tq_codebook_tables", "tq_quantize_append", "tq_quantize_cache",
           "tq_weights_quantize", "tq_lut_matmul_workspace_bytes", "tq_lut_matmul",
           "tq_decode_workspace_bytes", "tq_decode_attention", "tq_decode_attention_noalloc",
           "tq_rope_table", "tq_rope_append", "tq_tree_workspace_bytes", "tq_tree_attention",
           "tq_cache_compact", "tq_cache_copy", "tq_free", "tq_last_error")


class tq_params(C.Structure):
    _fields_ = [("head_dim", C.c_int), ("k_bits", C.c_int), ("v_bits", C.c_int),
                ("qjl", C.c_int), ("seed", C.c_uint64), ("codebook", C.c_int)]


# TQ_CODEBOOK_GAUSSIAN, TQ_CODEBOOK_SPHERE, TQ_CODEBOOK_AFFINE
CODEBOOKS = {"gaussian": 0, "sphere": 1, "affine": 2}


class tq_layout(C.Structure):
    _fields_ = [("k_code_bytes", C.c_size_t), ("v_code_bytes", C.c_size_t),
                ("k_sign_bytes", C.c_size_t), ("norm_halves", C.c_size_t)]


class tq_cache(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("v_codes", C.c_void_p), ("k_signs", C.c_void_p),
                ("k_norm", C.c_void_p), ("v_norm", C.c_void_p), ("k_rnorm", C.c_void_p),
                ("seq_lens", C.c_void_p), ("status", C.c_void_p), ("append_sync", C.c_void_p),
                ("batch", C.c_int), ("kv_heads", C.c_int), ("capacity", C.c_int)]


class tq_rope_params(C.Structure):
    _fields_ = [("rot_dim", C.c_int), ("interleaved", C.c_int), ("scaling", C.c_int),
                ("original_max", C.c_int), ("base", C.c_double), ("factor", C.c_double),
                ("beta_fast", C.c_double), ("beta_slow", C.c_double), ("low_freq", C.c_double),
                ("high_freq", C.c_double), ("attention_factor", C.c_double)]


# TQ_ROPE_NONE, TQ_ROPE_LINEAR, TQ_ROPE_NTK, TQ_ROPE_YARN, TQ_ROPE_BANDS
ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class tq_rope(C.Structure):
    _fields_ = [("table", C.c_void_p), ("max_pos", C.c_int), ("rot_dim", C.c_int),
                ("interleaved", C.c_int)]


class tq_heads(C.Structure):
    _fields_ = [("data", C.c_void_p), ("stride_b", C.c_int64), ("stride_h", C.c_int64),
                ("stride_t", C.c_int64)]


lib.tq_codebook_init.argtypes = [C.POINTER(tq_params), C.POINTER(C.c_void_p), C.POINTER(tq_layout)]
lib.tq_codebook_init.restype = C.c_int
lib.tq_codebook_tables.argtypes = [C.c_void_p] + [C.c_void_p] * 6
lib.tq_codebook_tables.restype = C.c_int
lib.tq_quantize_append.argtypes = [C.c_void_p, C.POINTER(tq_cache), C.c_void_p, C.c_void_p,
                                   C.c_int, C.c_int, C.c_void_p]
lib.tq_quantize_append.restype = C.c_int
lib.tq_quantize_cache.argtypes = [C.c_void_p, C.POINTER(tq_cache), C.c_void_p, C.c_void_p, C.c_int,
                                  C.c_int64, C.c_int64, C.c_int64, C.c_void_p, C.c_int, C.c_void_p]
lib.tq_quantize_cache.restype = C.c_int
lib.tq_weights_quantize.argtypes = [C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                    C.c_void_p, C.c_void_p]
lib.tq_weights_quantize.restype = C.c_int
lib.tq_lut_matmul_workspace_bytes.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int]
lib.tq_lut_matmul_workspace_bytes.restype = C.c_size_t
lib.tq_lut_matmul.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p,
                              C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
lib.tq_lut_matmul.restype = C.c_int
lib.tq_decode_workspace_bytes.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int]
lib.tq_decode_workspace_bytes.restype = C.c_size_t
lib.tq_decode_attention.argtypes = [C.c_void_p, C.POINTER(tq_cache), C.c_void_p, C.c_int, C.c_int,
                                    C.c_float, C.c_int, C.c_void_p, C.c_void_p, C.c_size_t,
                                    C.c_void_p]
lib.tq_decode_attention.restype = C.c_int
lib.tq_decode_attention_noalloc.argtypes = [C.c_void_p, C.POINTER(tq_cache), C.c_void_p, C.c_int,
                                            C.c_int, C.c_float, C.c_int, C.c_void_p, C.c_void_p]
lib.tq_decode_attention_noalloc.restype = C.c_int
lib.tq_rope_table.argtypes = [C.POINTER(tq_rope_params), C.c_int, C.c_void_p, C.c_void_p]
lib.tq_rope_table.restype = C.c_int
lib.tq_rope_append.argtypes = [C.c_void_p, C.POINTER(tq_cache), C.POINTER(tq_rope), C.POINTER(tq_heads),
                               C.c_int, C.POINTER(tq_heads), C.POINTER(tq_heads), C.c_int, C.c_int,
                               C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]
lib.tq_rope_append.restype = C.c_int
lib.tq_tree_workspace_bytes.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int]
lib.tq_tree_workspace_bytes.restype = C.c_size_t
lib.tq_tree_attention.argtypes = [C.c_void_p, C.POINTER(tq_cache), C.c_void_p, C.c_int, C.c_int, C.c_int,
                                  C.c_void_p, C.c_int64, C.c_float, C.c_int, C.c_void_p, C.c_void_p,
                                  C.c_size_t, C.c_void_p]
lib.tq_tree_attention.restype = C.c_int
lib.tq_cache_compact.argtypes = [C.c_void_p, C.POINTER(tq_cache), C.c_void_p, C.c_int64, C.c_int64,
                                 C.c_void_p, C.c_int, C.c_void_p, C.c_void_p]
lib.tq_cache_compact.restype = C.c_int
lib.tq_cache_copy.argtypes = [C.c_void_p, C.POINTER(tq_cache), C.POINTER(tq_cache), C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_int, C.c_int, C.c_void_p]
lib.tq_cache_copy.restype = C.c_int
lib.tq_free.argtypes = [C.c_void_p]
lib.tq_free.restype = None
lib.tq_last_error.argtypes = []
lib.tq_last_error.restype = C.c_char_p


class TQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status}: {tq_last_error()}")


def tq_last_error() -> str:
    return lib.tq_last_error().decode()


def _check(st: int, where: str):
    if st != TQ_OK:
        raise TQError(st, where)


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def kv_bits_split(kv_bits: float) -> tuple[int, int]:
    """Key/value widths for a fractional kv_bits (3.5 -> 3-bit keys, 4-bit values)."""
    return int(math.floor(kv_bits + 1e-9)), int(math.ceil(kv_bits - 1e-9))


class Codebook:
    """Owner of a tq_codebook handle (host memory; freed with tq_free)."""

    def __init__(self, head_dim: int, k_bits: int, v_bits: int, qjl: bool = False, seed: int = 0,
                 codebook: str = "gaussian"):
        """codebook: "gaussian" (Lloyd-Max for N(0,1)), "sphere" (Lloyd-Max for
        the exact distribution of a rotated coordinate, which depends on head_dim)
        or "affine" (the affine group-64 comparison codec: rotated keys, fp16
        scale and bias per group of 64 channels)."""
        if codebook not in CODEBOOKS:
            raise ValueError(f"codebook must be one of {sorted(CODEBOOKS)}")
        self.params = tq_params(head_dim, k_bits, v_bits, int(bool(qjl)), seed & ((1 << 64) - 1),
                                CODEBOOKS[codebook])
        self.layout = tq_layout()
        h = C.c_void_p()
        _check(lib.tq_codebook_init(C.byref(self.params), C.byref(h), C.byref(self.layout)),
               "tq_codebook_init")
        self.handle = h
        # elements of one slot: key codes, value codes, norms (or scales and biases), signs
        lay = self.layout
        self.slot_elements = (lay.k_code_bytes, lay.v_code_bytes, lay.norm_halves, lay.k_sign_bytes)

    @classmethod
    def from_kv_bits(cls, head_dim: int, kv_bits: float, qjl: bool = False, seed: int = 0,
                     codebook: str = "gaussian"):
        kb, vb = kv_bits_split(kv_bits)
        return cls(head_dim, kb, vb, qjl, seed, codebook)

    head_dim = property(lambda self: self.params.head_dim)
    k_bits = property(lambda self: self.params.k_bits)
    v_bits = property(lambda self: self.params.v_bits)
    qjl = property(lambda self: bool(self.params.qjl))
    affine = property(lambda self: self.params.codebook == CODEBOOKS["affine"])

    def tables(self) -> dict:
        """Host copies of the codebooks and rotation signs (tq_codebook_tables)."""
        lk, lv, d = 1 << self.k_bits, 1 << self.v_bits, self.head_dim
        kc, kb = (C.c_float * lk)(), (C.c_float * (lk - 1))()
        vc, vb = (C.c_float * lv)(), (C.c_float * (lv - 1))()
        s1, s2 = (C.c_int8 * d)(), (C.c_int8 * d)()
        _check(lib.tq_codebook_tables(self.handle, kc, kb, vc, vb, s1, s2), "tq_codebook_tables")
        to = lambda a, dt: torch.tensor(list(a), dtype=dt)
        return {"k_centroids": to(kc, torch.float32), "k_boundaries": to(kb, torch.float32),
                "v_centroids": to(vc, torch.float32), "v_boundaries": to(vb, torch.float32),
                "signs1": to(s1, torch.int8), "signs2": to(s2, torch.int8)}

    def __del__(self, _free=lib.tq_free):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            _free(h)
            self.handle = None


class Cache:
    """A compressed KV cache held in torch tensors (the caller owns them)."""

    def __init__(self, cb: Codebook, batch: int, kv_heads: int, capacity: int, device="cuda"):
        lay = cb.layout
        n = (batch, kv_heads, capacity)
        u8 = dict(dtype=torch.uint8, device=device)
        self.batch, self.kv_heads, self.capacity = batch, kv_heads, capacity
        self.k_codes = torch.zeros(*n, lay.k_code_bytes, **u8)
        self.v_codes = torch.zeros(*n, lay.v_code_bytes, **u8)
        self.k_signs = torch.zeros(*n, lay.k_sign_bytes, **u8) if cb.qjl else None
        # one fp16 norm per vector, or (scale, bias) per group for the affine codec
        nh = (lay.norm_halves,) if cb.affine else ()
        self.k_norm = torch.zeros(*n, *nh, dtype=torch.float16, device=device)
        self.v_norm = torch.zeros(*n, *nh, dtype=torch.float16, device=device)
        self.k_rnorm = torch.zeros(n, dtype=torch.float16, device=device) if cb.qjl else None
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.append_sync = torch.zeros(batch, dtype=torch.int32, device=device)

    def struct(self) -> tq_cache:
        p = lambda t: None if t is None else t.data_ptr()
        return tq_cache(p(self.k_codes), p(self.v_codes), p(self.k_signs), p(self.k_norm),
                        p(self.v_norm), p(self.k_rnorm), p(self.seq_lens), p(self.status),
                        p(self.append_sync), self.batch, self.kv_heads, self.capacity)

    def tensors(self) -> tuple:
        """Every array that it has."""
        ts = (self.k_codes, self.v_codes, self.k_signs, self.k_norm, self.v_norm, self.k_rnorm, self.seq_lens,
              self.status, self.append_sync)
        return tuple(t for t in ts if t is not None)

    def nbytes(self) -> int:
        ts = [self.k_codes, self.v_codes, self.k_signs, self.k_norm, self.v_norm, self.k_rnorm]
        return sum(t.numel() * t.element_size() for t in ts if t is not None)


def _on_device(where: str, device: torch.device, **tensors) -> None:
    """The library takes device pointers: every tensor handed to it must be a
    CUDA tensor on the device of the cache (or of the encoded weights)."""
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device != device):
            raise ValueError(f"{where}: {name} must be a CUDA tensor on {device}, not on {t.device}")


def _check_out(where: str, out: torch.Tensor, shape) -> None:
    if out.dtype != torch.float32 or tuple(out.shape) != tuple(shape) or not out.is_contiguous():
        raise ValueError(f"{where}: out must be a contiguous float32 tensor of shape {tuple(shape)}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def tq_quantize_append(cb: Codebook, cache: Cache, k: torch.Tensor, v: torch.Tensor,
                       stream=None) -> None:
    """k, v: [batch, kv_heads, n_new, head_dim] contiguous CUDA tensors of one dtype."""
    if k.shape != v.shape or k.dtype != v.dtype or k.dim() != 4:
        raise ValueError("k and v must be [batch, kv_heads, n_new, head_dim] of one dtype")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous")
    if k.shape[0] != cache.batch or k.shape[1] != cache.kv_heads or k.shape[3] != cb.head_dim:
        raise ValueError(f"k shape {tuple(k.shape)} does not match the cache")
    _on_device("tq_quantize_append", cache.seq_lens.device, cache=cache.seq_lens, k=k, v=v)
    cs = cache.struct()
    _check(lib.tq_quantize_append(cb.handle, C.byref(cs), k.data_ptr(), v.data_ptr(),
                                  _dtype_code(k), k.shape[2], _stream_ptr(stream)),
           "tq_quantize_append")


def tq_quantize_cache(cb: Codebook, cache: Cache, k: torch.Tensor, v: torch.Tensor,
                      lengths: torch.Tensor | None = None, stream=None) -> None:
    """Convert a dense cache: k, v are [batch, kv_heads, T, head_dim] CUDA tensors
    of one dtype with unit channel stride and any other strides (a view of a
    [batch, T, kv_heads, head_dim] cache transposed works in place); lengths is
    an int32 CUDA tensor [batch] (default: T for every row).  Sets seq_lens."""
    if k.shape != v.shape or k.dtype != v.dtype or k.dim() != 4:
        raise ValueError("k and v must be [batch, kv_heads, T, head_dim] of one dtype")
    if k.stride() != v.stride() or k.stride(3) != 1:
        raise ValueError("k and v must share strides, with unit channel stride")
    if k.shape[0] != cache.batch or k.shape[1] != cache.kv_heads or k.shape[3] != cb.head_dim:
        raise ValueError(f"k shape {tuple(k.shape)} does not match the cache")
    T = k.shape[2]
    if lengths is None:
        lengths = torch.full((cache.batch,), T, dtype=torch.int32, device=k.device)
    if lengths.dtype != torch.int32 or lengths.shape != (cache.batch,) or not lengths.is_contiguous():
        raise ValueError("lengths must be a contiguous int32 tensor [batch]")
    _on_device("tq_quantize_cache", cache.seq_lens.device, cache=cache.seq_lens, k=k, v=v,
               lengths=lengths)
    cs = cache.struct()
    _check(lib.tq_quantize_cache(cb.handle, C.byref(cs), k.data_ptr(), v.data_ptr(), _dtype_code(k),
                                 k.stride(0), k.stride(1), k.stride(2), lengths.data_ptr(), T,
                                 _stream_ptr(stream)),
           "tq_quantize_cache")


def tq_lut_matmul_workspace_bytes(cb: Codebook, rows: int, k: int, m: int) -> int:
    return int(lib.tq_lut_matmul_workspace_bytes(cb.handle, rows, k, m))


class QuantizedWeights:
    """A weight matrix [rows, k] encoded block by block (blocks of head_dim input
    channels, the key codec): codes [k/d, rows, k_bits*d/8], fp16 norms [k/d, rows]."""

    def __init__(self, cb: Codebook, w: torch.Tensor, stream=None):
        if w.dim() != 2 or not w.is_contiguous():
            raise ValueError("w must be a contiguous [rows, k] CUDA tensor")
        _on_device("tq_weights_quantize", w.device, w=w)
        self.cb, (self.rows, self.k) = cb, w.shape
        nb = self.k // cb.head_dim
        self.codes = torch.empty(nb, self.rows, cb.layout.k_code_bytes, dtype=torch.uint8, device=w.device)
        self.norms = torch.empty(nb, self.rows, dtype=torch.float16, device=w.device)
        _check(lib.tq_weights_quantize(cb.handle, w.data_ptr(), _dtype_code(w), self.rows, self.k,
                                       self.codes.data_ptr(), self.norms.data_ptr(), _stream_ptr(stream)),
               "tq_weights_quantize")

    def copy(self) -> "QuantizedWeights":
        """A second copy of the encoded weights (new device buffers)."""
        c = QuantizedWeights.__new__(QuantizedWeights)
        c.cb, c.rows, c.k = self.cb, self.rows, self.k
        c.codes, c.norms = self.codes.clone(), self.norms.clone()
        return c

    def matmul(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        """x [m, k] CUDA tensor -> float32 [m, rows] = x W_hat^T."""
        if x.dim() != 2 or x.shape[1] != self.k or not x.is_contiguous():
            raise ValueError(f"x must be a contiguous [m, {self.k}] tensor")
        _on_device("tq_lut_matmul", self.codes.device, x=x)
        m = x.shape[0]
        y = torch.empty(m, self.rows, dtype=torch.float32, device=x.device)
        nbytes = tq_lut_matmul_workspace_bytes(self.cb, self.rows, self.k, m)
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
        _check(lib.tq_lut_matmul(self.cb.handle, self.codes.data_ptr(), self.norms.data_ptr(), self.rows,
                                 self.k, x.data_ptr(), _dtype_code(x), m, y.data_ptr(), ws.data_ptr(),
                                 nbytes, _stream_ptr(stream)),
               "tq_lut_matmul")
        return y


def tq_decode_workspace_bytes(cb: Codebook, batch: int, q_heads: int, kv_heads: int,
                              max_ctx: int) -> int:
    return int(lib.tq_decode_workspace_bytes(cb.handle, batch, q_heads, kv_heads, max_ctx))


def tq_decode_attention(cb: Codebook, cache: Cache, q: torch.Tensor, out: torch.Tensor | None = None,
                        softmax_scale: float = 0.0, max_ctx: int | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q: [batch, q_heads, head_dim] CUDA tensor; returns float32 [batch, q_heads, head_dim]."""
    if q.dim() != 3 or q.shape[0] != cache.batch or q.shape[2] != cb.head_dim or not q.is_contiguous():
        raise ValueError("q must be contiguous [batch, q_heads, head_dim]")
    hq = q.shape[1]
    max_ctx = cache.capacity if max_ctx is None else max_ctx
    _on_device("tq_decode_attention", cache.seq_lens.device, cache=cache.seq_lens, q=q, out=out,
               workspace=workspace)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    _check_out("tq_decode_attention", out, q.shape)
    if workspace is None:   # (the library checks a caller's workspace size itself)
        need = tq_decode_workspace_bytes(cb, cache.batch, hq, cache.kv_heads, max_ctx)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous():
        raise ValueError("tq_decode_attention: workspace must be contiguous")
    cs = cache.struct()
    _check(lib.tq_decode_attention(cb.handle, C.byref(cs), q.data_ptr(), _dtype_code(q), hq,
                                   float(softmax_scale), int(max_ctx), out.data_ptr(),
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _stream_ptr(stream)),
           "tq_decode_attention")
    return out


def tq_decode_attention_noalloc(cb: Codebook, cache: Cache, q: torch.Tensor,
                                out: torch.Tensor | None = None, softmax_scale: float = 0.0,
                                max_ctx: int | None = None, stream=None) -> torch.Tensor:
    """tq_decode_attention without a workspace, for callers that cannot
    allocate device memory: the library's built-in static scratch (8 MiB) is
    used instead.  Calls share that scratch, so they must not overlap on the
    GPU; make the first call on a device before any stream capture.  `out`
    should be passed by such callers (allocating it here is only a
    convenience)."""
    if q.dim() != 3 or q.shape[0] != cache.batch or q.shape[2] != cb.head_dim or not q.is_contiguous():
        raise ValueError("q must be contiguous [batch, q_heads, head_dim]")
    max_ctx = cache.capacity if max_ctx is None else max_ctx
    _on_device("tq_decode_attention_noalloc", cache.seq_lens.device, cache=cache.seq_lens, q=q,
               out=out)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    _check_out("tq_decode_attention_noalloc", out, q.shape)
    cs = cache.struct()
    _check(lib.tq_decode_attention_noalloc(cb.handle, C.byref(cs), q.data_ptr(), _dtype_code(q),
                                           q.shape[1], float(softmax_scale), int(max_ctx),
                                           out.data_ptr(), _stream_ptr(stream)),
           "tq_decode_attention_noalloc")
    return out


# ---------------------------------------------------------------------------
# Speculative decoding over the compressed cache
# ---------------------------------------------------------------------------
class _on:
    """The device and stream of one call: a context in which the cache's device is
    current and what the call allocates belongs to the stream it runs on; it gives
    the stream's address.  Nothing is switched where both are current already.  Where
    the caller names a stream, the call's tensors (and its caches') are marked as used
    there, so that memory dropped after the call is not handed out again before it."""

    __slots__ = ("entered", "index")

    def __init__(self, device: torch.device, stream, *used):
        self.entered, self.index = (), device.index
        if stream is None and device.index == torch._C._cuda_getDevice():
            return
        self.entered = []
        if device.index != torch.cuda.current_device():
            self.entered.append(torch.cuda.device(device))
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self.entered.append(torch.cuda.stream(stream))
            for x in used:
                for t in x.tensors() if isinstance(x, Cache) else (x,):
                    if isinstance(t, torch.Tensor):
                        t.record_stream(stream)

    def __enter__(self) -> int:
        for c in self.entered:
            c.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.entered:
            for c in reversed(self.entered):
                c.__exit__(*exc)


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _refuse_device(where: str, name: str, t: torch.Tensor, device: torch.device):
    raise ValueError(f"{where}: {name} must be a CUDA tensor on {device}, not on {t.device}")


def _index_ptr(where: str, name: str, t: torch.Tensor | None, shape: tuple, device: torch.device):
    """The address of an int32 argument of this shape, None for none."""
    if t is None:
        return None
    if t.device != device:
        _refuse_device(where, name, t, device)
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous int32 tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _cache_struct(where: str, cb: Codebook, cache: Cache, device: torch.device) -> tq_cache:
    """The cache's arrays, each of its type, as large as the codebook asks for,
    contiguous and on the cache's device.  (Written out: it runs on every call.)"""
    if device.type != "cuda":
        _refuse_device(where, "cache", cache.seq_lens, device)
    i, (kb, vb, meta, sb) = device.index, cb.slot_elements
    b, h, c = cache.batch, cache.kv_heads, cache.capacity
    n = b * h * c
    kc, vc, kn, vn = cache.k_codes, cache.v_codes, cache.k_norm, cache.v_norm
    sl, st, sy = cache.seq_lens, cache.status, cache.append_sync
    try:
        good = (kc.numel() == n * kb and vc.numel() == n * vb and kn.numel() == vn.numel() == n * meta and
                sl.numel() == sy.numel() == b and st.numel() == 1 and
                kc.dtype is vc.dtype is torch.uint8 and kn.dtype is vn.dtype is torch.float16 and
                sl.dtype is sy.dtype is st.dtype is torch.int32 and
                kc.get_device() == vc.get_device() == kn.get_device() == vn.get_device() == sl.get_device() ==
                st.get_device() == sy.get_device() == i and
                kc.is_contiguous() and vc.is_contiguous() and kn.is_contiguous() and vn.is_contiguous() and
                sl.is_contiguous() and sy.is_contiguous())
        ks = kr = None
        if good and sb:
            ks, kr = cache.k_signs, cache.k_rnorm
            good = (ks.numel() == n * sb and kr.numel() == n and ks.dtype is torch.uint8 and
                    kr.dtype is torch.float16 and ks.get_device() == kr.get_device() == i and
                    ks.is_contiguous() and kr.is_contiguous())
            ks, kr = ks.data_ptr(), kr.data_ptr()
    except AttributeError:   # an array is None
        good = False
    if not good:
        raise ValueError(f"{where}: the cache's arrays must be contiguous tensors of the codebook's sizes and "
                         f"types on {device}")
    return tq_cache(kc.data_ptr(), vc.data_ptr(), ks, kn.data_ptr(), vn.data_ptr(), kr, sl.data_ptr(),
                    st.data_ptr(), sy.data_ptr(), b, h, c)


class Rope:
    """Rotary positions: the cosines and sines of ``max_pos`` positions for the
    first ``rot_dim`` channels of a head (tq_rope_table), kept on the device."""

    def __init__(self, rot_dim: int, max_pos: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: str | None = None, factor: float = 1.0, original_max: int = 0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, low_freq: float = 1.0,
                 high_freq: float = 4.0, attention_factor: float | None = None, device="cuda",
                 stream=None):
        """scaling: None, "linear", "ntk", "yarn" or "bands" (tq_rope_params gives the
        formulas); attention_factor multiplies cosine and sine (None: 0.1 ln(factor) + 1
        for yarn, else 1); interleaved pairs channels (2i, 2i + 1) instead of
        (i, i + rot_dim / 2)."""
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be None or one of {sorted(k for k in ROPE_SCALINGS if k)}")
        self.params = tq_rope_params(rot_dim, int(bool(interleaved)), ROPE_SCALINGS[scaling], original_max,
                                     base, factor, beta_fast, beta_slow, low_freq, high_freq,
                                     attention_factor or 0.0)
        self.rot_dim, self.max_pos, self.interleaved = rot_dim, max_pos, bool(interleaved)
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"Rope: the table lives on a CUDA device, not on {device}")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        with _on(device, stream) as s:
            self.table = torch.empty(max(max_pos, 1), max(rot_dim // 2, 1), 2, dtype=torch.float32, device=device)
            _check(lib.tq_rope_table(C.byref(self.params), max_pos, self.table.data_ptr(), s), "tq_rope_table")

    def struct(self) -> tq_rope:
        return tq_rope(self.table.data_ptr(), self.max_pos, self.rot_dim, int(self.interleaved))


def _heads(where: str, name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype,
           device: torch.device) -> tq_heads:
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{where}: {name} must be [batch, heads, n_new, head_dim] of one dtype, matching the cache")
    if t.device != device:
        _refuse_device(where, name, t, device)
    sb, sh, st, sc = t.stride()
    if sc != 1:
        raise ValueError(f"{where}: {name} must have a unit channel stride")
    b, h, n, _ = shape   # the stride of a dimension of one is free
    return tq_heads(t.data_ptr(), sb if b > 1 else 0, sh if h > 1 else 0, st if n > 1 else 0)


def tq_rope_append(cb: Codebook, cache: Cache, rope: Rope, k: torch.Tensor, v: torch.Tensor,
                   q: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                   relative: bool = False, start: torch.Tensor | None = None,
                   keys_out: bool | torch.Tensor = False, q_out: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor | None, torch.Tensor | None]:
    """tq_quantize_append with rotary positions.

    k, v: [batch, kv_heads, n_new, head_dim] and q: [batch, q_heads, n_new, head_dim]
    CUDA tensors of one dtype with unit channel stride and any other strides (views
    of a fused projection work in place).  positions: int32 [batch, n_new] (default:
    consecutive from the row's start); relative adds the row's start to them.
    start: int32 [batch], the slot of each row's first new token (default: seq_lens).
    Returns (rotated q [batch, n_new, q_heads, head_dim] or None, rotated k
    [batch, n_new, kv_heads, head_dim] if keys_out, else None)."""
    where, dev = "tq_rope_append", cache.seq_lens.device
    if k.dim() != 4 or k.shape[3] != cb.head_dim:
        raise ValueError(f"{where}: k must be [batch, kv_heads, n_new, head_dim {cb.head_dim}]")
    b, hk, n, d = shape = (cache.batch, cache.kv_heads, k.shape[2], cb.head_dim)
    dtype, hq = k.dtype, 0
    code = _dtype_code(k)
    kv = _heads(where, "k", k, shape, dtype, dev)
    vv = _heads(where, "v", v, shape, dtype, dev)
    qv = None
    if q is not None:
        hq = q.shape[1] if q.dim() == 4 else 0
        qv = _heads(where, "q", q, (b, hq, n, d), dtype, dev)
    if rope.table.device != dev:
        _refuse_device(where, "rope", rope.table, dev)
    pos = _index_ptr(where, "positions", positions, (b, n), dev)
    begin = _index_ptr(where, "start", start, (b,), dev)
    cs = _cache_struct(where, cb, cache, dev)
    with _on(dev, stream, cache, rope.table, k, v, q, positions, start, q_out, keys_out) as s:
        if q is None:
            q_out = None
        elif q_out is None:
            q_out = torch.empty((b, n, hq, d), dtype=dtype, device=dev)
        else:
            _check_like(where, "q_out", q_out, (b, n, hq, d), dtype, dev)
        k_out = None
        if isinstance(keys_out, torch.Tensor):
            k_out = keys_out
            _check_like(where, "keys_out", k_out, (b, n, hk, d), dtype, dev)
        elif keys_out:
            k_out = torch.empty((b, n, hk, d), dtype=dtype, device=dev)
        _check(lib.tq_rope_append(cb.handle, cs, rope.struct(), qv, hq, kv, vv, code, n, pos, int(bool(relative)), begin,
                                  _ptr(q_out), _ptr(k_out), s), where)
    return q_out, k_out


def _check_like(where: str, name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, device: torch.device):
    if t.device != device:
        _refuse_device(where, name, t, device)
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous {dtype} tensor {tuple(shape)}")


def pack_tree_mask(sees: torch.Tensor) -> torch.Tensor:
    """bool [..., n, n] (draft i attends draft j) -> the int32 words [..., n, ceil(n / 32)]
    that tq_tree_attention takes."""
    if sees.dtype != torch.bool or sees.dim() < 2 or sees.shape[-1] != sees.shape[-2]:
        raise ValueError("sees must be a bool tensor [..., n, n]")
    n = sees.shape[-1]
    words = (n + 31) // 32
    bits = torch.zeros(*sees.shape[:-1], 32 * words, dtype=torch.int64, device=sees.device)
    bits[..., :n] = sees
    w = (bits.unflatten(-1, (words, 32)) << torch.arange(32, device=sees.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def tq_tree_workspace_bytes(cb: Codebook, batch: int, q_heads: int, kv_heads: int, n_q: int, max_ctx: int) -> int:
    return int(lib.tq_tree_workspace_bytes(cb.handle, batch, q_heads, kv_heads, n_q, max_ctx))


def tq_tree_attention(cb: Codebook, cache: Cache, q: torch.Tensor, mask: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, softmax_scale: float = 0.0, max_ctx: int | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of the n_q tokens appended last: q [batch, n_q, q_heads, head_dim], a
    contiguous bf16 or fp16 CUDA tensor; mask int32 [n_q, ceil(n_q / 32)] or one per
    batch row (pack_tree_mask), None for a chain.  Returns q's shape and dtype."""
    where, dev = "tq_tree_attention", cache.seq_lens.device
    if q.dim() != 4 or q.shape[0] != cache.batch or q.shape[3] != cb.head_dim or not q.is_contiguous():
        raise ValueError(f"{where}: q must be contiguous [batch, n_q, q_heads, head_dim]")
    dtype = q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"{where}: q must be bfloat16 or float16, not {dtype}")
    if q.device != dev or dev.type != "cuda":
        _refuse_device(where, "q" if dev.type == "cuda" else "cache", q, dev)
    b, n, hq, _ = shape = q.shape
    max_ctx = cache.capacity if max_ctx is None else max_ctx
    bits, stride = None, 0
    if mask is not None:
        words = (n + 31) // 32
        bits = _index_ptr(where, "mask", mask, (n, words) if mask.dim() == 2 else (b, n, words), dev)
        stride = 0 if mask.dim() == 2 else n * words
    cs = _cache_struct(where, cb, cache, dev)
    with _on(dev, stream, cache, q, mask, out, workspace) as s:
        if out is None:
            out = torch.empty_like(q)
        else:
            _check_like(where, "out", out, shape, dtype, dev)
        if workspace is None:
            need = tq_tree_workspace_bytes(cb, b, hq, cache.kv_heads, n, max_ctx)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        elif workspace.device != dev:
            _refuse_device(where, "workspace", workspace, dev)
        elif not workspace.is_contiguous():
            raise ValueError(f"{where}: workspace must be contiguous")
        _check(lib.tq_tree_attention(cb.handle, cs, q.data_ptr(), _DTYPES[dtype], hq, n, bits, stride,
                                     softmax_scale, max_ctx, out.data_ptr(), workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), s), where)
    return out


def tq_cache_compact(cb: Codebook, cache: Cache, index: torch.Tensor, counts: torch.Tensor,
                     start: torch.Tensor | None = None, stream=None) -> None:
    """Keep slots start + index[b, (h,) i], i < counts[b], of every row, in order, and
    free the others: seq_lens becomes start + counts.  index int32 [batch, n] or
    [batch, kv_heads, n], ascending; counts int32 [batch]; start int32 [batch] (default 0)."""
    where, dev = "tq_cache_compact", cache.seq_lens.device
    b, h = cache.batch, cache.kv_heads
    if index.dim() not in (2, 3):
        raise ValueError(f"{where}: index must be [batch, n] or [batch, kv_heads, n]")
    n = index.shape[-1]
    per_head = index.dim() == 3
    cs = _cache_struct(where, cb, cache, dev)
    at = _index_ptr(where, "index", index, (b, h, n) if per_head else (b, n), dev)
    num = _index_ptr(where, "counts", counts, (b,), dev)
    begin = _index_ptr(where, "start", start, (b,), dev)
    with _on(dev, stream, cache, index, counts, start) as s:
        _check(lib.tq_cache_compact(cb.handle, cs, at, h * n if per_head else n, n if per_head else 0, num, n, begin, s),
               where)


def tq_cache_copy(cb: Codebook, dst: Cache, src: Cache, dst_rows: torch.Tensor, src_rows: torch.Tensor,
                  lengths: torch.Tensor | None = None, max_len: int | None = None, stream=None) -> None:
    """Row dst_rows[i] of dst becomes the first lengths[i] tokens (default: all) of row
    src_rows[i] of src; dst and src may be one cache.  Row lists and lengths are int32
    CUDA tensors [n]; max_len bounds the lengths (default: src's capacity)."""
    where, dev = "tq_cache_copy", dst.seq_lens.device
    if dst_rows.dim() != 1:
        raise ValueError(f"{where}: dst_rows must be [n]")
    n = dst_rows.shape[0]
    if src.seq_lens.device != dev:
        _refuse_device(where, "src", src.seq_lens, dev)
    cd = _cache_struct(where, cb, dst, dev)
    cs = cd if src is dst else _cache_struct(where, cb, src, dev)
    to = _index_ptr(where, "dst_rows", dst_rows, (n,), dev)
    come = _index_ptr(where, "src_rows", src_rows, (n,), dev)
    lens = _index_ptr(where, "lengths", lengths, (n,), dev)
    with _on(dev, stream, dst, src, dst_rows, src_rows, lengths) as s:
        _check(lib.tq_cache_copy(cb.handle, cd, cs, to, come, lens, n, src.capacity if max_len is None else max_len, s),
               where)


def tq_free(cb: Codebook) -> None:
    """Release a codebook's handle before the object's own end; it cannot be used afterwards."""
    cb.__del__()
