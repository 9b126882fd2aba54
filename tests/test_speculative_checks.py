"""Argument checks of the speculative-decoding calls (CPU only): the binding's, and
the library's own on addresses that it never reads."""
import ctypes as C

import pytest
import torch

from turboquant_kv_cache_rht_b200 import tq

FAKE = 0x10000


def _cache(**kw):
    a = dict(k_codes=FAKE, v_codes=FAKE, k_signs=None, k_norm=FAKE, v_norm=FAKE, k_rnorm=None, seq_lens=FAKE,
             status=FAKE, append_sync=FAKE, batch=2, kv_heads=2, capacity=64)
    a.update(kw)
    return tq.tq_cache(*a.values())


def _refused(status, needle, want=tq.TQ_ERR_INVALID):
    assert status == want, tq.tq_last_error()
    assert needle in tq.tq_last_error()


def _params(**kw):
    p = dict(rot_dim=128, interleaved=0, scaling=0, original_max=4096, base=1e4, factor=1.0, beta_fast=32.0,
             beta_slow=1.0, low_freq=1.0, high_freq=4.0, attention_factor=0.0)
    p.update(kw)
    return tq.tq_rope_params(*p.values())


@pytest.mark.parametrize("kw,needle", [
    (dict(rot_dim=0), "rot_dim"), (dict(rot_dim=7), "rot_dim"), (dict(rot_dim=258), "rot_dim"),
    (dict(scaling=5), "scaling"), (dict(scaling=-1), "scaling"), (dict(base=1.0), "base"),
    (dict(base=float("nan")), "base"), (dict(base=float("inf")), "base"), (dict(scaling=1, factor=0.5), "factor"),
    (dict(scaling=2, factor=float("nan")), "factor"), (dict(scaling=3, original_max=0), "original_max"),
    (dict(scaling=4, original_max=0), "original_max"), (dict(scaling=3, beta_fast=1.0), "beta_fast"),
    (dict(scaling=3, beta_slow=0.0), "beta_fast"), (dict(scaling=4, low_freq=4.0), "high_freq"),
    (dict(attention_factor=-1.0), "attention_factor"), (dict(attention_factor=float("inf")), "attention_factor")])
def test_rope_table_refusals(kw, needle):
    _refused(tq.lib.tq_rope_table(C.byref(_params(**kw)), 16, FAKE, None), needle)


def test_rope_table_arguments():
    _refused(tq.lib.tq_rope_table(None, 16, FAKE, None), "params")
    _refused(tq.lib.tq_rope_table(C.byref(_params()), 16, None, None), "table")
    _refused(tq.lib.tq_rope_table(C.byref(_params()), 16, FAKE + 4, None), "aligned")
    _refused(tq.lib.tq_rope_table(C.byref(_params()), 0, FAKE, None), "max_pos")
    with pytest.raises(ValueError):
        tq.Rope(128, 16, scaling="other")
    with pytest.raises(ValueError):
        tq.Rope(128, 16, device="cpu")


def _append(cache=None, rope=None, k=None, v=None, q=None, q_heads=4, dtype=1, n=4, positions=None, start=None,
            q_out=FAKE, k_out=None, cb=None):
    cb = cb or tq.Codebook(128, 3, 4)
    h = lambda **kw: tq.tq_heads(*{**dict(data=FAKE, b=2048, h=512, t=128), **kw}.values())
    k, v, q = (h(**(x or {})) for x in (k, v, q))
    rope = rope or tq.tq_rope(FAKE, 4096, 128, 0)
    return tq.lib.tq_rope_append(cb.handle, C.byref(cache or _cache()), C.byref(rope), C.byref(q), q_heads, C.byref(k),
                                 C.byref(v), dtype, n, positions, 0, start, q_out, k_out, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(cache=_cache(capacity=40)), "multiple of 16"), (dict(rope=tq.tq_rope(None, 4096, 128, 0)), "rope"),
    (dict(rope=tq.tq_rope(FAKE, 4096, 130, 0)), "rot_dim"), (dict(rope=tq.tq_rope(FAKE, 4096, 0, 0)), "rot_dim"),
    (dict(rope=tq.tq_rope(FAKE, 0, 128, 0)), "max_pos"), (dict(rope=tq.tq_rope(FAKE + 8, 16, 128, 0)), "aligned"),
    (dict(n=-1), "negative"), (dict(n=65), "capacity"), (dict(dtype=3), "dtype"), (dict(q_heads=0), "q_heads"),
    (dict(k=dict(data=None)), "NULL"), (dict(v=dict(data=None)), "NULL"), (dict(q=dict(data=None)), "q needs"),
    (dict(q_out=None), "q needs"), (dict(k=dict(t=129)), "strides of k"), (dict(v=dict(h=4)), "strides of v"),
    (dict(q=dict(b=-8)), "negative stride"), (dict(k=dict(data=FAKE + 2)), "k must be"),
    (dict(q_out=FAKE + 8), "q_out"), (dict(k_out=FAKE + 8), "q_out"), (dict(positions=FAKE + 2), "4-byte"),
    (dict(start=FAKE + 1), "4-byte")])
def test_rope_append_refusals(kw, needle):
    _refused(_append(**kw), needle)


def test_rope_append_of_nothing():
    assert _append(n=0) == tq.TQ_OK


def _tree(cb=None, cache=None, q=FAKE, dtype=1, q_heads=8, n=4, mask=None, stride=0, scale=0.0, max_ctx=64, out=FAKE,
          ws=FAKE, nbytes=1 << 40):
    cb = cb or tq.Codebook(128, 3, 4)
    return tq.lib.tq_tree_attention(cb.handle, C.byref(cache or _cache()), q, dtype, q_heads, n, mask, stride, scale,
                                    max_ctx, out, ws, nbytes, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(dtype=0), "bf16 or fp16"), (dict(dtype=9), "bf16 or fp16"),
    (dict(n=0), "n_q"), (dict(n=257), "n_q"), (dict(q_heads=0), "q_heads"), (dict(q_heads=7), "q_heads"),
    (dict(max_ctx=-1), "max_ctx"), (dict(max_ctx=65), "max_ctx"), (dict(q=FAKE + 8), "aligned"),
    (dict(out=FAKE + 8), "aligned"), (dict(mask=FAKE + 2), "aligned"), (dict(mask=FAKE, stride=3), "mask_stride"),
    (dict(mask=FAKE, stride=-4), "mask_stride"), (dict(scale=float("nan")), "softmax_scale")])
def test_tree_refusals(kw, needle):
    _refused(_tree(**kw), needle)


def test_tree_shapes_without_a_kernel():
    _refused(_tree(q_heads=6), "group", tq.TQ_ERR_UNSUPPORTED)
    _refused(_tree(cb=tq.Codebook(128, 4, 2)), "v_bits", tq.TQ_ERR_UNSUPPORTED)


def test_tree_workspace():
    cb = tq.Codebook(128, 3, 4)
    size = lambda **kw: tq.tq_tree_workspace_bytes(cb, *{**dict(batch=2, q_heads=8, kv_heads=2, n_q=4, max_ctx=64), **kw}.values())
    for bad in (dict(batch=0), dict(q_heads=0), dict(q_heads=7), dict(kv_heads=0), dict(n_q=0), dict(n_q=257), dict(max_ctx=-1)):
        assert size(**bad) == 0
    need = size()
    if need:
        _refused(_tree(nbytes=need - 1), "workspace", tq.TQ_ERR_CAPACITY)
        _refused(_tree(ws=None), "workspace", tq.TQ_ERR_CAPACITY)
        _refused(_tree(ws=FAKE + 4), "aligned")


def _compact(cache=None, index=FAKE, sb=8, sh=0, counts=FAKE, n=8, start=None):
    cb = tq.Codebook(128, 3, 4)
    return tq.lib.tq_cache_compact(cb.handle, C.byref(cache or _cache()), index, sb, sh, counts, n, start, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(index=None), "NULL"), (dict(counts=None), "NULL"), (dict(n=-1), "max_count"), (dict(n=65), "max_count"),
    (dict(sb=-1), "stride"), (dict(sh=-1), "stride"), (dict(index=FAKE + 2), "4-byte"), (dict(counts=FAKE + 2), "4-byte"),
    (dict(start=FAKE + 2), "4-byte"), (dict(cache=_cache(kv_heads=70000)), "kv_heads")])
def test_compact_refusals(kw, needle):
    _refused(_compact(**kw), needle)


def _copy(dst=None, src=None, to=FAKE, frm=FAKE, lengths=None, n=2, max_len=64):
    cb = tq.Codebook(128, 3, 4)
    return tq.lib.tq_cache_copy(cb.handle, C.byref(dst or _cache()), C.byref(src or _cache()), to, frm, lengths, n,
                                max_len, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(src=_cache(kv_heads=1)), "kv_heads"), (dict(n=-1), "n "), (dict(n=65536), "n "), (dict(max_len=-1), "max_len"),
    (dict(to=None), "NULL"), (dict(frm=None), "NULL"), (dict(lengths=FAKE + 2), "4-byte"),
    (dict(dst=_cache(capacity=24)), "multiple of 16"), (dict(src=_cache(v_codes=None)), "NULL")])
def test_copy_refusals(kw, needle):
    _refused(_copy(**kw), needle)


def test_copy_of_nothing():
    assert _copy(n=0) == tq.TQ_OK


def test_binding_checks():
    cb = tq.Codebook(128, 3, 4)
    c = tq.Cache(cb, 2, 2, 32, device="cpu")
    x = torch.zeros(2, 2, 4, 128)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    rope = tq.Rope.__new__(tq.Rope)
    rope.table, rope.rot_dim, rope.max_pos, rope.interleaved = torch.zeros(8, 64, 2), 128, 8, False
    for bad in (dict(k=x[..., :64]), dict(k=x[0]), dict(v=x.half()), dict(v=x[:, :, :3]), dict(v=x[:1]),
                dict(k=x.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            tq.tq_rope_append(cb, c, rope, **{**dict(k=x, v=x), **bad})
    q = torch.zeros(2, 4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        tq.tq_tree_attention(cb, c, q.float())
    for bad in (q[:1], q[..., :64], q[0], q.transpose(1, 2)):
        with pytest.raises(ValueError):
            tq.tq_tree_attention(cb, c, bad)
    with pytest.raises(ValueError, match="index must be"):
        tq.tq_cache_compact(cb, c, i32(4), i32(2))
    with pytest.raises(ValueError, match="dst_rows"):
        tq.tq_cache_copy(cb, c, c, i32(2, 1), i32(2))
    # host tensors never reach the library
    for call in (lambda: tq.tq_rope_append(cb, c, rope, x, x), lambda: tq.tq_tree_attention(cb, c, q),
                 lambda: tq.tq_cache_compact(cb, c, i32(2, 4), i32(2)), lambda: tq.tq_cache_copy(cb, c, c, i32(1), i32(1))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("n", [1, 5, 31, 32, 33, 64, 70])
def test_pack_tree_mask(n):
    sees = torch.rand(3, n, n, generator=torch.Generator().manual_seed(n)) < 0.5
    words = tq.pack_tree_mask(sees)
    assert words.dtype == torch.int32 and words.shape == (3, n, (n + 31) // 32)
    j = torch.arange(n)
    assert torch.equal(((words[..., j // 32].long() >> (j % 32)) & 1).bool(), sees)
    for bad in (sees.int(), sees[..., :1] if n > 1 else sees[0, 0]):
        with pytest.raises(ValueError):
            tq.pack_tree_mask(bad)
