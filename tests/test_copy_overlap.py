"""Copies between caches that share memory other than as one cache (CPU only: refused
before anything is read)."""
import ctypes as C

import pytest

from turboquant_kv_cache_rht_b200 import tq

ROWS, HEADS, CAP = 4, 2, 64
SLOTS = HEADS * CAP
# bytes of one row of each array: 3-bit keys, 4-bit values, head_dim 128, sketch
ROW = {"k_codes": SLOTS * 48, "v_codes": SLOTS * 64, "k_signs": SLOTS * 16, "k_norm": SLOTS * 2, "v_norm": SLOTS * 2,
       "k_rnorm": SLOTS * 2}
BASE = {name: 0x1000000 * (i + 1) for i, name in enumerate(ROW)}


def _cache(shift=None, batch=ROWS, capacity=CAP, **at):
    """A cache at BASE, all arrays moved by `shift` rows, or some of them by `at` bytes."""
    a = {name: BASE[name] + (shift or 0) * ROW[name] + at.get(name, 0) for name in ROW}
    return tq.tq_cache(*a.values(), 0x10, 0x20, 0x30, batch, HEADS, capacity)


def _copy(dst, src, n=0):
    cb = tq.Codebook(128, 3, 4, qjl=True)
    return tq.lib.tq_cache_copy(cb.handle, C.byref(dst), C.byref(src), 0x40, 0x50, None, n, 16, None)


@pytest.mark.parametrize("dst,src", [
    (_cache(1), _cache()), (_cache(), _cache(3)), (_cache(-3), _cache()),      # views of rows that overlap
    (_cache(capacity=32), _cache()), (_cache(), _cache(capacity=128)),         # rows of other sizes at one place
    (_cache(v_codes=1 << 30), _cache()), (_cache(k_rnorm=1 << 30), _cache()),  # some arrays shared, others not
    (_cache(k_codes=1 << 30), _cache()), (_cache(4, k_norm=-ROW["k_norm"]), _cache())])
def test_refused(dst, src):
    assert _copy(dst, src, n=1) == tq.TQ_ERR_INVALID
    assert "overlap" in tq.tq_last_error()
    assert _copy(src, dst, n=1) == tq.TQ_ERR_INVALID


@pytest.mark.parametrize("dst,src", [
    (_cache(), _cache()), (_cache(4), _cache()), (_cache(), _cache(-4)),
    (_cache(batch=2), _cache()), (_cache(), _cache(batch=1))])                 # one cache, or a view of its first rows
def test_allowed(dst, src):
    assert _copy(dst, src, n=0) == tq.TQ_OK
