"""Outputs of the rotary append that overlap what it reads, or one another (CPU only:
refused before anything is read)."""
import ctypes as C

import pytest

from turboquant_kv_cache_rht_b200 import tq

D, HQ, H, N, B = 128, 4, 2, 3, 2
ROW = (HQ + 2 * H) * D                      # elements of a token of a fused projection, 2 bytes each
BASE = 0x100000
SIZE = 2 * B * N * ROW                      # bytes of the projection
CACHE = tq.tq_cache(0x10000, 0x20000, None, 0x30000, 0x40000, None, 0x50000, 0x60000, 0x70000, B, H, 64)


def _heads(at):
    return tq.tq_heads(BASE + 2 * at * D, N * ROW, D, ROW)


def _append(q_out, k_out):
    cb = tq.Codebook(D, 3, 4)
    rope = tq.tq_rope(0x80000, 4096, D, 0)
    return tq.lib.tq_rope_append(cb.handle, C.byref(CACHE), C.byref(rope), C.byref(_heads(0)), HQ, C.byref(_heads(HQ)),
                                 C.byref(_heads(HQ + H)), 1, N, None, 0, None, q_out, k_out, None)


AWAY = BASE + SIZE
Q_OUT, K_OUT = 2 * B * N * HQ * D, 2 * B * N * H * D


@pytest.mark.parametrize("q_out,k_out", [
    (BASE, None), (BASE + 256, None), (BASE + SIZE - 2 * D, None), (BASE - Q_OUT + 16, None),
    (AWAY, BASE), (AWAY, BASE + 2 * HQ * D), (AWAY, BASE + SIZE - 16), (AWAY, AWAY), (AWAY, AWAY + Q_OUT - 16),
    (AWAY + 16, AWAY)])
def test_refused(q_out, k_out):
    assert _append(q_out, k_out) == tq.TQ_ERR_INVALID
    assert "overlap" in tq.tq_last_error()


@pytest.mark.parametrize("q_out,k_out", [(AWAY, None), (BASE - Q_OUT, None), (AWAY, AWAY + Q_OUT), (AWAY + K_OUT, AWAY)])
def test_not_refused(q_out, k_out):
    """Side by side (there is no GPU here: the launch is what fails)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert _append(q_out, k_out) in (tq.TQ_ERR_CUDA, tq.TQ_ERR_UNSUPPORTED)
