"""The binding's surface (CPU only): every entry point that the library exports and a
program calls has its function or class here, and a codebook can be released early."""
import pytest

from turboquant_kv_cache_rht_b200 import tq

# exports that the binding has under another name
CLASSES = {"tq_codebook_init": "Codebook", "tq_codebook_tables": "Codebook", "tq_weights_quantize": "QuantizedWeights",
           "tq_lut_matmul": "QuantizedWeights", "tq_rope_table": "Rope"}


@pytest.mark.parametrize("name", tq.EXPORTS)
def test_every_export_has_a_wrapper(name):
    assert callable(getattr(tq, CLASSES.get(name, name)))


def test_a_codebook_released_early():
    cb = tq.Codebook(64, 2, 2)
    tq.tq_free(cb)
    assert cb.handle is None
    tq.tq_free(cb)                                     # nothing is left to release
    with pytest.raises(Exception):
        cb.tables()
    cb.__del__()
    other = tq.Codebook(64, 2, 2)                      # and others are not touched
    assert other.tables()["signs1"].numel() == 64
