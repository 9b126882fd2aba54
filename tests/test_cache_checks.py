"""What the speculative-decoding calls check of a cache's arrays before the library sees
their addresses (CPU only: stand-ins that say they are on a GPU)."""
import pytest
import torch

from turboquant_kv_cache_rht_b200 import tq


class OnGpu:
    """A host tensor that answers as if it were on cuda:0, at an address that is never read."""

    def __init__(self, t, address=0x100000):
        self.t, self.address = t, address

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return 0

    def data_ptr(self):
        return self.address


DEVICE = torch.device("cuda", 0)
NAMES = ("k_codes", "v_codes", "k_signs", "k_norm", "v_norm", "k_rnorm", "seq_lens", "status", "append_sync")


def _cache(codebook="gaussian"):
    cb = tq.Codebook(64, 2, 3, qjl=True, codebook=codebook)
    c = tq.Cache(cb, 2, 2, 32, device="cpu")
    for name in NAMES:
        setattr(c, name, OnGpu(getattr(c, name)))
    return cb, c


def _struct(cb, c):
    return tq._cache_struct("here", cb, c, DEVICE)


@pytest.mark.parametrize("codebook", ["gaussian", "affine"])
def test_a_sound_cache(codebook):
    cb, c = _cache(codebook)
    s = _struct(cb, c)
    assert (s.batch, s.kv_heads, s.capacity) == (2, 2, 32) and s.k_rnorm == 0x100000


@pytest.mark.parametrize("name,dtype", [
    ("seq_lens", torch.int64), ("seq_lens", torch.int16), ("seq_lens", torch.float32), ("append_sync", torch.int64),
    ("append_sync", torch.uint8), ("status", torch.int64), ("status", torch.bool), ("k_norm", torch.uint8),
    ("v_norm", torch.uint8), ("k_norm", torch.float32), ("v_norm", torch.float32), ("k_rnorm", torch.uint8),
    ("k_rnorm", torch.float32), ("k_codes", torch.int16), ("v_codes", torch.float16), ("k_signs", torch.int32)])
@pytest.mark.parametrize("codebook", ["gaussian", "affine"])
def test_arrays_of_other_types(name, dtype, codebook):
    """The right number of elements, of a size that the kernels would pass or misread."""
    cb, c = _cache(codebook)
    setattr(c, name, OnGpu(getattr(c, name).t.to(dtype)))
    with pytest.raises(ValueError, match="arrays must be"):
        _struct(cb, c)


@pytest.mark.parametrize("name", NAMES)
def test_arrays_of_other_sizes(name):
    cb, c = _cache()
    t = getattr(c, name).t
    for bad in (OnGpu(t.flatten()[:-1]), OnGpu(torch.stack((t, t), -1)[..., 0]), None):
        if bad is not None and name == "status" and bad.t.numel() == 1:
            continue                                   # a view of one element is contiguous
        setattr(c, name, bad)
        with pytest.raises(ValueError, match="arrays must be"):
            _struct(cb, c)
