"""The binding refuses arrays whose elements are not those that the kernels read, or too few, before any
pointer is taken (no GPU)."""
import pytest
import torch

from paged_kv_cache_28_gb300 import _lib

B, HQ, HKV = 4, 8, 2
FAKE = 1 << 20


def shape():
    return _lib.make_shape(B, HQ, HKV, 128, 16, 64, 8, _lib.PA_KV_BF16)


def f32(n):
    return torch.zeros(n)


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


class Rows(int):
    """The address of 10 rows."""
    shape = (10,)


POOLS = (FAKE, FAKE, None, None, FAKE, FAKE)


def extend(offsets=FAKE, **kw):
    _lib.pa_extend_scored(shape(), FAKE, Rows(FAKE), offsets, *POOLS, 0.1, FAKE, **kw)


def decode(**kw):
    _lib.pa_decode_scored(shape(), FAKE, FAKE, *POOLS, 0.1, FAKE, **kw)


@pytest.mark.parametrize("bad", [f32(HKV), f32(HQ + 1), f32(HQ).double(), f32(HQ).bfloat16(), i32(HQ)])
def test_slopes(bad):
    for call in (extend, decode):
        with pytest.raises(ValueError, match="slopes"):
            call(slopes=bad)


@pytest.mark.parametrize("bad", [i32(B - 1), i32(B).long(), f32(B)])
def test_prefix_lens(bad):
    with pytest.raises(ValueError, match="prefix_lens"):
        extend(prefix_lens=bad)


@pytest.mark.parametrize("bad", [i32(B), i32(B + 1).long()])
def test_offsets(bad):
    with pytest.raises(ValueError, match="offsets"):
        extend(offsets=bad)
    with pytest.raises(ValueError, match="offsets"):
        read(bad, FAKE)


@pytest.mark.parametrize("bad", [i32(B - 1), i32(B).long()])
def test_starts(bad):
    with pytest.raises(ValueError, match="starts"):
        read(FAKE, bad)


def read(offsets, starts):
    _lib.pa_read_cache(shape(), None, None, *POOLS, offsets, starts)


def test_positions():
    for pos in (torch.zeros(3, B, dtype=torch.int64), torch.zeros(3, B)):
        with pytest.raises(ValueError, match="positions"):
            _lib.pa_rope_axes_and_cache(shape(), [0] * 16, torch.zeros(10, 32), pos, *(None,) * 8, None, None)


def test_arrays_that_fit_pass():
    """... to the next check: these are not on a GPU."""
    for kw in (dict(slopes=f32(HQ)), dict(prefix_lens=i32(B)), dict(prefix_lens=i32(B + 5))):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            extend(**kw)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        decode(slopes=f32(HQ).view(HKV, -1))
