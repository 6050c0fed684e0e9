"""pa_rope_axes_and_cache and pa_read_cache without a GPU: what they refuse before any CUDA call."""
import ctypes

import pytest

from paged_kv_cache_28_gb300 import _lib

FAKE = 1 << 20      # a 256-byte aligned non-null address: never dereferenced on these paths
BAD, NOT_BUILT, OK = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED, _lib.PA_OK


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_28_gb300 import build
    build.build()
    return _lib.load()


def shape(**kw):
    base = dict(B=4, Hq=8, Hkv=2, D=128, block_size=16, nblocks=64, max_blocks=8, kv_dtype=_lib.PA_KV_BF16)
    base.update(kw)
    return _lib.make_shape(**base)


def axes_call(lib, s, num_axes=3, pair_axis=(0, 1, 2), rotary=128, npos=100, stride=0, axes=True, **ptr):
    p = dict(cs=FAKE, pos=FAKE, qo=FAKE, q=FAKE, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, ks=None, vs=None, slots=FAKE)
    p.update(ptr)
    rope = _lib.pa_rope(rotary, 0, npos, stride, 0, 0)
    pair = bytes(pair_axis).ljust(64, b"\0")[:64]
    ax = _lib.pa_rope_axes(num_axes, (ctypes.c_uint8 * 64).from_buffer_copy(pair))
    return lib.pa_rope_axes_and_cache(ctypes.byref(s) if s else None, ctypes.byref(rope),
                                      ctypes.byref(ax) if axes else None, p["cs"], p["pos"], p["qo"], p["q"],
                                      p["k"], p["v"], p["kp"], p["vp"], p["ks"], p["vs"], p["slots"], None, None)


def test_axes_refuse(lib):
    s = shape()
    assert axes_call(lib, s, axes=False) == BAD
    assert axes_call(lib, None) == BAD
    for n in (0, -1, 5, 1 << 20):
        assert axes_call(lib, s, num_axes=n, pair_axis=()) == BAD, n
    assert axes_call(lib, s, num_axes=2) == BAD                       # a pair of axis 2
    assert axes_call(lib, s, pair_axis=[0] * 63 + [3]) == BAD
    assert axes_call(lib, shape(B=0), pair_axis=[0] * 16 + [9], rotary=32) == OK   # pairs past rotary_dim / 2
    assert axes_call(lib, s, rotary=0) == BAD and axes_call(lib, s, rotary=144) == BAD
    assert axes_call(lib, s, rotary=24) == NOT_BUILT
    assert axes_call(lib, s, npos=0) == BAD
    assert axes_call(lib, s, stride=4) == BAD and axes_call(lib, s, stride=8 * 128 + 4) == BAD
    for key in ("cs", "pos", "k", "v", "kp", "vp", "slots"):
        assert axes_call(lib, s, **{key: None}) == BAD, key
        assert axes_call(lib, s, **{key: FAKE + 4}) == BAD, key
    assert axes_call(lib, s, q=None) == BAD and axes_call(lib, s, qo=None) == BAD
    assert axes_call(lib, shape(kv_dtype=_lib.PA_KV_FP8_E4M3)) == BAD              # scales missing
    assert axes_call(lib, shape(Hq=6, Hkv=4)) == BAD and axes_call(lib, shape(D=96)) == NOT_BUILT


def test_axes_binding_checks_lengths():
    import torch
    pos, table = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(10, 32)
    args = (None,) * 2 + (None,) * 6
    for pair, p in (([0] * 15, pos), ([0] * 16, pos[0]), ([0] * 16, torch.zeros(3, 5, dtype=torch.int32))):
        with pytest.raises(ValueError):
            _lib.pa_rope_axes_and_cache(shape(), pair, table, p, *args, None, None)


def read(lib, s, T=10, **ptr):
    p = dict(ko=FAKE, vo=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE, sl=FAKE, off=FAKE, starts=FAKE)
    p.update(ptr)
    return lib.pa_read_cache(ctypes.byref(s) if s else None, p["ko"], p["vo"], p["k"], p["v"], p["ks"], p["vs"],
                             p["bt"], p["sl"], p["off"], T, p["starts"], None, None)


def test_read_refuses(lib):
    s = shape()
    assert read(lib, None) == BAD
    for kw, status in [(dict(D=96), NOT_BUILT), (dict(block_size=8), NOT_BUILT), (dict(kv_dtype=7), BAD),
                       (dict(B=-1), BAD), (dict(nblocks=0), BAD), (dict(max_blocks=0), BAD), (dict(B=20000), NOT_BUILT),
                       (dict(Hkv=4096), NOT_BUILT), (dict(B=4, max_blocks=1 << 29), BAD),
                       (dict(kv_dtype=_lib.PA_KV_FP8_E4M3, D=64), NOT_BUILT), (dict(kv_dtype=_lib.PA_KV_INT4), BAD)]:
        assert read(lib, shape(**kw)) == status, kw
    assert read(lib, s, T=-1) == BAD
    for key in ("k", "v", "bt", "sl", "off"):
        assert read(lib, s, **{key: None}) == BAD, key
        assert read(lib, s, **{key: FAKE + 4}) == BAD, key
    for key in ("ko", "vo", "starts"):
        assert read(lib, s, **{key: FAKE + 4}) == BAD, key
    q = shape(kv_dtype=_lib.PA_KV_FP8_E4M3)
    assert read(lib, q, ks=FAKE) == BAD and read(lib, q, vs=FAKE) == BAD
    # nothing to do: no pointer is looked at
    assert read(lib, shape(B=0), bt=None) == OK and read(lib, s, T=0, bt=None) == OK
    assert read(lib, s, ko=None, vo=None, bt=None) == OK
