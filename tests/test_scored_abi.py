"""pa_extend_scored and pa_decode_scored without a GPU: what they refuse before any CUDA call."""
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


def call(lib, name, s, T=10, window=0, cap=30.0, slopes=FAKE, prefix=FAKE, segments=7, ws_bytes=1 << 40,
         score=True, **ptr):
    p = dict(out=FAKE, q=FAKE, off=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE, sl=FAKE, ws=FAKE)
    p.update(ptr)
    s = ctypes.byref(s) if s else None
    sc = ctypes.byref(_lib.pa_score(cap, slopes, prefix)) if score else None
    pools = (p["k"], p["v"], p["ks"], p["vs"], p["bt"], p["sl"], window, sc, 0.1, p["ws"], ws_bytes)
    if name == "pa_extend_scored":
        return lib.pa_extend_scored(s, p["out"], p["q"], p["off"], T, *pools, None, None)
    return lib.pa_decode_scored(s, p["out"], p["q"], *pools, segments, None, None)


SHAPES = [(dict(Hq=6, Hkv=4), BAD), (dict(Hq=64, Hkv=2), NOT_BUILT), (dict(D=96), NOT_BUILT),
          (dict(block_size=8), NOT_BUILT), (dict(kv_dtype=_lib.PA_KV_FP8_E4M3, D=64), NOT_BUILT),
          (dict(kv_dtype=7), BAD), (dict(B=-1), BAD), (dict(nblocks=0), BAD), (dict(B=20000), NOT_BUILT),
          (dict(B=2, max_blocks=1 << 30), BAD)]


@pytest.mark.parametrize("name", ["pa_extend_scored", "pa_decode_scored"])
def test_refuses(lib, name):
    for kw, status in SHAPES:
        assert call(lib, name, shape(**kw)) == status, kw
    assert call(lib, name, None) == BAD
    assert call(lib, name, shape(), score=False) == BAD
    for cap in (-1.0, float("nan"), float("inf"), 1e-11, 1e11, -float("inf")):
        assert call(lib, name, shape(), cap=cap) == BAD, cap
    assert call(lib, name, shape(), slopes=FAKE + 2) == BAD
    assert call(lib, name, shape(), prefix=FAKE + 1) == BAD
    assert call(lib, name, shape(), window=-1) == BAD
    for key in ("out", "q", "k", "v", "bt", "sl", "ws"):
        assert call(lib, name, shape(), **{key: None}) == BAD, key
        assert call(lib, name, shape(), **{key: FAKE + 4}) == BAD, key
    assert call(lib, name, shape(), ws=FAKE + 16) == BAD             # not 256-byte aligned
    assert call(lib, name, shape(kv_dtype=_lib.PA_KV_FP8_E4M3)) == BAD             # scales missing
    assert call(lib, name, shape(kv_dtype=_lib.PA_KV_INT4), ks=FAKE) == BAD
    assert call(lib, name, shape(B=0), q=None) == OK                 # nothing to do
    if name == "pa_extend_scored":
        assert call(lib, name, shape(), off=None) == BAD
        assert call(lib, name, shape(), T=-1) == BAD
        assert call(lib, name, shape(), T=0, q=None) == OK
        assert call(lib, name, shape(), T=0, cap=-1.0) == BAD
    else:
        assert call(lib, name, shape(), segments=-1) == BAD and call(lib, name, shape(), segments=65537) == BAD
        need = _lib.pa_decode_workspace_bytes(shape(), 7)
        assert call(lib, name, shape(), ws_bytes=need - 1) == BAD
