"""pa_rope_and_cache, pa_extend and pa_cross_attend without a GPU: what they refuse before any
CUDA call, and the workspace's size."""
import ctypes

import pytest

from paged_kv_cache_28_gb300 import _lib

FAKE = 1 << 20      # a 256-byte aligned non-null address: never dereferenced on these paths
BAD, NOT_BUILT = _lib.PA_ERR_INVALID_ARG, _lib.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_28_gb300 import build
    build.build()
    return _lib.load()


def shape(**kw):
    base = dict(B=4, Hq=8, Hkv=2, D=128, block_size=16, nblocks=64, max_blocks=8, kv_dtype=_lib.PA_KV_BF16)
    base.update(kw)
    return _lib.make_shape(**base)


def attend(lib, s, name="pa_extend", T=10, window=0, ws_bytes=1 << 40, **ptr):
    p = dict(out=FAKE, q=FAKE, off=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE, sl=FAKE, ws=FAKE)
    p.update(ptr)
    args = [ctypes.byref(s) if s else None, p["out"], p["q"], p["off"], T, p["k"], p["v"], p["ks"], p["vs"],
            p["bt"], p["sl"]]
    if name == "pa_extend":
        args.append(window)
    return getattr(lib, name)(*args, 0.1, p["ws"], ws_bytes, None, None)


SHAPES = [(dict(Hq=6, Hkv=4), BAD), (dict(Hq=64, Hkv=2), NOT_BUILT), (dict(D=96), NOT_BUILT),
          (dict(block_size=8), NOT_BUILT), (dict(kv_dtype=_lib.PA_KV_FP8_E4M3, D=64), NOT_BUILT),
          (dict(kv_dtype=7), BAD), (dict(B=-1), BAD), (dict(nblocks=0), BAD), (dict(B=20000), NOT_BUILT),
          (dict(B=1, max_blocks=1 << 26), BAD)]     # 2^30 positions


@pytest.mark.parametrize("name", ["pa_extend", "pa_cross_attend"])
def test_attend_refuses(lib, name):
    for kw, status in SHAPES:
        assert attend(lib, shape(**kw), name) == status, kw
        assert _lib.pa_attend_workspace_bytes(shape(**kw), 10, 152) == 0
    assert attend(lib, None, name) == BAD
    for key in ("out", "q", "off", "k", "v", "bt", "sl", "ws"):
        assert attend(lib, shape(), name, **{key: None}) == BAD, key
        assert attend(lib, shape(), name, **{key: FAKE + 4}) == BAD, key
    assert attend(lib, shape(), name, ws=FAKE + 16) == BAD           # not 256-byte aligned
    assert attend(lib, shape(), name, T=-1) == BAD
    assert attend(lib, shape(), name, T=1 << 28) == BAD              # 2^31 query rows
    assert attend(lib, shape(kv_dtype=_lib.PA_KV_FP8_E4M3), name) == BAD          # scales missing
    assert attend(lib, shape(kv_dtype=_lib.PA_KV_INT4), name, ks=FAKE) == BAD
    # nothing to do: no pointer is looked at
    assert attend(lib, shape(B=0), name, q=None) == _lib.PA_OK
    assert attend(lib, shape(), name, T=0, q=None) == _lib.PA_OK
    if name == "pa_extend":
        assert attend(lib, shape(), name, window=-1) == BAD


def test_attend_workspace(lib):
    s = shape(Hq=64, Hkv=8)
    # two pieces per worker of rows x (D + 2) floats, and a record per worker
    few = _lib.pa_attend_workspace_bytes(s, 4, 152)                  # 4 tokens x 8 heads: 32 rows
    assert 0 <= few - (2 * 304 * 32 * 130 * 4 + 304 * 16) < 1024
    many = _lib.pa_attend_workspace_bytes(s, 1000, 152)
    assert 0 <= many - (2 * 152 * 256 * 130 * 4 + 152 * 16) < 1024
    assert _lib.pa_attend_workspace_bytes(s, 10, 0) == 0
    # a million query tokens, each over a block table of 2^29 positions: too many tiles to count
    far = shape(Hq=64, Hkv=8, B=1, max_blocks=1 << 25)
    assert _lib.pa_attend_workspace_bytes(far, 1 << 20, 152) == 0
    assert _lib.pa_attend_workspace_bytes(far, 1 << 10, 152) > 0
    assert _lib.pa_attend_workspace_bytes(s, -1, 152) == 0


def rope(lib, s, r=128, interleaved=0, rows=100, strides=(0, 0, 0), no_rope=False, **ptr):
    p = dict(cs=FAKE, pos=FAKE, qo=FAKE, q=2 * FAKE, k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, ks=None, vs=None,
             slots=FAKE)
    p.update(ptr)
    how = _lib.pa_rope(r, interleaved, rows, *strides)
    return lib.pa_rope_and_cache(ctypes.byref(s) if s else None, None if no_rope else ctypes.byref(how), p["cs"],
                                 p["pos"], p["qo"], p["q"], p["k"], p["v"], p["kp"], p["vp"], p["ks"], p["vs"],
                                 p["slots"], None, None)


def test_rope_refuses(lib):
    assert rope(lib, None) == BAD and rope(lib, shape(), no_rope=True) == BAD
    assert rope(lib, shape(Hq=6, Hkv=4)) == BAD
    assert rope(lib, shape(D=96)) == NOT_BUILT
    for r, status in ((0, BAD), (-16, BAD), (130, BAD), (144, BAD), (24, NOT_BUILT), (8, NOT_BUILT)):
        assert rope(lib, shape(), r=r) == status, r
    assert rope(lib, shape(), rows=0) == BAD
    for strides in ((1000, 0, 0), (0, 128, 0), (0, 0, 260 + 2), (-1024, 0, 0)):
        assert rope(lib, shape(), strides=strides) == BAD, strides
    for key in ("cs", "pos", "k", "v", "kp", "vp", "slots"):
        assert rope(lib, shape(), **{key: None}) == BAD, key
        assert rope(lib, shape(), **{key: FAKE + 8}) == BAD, key
    assert rope(lib, shape(), q=None) == BAD and rope(lib, shape(), qo=None) == BAD
    assert rope(lib, shape(), q=FAKE, strides=(2048, 0, 0)) == BAD   # in place, but not dense
    assert rope(lib, shape(kv_dtype=_lib.PA_KV_FP8_E4M3)) == BAD     # scales missing
    assert rope(lib, shape(B=0), q=None, qo=None, k=None) == _lib.PA_OK


def test_binding_takes_slices_of_a_fused_projection():
    torch = pytest.importorskip("torch")
    x = torch.zeros(5, 12, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        _lib._token_ptr(x)
    assert _lib._token_ptr(None) == (None, 0)


def test_writes_of_many_tokens_beside_a_wide_block_table(lib):
    """A write's B counts tokens: its size has nothing to do with the block table's width."""
    for kw in (dict(B=32768, Hkv=8, Hq=64, max_blocks=8192), dict(B=16384, Hkv=16, Hq=16, max_blocks=8192),
               dict(B=1 << 20, max_blocks=1 << 20)):
        # (a rotation that is not built is found after the shape, before any CUDA call)
        assert rope(lib, shape(**kw), r=24) == NOT_BUILT, kw
        # the same shape as a batch of sequences has too many tiles to count
        assert attend(lib, shape(**kw)) in (BAD, NOT_BUILT)
        assert _lib.pa_attend_workspace_bytes(shape(**kw), 10, 152) == 0
    assert rope(lib, shape(B=32768, max_blocks=0), r=24) == BAD
