"""Scored attention over code pools whose V scales are zero or far apart, and whose scores leave the
biased softmax's reference far above the largest exponent.

Tolerances: those of test_gpu_scored.py, and what the reference may lose.  It is a bound of the largest
exponent, at most 62 octaves above it (31 keys of 2 octaves each); V's scale takes up to 24 octaves more in
the exponent; the exponential gives 0 below 2^-126.  So weights below 2^-40 of a row's largest may be lost, in
the numerator and in the sum: with largest value V and N keys, 2 N 2^-40 V.
"""
import pytest
import torch
from test_gpu_scored import Scored

import paged_kv_cache_28_gb300 as pa

pytestmark = pytest.mark.gpu

BIASED = {"bias": {}, "both": dict(cap=50.0)}
STEEP = [0.5, 0.6, 0.7, 0.8, 0.917, 1.0, 1.15, 1.3]     # octaves a key: 0.7 to 1.9


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


class Spread(Scored):
    def reference(self):
        ref, size = super().reference()
        top = self.values(self.v, self.v_scale).nan_to_num(0.0).abs().amax()
        return ref, size + 2 * max(self.L) * 2.0 ** -40 * top


def codes_of(b, x):
    """Codes of the whole number x, as the pool's kind holds it in its first channel."""
    return x + 8 if b.kind == "int4" else int(torch.tensor(float(x)).to(torch.float8_e4m3fn).view(torch.uint8))


def scores(b, low, high, every):
    """Every key scores 4 low, but every `every`-th of a sequence 4 high, whatever its query."""
    b.q.zero_()
    b.q[..., 0] = 1.0
    b.scale = 1.0
    b.k_scale.fill_(4.0)
    mask = 15 if b.kind == "int4" else 0xFF
    for s in range(b.B):
        pos = torch.arange(b.L[s], device="cuda")
        rows = b.block_tables[s, pos // b.bs].long() * b.bs + pos % b.bs
        first = b.k.view(-1, b.Hkv, b.k.shape[-1])[rows]
        code = torch.where(pos % every == 0, codes_of(b, high), codes_of(b, low)).to(torch.uint8)
        first[..., 0] = (first[..., 0] & (0xFF ^ mask)) | code[:, None]
        b.k.view(-1, b.Hkv, b.k.shape[-1])[rows] = first


def pages(b, s):
    return b.block_tables[s, :-(-b.L[s] // b.bs)].long()


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("change", BIASED.values(), ids=BIASED)
@pytest.mark.parametrize("n,L", [([1], [256]), ([4, 1], [260, 640]), ([150], [400]), ([300, 2, 33], [300, 512, 700])])
def test_the_largest_weights_on_pages_without_values(n, L, kind, change):
    """One key of 24 in 32 of -20, on pages whose V scale is 0: a row whose nearest such key is 31 back
    has a reference 31 slopes above its largest exponent, and nearly all its weight where V is 0."""
    for slopes in (STEEP, "usual"):
        b = Spread(n, L, 1, 8, 128, 16, kind, slopes=slopes, seed=61, **change)
        scores(b, -5, 6, 32)
        for s in range(b.B):
            b.v_scale[pages(b, s)[::2]] = 0.0
        b.check()


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("change", BIASED.values(), ids=BIASED)
@pytest.mark.parametrize("small", [0.0, 1e-25, 1e-12, 1e-7])
def test_the_reference_follows_from_pages_without_values(small, kind, change):
    """The newest tile's pages weigh nothing in V, an older key scores far more than all of theirs."""
    for n, L in (([1], [256]), ([3, 200], [259, 384])):
        b = Spread(n, L, 1, 8, 128, 16, kind, slopes=STEEP, seed=62, **change)
        scores(b, -5, 6, 32)
        for s in range(b.B):
            b.v_scale[pages(b, s)[-8:]] = small
            b.k_scale[pages(b, s)[-10]] = 70.0
        b.check()


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("change", [*BIASED.values(), dict(cap=50.0, slopes=None)], ids=[*BIASED, "cap"])
@pytest.mark.parametrize("n", [[3, 1], [200]])
def test_zero_scales(n, kind, change):
    for slopes in ("usual", STEEP):
        for qmul in (1.0, 12.0):
            b = Spread(n, [600] * len(n), 1, 8, 128, 16, kind, qmul=qmul, seed=63, **{"slopes": slopes, **change})
            b.k_scale[::3] = 0
            b.v_scale[::2] = 0
            b.check()


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("change", BIASED.values(), ids=BIASED)
@pytest.mark.parametrize("decades", [(-3, 4), (-25, 1), (-8, -6)])
def test_scales_over_many_decades(decades, kind, change):
    for slopes in ("usual", STEEP):
        b = Spread([40, 5], [700, 900], 1, 8, 128, 16, kind, slopes=slopes, qmul=6.0, seed=64, **change)
        g = torch.Generator(device="cuda").manual_seed(64)
        b.v_scale *= 10.0 ** torch.randint(*decades, b.v_scale.shape, generator=g, device="cuda")
        b.check()


def test_decode_too():
    """pa_decode_scored's reference is the largest exponent itself; the same pools through it."""
    for kind in ("fp8", "int4"):
        for change in BIASED.values():
            b = Spread([1] * 3, [256, 640, 77], 1, 8, 128, 16, kind, slopes=STEEP, decode=True, seed=65, **change)
            scores(b, -5, 6, 32)
            for s in range(b.B):
                b.v_scale[pages(b, s)[::2]] = 0.0
            b.check()
    assert pa.pa_read_error_flag(b.err) == 0
