"""Capped scores whose product of query and key is huge beside a scale that is tiny or 0, on a GPU against
the formula in 64 bits (tolerances as in test_gpu_scored.py)."""
import pytest
import torch
from test_gpu_scored import Scored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("bf16", 64), ("fp8", 128)])
@pytest.mark.parametrize("power,scale", [(10, 0.0), (10, 1e-24), (10, 1e-21), (10, 1e-20), (10, 2e-19), (16, 0.0),
                                         (16, 1e-33), (16, 1e-31), (7, 1e-14), (7, 3e-13)])
def test_huge_products(power, scale, kind, D, decode):
    """Products around 10^(2 power), whose squares pass the largest number, and scores of 0 to some tens."""
    for n in ([1, 1], [200, 1])[:1 if decode else 2]:
        for change in (dict(cap=50.0), dict(cap=1e-3), dict(cap=30.0, slopes="usual")):
            b = Scored(n, [700, 90], 2, 8, D, 16, kind, qmul=10.0 ** power, decode=decode, seed=71, **change)
            if kind == "bf16":
                b.k *= 10.0 ** power
            else:
                b.k_scale *= 10.0 ** power
            b.scale = scale
            b.check()


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("scale", [0.0, 1e-32])
def test_zero_scales_beside_huge_queries(scale, kind, decode):
    """A block whose K scale is 0 scores 0, however large its codes' products are."""
    for n in ([1, 1], [200, 1])[:1 if decode else 2]:
        for change in (dict(cap=50.0), dict(cap=30.0, slopes="usual")):
            b = Scored(n, [700, 90], 2, 8, 128, 16, kind, qmul=1e30, decode=decode, seed=72, **change)
            b.k_scale[::2] = 0.0
            b.scale = scale
            b.check()


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("scale", [1e29, -3e38])
def test_a_scale_far_above_its_cap(scale, kind, decode):
    """Every product but 0 passes the cap: queries of zeros score 0, the others the cap (and what their
    scores' fp32 products are off by does not count there)."""
    for n in ([1, 1], [200, 1])[:1 if decode else 2]:
        b = Scored(n, [700, 90], 2, 8, 128, 16, kind, qmul=1.0, cap=1e-10, decode=decode, seed=73)
        b.q[::2] = 0.0
        b.scale = scale
        out = b.run()
        # scores of +-1e-10: every weight is 1 to 2e-10, so the rows are the means of V (u: weights of 1, rounded
        # once each way; sums over N keys)
        v = b.values(b.v, b.v_scale)
        at = 0
        for s in range(b.B):
            pos = torch.arange(b.L[s], device="cuda")
            rows = v.view(-1, 2, 128)[b.block_tables[s, pos // 16].long() * 16 + pos % 16]
            for i in range(b.n[s]):
                seen = rows[:b.L[s] - b.n[s] + i + 1]
                mean = seen.mean(0)[:, None].expand(2, 8, 128).reshape(16, 128)
                size = seen.abs().mean(0)[:, None].expand(2, 8, 128).reshape(16, 128)
                off = 2.0 ** -8 * mean.abs() + (2.0 ** -8 + 2 * len(seen) * 2.0 ** -24 + 1e-9) * size
                assert ((out[at + i].double() - mean).abs() <= off).all(), (s, i)
            at += b.n[s]
