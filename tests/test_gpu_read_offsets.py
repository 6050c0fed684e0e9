"""pa_read_cache with offsets that fall or leave the rows: such a sequence is skipped, whatever the search
for a row's sequence meets on its way, and every other one is read."""
import numpy as np
import pytest
import torch
from test_gpu_axes_read import cache, check_rows, read

import paged_kv_cache_28_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def claimed(offsets, T):
    """The sequences that claim each row, bad ones left out."""
    rows = [[] for _ in range(T)]
    for b, (q0, q1) in enumerate(zip(offsets, offsets[1:])):
        if 0 <= q0 <= q1 <= T:
            for t in range(q0, q1):
                rows[t].append(b)
    return rows


def check(c, out, offsets, T):
    rows = claimed(offsets, T)
    for x, got in out.items():
        pool = c[x][0].view(-1, c["Hkv"], c["D"])
        for t, by in enumerate(rows):
            if not by:
                assert (got[t] == -3.0).all(), (x, t)
                continue
            want = [pool[int(c["bt"][b, (t - offsets[b]) // c["bs"]]) * c["bs"] + (t - offsets[b]) % c["bs"]] for b in by]
            assert any(torch.equal(got[t], w) for w in want), (x, t, by)


@pytest.mark.parametrize("offsets,T", [
    ([0, 4, 8, 13], 12), ([-1, 4, 8, 12], 12), ([-3, -1, 8, 12], 12), ([0, 10, 5, 12], 12), ([5, 4, 3, 2], 12),
    ([0, 4, 100, 12], 12), ([0, 30, 4, 12], 12), ([2 ** 31 - 1, 3, 6, 12], 12), ([0, 4, -2 ** 31, 12], 12),
    ([3, 3, 3, 40], 40), ([0, 0, 41, 41], 40), ([20, 40, 0, 20], 40),
])
def test_bad_offsets(offsets, T):
    c = cache([40, 41, 40], 2, 64, 16, "bf16", seed=81)
    out = read(c, offsets, T)
    bad = any(not 0 <= a <= b <= T for a, b in zip(offsets, offsets[1:]))
    assert pa.pa_read_error_flag(c["err"]) == (pa.PA_DEVERR_QUERY if bad else 0)
    check(c, out, offsets, T)


@pytest.mark.parametrize("B,T", [(40, 400), (1100, 3300)])
def test_bad_offsets_among_many_sequences(B, T):
    """More sequences than a warp looks at in one step, one to three of their offsets out of order."""
    c = cache([10] * B, 1, 64, 16, "bf16", seed=82)
    r = np.random.default_rng(B)
    good = np.sort(r.integers(0, T + 1, B + 1))
    for trial in range(12):
        offsets = good.copy()
        for i in r.integers(0, B + 1, 1 + trial % 3):
            offsets[i] = r.choice([-5, 0, T, T + 9, 2 ** 31 - 1, -2 ** 31, int(r.integers(0, T))])
        # a sequence of more rows than it has tokens reads zeros there
        offsets = offsets.tolist()
        c["err"].zero_()
        out = read(c, offsets, T)
        bad = any(not 0 <= a <= b <= T for a, b in zip(offsets, offsets[1:]))
        assert bool(pa.pa_read_error_flag(c["err"]) & pa.PA_DEVERR_QUERY) == bad
        rows = claimed(offsets, T)
        pool = c["k"][0].view(-1, 1, 64)
        got = out["k"].cpu()
        bt, host = c["bt"].cpu(), pool.cpu()
        for t, by in enumerate(rows):
            want = [host[int(bt[b, 0]) * 16 + t - offsets[b]] if t - offsets[b] < 10 else torch.zeros(1, 64).bfloat16()
                    for b in by] or [torch.full((1, 64), -3.0).bfloat16()]
            assert any(torch.equal(got[t], w) for w in want), (trial, t, by)


def test_rows_before_and_behind_many_sequences():
    """Good offsets with rows of no sequence on both sides, as a padded batch has them."""
    L = [3, 0, 1] * 200
    c = cache(L, 2, 128, 32, "fp8", seed=83)
    offsets = (100 + np.concatenate([[0], np.cumsum(L)])).tolist()
    out = read(c, offsets, offsets[-1] + 3000)
    assert pa.pa_read_error_flag(c["err"]) == 0
    check_rows(c, out, offsets, None)
