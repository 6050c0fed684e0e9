"""DeviceBatch's scored calls, its rotation by several axes and its reading back, on another stream than the
current one while that one is busy: the bits of calls on an idle GPU.  An output that was filled, or a buffer
that was taken, in the current stream's order would hold something else."""
import pytest
import torch

from paged_kv_cache_28_gb300 import workload as wl
from paged_kv_cache_28_gb300.device import DeviceBatch, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


@pytest.mark.parametrize("name", ["rope", "extend", "decode", "read"])
@pytest.mark.parametrize("raw", [False, True])
def test_bits_on_a_stream_beside_a_busy_one(name, raw):
    batch = wl.make("tiny")
    dev = DeviceBatch(batch, device="cuda")
    rows = torch.arange(batch.B + 1, dtype=torch.int32, device="cuda")
    offsets = torch.cat([rows[:1] * 0, dev.seq_lens.cumsum(0).int()]) + 2
    total = int(offsets[-1]) + 3                         # rows of no sequence on both sides: zeros
    slopes = torch.linspace(0.01, 0.5, batch.Hq, device="cuda")
    positions = torch.stack([dev.seq_lens - 1, dev.seq_lens % 7]).int()
    pair = [j % 2 for j in range(batch.D // 2)]
    table = rope_table(int(dev.seq_lens.max()) + 1, batch.D)
    q = torch.cat([dev.q, dev.q])                        # rows of no sequence here, too
    calls = dict(
        rope=lambda st: dev.rope_axes_and_cache(dev.q, dev.k_new, dev.v_new, pair, positions, dev.slot_mapping,
                                                table, stream=st),
        extend=lambda st: dev.extend_scored(q, rows, softcap=9.0, slopes=slopes, stream=st),
        decode=lambda st: dev.decode_scored(softcap=9.0, slopes=slopes, stream=st),
        read=lambda st: dev.read_cache(offsets, total, stream=st))
    calls["rope"](None)                                  # (later calls write the same tokens anew)
    want = calls[name](None)
    torch.cuda.synchronize()
    side, junk = torch.cuda.Stream(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for i in range(12):
            junk.fill_(i)
        got = calls[name](side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        del got, a
    assert dev.read_err() == 0
