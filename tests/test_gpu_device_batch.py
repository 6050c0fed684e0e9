"""DeviceBatch's calls with several tokens per sequence on streams other than the current one.

The current stream is kept busy ahead of a call on another stream: whatever the call puts on the
current one comes after its kernels.  Results are compared bit for bit with the same call on the
current stream, so no tolerance is needed.
"""
import numpy as np
import pytest
import torch

from paged_kv_cache_28_gb300 import _lib, workload
from paged_kv_cache_28_gb300.device import DeviceBatch, rope_table

pytestmark = pytest.mark.gpu

BUSY = 100_000_000          # clock cycles, about 50 ms


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def device_batch(lens=(300, 700, 90, 1500), Hq=8, Hkv=2, D=64, seed=1):
    lens = np.array(lens, dtype=np.int32)
    return DeviceBatch(workload.build_batch("ragged", lens, Hq=Hq, Hkv=Hkv, D=D, block_size=16, seed=seed))


def queries(dev, n, seed):
    """n query tokens of each sequence, and their offsets."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = dev.batch
    q = torch.randn(n * b.B, b.Hq, b.D, generator=g, device="cuda").bfloat16()
    return q, torch.arange(0, n * b.B + 1, n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["extend", "cross_attend"])
def test_a_new_output_is_made_on_the_calls_stream(name, raw):
    dev = device_batch()
    q, offsets = queries(dev, 5, 2)
    call = getattr(dev, name)
    want = call(q, offsets).clone()
    assert (want != 0).any(-1).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(BUSY)
        out = call(q, offsets, stream=side.cuda_stream if raw else side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert dev.read_err() == 0


def stream_of(t):
    """The stream whose memory torch gave a tensor."""
    at = t.data_ptr()
    return next(x["stream"] for x in torch.cuda.memory_snapshot()
                if x["address"] <= at < x["address"] + x["total_size"])


def test_new_tensors_belong_to_the_calls_stream():
    """A new tensor's memory goes back to the stream that wrote it, not to one that may hand it out
    while the kernel still writes."""
    dev = device_batch()
    T, b = 64, dev.batch
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(T, b.Hq + 2 * b.Hkv, b.D, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :b.Hq], qkv[:, b.Hq:b.Hq + b.Hkv], qkv[:, b.Hq + b.Hkv:]
    args = (q, k, v, torch.arange(T, dtype=torch.int32, device="cuda"),
            torch.arange(T, dtype=torch.int64, device="cuda"), rope_table(T, b.D))
    want = dev.rope_and_cache(*args).clone()
    rows, offsets = queries(dev, 3, 4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        out = dev.rope_and_cache(*args, stream=stream)
        assert stream_of(out) == side.cuda_stream
        side.synchronize()
        assert torch.equal(out, want)
        assert stream_of(dev.extend(rows, offsets, stream=stream)) == side.cuda_stream
    assert stream_of(dev.rope_and_cache(*args)) == torch.cuda.current_stream().cuda_stream
    assert stream_of(dev.rope_and_cache(*args, stream=0)) == 0
    torch.cuda.synchronize()


class Spy:
    """Stands before a binding's call and keeps the workspaces it is given."""

    def __init__(self, monkeypatch, name):
        self.seen, self.call = [], getattr(_lib, name)
        monkeypatch.setattr(_lib, name, self)

    def __call__(self, shape, out, q, offsets, k, v, ks, vs, bt, sl, scale, workspace, *rest, **kw):
        self.seen.append((workspace.data_ptr(), workspace.numel()))
        return self.call(shape, out, q, offsets, k, v, ks, vs, bt, sl, scale, workspace, *rest, **kw)


def apart(a, b):
    return a[0] + a[1] <= b[0] or b[0] + b[1] <= a[0]


@pytest.mark.parametrize("name", ["extend", "cross_attend"])
def test_calls_that_may_overlap_have_a_workspace_each(name, monkeypatch):
    dev = device_batch((9000, 7000, 11000))
    spy = Spy(monkeypatch, "pa_" + name)
    sides = [torch.cuda.Stream() for _ in range(2)]
    work = [queries(dev, 40, 5), queries(dev, 3, 6)]
    call = getattr(dev, name)
    want = [call(q, offsets).clone() for q, offsets in work]
    torch.cuda.synchronize()
    spy.seen.clear()
    outs = [[call(q, offsets, stream=s) for (q, offsets), s in zip(work, sides)] for _ in range(30)]
    torch.cuda.synchronize()
    for pair in outs:
        for out, w in zip(pair, want):
            assert torch.equal(out, w)
    first, second = spy.seen[0::2], spy.seen[1::2]
    assert all(apart(a, b) for a in first for b in second)


def test_captured_calls_keep_their_workspaces(monkeypatch):
    """Two graphs of one DeviceBatch share no workspace with each other nor with later eager calls,
    larger ones among them."""
    dev = device_batch((9000, 7000, 11000))
    spy = Spy(monkeypatch, "pa_extend")
    work = [queries(dev, 3, 7), queries(dev, 4, 8)]
    want = [dev.extend(q, offsets).clone() for q, offsets in work]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    spy.seen.clear()
    graphs = []
    for (q, offsets), out in zip(work, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            dev.extend(q, offsets, out)
    large = queries(dev, 200, 9)
    dev.extend(*large)
    dev.extend(*work[0])
    assert apart(*spy.seen[:2])
    assert all(apart(a, b) for a in spy.seen[:2] for b in spy.seen[2:])
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                g.replay()
        dev.extend(*large)
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out, w)


def test_a_workspace_of_the_callers():
    dev = device_batch()
    q, offsets = queries(dev, 5, 10)
    ws = dev.attend_workspace(q.shape[0])
    ws.fill_(0xFF)
    for name in ("extend", "cross_attend"):
        call = getattr(dev, name)
        assert torch.equal(call(q, offsets, workspace=ws), call(q, offsets))
    with pytest.raises(_lib.PAError, match="PA_ERR_INVALID_ARG"):
        dev.extend(q, offsets, workspace=ws[:-256])


def test_quest_buffers_are_made_on_the_calls_stream():
    dev = device_batch((3000, 900, 5000))
    dev.quest_build_summaries()
    summaries = dev.key_summaries.clone()
    dev.quest_buffers(9)
    pages = dev.quest_select(9).clone()
    assert (summaries != 0).any() and (pages >= 0).any()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(BUSY)
        dev.quest_build_summaries(stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(dev.key_summaries, summaries)
        del dev.selected_pages
        scores = dev.page_scores.clone()
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        got = dev.quest_select(9, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, pages) and torch.equal(dev.page_scores, scores)
    assert dev.read_err() == 0


def test_long_prompt_beside_a_wide_block_table():
    """32,768 tokens in one call, with a block table of 131,072 positions: the same bytes as in two calls
    of half as many."""
    T, D, Hkv = 32768, 64, 8
    batch = workload.build_batch("long", [T], Hq=8, Hkv=Hkv, D=D, block_size=16, max_blocks=8192, seed=11,
                                 with_pools=False)
    g = torch.Generator(device="cuda").manual_seed(12)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    pools = [rand(batch.nblocks, 16, Hkv, D) for _ in range(2)]
    whole = DeviceBatch(batch, pools=[x.clone() for x in pools] + [None, None])
    half = DeviceBatch(batch, pools=[x.clone() for x in pools] + [None, None])
    q, k, v = rand(T, 8, D), rand(T, Hkv, D), rand(T, Hkv, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = whole.block_tables[0, (pos // 16).long()].long() * 16 + pos.long() % 16
    table = rope_table(T, D)
    out = whole.rope_and_cache(q, k, v, pos, slots, table)
    outs = [half.rope_and_cache(q[i:i + T // 2], k[i:i + T // 2], v[i:i + T // 2], pos[i:i + T // 2],
                                slots[i:i + T // 2], table) for i in (0, T // 2)]
    assert torch.equal(out, torch.cat(outs))
    assert torch.equal(whole.k_pool, half.k_pool) and torch.equal(whole.v_pool, half.v_pool)
    # the plain write and the page summaries of as many tokens
    shape = _lib.make_shape(T, 8, Hkv, D, 16, batch.nblocks, 8192, _lib.PA_KV_BF16)
    _lib.pa_reshape_and_cache(shape, k, v, whole.k_pool, whole.v_pool, None, None, slots, whole.err)
    assert torch.equal(whole.k_pool.view(-1, Hkv, D)[slots], k)
    assert torch.equal(whole.v_pool.view(-1, Hkv, D)[slots], v)
    summaries = torch.zeros(batch.nblocks, Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    _lib.pa_quest_summarize(shape, whole.k_pool, None, summaries, slots, whole.err)
    page = k.view(T // 16, 16, Hkv, D)
    assert torch.equal(summaries[slots[::16] // 16], torch.stack([page.amin(1), page.amax(1)], 2))
    assert whole.read_err() == 0 and half.read_err() == 0
