"""pa_rope_axes_and_cache and pa_read_cache on a GPU.

Tolerances.  A rotated channel is a sum of two products in fp32, each rounded (3 roundings of at most
2^-24 of |a c| + |b s|), then one rounding to bf16 (2^-8 of the value, and of what the first three
moved it by).  A restored code is an fp32 product (2^-24) rounded to bf16 (2^-8); rows of bf16 pools
and copied channels are compared bit for bit.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_28_gb300 as pa
from paged_kv_cache_28_gb300.device import rope_table

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -24
KINDS = {"bf16": pa.PA_KV_BF16, "fp8": pa.PA_KV_FP8_E4M3, "int4": pa.PA_KV_INT4}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def bits(x):
    return x.contiguous().view(torch.int16 if x.dtype == torch.bfloat16 else torch.uint8)


def pools(nblocks, bs, Hkv, D, kind, g):
    """K or V pool and scales with every code, or every kind of bf16, in it."""
    if kind == "bf16":
        return torch.randn(nblocks, bs, Hkv, D, generator=g, device="cuda").bfloat16(), None
    w = D if kind == "fp8" else D // 2
    pool = torch.randint(0, 256, (nblocks, bs, Hkv, w), generator=g, device="cuda", dtype=torch.uint8)
    if kind == "fp8":
        pool[(pool & 0x7F) == 0x7F] = 0x7E               # no NaN codes
    scale = 10.0 ** torch.empty(nblocks, Hkv, device="cuda").uniform_(-4, 1, generator=g)
    scale[0] = 0.0
    return pool, scale


# ------------------------------------------------------------------ several position axes

def arrangements(half, axes):
    yield "runs", sorted(j % axes for j in range(half))
    yield "turns", [j % axes for j in range(half)]
    yield "uneven", [min(axes - 1, (j * j) % 7 // 2) for j in range(half)]


def append(T, Hq, Hkv, D, bs, kind, rotary, seed=0, npos=97):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nblocks = -(-T // bs) + 2
    x = dict(T=T, Hq=Hq, Hkv=Hkv, D=D, bs=bs, kind=kind, g=g)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    x["q"], x["k"], x["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    order = torch.randperm(nblocks, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    x["slots"] = order[t // bs] * bs + t % bs
    x["table"] = rope_table(npos, rotary, 10000.0)
    x["shape"] = pa.make_shape(T, Hq, Hkv, D, bs, nblocks, 1, KINDS[kind])
    x["pools"] = [pools(nblocks, bs, Hkv, D, kind, g) for _ in "kv"]
    x["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return x


def call(x, axis, positions, interleaved, fn=None, table=None, **kw):
    """(q_out, k pool, v pool, k scale, v scale) after the call, the case's own left alone."""
    (kp, ks), (vp, vs) = [(p.clone(), None if s is None else s.clone()) for p, s in x["pools"]]
    out = torch.full((x["T"], x["Hq"], x["D"]), -3.0, dtype=torch.bfloat16, device="cuda")
    table = x["table"] if table is None else table
    rest = (out, x["q"], x["k"], x["v"], kp, vp, ks, vs, x["slots"], x["err"])
    if axis is None:
        pa.pa_rope_and_cache(x["shape"], table, positions, *rest, interleaved=interleaved, **kw)
    else:
        pa.pa_rope_axes_and_cache(x["shape"], axis, table, positions, *rest, interleaved=interleaved, **kw)
    return out, kp, vp, ks, vs


def own_table(table, positions, axis):
    """A table with a row for each token: pair j's angles from the row of its axis."""
    half = table.shape[1] // 2
    at = positions.long()[torch.tensor(list(axis), device="cuda")].T
    j = torch.arange(half, device="cuda")
    return torch.cat([table[at, j], table[at, half + j]], 1).contiguous()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,bs,kind,rotary,axes", [
    (1, 8, 2, 64, 16, "bf16", 64, 3), (5, 4, 4, 128, 32, "bf16", 128, 4), (77, 24, 8, 128, 16, "bf16", 96, 2),
    (300, 7, 7, 64, 16, "bf16", 16, 3), (1, 64, 8, 128, 16, "fp8", 128, 3), (39, 16, 1, 128, 32, "fp8", 128, 3),
    (1100, 8, 4, 128, 16, "fp8", 48, 4), (2100, 8, 1, 128, 16, "int4", 128, 3), (33, 6, 2, 128, 32, "int4", 32, 1),
])
def test_axes_match_a_table_row_per_token(T, Hq, Hkv, D, bs, kind, rotary, axes, interleaved):
    """The same bits as the one-axis call whose table has each token's own angles as a row."""
    x = append(T, Hq, Hkv, D, bs, kind, rotary, seed=T)
    pos = torch.randint(0, 97, (axes, T), generator=x["g"], device="cuda", dtype=torch.int32)
    for name, axis in arrangements(rotary // 2, axes):
        got = call(x, axis, pos, interleaved)
        want = call(x, None, torch.arange(T, dtype=torch.int32, device="cuda"), interleaved,
                    table=own_table(x["table"], pos, axis))
        for a, b in zip(got, want):
            if a is not None:
                assert torch.equal(a if a.dtype == torch.float32 else bits(a),
                                   b if b.dtype == torch.float32 else bits(b)), name
    assert pa.pa_read_error_flag(x["err"]) == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rotary", [(64, 64), (128, 80)])
def test_axes_against_the_formula(D, rotary, interleaved):
    x = append(50, 8, 2, D, 16, "bf16", rotary, seed=3)
    half = rotary // 2
    axis = [(j * 5) % 3 for j in range(half)]
    pos = torch.randint(0, 97, (3, 50), generator=x["g"], device="cuda", dtype=torch.int32)
    out, kp, vp, _, _ = call(x, axis, pos, interleaved)
    c, s = own_table(x["table"], pos, axis).double().view(50, 1, 2, half).unbind(2)
    ia = torch.arange(half, device="cuda") * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else half)
    k = kp.view(-1, 2, D)[x["slots"]]
    for src, got in ((x["q"], out), (x["k"], k)):
        a, b = src.double()[..., ia], src.double()[..., ib]
        for want, size, ch in ((a * c - b * s, (a * c).abs() + (b * s).abs(), ia),
                               (b * c + a * s, (b * c).abs() + (a * s).abs(), ib)):
            moved = 3 * E * size
            assert ((got.double()[..., ch] - want).abs() <= U * (want.abs() + moved) + moved).all()
        assert torch.equal(bits(got[..., rotary:]), bits(src[..., rotary:]))
    assert torch.equal(bits(vp.view(-1, 2, D)[x["slots"]]), bits(x["v"]))


def test_axes_skip_padding_and_bad_positions():
    for kind in KINDS:
        x = append(40, 8, 2, 128, 16, kind, 128, seed=7)
        axis = [j % 3 for j in range(64)]
        pos = torch.randint(0, 97, (3, 40), generator=x["g"], device="cuda", dtype=torch.int32)
        pos[0, 3], pos[1, 17], pos[2, 39] = -1, 97, 2 ** 30          # one axis each
        x["slots"][20] = -1
        skipped = [3, 17, 20, 39]
        kept = [t for t in range(40) if t not in skipped]
        got = call(x, axis, pos, False)
        assert pa.pa_read_error_flag(x["err"]) == pa.PA_DEVERR_POSITION
        assert (got[0][skipped] == -3.0).all() and not (got[0][kept] == -3.0).all(-1).any()
        # the same as those tokens being padding, with good positions
        y = dict(x, err=torch.zeros_like(x["err"]), slots=x["slots"].clone())
        y["slots"][skipped] = -1
        want = call(y, axis, pos.clamp(0, 96), False)
        for a, b in zip(got, want):
            if a is not None:
                assert torch.equal(a if a.dtype == torch.float32 else bits(a),
                                   b if b.dtype == torch.float32 else bits(b))
        assert pa.pa_read_error_flag(y["err"]) == 0


def test_axes_keys_only_captured_on_another_stream():
    x = append(64, 8, 2, 128, 16, "fp8", 128, seed=9)
    axis = bytes(j % 3 for j in range(64))
    pos = torch.randint(0, 97, (3, 64), generator=x["g"], device="cuda", dtype=torch.int32)
    want = call(x, axis, pos, True)
    (kp, ks), (vp, vs) = [(p.clone(), s.clone()) for p, s in x["pools"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_rope_axes_and_cache(x["shape"], axis, x["table"], pos, None, None, x["k"], x["v"], kp, vp, ks, vs,
                                  x["slots"], x["err"], interleaved=True)
    for _ in range(2):                  # offset 0 starts a block's scale anew: twice gives the same
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((kp, vp, ks, vs), want[1:]):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ reading the cache

def restored(pool, scale, kind):
    if kind == "bf16":
        return pool
    if kind == "fp8":
        x = pool.view(torch.float8_e4m3fn).double()
    else:
        x = torch.stack([(pool & 15).double() - 8, (pool >> 4).double() - 8], -1).flatten(-2)
    return x * scale.double()[:, None, :, None]


def cache(L, Hkv, D, bs, kind, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-x // bs) for x in L]
    nblocks, width = sum(need) + 3, max(need + [1]) + 1
    order = torch.randperm(nblocks, generator=g, device="cuda").int()
    bt = torch.full((len(L), width), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        bt[b, :k] = order[at:at + k]
        at += k
    (kp, ks), (vp, vs) = (pools(nblocks, bs, Hkv, D, kind, g) for _ in "kv")
    shape = pa.make_shape(len(L), Hkv, Hkv, D, bs, nblocks, width, KINDS[kind])
    return dict(L=L, Hkv=Hkv, D=D, bs=bs, kind=kind, bt=bt, k=(kp, ks), v=(vp, vs), shape=shape,
                sl=torch.tensor(L, dtype=torch.int32, device="cuda"),
                err=torch.zeros(1, dtype=torch.int32, device="cuda"))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def read(c, offsets, T, starts=None, shift=0, which="kv", **kw):
    """Rows -3 where nothing is written; shift: bf16 elements past a 32-byte boundary."""
    out = {}
    for x in which:
        flat = torch.full((T * c["Hkv"] * c["D"] + 16,), -3.0, dtype=torch.bfloat16, device="cuda")
        out[x] = flat[shift:shift + T * c["Hkv"] * c["D"]].view(T, c["Hkv"], c["D"])
    pa.pa_read_cache(c["shape"], out.get("k"), out.get("v"), c["k"][0] if "k" in which else None,
                     c["v"][0] if "v" in which else None, c["k"][1] if "k" in which else None,
                     c["v"][1] if "v" in which else None, c["bt"], c["sl"], ints(offsets),
                     None if starts is None else ints(starts), c["err"], **kw)
    return out


def check_rows(c, out, offsets, starts, zeros=()):
    """zeros: (sequence, position) that read zeros."""
    for x, got in out.items():
        pool, scale = c[x]
        all_rows = restored(pool, scale, c["kind"]).reshape(-1, c["Hkv"], c["D"])
        T = got.shape[0]
        touched = torch.zeros(T, dtype=torch.bool, device="cuda")
        for b in range(len(c["L"])):
            q0, q1 = offsets[b], offsets[b + 1]
            touched[q0:q1] = True
            pos = torch.arange(q1 - q0, device="cuda") + (starts[b] if starts is not None else 0)
            bad = torch.tensor([(b, int(p)) in zeros for p in pos], dtype=torch.bool, device="cuda")
            rows = c["bt"][b, (pos // c["bs"]).clamp(0, c["bt"].shape[1] - 1)].long() * c["bs"] + pos % c["bs"]
            want = all_rows[torch.where(bad, 0, rows)]
            want = torch.where(bad[:, None, None], torch.zeros((), dtype=want.dtype, device="cuda"), want)
            mine = got[q0:q1]
            if c["kind"] == "bf16":
                assert torch.equal(bits(mine), bits(want)), (x, b)
            else:
                assert ((mine.double() - want).abs() <= (U + 2 * E) * want.abs()).all(), (x, b)
        assert (got[~touched] == -3.0).all()


@pytest.mark.parametrize("kind,D", [("bf16", 64), ("bf16", 128), ("fp8", 128), ("int4", 128)])
@pytest.mark.parametrize("L,Hkv,bs,shift", [
    ([1], 1, 16, 0), ([0, 5, 0], 2, 32, 8), ([16, 17, 15, 33], 3, 16, 0), ([700, 1, 0, 0, 260], 8, 32, 0),
    ([40] * 45, 1, 16, 8), ([2, 0, 1] * 400, 2, 16, 0), ([90], 160, 16, 0),
])
def test_read_whole_sequences(L, Hkv, bs, shift, kind, D):
    c = cache(L, Hkv, D, bs, kind, seed=sum(L))
    offsets = np.concatenate([[3], 3 + np.cumsum(L)]).tolist()      # three rows before, two behind
    out = read(c, offsets, offsets[-1] + 2, shift=shift)
    assert pa.pa_read_error_flag(c["err"]) == 0
    check_rows(c, out, offsets, None)


@pytest.mark.parametrize("kind", list(KINDS))
def test_read_ranges_and_one_tensor(kind):
    L, n, start = [100, 37, 64, 5], [31, 0, 64, 1], [69, 12, 0, 4]
    c = cache(L, 4, 128, 16, kind, seed=2)
    offsets = np.concatenate([[0], np.cumsum(n)]).tolist()
    both = read(c, offsets, offsets[-1], start)
    check_rows(c, both, offsets, start)
    for x in "kv":
        one = read(c, offsets, offsets[-1], start, which=x)
        assert torch.equal(bits(one[x]), bits(both[x]))
    assert pa.pa_read_error_flag(c["err"]) == 0


@pytest.mark.parametrize("kind", list(KINDS))
def test_read_outside_gives_zeros(kind):
    L = [40, 20, 30]
    c = cache(L, 2, 128, 16, kind, seed=4)
    # past the length, before the first position
    offsets, start = [0, 10, 25, 30], [35, -5, 25]
    out = read(c, offsets, 30, start)
    assert pa.pa_read_error_flag(c["err"]) == pa.PA_DEVERR_SEQ_LEN
    check_rows(c, out, offsets, start, {(0, p) for p in range(40, 45)} | {(1, p) for p in range(-5, 0)})
    # a bad block
    c["err"].zero_()
    c["bt"][1, 0] = -1
    c["bt"][2, 1] = c["shape"].nblocks
    offsets = [0, 0, 20, 50]
    out = read(c, offsets, 50)
    assert pa.pa_read_error_flag(c["err"]) == pa.PA_DEVERR_BLOCK_ID
    check_rows(c, out, offsets, None, {(1, p) for p in range(16)} | {(2, p) for p in range(16, 30)})
    # a length beyond the block table, the largest start
    c["err"].zero_()
    c["sl"][0] = 2 ** 31 - 1
    width = c["bt"].shape[1] * 16
    out = read(c, [0, 3, 6, 6], 6, [width - 1, 2 ** 31 - 1, 0])
    assert pa.pa_read_error_flag(c["err"]) & pa.PA_DEVERR_SEQ_LEN
    assert (out["k"][1:] == 0).all() and (out["v"][1:] == 0).all()


def test_read_reports_bad_offsets():
    c = cache([40, 20, 30], 2, 64, 16, "bf16", seed=5)
    for offsets in ([0, 10, 5, 12], [-1, 4, 8, 12], [0, 4, 8, 13], [5, 4, 3, 2]):
        c["err"].zero_()
        read(c, offsets, 12)
        assert pa.pa_read_error_flag(c["err"]) & pa.PA_DEVERR_QUERY, offsets


def test_read_keeps_nan_and_infinity():
    c = cache([64], 1, 128, 16, "bf16", seed=6)
    c["k"][0].view(torch.int16).copy_(torch.arange(5 * 16 * 128 * 2, device="cuda")[:c["k"][0].numel()].view_as(
        c["k"][0]).to(torch.int16))
    check_rows(c, read(c, [0, 64], 64), [0, 64], None)
    c = cache([16], 1, 128, 16, "fp8", seed=6)
    block = int(c["bt"][0, 0])
    c["k"][0][block, 3, 0, 5] = 0x7F
    c["k"][1][block] = float("inf")
    got = read(c, [0, 16], 16)["k"]
    code = c["k"][0][block].view(torch.float8_e4m3fn).float()
    want = code * float("inf")
    assert torch.equal(got.float().nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))


def test_read_beyond_4_gib():
    """Rows at the end of a pool of 4.3 GB, and output rows past 2^31 bytes."""
    nblocks, bs, Hkv, D = 66000, 32, 8, 128
    g = torch.Generator(device="cuda").manual_seed(8)
    pool = torch.empty(nblocks, bs, Hkv, D, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(40, bs, Hkv, D, generator=g, device="cuda").bfloat16()
    pool[-40:] = last
    T = 1_100_000
    width = -(-T // bs)
    bt = torch.randint(nblocks - 40, nblocks, (1, width), generator=g, device="cuda", dtype=torch.int32)
    shape = pa.make_shape(1, Hkv, Hkv, D, bs, nblocks, width, pa.PA_KV_BF16)
    out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_read_cache(shape, out, None, pool, None, None, None, bt, ints([T]), ints([0, T]), None, err)
    assert pa.pa_read_error_flag(err) == 0
    t = torch.arange(T - 5000, T, device="cuda")
    want = last[bt[0, t // bs].long() - (nblocks - 40), t % bs]
    assert torch.equal(bits(out[-5000:]), bits(want))


def test_read_after_writing_in_a_graph_on_another_stream():
    """A prompt is rotated, written and read back, captured and replayed twice."""
    x = append(70, 8, 2, 128, 16, "int4", 128, seed=11)
    axis = [j % 3 for j in range(64)]
    pos = torch.randint(0, 97, (3, 70), generator=x["g"], device="cuda", dtype=torch.int32)
    want = call(x, axis, pos, False)
    (kp, ks), (vp, vs) = [(p.clone(), s.clone()) for p, s in x["pools"]]
    order = (x["slots"][::16] // 16).int()[None].contiguous()
    shape = pa.make_shape(1, 8, 2, 128, 16, x["shape"].nblocks, order.shape[1], pa.PA_KV_INT4)
    ko, vo = (torch.full((70, 2, 128), -3.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    sl, off = ints([70]), ints([0, 70])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_rope_axes_and_cache(x["shape"], axis, x["table"], pos, None, None, x["k"], x["v"], kp, vp, ks, vs,
                                  x["slots"], x["err"])
        pa.pa_read_cache(shape, ko, vo, kp, vp, ks, vs, order, sl, off, None, x["err"])
    for _ in range(2):
        ko.fill_(-3.0)
        graph.replay()
    torch.cuda.synchronize()
    for got, pool, scale in ((ko, want[1], want[3]), (vo, want[2], want[4])):
        ref = restored(pool, scale, "int4").view(-1, 2, 128)[x["slots"]]
        assert ((got.double() - ref).abs() <= (U + 2 * E) * ref.abs()).all()
    assert pa.pa_read_error_flag(x["err"]) == 0
