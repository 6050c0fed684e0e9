"""pa_rope_and_cache, pa_extend and pa_cross_attend on a GPU against plain 64-bit forms.

Tolerances.  A rounding to bf16 is off by at most u = 2^-8 of the value (half a step).  The
attention rounds each weight to bf16 before the second product (error <= u sum_j w_j |V_j| / sum_j
w_j = u A) and its result once (<= u |out|).  What 32 bits add: a score is a sum of D <= 128
products and its rounding, off by <= D 2^-24 s with s = scale sum |q k|, which is the relative
error of its weight, above and below the fraction; sums over N keys add N 2^-24 of A on each side:
    |out - ref| <= u |ref| + (u + 2 (D s + N + 16) 2^-24) A
(16: the exponential's own error and the scale factors).  Where every weight is exactly 1 (q = 0)
only the sums and the last rounding are left.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_28_gb300 as pa
from paged_kv_cache_28_gb300.device import rope_table

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
KINDS = {"bf16": pa.PA_KV_BF16, "fp8": pa.PA_KV_FP8_E4M3, "int4": pa.PA_KV_INT4}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def restore(pool, scale, kind):
    """The values of a pool [nblocks, bs, Hkv, D] in 64 bits."""
    if kind == "bf16":
        return pool.double()
    if kind == "fp8":
        x = pool.view(torch.float8_e4m3fn).double()
    else:
        x = torch.stack([(pool & 15).double() - 8, (pool >> 4).double() - 8], -1).flatten(-2)
    return x * scale.double()[:, None, :, None]


class Batch:
    """Ragged sequences over a pool whose every row that no token sees is NaN (bf16 and E4M3)."""

    def __init__(self, n, L, Hkv, G, D=128, bs=16, kind="bf16", window=0, causal=True, seed=0, qmul=1.0,
                 extra_rows=3, max_blocks=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.L, self.Hkv, self.G, self.D, self.bs = n, L, Hkv, G, D, bs
        self.kind, self.window, self.causal = kind, window, causal
        self.Hq, self.B = Hkv * G, len(n)
        need = [-(-x // bs) for x in L]
        self.nblocks = sum(need) + 4
        self.max_blocks = max_blocks or max(need + [1]) + 2
        order = torch.randperm(self.nblocks, generator=g, device="cuda").int()
        bt = torch.full((self.B, self.max_blocks), -7, dtype=torch.int32, device="cuda")
        at = 0
        for b, k in enumerate(need):
            bt[b, :k] = order[at:at + k]
            at += k
        self.block_tables = bt
        shape = (self.nblocks, bs, Hkv, D)
        self.k_scale = self.v_scale = None
        if kind == "bf16":
            self.k = torch.randn(shape, generator=g, device="cuda").bfloat16()
            self.v = torch.randn(shape, generator=g, device="cuda").bfloat16()
        elif kind == "fp8":
            self.k = (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(
                torch.float8_e4m3fn).view(torch.uint8)
            self.v = (torch.randn(shape, generator=g, device="cuda") * 100).clamp(-448, 448).to(
                torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.k, self.v = (torch.randint(0, 256, (*shape[:3], D // 2), generator=g, device="cuda",
                                            dtype=torch.uint8) for _ in range(2))
            for x in (self.k, self.v):           # nibbles 1..15
                x |= ((x & 15) == 0).to(torch.uint8) | (((x >> 4) == 0).to(torch.uint8) << 4)
        if kind != "bf16":
            unit = 0.01 if kind == "fp8" else 0.25
            self.k_scale, self.v_scale = (unit * (0.5 + torch.rand(self.nblocks, Hkv, generator=g,
                                                                   device="cuda")) for _ in range(2))
        # rows that some token sees
        seen = torch.zeros(self.nblocks * bs, dtype=torch.bool, device="cuda")
        for b in range(self.B):
            lo = max(0, L[b] - n[b] - window + 1) if causal and window else 0
            pos = torch.arange(lo, L[b], device="cuda")
            seen[bt[b, pos // bs].long() * bs + pos % bs] = True
        self.seen = seen
        if kind != "int4":
            for x in (self.k, self.v):
                x.view(-1, Hkv, D)[~seen] = float("nan") if kind == "bf16" else 0x7F
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        self.seq_lens = torch.tensor(L, dtype=torch.int32, device="cuda")
        self.T = sum(n) + extra_rows
        self.q = (torch.randn(self.T, self.Hq, D, generator=g, device="cuda") * qmul).bfloat16()
        self.scale = D ** -0.5
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.shape = pa.make_shape(self.B, self.Hq, Hkv, D, bs, self.nblocks, self.max_blocks, KINDS[kind])
        self.ws = workspace(self.shape, self.T)

    def run(self, out=None, stream=None):
        out = torch.full((self.T, self.Hq, self.D), -3.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        args = (self.shape, out, self.q, self.offsets, self.k, self.v, self.k_scale, self.v_scale,
                self.block_tables, self.seq_lens, self.scale, self.ws, self.err, stream)
        if self.causal:
            pa.pa_extend(*args, window=self.window)
        else:
            pa.pa_cross_attend(*args)
        return out

    def reference(self):
        """The result in 64 bits, and the bound's second term."""
        ref = torch.full((self.T, self.Hq, self.D), -3.0, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(ref)
        kd, vd = restore(self.k, self.k_scale, self.kind), restore(self.v, self.v_scale, self.kind)
        at = 0
        for b in range(self.B):
            n, L = self.n[b], self.L[b]
            pos = torch.arange(L, device="cuda")
            rows = self.block_tables[b, pos // self.bs].long() * self.bs + pos % self.bs
            ok = self.seen[rows][:, None, None]
            zero = torch.zeros((), dtype=torch.float64, device="cuda")
            k = torch.where(ok, kd.view(-1, self.Hkv, self.D)[rows], zero)
            v = torch.where(ok, vd.view(-1, self.Hkv, self.D)[rows], zero)
            q = self.q[at:at + n].double().view(n, self.Hkv, self.G, self.D)
            s = torch.einsum("ihgd,jhd->hgij", q, k) * self.scale
            slack = 0.0
            if n and L:
                top = float(torch.einsum("ihgd,jhd->hgij", q.abs(), k.abs()).max()) * abs(self.scale)
                slack = 2 * (self.D * top + L + 16) * 2.0 ** -24
            if self.causal:
                me = torch.arange(n, device="cuda")[:, None] + (L - n)
                hide = pos > me
                if self.window:
                    hide |= pos <= me - self.window
                s = s.masked_fill(hide, -math.inf)
            if L:
                w = s.softmax(-1)
                ref[at:at + n] = torch.einsum("hgij,jhd->ihgd", w, v).reshape(n, self.Hq, self.D)
                size[at:at + n] = (U + slack) * torch.einsum("hgij,jhd->ihgd", w, v.abs()).reshape(
                    n, self.Hq, self.D)
            else:
                ref[at:at + n] = 0
            at += n
        return ref, size

    def check(self, out=None):
        out = self.run() if out is None else out
        torch.cuda.synchronize()
        assert pa.pa_read_error_flag(self.err) == 0
        ref, size = self.reference()
        bad = ~((out.double() - ref).abs() <= U * ref.abs() + size)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off; first {bad.nonzero()[0].tolist()}"


def workspace(shape, T):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return torch.full((pa.pa_attend_workspace_bytes(shape, T, sms),), 0xFF, dtype=torch.uint8, device="cuda")


HEADS = [(2, 4, 64, 16), (1, 8, 128, 16), (3, 1, 128, 32), (2, 3, 64, 32), (1, 5, 128, 16), (2, 16, 128, 32)]
LENGTHS = {
    "one": ([1], [1]),
    "one of many": ([1], [700]),
    "few": ([4], [100]),
    "tile edges": ([127, 1, 16], [128, 129, 127]),
    "prompt": ([300], [300]),
    "ragged": ([5, 0, 33, 1, 130], [5, 40, 1000, 257, 131]),
    "page ends": ([17, 31, 1], [17, 47, 33]),
    "many short": ([1, 2, 3, 1, 2, 3] * 30, [1, 2, 30, 17, 60, 129] * 30),
}


def kinds_of(D):
    return ["bf16"] if D == 64 else ["bf16", "fp8", "int4"]


CASES = [(h, name, kind) for h in HEADS for name in LENGTHS for kind in kinds_of(h[2])]


@pytest.mark.parametrize("heads,name,kind", CASES)
def test_extend(heads, name, kind):
    Hkv, G, D, bs = heads
    n, L = LENGTHS[name]
    Batch(n, L, Hkv, G, D, bs, kind, seed=3).check()


@pytest.mark.parametrize("heads,name,kind", CASES)
def test_cross_attend(heads, name, kind):
    Hkv, G, D, bs = heads
    n, L = LENGTHS[name]
    L = L[::-1]
    L[0] = 0 if len(L) > 2 else L[0]             # a sequence without states gives zeros
    Batch(n, L, Hkv, G, D, bs, kind, causal=False, seed=4).check()


@pytest.mark.parametrize("window", [1, 16, 100, 128, 129, 1000])
@pytest.mark.parametrize("G,kind", [(8, "bf16"), (3, "bf16"), (4, "fp8"), (8, "int4")])
def test_extend_window(window, G, kind):
    Batch([200, 3, 1, 140], [900, 600, 513, 140], 2, G, 128, 16, kind, window=window, seed=5).check()


def counting(b):
    """q = 0 makes every weight 1 and V[j] the unit vector of j mod D: channel d of a row times the
    number of keys it sees is the number of them that are d mod D, which shows every key."""
    b.q.zero_()
    for s in range(b.B):
        pos = torch.arange(b.L[s], device="cuda")
        rows = b.block_tables[s, pos // b.bs].long() * b.bs + pos % b.bs
        keep = b.seen[rows]
        one = torch.nn.functional.one_hot(pos % b.D, b.D)[:, None].expand(-1, b.Hkv, -1).bfloat16()
        b.v.view(-1, b.Hkv, b.D)[rows[keep]] = one[keep]
    out = b.run().double()
    assert pa.pa_read_error_flag(b.err) == 0
    at = 0
    for s in range(b.B):
        n, L = b.n[s], b.L[s]
        i = torch.arange(n, device="cuda")[:, None]
        d = torch.arange(b.D, device="cuda")[None]
        hi = (L - n + i + 1) if b.causal else torch.full_like(i, L)
        lo = (hi - b.window).clamp(min=0) if b.causal and b.window else torch.zeros_like(i)
        upto = lambda x: (x - d + b.D - 1).div(b.D, rounding_mode="floor").clamp(min=0)  # noqa: E731
        want = upto(hi) - upto(lo)
        got = out[at:at + n] * (hi - lo)[:, None].double()
        if n and L:
            assert float(want.max()) * U < 0.49  # a count is told from its neighbours
            assert torch.equal(got.round(), want[:, None].expand_as(got).double()), s
        at += n
    assert (out[at:] == -3.0).all()


@pytest.mark.parametrize("n,L,G,bs,window", [
    ([1], [9000], 8, 16, 0), ([3], [12001], 5, 32, 0), ([700], [8000], 8, 16, 0),
    ([260, 1, 77], [4001, 15999, 300], 8, 32, 0), ([2000], [5003], 1, 16, 0),
    ([513, 9], [6000, 7000], 7, 16, 2500), ([2048], [2048], 16, 16, 300),
    ([40, 300, 0, 1, 5], [10000, 300, 7, 1, 6001], 2, 16, 0),
])
def test_extend_sees_every_key(n, L, G, bs, window):
    counting(Batch(n, L, 2, G, 128, bs, window=window, seed=6))


@pytest.mark.parametrize("n,L,G,D", [([1] * 40, list(range(1, 1600, 40)), 1, 64),
                                     ([448, 60, 3], [1500, 700, 7000], 1, 64),
                                     ([300, 5], [0, 12345], 4, 128)])
def test_cross_attend_sees_every_key(n, L, G, D):
    counting(Batch(n, L, 4, G, D, 16, causal=False, seed=7))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("qmul", [0.0, 8.0, 64.0, -64.0])
def test_large_and_equal_scores(qmul, causal):
    """The reference maximum moves between tiles; a negative sm_scale turns the order around."""
    b = Batch([70, 3], [900, 1300], 2, 8, qmul=abs(qmul), causal=causal, seed=8)
    if qmul < 0:
        b.scale = -b.scale
    b.check()


def test_zero_scale_is_the_mean():
    b = Batch([20], [300], 1, 4, seed=9)
    b.scale = 0.0
    b.check()


def test_rows_outside_the_batch_stay():
    b = Batch([5, 0, 3], [50, 10, 3], 2, 4, seed=10, extra_rows=0)
    b.offsets += 2                               # two rows before the first sequence
    b.T += 4
    b.q = torch.randn(b.T, b.Hq, b.D, device="cuda").bfloat16()
    b.ws = workspace(b.shape, b.T)
    out = b.run()
    assert (out[:2] == -3).all() and (out[10:] == -3).all()
    inner = b.q
    b.q, b.offsets, b.T = inner[2:10].contiguous(), b.offsets - 2, 8
    b.check(out[2:10])


def test_same_bits_on_every_call_and_with_any_workspace_contents():
    b = Batch([40, 1, 7, 300], [3000, 9000, 100, 300], 2, 8, seed=11)
    first = b.run().clone()
    for fill in (0, 0x7F, 0xFF):
        b.ws.fill_(fill)
        assert torch.equal(b.run(), first)


def test_capture_and_replay_with_new_lengths():
    b = Batch([16, 8], [2000, 500], 2, 8, seed=12)
    out = b.run()
    want = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.run(out, stream=torch.cuda.current_stream())
    out.fill_(-3.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    b.L = [300, 444]                             # other lengths in the same buffers
    b.seq_lens.copy_(torch.tensor(b.L, dtype=torch.int32))
    b.k.nan_to_num_()
    b.v.nan_to_num_()
    b.seen[:] = True
    out.fill_(-3.0)
    g.replay()
    b.check(out)


def test_two_streams_at_once():
    bs = [Batch([200], [2000], 2, 8, seed=13), Batch([3] * 20, [700] * 20, 2, 8, seed=14, causal=False)]
    want = [b.run().clone() for b in bs]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(10):
        for b, o, s in zip(bs, outs, streams):
            b.run(o, stream=s)
    torch.cuda.synchronize()
    for b, o, w in zip(bs, outs, want):
        k = sum(b.n)
        assert torch.equal(o[:k], w[:k])


def test_device_errors():
    # a block id outside the pool reads zeros: its keys score 0 and its values add nothing
    b = Batch([1], [40], 1, 2, seed=15)
    b.block_tables[0, 1] = b.nblocks + 5
    b.run()
    assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_BLOCK_ID
    # more query tokens than cached tokens: zeros, and the other sequence as ever
    b = Batch([4, 3], [20, 30], 1, 2, seed=16)
    want = b.run().clone()
    b.seq_lens[0] = 3
    out = b.run()
    assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_SEQ_LEN
    assert (out[:4] == 0).all() and torch.equal(out[4:], want[4:])
    # negative length, length beyond the table
    for bad in (-5, 10 ** 8):
        b.err.zero_()
        b.seq_lens[0] = bad
        b.k.nan_to_num_()
        b.block_tables[0] = b.block_tables[0, 0]
        assert torch.equal(b.run()[4:], want[4:])
        assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_SEQ_LEN
    # offsets that fall, or leave the rows: that sequence is skipped
    for offsets in ([0, 7, 5], [0, 4, 4 + 3 + 4]):
        b = Batch([4, 3], [20, 30], 1, 2, seed=16)
        b.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        out = b.run()
        assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_QUERY
        assert (out[7:] == -3).all()


def test_output_and_queries_on_a_16_byte_boundary():
    """16-byte aligned tensors, not 32: the narrow stores."""
    for n, L in (([40, 3], [300, 5000]), ([300], [300])):
        b = Batch(n, L, 2, 4, seed=25)
        k = b.T * b.Hq * b.D
        b.q = torch.cat([b.q.new_zeros(8), b.q.flatten()])[8:].view(b.q.shape)
        out = torch.full((k + 8,), -3.0, dtype=torch.bfloat16, device="cuda")[8:].view(b.q.shape)
        assert b.q.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16
        b.check(b.run(out))
        assert (out[sum(n):] == -3.0).all()


def test_sequences_that_share_blocks():
    b = Batch([5, 70, 1], [900, 900, 900], 2, 4, seed=26, causal=False)
    b.block_tables[:] = b.block_tables[0]
    b.check()


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("n", [[3, 1], [200]])
def test_zero_scales_restore_to_zero(kind, n):
    """A block whose scale is 0 scores 0 and adds nothing, whatever its codes are."""
    b = Batch(n, [600] * len(n), 2, 4, kind=kind, seed=27)
    b.k_scale[::3] = 0
    b.v_scale[::2] = 0
    b.check()


@pytest.mark.parametrize("kind", ["fp8", "int4"])
def test_scales_over_six_decades(kind):
    """Pages with large V scales among small ones; scores stay within a few units."""
    b = Batch([40, 5], [700, 900], 2, 4, kind=kind, seed=28)
    g = torch.Generator(device="cuda").manual_seed(28)
    b.v_scale *= 10.0 ** torch.randint(-3, 4, b.v_scale.shape, generator=g, device="cuda")
    b.check()


def test_the_most_kv_heads():
    Batch([3, 1], [40, 300], 2048, 1, 64, seed=29).check()


@pytest.mark.parametrize("most", [3, 200])
def test_thousands_of_sequences(most):
    """More than 32 groups of 32 sequences: the places of the segments are found in two steps."""
    r = np.random.default_rng(30)
    n = [int(x) for x in r.integers(0, most, 2500)]
    counting(Batch(n, [a + int(x) for a, x in zip(n, r.integers(1, 60, 2500))], 1, 4, 64, seed=30))


def test_rows_past_4_gib_of_a_pool():
    """Blocks at the end of a 5 GB pool, written by pa_rope_and_cache and read by pa_extend."""
    b = Batch([50, 2], [400, 90], 8, 2, seed=31)
    blocks = 5 * 2 ** 30 // (16 * 8 * 128 * 2)
    far = torch.arange(blocks - b.nblocks, blocks, device="cuda", dtype=torch.int32)
    pools = []
    for x in (b.k, b.v):
        pool = torch.empty(blocks, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
        pool[far.long()] = x
        pools.append(pool)
    want = b.run().clone()
    b.block_tables = torch.where(b.block_tables >= 0, far[b.block_tables.clamp(min=0).long()], -7)
    b.k, b.v = pools
    b.shape = pa.make_shape(b.B, b.Hq, 8, 128, 16, blocks, b.max_blocks, KINDS["bf16"])
    assert torch.equal(b.run(), want)
    a = Append(20, 8, 8, nblocks=8, seed=31)
    small = [x.clone() for x in a.pools]
    a.run()
    lift = torch.where(a.slots >= 0, a.slots + (blocks - 8) * 16, -1)
    for pool, x in zip(pools, small):
        pool[-8:] = x
    pa.pa_rope_and_cache(pa.make_shape(20, 8, 8, 128, 16, blocks, 1, KINDS["bf16"]), a.cos_sin, a.pos, a.q_out, a.q,
                         a.k, a.v, *pools, None, None, lift, a.err)
    for pool, x in zip(pools, a.pools):
        assert torch.equal(pool[-8:], x)
    assert pa.pa_read_error_flag(a.err) == 0


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    r = np.random.default_rng(100 + seed)
    kind = ["bf16", "fp8", "int4"][seed % 3]
    D = 128 if kind != "bf16" or seed % 2 else 64
    B = int(r.integers(1, 9))
    top = int(r.choice([6, 60, 400]))
    n = [int(x) for x in r.integers(0, top, B)]
    L = [a + int(x) for a, x in zip(n, r.integers(0, 1500, B))]
    causal = bool(r.integers(0, 3))
    window = int(r.choice([0, 0, 1, 50, 700, 2 ** 31 - 1])) if causal else 0
    Batch(n, L if causal else L[::-1], int(r.choice([1, 2, 5])), int(r.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])), D,
          int(r.choice([16, 32])), kind, window=window, causal=causal, seed=seed).check()


def test_refuses_a_short_workspace():
    b = Batch([4], [20], 1, 2, seed=17)
    b.ws = b.ws[:-256]
    with pytest.raises(pa.PAError, match="PA_ERR_INVALID_ARG"):
        b.run()


def test_a_batch_without_tokens():
    b = Batch([0, 0], [10, 0], 1, 2, seed=18)
    assert (b.run() == -3).all()
    b = Batch([0], [10], 1, 2, seed=18, extra_rows=0)
    assert b.run().numel() == 0


# ------------------------------------------------------------------ rotation and write

def rotated(x, cos_sin, pos, interleaved):
    """The written formula in the type of cos_sin, not rounded."""
    r = cos_sin.shape[1]
    c, s = cos_sin[pos][:, None, :r // 2], cos_sin[pos][:, None, r // 2:]
    x = x.to(cos_sin.dtype)
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, v = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = u, v
    else:
        y[..., :r // 2], y[..., r // 2:r] = u, v
    return y


def write_codes(x, pool, scale, slots, bs, kind):
    """The quantised write in the order of the tokens, one after the other, in fp32."""
    top = {"fp8": 448.0, "int4": 7.0}[kind]
    per_code = torch.tensor(1.0 / top, dtype=torch.float32, device="cuda")
    code = restore(pool, torch.ones_like(scale), kind).float()

    def encode(v, s):
        y = torch.where(s == 0, torch.zeros_like(v), v / torch.where(s == 0, torch.ones_like(s), s))
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).float() if kind == "fp8" else y.round().clamp(-7, 7)

    for t, slot in enumerate(slots.tolist()):
        if slot < 0:
            continue
        blk, off = divmod(slot, bs)
        v, old = x[t].float(), scale[blk].clone()
        cand = v.abs().amax(-1) * per_code
        new = cand if off == 0 else torch.maximum(old, cand)
        if off:
            again = encode(code[blk, :off] * old[:, None], new[:, None])
            code[blk, :off] = torch.where((new > old)[:, None], again, code[blk, :off])
        code[blk, off] = encode(v, new[:, None])
        scale[blk] = new
    if kind == "fp8":
        pool.copy_(code.to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        u = (code + 8).to(torch.uint8)
        pool.copy_(u[..., 0::2] | (u[..., 1::2] << 4))


class Append:
    def __init__(self, T, Hq, Hkv, D=128, bs=16, kind="bf16", r=None, interleaved=False, fused=False, seed=0,
                 order="runs", nblocks=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.T, self.Hq, self.Hkv, self.D, self.bs, self.kind = T, Hq, Hkv, D, bs, kind
        self.interleaved, self.r = interleaved, r or D
        self.nblocks = nblocks or T // 4 + 5
        blocks = rng.permutation(self.nblocks)
        if order == "runs":                      # runs of consecutive slots, starting inside blocks
            slots, at = [], 0
            while len(slots) < T:
                start = int(rng.integers(0, bs))
                k = min(int(rng.integers(1, 3 * bs)), T - len(slots), (len(blocks) - at) * bs - start)
                for i in range(start, start + k):
                    slots.append(int(blocks[at + i // bs]) * bs + i % bs)
                at = at + (start + k - 1) // bs + 1
                if at >= len(blocks):
                    slots += [-1] * (T - len(slots))
        else:                                    # every slot of some blocks, shuffled
            k = -(-T // bs)
            slots = rng.permutation(np.concatenate([b * bs + np.arange(bs) for b in blocks[:k]]))[:T].tolist()
        self.slots = torch.tensor(slots, dtype=torch.int64, device="cuda")
        self.npos = 5000
        self.pos = torch.from_numpy(rng.integers(0, self.npos, T).astype(np.int32)).cuda()
        self.cos_sin = rope_table(self.npos, self.r, 500000.0)
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
        parts = [qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]]
        self.q, self.k, self.v = parts if fused else [x.contiguous() for x in parts]
        shape = (self.nblocks, bs, Hkv, {"bf16": D, "fp8": D, "int4": D // 2}[kind])
        if kind == "bf16":
            self.pools = [torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2)]
            self.scales = [None, None]
        else:
            self.pools = [torch.randint(0, 0x7F if kind == "fp8" else 256, shape, generator=g, device="cuda",
                                        dtype=torch.uint8) for _ in range(2)]
            self.scales = [torch.rand(self.nblocks, Hkv, generator=g, device="cuda") * 0.02 for _ in range(2)]
        self.shape = pa.make_shape(T, Hq, Hkv, D, bs, self.nblocks, 1, KINDS[kind])
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q_out = torch.full((T, Hq, D), -3.0, dtype=torch.bfloat16, device="cuda")

    def run(self, q="own", q_out=None):
        pa.pa_rope_and_cache(self.shape, self.cos_sin, self.pos, self.q_out if q_out is None else q_out,
                             self.q if isinstance(q, str) else q, self.k, self.v, *self.pools, *self.scales,
                             self.slots, self.err, interleaved=self.interleaved)

    def check(self, keep=None):
        """Queries against 64 bits; keys and values: the bytes of the plain formula (bf16 pools: of
        pa_reshape_and_cache)."""
        keep = self.slots >= 0 if keep is None else keep
        pools = [x.clone() for x in self.pools]
        scales = [None if x is None else x.clone() for x in self.scales]
        self.run()
        k = rotated(self.k, self.cos_sin, self.pos.long().clamp(0, self.npos - 1), self.interleaved).bfloat16()
        slots = torch.where(keep, self.slots, -1)
        if self.kind == "bf16":
            pa.pa_reshape_and_cache(self.shape, k, self.v.contiguous(), *pools, None, None, slots, None)
        else:
            write_codes(k, pools[0], scales[0], slots, self.bs, self.kind)
            write_codes(self.v, pools[1], scales[1], slots, self.bs, self.kind)
        torch.cuda.synchronize()
        for x, y in zip(self.pools + self.scales, pools + scales):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        q = self.q[keep]
        pos = self.pos[keep].long()
        ref = rotated(q, self.cos_sin.double(), pos, self.interleaved)
        # products and their sum in 32 bits: three roundings of parts no larger than |a| + |b|
        part = rotated(q.abs(), torch.ones_like(self.cos_sin).double(), pos, self.interleaved).abs() + 2 * q.abs().double()
        assert ((self.q_out[keep].double() - ref).abs() <= U * ref.abs() + 3 * 2.0 ** -24 * part).all()
        assert (self.q_out[~keep] == -3.0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("T,Hq,Hkv,bs,order", [(1, 8, 1, 16, "runs"), (37, 6, 2, 32, "runs"),
                                               (300, 64, 8, 16, "runs"), (600, 10, 5, 32, "shuffled"),
                                               (257, 16, 16, 16, "shuffled")])
@pytest.mark.parametrize("interleaved,r,fused", [(False, 128, False), (True, 128, True), (False, 32, True),
                                                 (True, 16, False), (False, 112, False)])
def test_rope_and_cache(kind, T, Hq, Hkv, bs, order, interleaved, r, fused):
    Append(T, Hq, Hkv, 128, bs, kind, r, interleaved, fused, seed=T + r, order=order).check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("T,Hq,Hkv,bs,order", [(1024, 12, 12, 16, "runs"), (2047, 4, 2, 16, "shuffled"),
                                               (2048, 6, 3, 32, "runs"), (2055, 5, 5, 32, "shuffled"),
                                               (4100, 2, 2, 16, "shuffled")])
def test_rope_and_cache_of_long_calls(kind, T, Hq, Hkv, bs, order):
    """Calls whose CTAs take all heads, and several tokens each: padding and bad tokens among them,
    a slot that two tokens far apart write, a block's tokens in either order."""
    a = Append(T, Hq, Hkv, 128, bs, kind, seed=T, order=order)
    a.slots[100:118] = -1
    a.slots[9::41] = -1
    a.pos[9::41] = a.npos + 7
    a.slots[333] = a.nblocks * a.bs + 5
    a.pos[700] = -4
    keep = a.slots >= 0
    bad = int(keep[700])
    keep[333] = keep[700] = False
    quantised = kind != "bf16"
    if quantised:
        good = keep.nonzero().flatten()
        a.slots[good[-1]] = a.slots[good[3]]
    a.check(keep)
    assert pa.pa_read_error_flag(a.err) == (pa.PA_DEVERR_SLOT | bad * pa.PA_DEVERR_POSITION
                                            | quantised * pa.PA_DEVERR_FP8_CONFLICT)


@pytest.mark.parametrize("kind", ["fp8", "int4"])
def test_scales_agree_with_reshape_and_cache(kind):
    """The scales of the two writers are off by one unit in the last place at most."""
    a = Append(300, 8, 4, kind=kind, seed=9)
    k = rotated(a.k, a.cos_sin, a.pos.long(), False).bfloat16()
    pools, scales = [x.clone() for x in a.pools], [x.clone() for x in a.scales]
    a.run()
    pa.pa_reshape_and_cache(a.shape, k, a.v, *pools, *scales, a.slots, None)
    for x, y in zip(a.scales, scales):
        assert ((x - y).abs() <= 2.0 ** -23 * y).all()


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("spread", [3, 40, 100])
def test_rope_codes_of_far_apart_values(kind, spread):
    """Codes are correctly rounded quotients whatever the scale: values over 2^-spread .. 2^spread, a
    block of zeros, and scales near the ends of the range."""
    a = Append(400, 4, 4, kind=kind, seed=40 + spread, order="shuffled")
    g = torch.Generator(device="cuda").manual_seed(spread)
    for x in (a.k, a.v):
        x.copy_((x.float() * 2.0 ** torch.randint(-spread, spread + 1, (400, 4, 1), generator=g, device="cuda")).bfloat16())
        x[:, 1] *= 2.0 ** -spread
        x[:, 2] = 0
    for s in a.scales:
        s.zero_()
    for x in a.pools:
        x.fill_(0x38 if kind == "fp8" else 0x88)
    a.check()


@pytest.mark.parametrize("interleaved,r", [(False, 64), (True, 64), (False, 48), (True, 16)])
def test_rope_and_cache_small_heads(interleaved, r):
    Append(77, 9, 3, 64, 16, "bf16", r, interleaved, True, seed=r).check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_rope_skips_padding_and_bad_tokens(kind):
    a = Append(120, 8, 2, kind=kind, seed=3, order="shuffled")
    a.slots[::7] = -1
    a.pos[::7] = -9                              # a padded token's position means nothing
    a.slots[5] = a.nblocks * a.bs
    a.pos[11] = a.npos
    a.pos[24] = -1
    keep = a.slots >= 0
    keep[5] = keep[11] = keep[24] = False
    a.check(keep)
    assert pa.pa_read_error_flag(a.err) == pa.PA_DEVERR_SLOT | pa.PA_DEVERR_POSITION


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_rope_in_place_and_without_queries(kind):
    a = Append(50, 8, 2, kind=kind, seed=4)
    a.run()
    q = a.q.clone()
    keep = a.slots >= 0
    a.run(q, q)
    assert torch.equal(q[keep], a.q_out[keep]) and torch.equal(q[~keep], a.q[~keep])
    b = Append(50, 8, 2, kind=kind, seed=4)
    pa.pa_rope_and_cache(b.shape, b.cos_sin, b.pos, None, None, b.k, b.v, *b.pools, *b.scales, b.slots, b.err)
    c = Append(50, 8, 2, kind=kind, seed=4)
    c.run()
    for x, y in zip(b.pools, c.pools):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("kind", ["fp8", "int4"])
def test_rope_two_tokens_in_one_slot(kind):
    a = Append(700, 4, 2, kind=kind, seed=5, order="shuffled")
    a.slots[650] = a.slots[3]
    a.slots[4] = a.slots[3]
    a.check()
    assert pa.pa_read_error_flag(a.err) == pa.PA_DEVERR_FP8_CONFLICT


def test_rope_far_positions():
    """A table row of a far position holds the angle to 32 bits, and the kernel adds no error."""
    a = Append(40, 4, 2, seed=6)
    a.npos = 1 << 20
    a.cos_sin = rope_table(a.npos, 128, 10000.0)
    a.pos = torch.randint(a.npos - 1000, a.npos, (40,), dtype=torch.int32, device="cuda")
    f = 10000.0 ** -(torch.arange(0, 128, 2, dtype=torch.float64, device="cuda") / 128)
    angle = a.pos.double()[:, None] * f
    row = a.cos_sin[a.pos.long()].double()
    assert (row - torch.cat([angle.cos(), angle.sin()], 1)).abs().max() < 2.0 ** -24 + 2.0 ** -32
    a.check()


# ------------------------------------------------------------------ as they are used together

@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_prompt_in_chunks_then_decode(kind):
    """Three sequences of different lengths: their prompts in two chunks through pa_rope_and_cache
    and pa_extend, then a decode step through pa_rope_and_cache and pa_decode.  Every attention is
    checked against 64 bits on the cache that it read."""
    Hkv, G, D, bs, B = 2, 4, 128, 16, 3
    b = Batch([40, 17, 90], [150, 33, 200], Hkv, G, D, bs, kind, seed=20, max_blocks=14)
    spare = torch.arange(B * 14, device="cuda").view(B, 14).int()
    b.block_tables = spare                       # every sequence has 14 blocks of its own
    b.nblocks = B * 14
    pools = [torch.zeros(b.nblocks, bs, Hkv, D if kind != "int4" else D // 2, device="cuda",
                         dtype=torch.bfloat16 if kind == "bf16" else torch.uint8) for _ in range(2)]
    b.k, b.v = pools
    if kind != "bf16":
        b.k_scale, b.v_scale = (torch.zeros(b.nblocks, Hkv, device="cuda") for _ in range(2))
    b.shape = pa.make_shape(B, b.Hq, Hkv, D, bs, b.nblocks, 14, KINDS[kind])
    b.seen = torch.ones(b.nblocks * bs, dtype=torch.bool, device="cuda")
    cos_sin = rope_table(400, D)
    g = torch.Generator(device="cuda").manual_seed(21)
    done = [0] * B
    for chunk in ([110, 16, 110], [40, 17, 90], [1, 1, 1]):
        T = sum(chunk)
        qkv = torch.randn(T, b.Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
        q, k, v = qkv[:, :b.Hq], qkv[:, b.Hq:b.Hq + Hkv], qkv[:, b.Hq + Hkv:]
        pos = torch.cat([torch.arange(d, d + c, device="cuda") for d, c in zip(done, chunk)]).int()
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(chunk, device="cuda"))
        slots = b.block_tables[seq, (pos // bs).long()].long() * bs + pos.long() % bs
        q_out = torch.empty(T, b.Hq, D, dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_and_cache(pa.make_shape(T, b.Hq, Hkv, D, bs, b.nblocks, 14, KINDS[kind]), cos_sin, pos, q_out,
                             q, k, v, b.k, b.v, b.k_scale, b.v_scale, slots, b.err)
        done = [d + c for d, c in zip(done, chunk)]
        b.n, b.L, b.T, b.q = chunk, list(done), T, q_out
        b.offsets = torch.tensor(np.concatenate([[0], np.cumsum(chunk)]), dtype=torch.int32, device="cuda")
        b.seq_lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        b.ws = workspace(b.shape, T)
        b.check()
        if kind == "bf16":                       # what went into the cache is the rotated key
            want = rotated(k, cos_sin, pos.long(), False).bfloat16()
            assert torch.equal(b.k.view(-1, Hkv, D)[slots], want)
    out = torch.empty(B, b.Hq, D, device="cuda")
    pa.pa_decode(b.shape, out, b.q, b.k, b.v, b.k_scale, b.v_scale, b.block_tables, b.seq_lens, b.scale, b.err)
    ref, size = b.reference()
    assert ((out.double() - ref).abs() <= (1e-3 if kind == "bf16" else 2e-2) * (1 + ref.abs())).all()


def write_codes_nan(x, pool, scale, slots, bs, kind):
    """write_codes for values with NaN: a maximum leaves NaN out unless a vector holds nothing else, a
    comparison with NaN is false, and the code of a NaN is E4M3's NaN or the lowest 4-bit code."""
    top = {"fp8": 448.0, "int4": 7.0}[kind]
    per_code = np.float32(1.0 / top)
    code = restore(pool, torch.ones_like(scale), kind).float().cpu().numpy()
    xs, sc = x.float().cpu().numpy(), scale.cpu().numpy()

    def encode(v, s):
        with np.errstate(all="ignore"):
            y = np.where(s == 0, np.float32(0), v / s)
        if kind == "fp8":
            return torch.from_numpy(y).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
        return np.where(np.isnan(y), np.float32(-7), np.clip(np.rint(y), -7, 7))

    for t, slot in enumerate(slots.tolist()):
        if slot < 0:
            continue
        blk, off = divmod(slot, bs)
        for h in range(xs.shape[1]):
            v, old = xs[t, h], sc[blk, h]
            cand = np.fmax.reduce(np.abs(v)) * per_code
            new = cand if off == 0 or cand > old else old
            if off and new > old:
                code[blk, :off, h] = encode(code[blk, :off, h] * old, new)
            code[blk, off, h] = encode(v, new)
            sc[blk, h] = new
    code = torch.from_numpy(code).cuda()
    if kind == "fp8":
        pool.copy_(code.to(torch.float8_e4m3fn).view(torch.uint8))
    else:
        u = (code + 8).to(torch.uint8)
        pool.copy_(u[..., 0::2] | (u[..., 1::2] << 4))
    scale.copy_(torch.from_numpy(sc).cuda())


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("T,Hkv,order", [(60, 2, "runs"), (2100, 1, "shuffled")])
def test_rope_leaves_nan_out_of_the_scale(kind, T, Hkv, order):
    """A NaN channel costs itself alone, at a block's first row and at others, as in
    pa_reshape_and_cache; only a vector of nothing but NaN sets a NaN scale, and only at offset 0."""
    a = Append(T, 4, Hkv, kind=kind, seed=T, order=order)
    g = torch.Generator(device="cuda").manual_seed(T)
    first = (a.slots % a.bs == 0) & (a.slots >= 0)
    for x in (a.k, a.v):
        one = torch.randint(0, 128, (T, Hkv, 1), generator=g, device="cuda")
        some = (torch.rand(T, Hkv, 1, generator=g, device="cuda") < 0.3) | first[:, None, None]
        x.masked_fill_((torch.arange(128, device="cuda") == one) & some, float("nan"))
        x[::17] = float("nan")
        x[5::23] = -x[5::23].abs() * 8           # raised scales after them
    assert (a.k[first].isnan().any(-1) & ~a.k[first].isnan().all(-1)).any()
    k = rotated(a.k, a.cos_sin, a.pos.long(), False).bfloat16()
    pools, scales = [x.clone() for x in a.pools], [x.clone() for x in a.scales]
    other, others = [x.clone() for x in a.pools], [x.clone() for x in a.scales]
    a.run()
    for x, pool, scale in zip((k, a.v), pools, scales):
        write_codes_nan(x, pool, scale, a.slots, a.bs, kind)
    pa.pa_reshape_and_cache(a.shape, k, a.v, *other, *others, a.slots, None)
    torch.cuda.synchronize()
    assert pa.pa_read_error_flag(a.err) == 0
    for mine, plain, theirs in zip(a.scales, scales, others):
        assert torch.equal(mine.nan_to_num(-1.0), plain.nan_to_num(-1.0))
        assert torch.equal(mine.isnan(), theirs.isnan())
        assert ((mine - theirs).abs() <= 2.0 ** -23 * theirs).logical_or(mine.isnan()).all()
    one_nan = (lambda x: torch.where(x == 0xFF, 0x7F, x)) if kind == "fp8" else (lambda x: x)  # noqa: E731
    for mine, plain in zip(a.pools, pools):
        assert torch.equal(one_nan(mine), one_nan(plain))


@pytest.mark.parametrize("bad", ["nblocks", "far", 2 ** 31 - 1, -1, -2 ** 31, -2 ** 31 + 2])
@pytest.mark.parametrize("kind,n,L,causal", [("bf16", [3, 1], [400, 90], True), ("bf16", [200], [500], True),
                                             ("bf16", [1, 2], [300, 20], False), ("fp8", [3, 1], [400, 90], True),
                                             ("fp8", [200], [500], True), ("int4", [3, 1], [400, 90], True),
                                             ("int4", [200], [500], False)])
def test_blocks_outside_the_pool_read_zeros(kind, n, L, causal, bad):
    """Keys of a block id outside the pool, of either sign, score 0 and count in the softmax's sum, and
    their values add nothing: the same result as for a block of zeros."""
    b = Batch(n, L, 2, 4, kind=kind, causal=causal, seed=32)
    used = set(b.block_tables.flatten().tolist())
    zero = next(i for i in range(b.nblocks) if i not in used)
    for x in (b.k, b.v):
        x[zero] = 0x88 if kind == "int4" else 0
    b.seen.view(b.nblocks, b.bs)[zero] = True
    b.block_tables[0, 1] = zero
    b.check()                                    # with the block of zeros
    ref, size = b.reference()
    b.block_tables[0, 1] = {"nblocks": b.nblocks, "far": b.nblocks + 5}.get(bad, bad)
    out = b.run()
    assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_BLOCK_ID
    assert ((out.double() - ref).abs() <= U * ref.abs() + size).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind,n,L", [("bf16", [3, 2], [400, 9000]), ("bf16", [200, 3], [700, 4000]),
                                      ("fp8", [3, 2], [400, 9000]), ("int4", [200, 3], [700, 4000]),
                                      ("bf16", [3, 2] * 150, [100, 128] * 150),
                                      ("bf16", [40, 60] * 60, [90, 120] * 60),
                                      ("fp8", [3, 2] * 150, [100, 128] * 150),
                                      ("int4", [40, 60] * 60, [90, 120] * 60)])
def test_a_nan_in_a_query_shows(kind, n, L, causal):
    """A query head with a NaN has no weights: its output is NaN, whether its unit was cut or not, and
    every other row is what it was."""
    b = Batch(n, L, 2, 4, kind=kind, causal=causal, seed=33)
    want = b.run().clone()
    hit = torch.zeros(b.T, b.Hq, dtype=torch.bool, device="cuda")
    for row, head, d in ((0, 0, 0), (1, 5, 127), (n[0] - 1, 2, 64), (n[0], 7, 3), (sum(n) - 1, 4, 31)):
        b.q[row, head, d] = float("nan")
        hit[row, head] = True
    out = b.run()
    assert pa.pa_read_error_flag(b.err) == 0
    assert out[hit].isnan().all()
    assert torch.equal(out[~hit], want[~hit])
    b.seq_lens.zero_()                           # nothing to see: zeros all the same
    b.err.zero_()
    assert (b.run()[:sum(n)] == 0).all()


@pytest.mark.parametrize("kind", ["fp8", "int4"])
@pytest.mark.parametrize("causal", [True, False])
def test_half_empty_units_between_full_ones(kind, causal):
    """Shared form: units whose second row tile has no tokens lie between full ones, with more key tiles
    than the scales of a stream are held for."""
    n = [65, 1, 100, 10, 128, 70, 2, 97] * 3
    L = [1500, 2900, 1400, 700, 2300, 900, 5000, 1111] * 3
    Batch(n, L, 2, 8, kind=kind, causal=causal, seed=34).check()


@pytest.mark.parametrize("kind", ["fp8", "subnormal", "int4"])
@pytest.mark.parametrize("n", [[3, 1], [200]])
def test_every_code(kind, n):
    """All finite E4M3 codes, its subnormal ones and zeros by themselves, and all 4-bit codes, in K and V."""
    b = Batch(n, [600] * len(n), 2, 4, kind="fp8" if kind == "subnormal" else kind, seed=35)
    for m, (x, scale) in enumerate(((b.k, b.k_scale), (b.v, b.v_scale))):
        i = torch.arange(x.numel(), device="cuda").view(x.shape) * 7919 + m
        sign = (i // 13 % 2 * 128).to(torch.uint8)
        if kind == "subnormal":                  # up to 7 / 512
            x.copy_((i % 8).to(torch.uint8) | sign)
            scale.fill_(64.0)
        elif kind == "fp8":
            x.copy_((i % 127).to(torch.uint8) | sign)
            scale.fill_(2.0 ** -7)
        else:
            x.copy_((i % 256).to(torch.uint8))
    b.check()
