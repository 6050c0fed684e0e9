"""pa_extend_scored and pa_decode_scored on a GPU against the formula in 64 bits.

Tolerances.  As for pa_extend a weight is rounded to bf16 once (u = 2^-8; pa_decode_scored's are finer)
and the result once.  The exponent of key j's weight, a_j - m, is off by delta_j at most:
    D e s_j          the product of D <= 128 terms, e = 2^-24, s_j = |scale| sum |q k| (a cap only shrinks it)
    2^-20 |a_j|      a capped score (2^-20.7 of its fit and a few e)
    16 e (|a_j| + |bias_j| + |M| + 32)   the bias, the changes of logarithm, the reference's steps (each of
                     more than 8 octaves, so that few of them touch a weight that counts) and the exponential
With A = sum_j w_j |V_j| over the normalised weights and sums over N keys:
    |out - ref| <= u |ref| + u A + sum_j w_j delta_j (|V_j| + |ref|) + 2 N e A
The exponential gives 0 below 2^-126, and the reference lies up to 8 octaves under the largest score, so
weights below 2^-118 of the largest may be lost: with largest value V, N 2^-118 V (a steep slope leaves a
query its own key and, where that key's value is 0, values of e^-100: they count as 0).
A quantised pa_decode_scored holds its weights, 1 for the largest, as f16 numbers whose smallest step is
2^-24: half of it for each of N keys of a largest restored value V adds N 2^-25 V.
"""
import math

import pytest
import torch
from test_gpu_extend import Batch, workspace

import paged_kv_cache_28_gb300 as pa

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Scored(Batch):
    """A batch of pa_extend_scored, or (decode) one token per sequence of pa_decode_scored."""

    def __init__(self, n, L, Hkv, G, *args, cap=0.0, slopes=None, prefix=None, decode=False, **kw):
        kw.setdefault("qmul", 4.0)
        super().__init__(n, L, Hkv, G, *args, **kw)
        self.cap, self.decode = cap, decode
        self.prefix = None if prefix is None else ints(prefix)
        if slopes == "usual":
            slopes = [2.0 ** (-8.0 * (h + 1) / self.Hq) for h in range(self.Hq)]
        self.slopes = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
        if decode:
            self.T = self.B
            self.q = self.q[:self.B].contiguous()
            self.ws = self.decode_workspace()

    def decode_workspace(self, segments=0):
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        n = pa.pa_decode_workspace_bytes(self.shape, segments or pa.pa_default_num_segments(self.shape, sms))
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, out=None, stream=None, ws=None, **kw):
        out = torch.full((self.T, self.Hq, self.D), -3.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        ws = self.ws if ws is None else ws
        pools = (self.k, self.v, self.k_scale, self.v_scale, self.block_tables, self.seq_lens)
        if self.decode:
            pa.pa_decode_scored(self.shape, out, self.q, *pools, self.scale, ws, self.err, stream,
                                window=self.window, softcap=self.cap, slopes=self.slopes, **kw)
        else:
            pa.pa_extend_scored(self.shape, out, self.q, self.offsets, *pools, self.scale, ws, self.err, stream,
                                window=self.window, softcap=self.cap, slopes=self.slopes,
                                prefix_lens=self.prefix, **kw)
        return out

    def values(self, pool, scale):
        if self.kind == "bf16":
            return pool.double()
        if self.kind == "fp8":
            x = pool.view(torch.float8_e4m3fn).double()
        else:
            x = torch.stack([(pool & 15).double() - 8, (pool >> 4).double() - 8], -1).flatten(-2)
        return x * scale.double()[:, None, :, None]

    def reference(self):
        ref = torch.full((self.T, self.Hq, self.D), -3.0, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(ref)
        kd, vd = self.values(self.k, self.k_scale), self.values(self.v, self.v_scale)
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        at = 0
        for b in range(self.B):
            n, L = self.n[b], self.L[b]
            pos = torch.arange(L, device="cuda")
            rows = self.block_tables[b, pos // self.bs].long() * self.bs + pos % self.bs
            ok = self.seen[rows][:, None, None]
            k = torch.where(ok, kd.view(-1, self.Hkv, self.D)[rows], zero)
            v = torch.where(ok, vd.view(-1, self.Hkv, self.D)[rows], zero)
            for i0 in range(0, n, 128):
                i1 = min(n, i0 + 128)
                if L == 0:
                    ref[at + i0:at + i1] = 0
                    continue
                q = self.q[at + i0:at + i1].double().view(i1 - i0, self.Hkv, self.G, self.D)
                me = torch.arange(i0, i1, device="cuda")[:, None] + (L - n)
                s_abs = torch.einsum("ihgd,jhd->hgij", q.abs(), k.abs()) * abs(self.scale)
                a = torch.einsum("ihgd,jhd->hgij", q, k) * self.scale
                if self.cap:
                    a = self.cap * torch.tanh(a / self.cap)
                bias = torch.zeros_like(a)
                if self.slopes is not None:
                    bias = -self.slopes.double().view(self.Hkv, self.G, 1, 1) * (me - pos).abs()
                hide = pos > (me if self.prefix is None else me.clamp(min=int(self.prefix[b]) - 1))
                if self.window:
                    hide = hide | (pos <= me - self.window)
                x = (a + bias).masked_fill(hide, -math.inf)
                w = x.softmax(-1)
                M = x.amax(-1, keepdim=True).abs()
                delta = E * self.D * s_abs + 16 * E * (a.abs() + bias.abs() + M + 32)
                if self.cap:
                    delta = delta + 2.0 ** -20 * a.abs()
                wd = w * torch.where(w > 0, delta, zero)
                out = torch.einsum("hgij,jhd->ihgd", w, v)
                A = torch.einsum("hgij,jhd->ihgd", w, v.abs())
                off = (U + 2 * L * E) * A + torch.einsum("hgij,jhd->ihgd", wd, v.abs()) + \
                    wd.sum(-1).permute(2, 0, 1)[..., None] * out.abs()
                off = off + L * 2.0 ** -118 * v.abs().amax()
                if self.decode and self.kind != "bf16":
                    off = off + L * E / 2 * v.abs().amax()
                ref[at + i0:at + i1] = out.reshape(i1 - i0, self.Hq, self.D)
                size[at + i0:at + i1] = off.reshape(i1 - i0, self.Hq, self.D)
            at += n
        return ref, size


CHANGES = {
    "cap": dict(cap=20.0),
    "bias": dict(slopes="usual"),
    "both": dict(cap=7.0, slopes="usual"),
}
HEADS = [(2, 4, 64, 16), (1, 8, 128, 16), (3, 1, 128, 32), (1, 5, 128, 16), (2, 16, 128, 32)]
LENGTHS = {
    "one": ([1], [1]),
    "few": ([4], [100]),
    "tile edges": ([127, 1, 16], [128, 129, 127]),
    "prompt": ([300], [300]),
    "ragged": ([5, 0, 33, 1, 130], [5, 40, 1000, 257, 131]),
    "many short": ([1, 2, 3, 1, 2, 3] * 30, [1, 2, 30, 17, 60, 129] * 30),
}


def kinds_of(D):
    return ["bf16"] if D == 64 else ["bf16", "fp8", "int4"]


CASES = [(h, name, kind, c) for h in HEADS for name in LENGTHS for kind in kinds_of(h[2]) for c in CHANGES]


# ------------------------------------------------------------------ several tokens per sequence

@pytest.mark.parametrize("heads,name,kind,change", CASES)
def test_extend(heads, name, kind, change):
    Hkv, G, D, bs = heads
    n, L = LENGTHS[name]
    Scored(n, L, Hkv, G, D, bs, kind, seed=3, **CHANGES[change]).check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("change", [{}, *CHANGES.values()], ids=["none", *CHANGES])
@pytest.mark.parametrize("n,L,prefix", [
    ([200, 40, 90], [300, 40, 400], [250, 40, 10]),      # ends among the new tokens, whole, before them
    ([200, 3, 1], [200, 900, 500], [128, 900, -5]),      # at a tile's edge, the whole sequence, none
    ([400], [700], [2 ** 31 - 1]),                       # beyond the sequence: all of it
    ([2, 5, 1], [300, 200, 129], [299, 197, 129]),       # few tokens
    ([33, 270, 64], [33, 300, 1000], [1, 0, 937]),
])
def test_prefixes(n, L, prefix, kind, change):
    for G in (8, 3):
        Scored(n, L, 2, G, 128, 16, kind, prefix=prefix, seed=7, **change).check()


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("window", [1, 100, 129])
def test_prefix_with_a_window(window, kind):
    """The window bounds what a token sees behind it; its prefix, what it sees ahead."""
    n, L = [200, 3, 140, 310], [900, 600, 140, 310]
    for change in ({}, dict(cap=10.0, slopes="usual")):
        Scored(n, L, 2, 8, 128, 16, kind, window=window, prefix=[800, 599, 70, 310], seed=8, **change).check()


@pytest.mark.parametrize("G", [1, 8, 7])
@pytest.mark.parametrize("S", [16, 300])
def test_every_key_of_a_prefix_is_seen(G, S):
    """q = 0 and V[j] the unit vector of j mod D: a row's channels count the keys it sees."""
    g = torch.Generator().manual_seed(S + G)
    n = [int(x) for x in torch.randint(1, S, (9,), generator=g)]
    L = [x + int(torch.randint(0, 900, (1,), generator=g)) for x in n]
    prefix = [int(torch.randint(0, x + 40, (1,), generator=g)) for x in L]
    b = Scored(n, L, 2, G, 128, 32, "bf16", prefix=prefix, seed=S)
    b.q.zero_()
    for s in range(b.B):
        pos = torch.arange(b.L[s], device="cuda")
        rows = b.block_tables[s, pos // 32].long() * 32 + pos % 32
        b.v.view(-1, 2, 128)[rows] = torch.nn.functional.one_hot(pos % 128, 128)[:, None].expand(
            -1, 2, -1).bfloat16()
    out = b.run().double()
    assert pa.pa_read_error_flag(b.err) == 0
    at = 0
    for s in range(b.B):
        last = torch.maximum(torch.arange(L[s] - n[s], L[s]), torch.tensor(min(prefix[s], L[s]) - 1))
        j = torch.arange(L[s])
        for i in range(n[s]):
            count = torch.bincount(j[:int(last[i]) + 1] % 128, minlength=128).double()
            want = (count / count.sum()).cuda()
            # the weights are exactly 1: sums of whole numbers, one quotient, one rounding
            assert ((out[at + i] - want).abs() <= (U + 4 * E) * want).all(), (s, i)
        at += n[s]


def test_unchanged_scores_are_pa_extend():
    for n, L in (([300, 7], [400, 900]), ([3, 1], [1000, 50])):
        for kind in ("bf16", "fp8", "int4"):
            b = Scored(n, L, 2, 8, 128, 16, kind, seed=5)
            want = Batch.run(b)
            assert torch.equal(b.run().view(torch.int16), want.view(torch.int16))
            b.prefix = ints([0, L[1] - n[1] + 1])        # a prefix that adds nothing: other sums, same formula
            b.check()


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("cap,qmul", [(1e-3, 1.0), (1.0, 8.0), (50.0, 64.0), (5.0, -300.0), (1e10, 1.0), (1e-10, 1.0)])
def test_small_and_large_caps(cap, qmul, kind, decode):
    """Scores far below their cap, around it and far past it."""
    for n in ([1, 1], [200, 1])[:1 if decode else 2]:
        Scored(n, [700, 90], 2, 8, 128, 16, kind, cap=cap, qmul=qmul, decode=decode, seed=9).check()


@pytest.mark.parametrize("decode", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("slopes", [[0.0] * 8, [1e-4, 0.5, 3.0, 100.0, 1e6, 1e30, 0.01, 0.0],
                                    [-1e-3, -0.25, 0.25, -2.0, 0.0, 1.0, -10.0, 0.1]])
def test_slopes_of_any_size_and_sign(slopes, kind, decode):
    for n in ([1, 1], [200, 1])[:1 if decode else 2]:
        Scored(n, [900, 130], 1, 8, 128, 16, kind, slopes=slopes, qmul=1.0, decode=decode, seed=10).check()


@pytest.mark.parametrize("factor", [-1.0, 0.0, 1e-4, 300.0])
def test_scales_of_any_size_and_sign(factor):
    for kind in ("bf16", "fp8"):
        for decode in (False, True):
            for change in CHANGES.values():
                b = Scored([1, 1] if decode else [150, 1], [400, 300], 2, 4, 128, 16, kind, decode=decode, seed=11,
                           **change)
                b.scale *= factor
                b.check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_a_nan_in_a_query_shows(kind):
    for n, L in (([3, 2], [400, 900]), ([200, 3], [700, 400])):
        for change in CHANGES.values():
            b = Scored(n, L, 2, 8, 128, 16, kind, prefix=[300, 20], seed=12, **change)
            want = b.run()
            row, head = n[0] - 1, 5
            b.q[row, head, 7] = float("nan")
            got = b.run()
            assert got[row, head].isnan().all()
            got[row, head] = want[row, head]
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_extend_device_errors():
    """As pa_extend: a sequence with more query than cached tokens gives zeros, its prefix or not; a
    prefix of a sequence whose length is out of range does no harm."""
    b = Scored([5, 40, 3], [50, 40, 60], 2, 8, 128, 16, "bf16", prefix=[50, 40, 60], cap=10.0, seed=13)
    want = b.run()
    b.seq_lens[1] = 39
    out = b.run()
    assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_SEQ_LEN
    assert (out[5:45] == 0).all()
    keep = [*range(5), *range(45, 48)]
    assert torch.equal(out[keep].view(torch.int16), want[keep].view(torch.int16))
    b.err.zero_()
    b.seq_lens[1] = -2 ** 31
    assert (b.run()[5:45] == 0).all()
    assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_SEQ_LEN
    b.err.zero_()
    b.seq_lens[1] = 40
    b.offsets[1:3] = ints([45, 5])                       # falls
    b.run()
    assert pa.pa_read_error_flag(b.err) & pa.PA_DEVERR_QUERY


@pytest.mark.parametrize("seed", range(16))
def test_random_batches(seed):
    g = torch.Generator().manual_seed(seed)

    def pick(lo, hi):
        return int(torch.randint(lo, hi, (1,), generator=g))

    kind = ["bf16", "fp8", "int4"][seed % 3]
    B, G = pick(1, 40), [1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 16][pick(0, 11)]
    most = [6, 60, 400][pick(0, 3)]
    n = [pick(0, most) for _ in range(B)]
    L = [x + pick(0, [10, 300, 1500][pick(0, 3)]) for x in n]
    prefix = [pick(-3, x + 20) for x in L] if seed % 4 < 2 else None
    Scored(n, L, pick(1, 4), G, 128, [16, 32][seed % 2], kind, seed=seed, window=[0, 0, pick(1, 700)][pick(0, 3)],
           prefix=prefix, cap=[0.0, 15.0][pick(0, 2)], slopes=[None, "usual"][pick(0, 2)]).check()


# ------------------------------------------------------------------ one token per sequence

@pytest.mark.parametrize("heads", HEADS + [(2, 8, 128, 16), (4, 8, 128, 32), (1, 12, 128, 16)])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("change", [{}, *CHANGES.values()], ids=["none", *CHANGES])
def test_decode(heads, kind, change):
    Hkv, G, D, bs = heads
    if kind not in kinds_of(D):
        return
    for L in ([1], [4000], [0, 5, 16, 17, 0, 900, 33], [7] * 50):
        Scored([1] * len(L), L, Hkv, G, D, bs, kind, decode=True, seed=21, **change).check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("window", [1, 16, 100, 513])
def test_decode_window(window, kind):
    for change in CHANGES.values():
        Scored([1] * 4, [900, 100, 513, 8], 2, 8, 128, 16, kind, window=window, decode=True, seed=22, **change).check()


@pytest.mark.parametrize("segments", [1, 2, 7, 1000])
def test_decode_any_number_of_segments(segments):
    for kind in ("bf16", "fp8"):
        b = Scored([1] * 5, [900, 0, 40, 3000, 17], 2, 8, 128, 16, kind, cap=10.0, slopes="usual", decode=True, seed=23)
        b.check(b.run(ws=b.decode_workspace(segments), num_segments=segments))


def test_decode_agrees_with_extend():
    """One token per sequence through both calls: the same formula, each within its own bound."""
    for kind in ("bf16", "int4"):
        for change in CHANGES.values():
            b = Scored([1] * 6, [900, 1, 40, 300, 17, 2000], 2, 8, 128, 16, kind, decode=True, seed=24, **change)
            b.check()
            b.decode, b.ws = False, workspace(b.shape, b.T)
            b.check()


def test_decode_device_errors():
    b = Scored([1] * 3, [50, 40, 60], 2, 8, 128, 16, "bf16", cap=10.0, slopes="usual", decode=True, seed=25)
    want = b.run()
    b.seq_lens[1] = -4
    out = b.run()
    assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_SEQ_LEN
    assert (out[1] == 0).all()
    assert torch.equal(out[[0, 2]].view(torch.int16), want[[0, 2]].view(torch.int16))
    b.err.zero_()
    b.seq_lens[1] = 40
    b.block_tables[1, 0] = b.nblocks
    b.run()
    assert pa.pa_read_error_flag(b.err) == pa.PA_DEVERR_BLOCK_ID


# ------------------------------------------------------------------ how the calls are made

@pytest.mark.parametrize("decode", [False, True])
def test_same_bits_captured_and_on_two_streams(decode):
    """Two captured calls with a workspace each, replayed together on two streams with new lengths."""
    batches = [Scored([1] * 4 if decode else [150, 1, 20, 3], [900, 40, 300, 77], 2, 8, 128, 16, kind, cap=12.0,
                      slopes="usual", prefix=None if decode else [800, 40, 0, 76], decode=decode, seed=31)
               for kind in ("bf16", "fp8")]
    graphs = []
    for b in batches:
        b.out = torch.full_like(b.q, -3.0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.run(out=b.out)
        graphs.append((graph, side))
    for step in range(3):
        for b in batches:
            b.out.fill_(-3.0)
            b.ws.fill_(step)
        torch.cuda.synchronize()
        for graph, side in graphs:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for b in batches:
            assert torch.equal(b.out.view(torch.int16), b.run().view(torch.int16)), step
            b.check(b.out)
            b.L = [x - 1 for x in b.L] if decode else b.L
            if decode:
                b.seq_lens -= 1


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_same_bits_whatever_ran_before(kind):
    """What an earlier call left in shared memory and beyond a sequence's length is no part of a result:
    the form that a tile takes may not depend on it."""
    for change in CHANGES.values():
        for decode in (False, True):
            n, L = ([1] * 3, [130, 7, 300]) if decode else ([90, 3, 200], [130, 7, 300])
            b = Scored(n, L, 2, 8, 128, 16, kind, qmul=1.0, decode=decode, seed=41, **change)
            other = Scored(n, [x + 77 for x in L], 2, 8, 128, 16, kind, qmul=200.0, decode=decode, seed=42, **change)
            want = b.run()
            b.check(want)
            for _ in range(3):
                other.run()
                assert torch.equal(b.run().view(torch.int16), want.view(torch.int16))


def test_outputs_on_a_16_byte_boundary():
    for decode in (False, True):
        b = Scored([1] * 2 if decode else [40, 1], [300, 40], 2, 3, 64, 16, "bf16", cap=9.0, decode=decode, seed=33)
        flat = torch.full((b.q.numel() + 8,), -3.0, dtype=torch.bfloat16, device="cuda")
        b.check(b.run(out=flat[8:].view_as(b.q)))
        assert (flat[:8] == -3.0).all()


def test_positions_past_2_to_the_20():
    """A long cache whose blocks repeat: distances of more than a million, the last keys weighing most."""
    bs, Hkv, G, D, L = 32, 1, 8, 128, 1_200_003
    g = torch.Generator(device="cuda").manual_seed(40)
    nblocks, width = 512, -(-L // bs)
    k, v = (torch.randn(nblocks, bs, Hkv, D, generator=g, device="cuda").bfloat16() for _ in "kv")
    bt = torch.randint(0, nblocks, (1, width), generator=g, device="cuda", dtype=torch.int32)
    slopes = (2.0 ** -torch.arange(2.0, 18.0, 2.0, device="cuda")).float()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pos = torch.arange(L, device="cuda")
    rows = bt[0, pos // bs].long() * bs + pos % bs
    kd, vd = k.view(-1, D)[rows].double(), v.view(-1, D)[rows].double()
    for n in (1, 5):
        q = torch.randn(n, G, D, generator=g, device="cuda").bfloat16()
        shape = pa.make_shape(1, G, Hkv, D, bs, nblocks, width, pa.PA_KV_BF16)
        me = torch.arange(L - n, L, device="cuda")
        a = torch.einsum("igd,jd->gij", q.double(), kd) * D ** -0.5
        a = a - slopes.double()[:, None, None] * (me[:, None] - pos)
        w = a.masked_fill(pos > me[:, None], -math.inf).softmax(-1)
        ref = torch.einsum("gij,jd->igd", w, vd)
        size = torch.einsum("gij,jd->igd", w, vd.abs())
        # the weights that count lie within 30 / slope <= 2^21 positions: |bias| <= 40
        bound = U * ref.abs() + (U + 2 * L * E + 2 * (128 * 40 + 16 * 120) * E) * size
        outs = [torch.empty_like(q)]
        pa.pa_extend_scored(shape, outs[0], q, ints([0, n]), k, v, None, None, bt, ints([L]), D ** -0.5,
                            workspace(shape, n), err, slopes=slopes)
        if n == 1:
            outs.append(torch.empty_like(q))
            ws = torch.empty(pa.pa_decode_workspace_bytes(shape, pa.pa_default_num_segments(shape, sms)),
                             dtype=torch.uint8, device="cuda")
            pa.pa_decode_scored(shape, outs[1], q, k, v, None, None, bt, ints([L]), D ** -0.5, ws, err, slopes=slopes)
        assert pa.pa_read_error_flag(err) == 0
        for out in outs:
            assert ((out.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_a_layer_from_its_prompt_to_its_next_tokens(kind):
    """Positions with several axes, the write, capped attention of a prompt whose image sees all of
    itself, a decode step behind it and the cache read back, as a model's layer would run them."""
    from paged_kv_cache_28_gb300.device import rope_table
    Hkv, G, D, bs, L, image = 2, 4, 128, 16, 150, 100
    Hq, total = Hkv * G, 152
    g = torch.Generator(device="cuda").manual_seed(50)
    pool_kind = {"bf16": pa.PA_KV_BF16, "fp8": pa.PA_KV_FP8_E4M3, "int4": pa.PA_KV_INT4}[kind]
    nblocks = 14
    row = {"bf16": (D, torch.bfloat16), "fp8": (D, torch.uint8), "int4": (D // 2, torch.uint8)}[kind]
    k, v = (torch.zeros(nblocks, bs, Hkv, row[0], dtype=row[1], device="cuda") for _ in "kv")
    ks = vs = None
    if kind != "bf16":
        ks, vs = (torch.zeros(nblocks, Hkv, device="cuda") for _ in "kv")
    bt = torch.randperm(nblocks, generator=g, device="cuda")[None, :10].int().contiguous()
    qkv = torch.randn(total, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    q, kn, vn = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = torch.arange(total, device="cuda")
    axes = torch.stack([pos.clamp(min=image), pos // 10, pos % 10]).int()
    slots = bt[0, pos // bs].long() * bs + pos % bs
    table, pair = rope_table(200, D), [j % 3 for j in range(D // 2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, q_out = torch.empty(total, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(q).contiguous()
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def shape(B, width=10):
        return pa.make_shape(B, Hq, Hkv, D, bs, nblocks, width, pool_kind)

    steps = [(0, L), (L, L + 1), (L + 1, total)]
    for t0, t1 in steps:
        n = t1 - t0
        pa.pa_rope_axes_and_cache(shape(n), pair, table, axes[:, t0:t1].contiguous(), q_out[t0:t1], q[t0:t1],
                                  kn[t0:t1], vn[t0:t1], k, v, ks, vs, slots[t0:t1].clone(), err)
        if n > 1:
            pa.pa_extend_scored(shape(1), out[t0:t1], q_out[t0:t1], ints([0, n]), k, v, ks, vs, bt, ints([t1]),
                                D ** -0.5, workspace(shape(1), n), err, softcap=5.0, prefix_lens=ints([image]))
        else:
            ws = torch.empty(pa.pa_decode_workspace_bytes(shape(1), pa.pa_default_num_segments(shape(1), sms)),
                             dtype=torch.uint8, device="cuda")
            pa.pa_decode_scored(shape(1), out[t0:t1], q_out[t0:t1], k, v, ks, vs, bt, ints([t1]), D ** -0.5, ws, err,
                                softcap=5.0)
        # against the cache as it is read back (its rounding to bf16 apart from the kernels' own)
        kr, vr = (torch.empty(t1, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        pa.pa_read_cache(shape(1), kr, vr, k, v, ks, vs, bt, ints([t1]), ints([0, t1]), None, err)
        assert pa.pa_read_error_flag(err) == 0
        qd = q_out[t0:t1].double().view(n, Hkv, G, D)
        a = torch.einsum("ihgd,jhd->hgij", qd, kr.double()) * D ** -0.5
        s_abs = float((torch.einsum("ihgd,jhd->hgij", qd.abs(), kr.double().abs()) * D ** -0.5).max())
        me, j = torch.arange(t0, t1, device="cuda")[:, None], torch.arange(t1, device="cuda")
        w = (5.0 * torch.tanh(a / 5.0)).masked_fill(j > me.clamp(min=image - 1), -math.inf).softmax(-1)
        ref = torch.einsum("hgij,jhd->ihgd", w, vr.double()).reshape(n, Hq, D)
        size = torch.einsum("hgij,jhd->ihgd", w, vr.double().abs()).reshape(n, Hq, D)
        read_off = 0.0 if kind == "bf16" else 2 * U          # V's and K's rows as read are rounded to bf16
        bound = U * ref.abs() + (U + read_off / 2 + 2 * read_off / 2 * s_abs + 2.0 ** -17) * size
        if kind != "bf16":
            bound = bound + t1 * E / 2 * float(vr.abs().max())
        assert ((out[t0:t1].double() - ref).abs() <= bound).all(), (t0, t1)


def test_device_batch_on_a_stream_beside_a_busy_one():
    """DeviceBatch's calls on another stream, whose new tensors are made in its order."""
    from paged_kv_cache_28_gb300 import workload as wl
    from paged_kv_cache_28_gb300.device import DeviceBatch, rope_table
    batch = wl.make("tiny")
    dev = DeviceBatch(batch, device="cuda")
    dev.reshape_and_cache()
    B, Hq = batch.B, batch.Hq
    rows = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    offsets = torch.cat([rows[:1] * 0, dev.seq_lens.cumsum(0).int()])
    total = int(offsets[-1])
    slopes = torch.linspace(0.01, 0.5, Hq, device="cuda")
    positions = torch.stack([dev.seq_lens - 1, dev.seq_lens % 7]).int()
    pair = [j % 2 for j in range(batch.D // 2)]
    table = rope_table(int(dev.seq_lens.max()) + 1, batch.D)
    calls = dict(
        extend=lambda st: dev.extend_scored(dev.q, rows, softcap=9.0, slopes=slopes, stream=st),
        decode=lambda st: dev.decode_scored(softcap=9.0, slopes=slopes, stream=st),
        read=lambda st: torch.cat(dev.read_cache(offsets, total, stream=st)),
        rope=lambda st: dev.rope_axes_and_cache(dev.q, dev.k_new, dev.v_new, pair, positions, dev.slot_mapping,
                                                table, stream=st))
    first = dev.k_pool.view(-1, batch.Hkv, batch.D)[int(batch.block_tables[0, 0]) * batch.block_size].clone()
    want = {k: f(None) for k, f in calls.items()}        # (rope, the last, writes the same tokens anew)
    assert dev.read_err() == 0
    assert torch.equal(want["read"][0], first)
    torch.cuda.synchronize()
    side, junk = torch.cuda.Stream(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for stream in (side, side.cuda_stream):
        for name in ("extend", "decode", "rope"):        # (before rope writes its keys again: the same bits)
            for i in range(4):
                junk.fill_(i)                            # the current stream is busy
            got = calls[name](stream)
            side.synchronize()
            if name == "rope":
                assert torch.equal(got.view(torch.int16), want[name].view(torch.int16))
            else:
                assert got.isfinite().all()
    assert dev.read_err() == 0
    after = {k: calls[k](None) for k in ("extend", "decode")}
    for name in after:
        assert torch.equal(calls[name](side).view(torch.int16), after[name].view(torch.int16))
