"""What is timed of the operators for changed scores, several position axes and reading the cache
back, and their plain forms.

Four operators around the paged cache of this package:

  extend   pa_extend_scored: attention of the tokens that a call appends, whose scores are capped
           by a tanh, get a bias that falls with distance, or whose prefix sees all of itself
  decode   pa_decode_scored: the same for one token per sequence
  append   pa_rope_axes_and_cache: the rotation by positions with several axes (time, height,
           width of images and video) and the slot-mapped write
  read     pa_read_cache: cached rows, restored, as dense bf16 tensors

`run` computes them in elementary torch operations (own = False) or through the package's
entry points (own = True).  A case fixes its sizes; its lengths are drawn from the number
`lens` in it, everything else from prepare()'s seed.
"""
import math
import random

import numpy as np
import torch

own = False

MAX_CODE = {"fp8": 448.0, "int4": 7.0}
# which axis of (time, height, width) a pair of channels turns by: in runs of a quarter and two
# times three eighths of the pairs, or in turn until the runs' numbers are used up
ARRANGEMENTS = ("runs", "turns")


def listed():
    # the layer shape of the 70B-class workloads of this repository
    big = {"Hq": 64, "Hkv": 8, "D": 128, "bs": 16}
    tiny = {"Hq": 8, "Hkv": 2, "D": 64, "bs": 16}
    return [
        # the smallest call: four speculated tokens of one short sequence, little heads
        case("extend cap tiny", "extend", "bf16", tiny, B=1, n=(4, 4), L=(100, 100), lens=1, cap=50.0),
        # whole prompts around the median length after the system prompt's 900 tokens, capped scores
        case("extend cap prompts", "extend", "bf16", big, B=4, n=(1210, 2400), L=(2110, 3300), lens=2,
             cap=50.0),
        # one chunk of a long prompt, scores falling with distance
        case("extend bias chunk", "extend", "bf16", big, B=1, n=(2048, 2048), L=(18000, 18000), lens=3,
             bias=True),
        # images and instructions that see all of themselves, capped, a windowed layer, E4M3 cache
        case("extend prefix fp8", "extend", "fp8", big, B=5, n=(301, 1500), L=(900, 4000), lens=4,
             cap=30.0, window=1024, prefix=True),
        # one decode step of a batch, capped scores, E4M3 cache
        case("decode cap fp8", "decode", "fp8", big, B=64, n=(1, 1), L=(150, 8000), lens=5, cap=50.0),
        # a few very long sequences, scores falling with distance: few rows, a long axis
        case("decode bias long", "decode", "bf16", dict(big, bs=32), B=3, n=(1, 1), L=(100001, 131072),
             lens=6, bias=True),
        # a windowed and capped layer of a small batch, 4-bit cache
        case("decode window int4", "decode", "int4", big, B=9, n=(1, 1), L=(700, 12000), lens=7, cap=30.0,
             window=4096),
        # one decode step of a batch of 64: its new tokens, each in a block of its own
        case("append step", "append", "bf16", big, B=64, n=(1, 1), L=(1, 32768), lens=8, axes="turns"),
        # a long prompt of text and images at once, from a fused QKV projection
        case("append prompt", "append", "bf16", big, B=1, n=(16384, 16384), L=(16384, 16384), lens=9,
             fused=True, axes="runs"),
        # ragged chunks of prompts into an E4M3 cache, starting inside blocks
        case("append chunks fp8", "append", "fp8", big, B=7, n=(400, 2011), L=(2100, 18000), lens=10,
             axes="runs"),
        # a batch's prompts leave an E4M3 cache, to be sent elsewhere
        case("read prompts fp8", "read", "fp8", big, B=16, n=(900, 8000), L=(900, 8000), lens=11),
        # the newest tokens of short sequences of a 4-bit cache
        case("read tails int4", "read", "int4", big, B=32, n=(1, 70), L=(100, 3000), lens=12),
    ]


def case(name, op, kv, heads, **more):
    c = {"name": name, "op": op, "kv": kv, **heads}
    for k, v in more.items():
        if isinstance(v, tuple):
            c[k + "_min"], c[k + "_max"] = v
        else:
            c[k] = v
    return c


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["extend", "extend", "decode", "append", "read"])
    kv = rng.choice(["bf16", "bf16", "fp8", "int4"])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    heads = {"Hq": Hkv * G, "Hkv": Hkv, "D": rng.choice([64, 128]) if kv == "bf16" else 128,
             "bs": rng.choice([16, 32])}
    lens = rng.randrange(1 << 30)
    if op == "append":
        B = log(1, 128)
        n = log(1, max(1, min(4096, 16384 // B)))
        c = case("", op, kv, heads, B=B, n=(max(1, n // 3), n), L=(n, n + log(1, 30000)), lens=lens,
                 fused=rng.random() < 0.5, interleaved=rng.random() < 0.3, axes=rng.choice(ARRANGEMENTS))
    elif op == "read":
        B = log(1, 128)
        L = log(1, max(2, min(32768, 70000 // B)))
        n = log(1, L)
        c = case("", op, kv, heads, B=B, n=(max(1, n // 3), n), L=(max(1, L // 3), L), lens=lens)
    else:
        B = log(1, 64)
        n = 1 if op == "decode" else log(1, 2048)
        # queries x keys x heads of the padded batch, and the cache, stay below the largest listed case's
        Lmax = int(min(131072, 2.2e9 / (B * n * heads["Hq"]), 3e8 / (B * Hkv * heads["D"])))
        n = min(n, max(1, Lmax // 2))
        L = log(max(n, 16), max(n + 1, Lmax))
        c = case("", op, kv, heads, B=B, n=(max(1, n // 4), n), L=(max(n, L // 3), max(n, L)), lens=lens)
        kind = rng.choice(["cap", "bias", "both", "prefix"] if op == "extend" else ["cap", "bias", "both"])
        if kind in ("cap", "both") or (kind == "prefix" and rng.random() < 0.5):
            c["cap"] = rng.choice([20.0, 30.0, 50.0])
        if kind in ("bias", "both"):
            c["bias"] = True
        if kind == "prefix":
            c["prefix"] = True
        if rng.random() < 0.3:
            c["window"] = log(1, 2 * c["L_max"])
    return {k: v for k, v in c.items() if k != "name"}


def lengths(case):
    """Tokens of the call and cached tokens of each sequence, from the case alone; the first
    sequence has the longest of both."""
    r = random.Random(case["lens"])
    n = [case["n_max"]] + [r.randint(case["n_min"], case["n_max"]) for _ in range(case["B"] - 1)]
    lo, hi = case["L_min"], case["L_max"]
    L = [hi] + [int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))) for _ in range(case["B"] - 1)]
    return n, [max(a, b) for a, b in zip(n, L)]     # the call's tokens are the last cached ones


def prefixes(case):
    """Tokens of each sequence's prefix: from none to some of the call's own tokens."""
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, 1) * (b - a + r.randint(1, a)) for a, b in zip(*lengths(case))]


def pair_axes(case):
    half = case["D"] // 2
    count = [half - 2 * (3 * half // 8), 3 * half // 8, 3 * half // 8]
    if case["axes"] == "runs":
        return [a for a in range(3) for _ in range(count[a])]
    # in turn while height and width have pairs left, the others by time
    return [j % 3 if j % 3 and j // 3 < count[j % 3] else 0 for j in range(half)]


def row_bytes(case):
    """Bytes of one token's K (or V) row over the KV heads."""
    return case["Hkv"] * case["D"] * {"bf16": 2.0, "fp8": 1.0, "int4": 0.5}[case["kv"]]


def blocks_touched(n, L, bs):
    return -(-L // bs) - (L - n) // bs


def work(case):
    n, L = lengths(case)
    T, Hq, Hkv, D, bs = sum(n), case["Hq"], case["Hkv"], case["D"], case["bs"]
    quant = case["kv"] != "bf16"
    if case["op"] == "append":
        pairs = T * (Hq + Hkv) * D // 2
        nbytes = 2 * T * Hq * D * 2 + 2 * T * Hkv * D * 2 + 2 * T * row_bytes(case) + T * (D * 4 + 20)
        if quant:                    # the scales of the blocks written, read and written
            nbytes += 2 * 2 * 4 * Hkv * sum(blocks_touched(a, b, bs) for a, b in zip(n, L))
        return {"bytes": nbytes, "flops": 6 * pairs}
    if case["op"] == "read":
        blocks = sum(blocks_touched(a, b, bs) for a, b in zip(n, L))
        nbytes = 2 * T * row_bytes(case) + 2 * T * Hkv * D * 2 + 4 * blocks + 12 * case["B"]
        if quant:
            nbytes += 2 * 4 * Hkv * blocks
        return {"bytes": nbytes, "flops": 2 * T * Hkv * D if quant else 0}
    W = case.get("window", 0)
    P = prefixes(case) if case.get("prefix") else [0] * case["B"]
    keys = pairs = blocks = 0
    for a, b, pre in zip(n, L, P):
        first = b - a                # position of the first query token
        lo = max(0, first - W + 1) if W else 0
        keys, blocks = keys + b - lo, blocks + -(-b // bs) - lo // bs
        for p in range(first, b):
            pairs += max(p + 1, pre) - (max(0, p - W + 1) if W else 0)
    nbytes = 2 * keys * row_bytes(case) + 2 * T * Hq * D * 2 + 4 * blocks + 12 * case["B"] + 4 * Hq
    if quant:
        nbytes += 2 * 4 * Hkv * blocks
    return {"bytes": nbytes, "flops": 4 * D * Hq * pairs}


class State(dict):
    __getattr__ = dict.__getitem__


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    n, L = lengths(case)
    B, Hq, Hkv, D, bs, kv, op = (case[k] for k in ("B", "Hq", "Hkv", "D", "bs", "kv", "op"))
    T = sum(n)
    s = State(case=case, T=T, n_max=max(n), L_max=max(L))
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device=dev)  # noqa: E731
    normal = lambda *sh: torch.randn(*sh, generator=g, device=dev, dtype=torch.float32).bfloat16()  # noqa: E731
    s["offsets"] = ints(np.concatenate([[0], np.cumsum(n)]).tolist())
    s["seq_lens"] = ints(L)
    pos = np.concatenate([np.arange(b - a, b) for a, b in zip(n, L)])
    if op == "append":
        # only the blocks that the call touches are held: block j of sequence b is the j-th of
        # them, at a random place of the pool
        first = [(b - a) // bs for a, b in zip(n, L)]
        count = [blocks_touched(a, b, bs) for a, b in zip(n, L)]
        nblocks = sum(count) + 3
        place = torch.randperm(nblocks, generator=g, device=dev)
        base = np.concatenate([[0], np.cumsum(count)])
        blk = np.concatenate([base[i] + np.arange(b - a, b) // bs - first[i]
                              for i, (a, b) in enumerate(zip(n, L))])
        s["slots"] = place[ints(blk.tolist(), torch.int64)] * bs + ints((pos % bs).tolist(), torch.int64)
        # text, then an image of 24 x 32 patches, in turn: text has one position on all axes, an
        # image's patches the image's time and their row and column after it
        at = ints(pos.tolist(), torch.int64)
        inside = at % 1200 - 432
        image, start = inside >= 0, at - inside
        s["positions"] = torch.stack([torch.where(image, start, at),
                                      torch.where(image, start + inside // 32, at),
                                      torch.where(image, start + inside % 32, at)]).int()
        qkv = normal(T, Hq + 2 * Hkv, D)
        parts = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q"], s["k"], s["v"] = parts if case.get("fused") else (p.contiguous() for p in parts)
        s["axis"] = pair_axes(case)
        s["interleaved"] = bool(case.get("interleaved"))
        # the table that a program builds once: cos, then sin, of every position (base 500000)
        f = torch.arange(0, D, 2, device=dev, dtype=torch.float64) / D
        angle = torch.arange(max(L), device=dev, dtype=torch.float64)[:, None] * 500000.0 ** -f
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        B = T                        # the cache write's shape counts tokens
        max_blocks = 1
    else:
        count = [-(-b // bs) for b in L]
        max_blocks = max(count)
        nblocks = sum(count) + 5
        place = torch.randperm(nblocks, generator=g, device=dev, dtype=torch.int32)
        base = torch.tensor(np.concatenate([[0], np.cumsum(count)[:-1]]), device=dev)
        j = torch.arange(max_blocks, device=dev)
        held = j[None, :] < ints(count, torch.int64)[:, None]
        s["block_tables"] = torch.where(held, place[(base[:, None] + j).clamp(max=nblocks - 1)], 0).contiguous()
    if op == "read":
        s["starts"] = ints([b - a for a, b in zip(n, L)])
        s["k"], s["v"] = (torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=dev) for _ in "kv")
    if op in ("extend", "decode"):
        # scores spread over +-25 and more, as a cap is made for
        s["q"] = normal(T, Hq, D) * 6
        s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        s["sm_scale"] = D ** -0.5
        # the usual slopes: 2^(-8 / Hq) and its powers
        s["slopes"] = (2.0 ** (-8.0 / Hq * torch.arange(1, Hq + 1, device=dev, dtype=torch.float64))
                       ).float() if case.get("bias") else None
        s["prefix"] = ints(prefixes(case)) if case.get("prefix") else None
    s["k_scale"] = s["v_scale"] = None
    if kv == "bf16":
        s["k_pool"], s["v_pool"] = normal(nblocks, bs, Hkv, D), normal(nblocks, bs, Hkv, D)
    else:
        top = MAX_CODE[kv]
        for x in "kv":               # codes of N(0,1) values whose block maximum lies near 4
            codes = torch.randn(nblocks, bs, Hkv, D, generator=g, device=dev).clamp(-4, 4) * (top / 4)
            if kv == "fp8":
                s[x + "_pool"] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                c = (codes.round().int() + 8).to(torch.uint8)
                s[x + "_pool"] = (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()
            s[x + "_scale"] = 4 / top * (0.8 + 0.4 * torch.rand(nblocks, Hkv, generator=g, device=dev))
    s["err"] = torch.zeros(1, dtype=torch.int32, device=dev)
    if own:
        import paged_kv_cache_28_gb300 as pa
        kind = {"bf16": pa.PA_KV_BF16, "fp8": pa.PA_KV_FP8_E4M3, "int4": pa.PA_KV_INT4}[kv]
        s["shape"] = pa.make_shape(B, Hq, Hkv, D, bs, nblocks, max_blocks, kind)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        if op == "extend":
            nbytes = pa.pa_attend_workspace_bytes(s.shape, T, sms)
        elif op == "decode":
            nbytes = pa.pa_decode_workspace_bytes(s.shape, pa.pa_default_num_segments(s.shape, sms))
        if op in ("extend", "decode"):
            s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return s


def run(s):
    c = s.case
    if c["op"] == "append":
        if own:
            import paged_kv_cache_28_gb300 as pa
            pa.pa_rope_axes_and_cache(s.shape, s.axis, s.cos_sin, s.positions, s.q_out, s.q, s.k, s.v,
                                      s.k_pool, s.v_pool, s.k_scale, s.v_scale, s.slots, s.err,
                                      interleaved=s.interleaved)
        else:
            append_plain(s)
        if c["kv"] == "fp8":         # the codes as the E4M3 numbers that they are, and the scales
            return {"q": s.q_out, "k": s.k_pool.view(torch.float8_e4m3fn),
                    "v": s.v_pool.view(torch.float8_e4m3fn), "k_scale": s.k_scale, "v_scale": s.v_scale}
        if c["kv"] == "int4":
            return {"q": s.q_out, "k": s.k_pool, "v": s.v_pool, "k_scale": s.k_scale, "v_scale": s.v_scale}
        return {"q": s.q_out, "k": s.k_pool, "v": s.v_pool}
    if c["op"] == "read":
        if own:
            import paged_kv_cache_28_gb300 as pa
            pa.pa_read_cache(s.shape, s.k, s.v, s.k_pool, s.v_pool, s.k_scale, s.v_scale, s.block_tables,
                             s.seq_lens, s.offsets, s.starts, s.err)
        else:
            read_plain(s)
        return {"k": s.k, "v": s.v}
    if not own:
        return attend_plain(s)
    import paged_kv_cache_28_gb300 as pa
    if c["op"] == "extend":
        pa.pa_extend_scored(s.shape, s.out, s.q, s.offsets, s.k_pool, s.v_pool, s.k_scale, s.v_scale,
                            s.block_tables, s.seq_lens, s.sm_scale, s.workspace, s.err,
                            window=c.get("window", 0), softcap=c.get("cap", 0.0), slopes=s.slopes,
                            prefix_lens=s.prefix)
    else:
        pa.pa_decode_scored(s.shape, s.out, s.q, s.k_pool, s.v_pool, s.k_scale, s.v_scale,
                            s.block_tables, s.seq_lens, s.sm_scale, s.workspace, s.err,
                            window=c.get("window", 0), softcap=c.get("cap", 0.0), slopes=s.slopes)
    return s.out


# ------------------------------------------------------------------ plain forms

def rotate(x, c, sn, interleaved):
    """x [T, H, D] fp32 rotated by the angles of c, sn [T, 1, D / 2]."""
    half = x.shape[-1] // 2
    y = torch.empty_like(x)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    ya, yb = a * c - b * sn, b * c + a * sn
    if interleaved:
        y[..., 0::2], y[..., 1::2] = ya, yb
    else:
        y[..., :half], y[..., half:] = ya, yb
    return y


def append_plain(s):
    c, kv, half = s.case, s.case["kv"], s.case["D"] // 2
    axis = torch.tensor(s.axis, device=s.q.device)
    at = s.positions.long()[axis].T                       # [T, D / 2]: the row of each pair
    pair = torch.arange(half, device=at.device)
    cos, sin = s.cos_sin[at, pair][:, None], s.cos_sin[at, half + pair][:, None]
    s.q_out.copy_(rotate(s.q.float(), cos, sin, s.interleaved))
    k = rotate(s.k.float(), cos, sin, s.interleaved).bfloat16()
    if kv == "bf16":
        s.k_pool.view(-1, c["Hkv"], c["D"])[s.slots] = k
        s.v_pool.view(-1, c["Hkv"], c["D"])[s.slots] = s.v
        return
    write_codes(k, s.k_pool, s.k_scale, s.slots, c["bs"], kv)
    write_codes(s.v, s.v_pool, s.v_scale, s.slots, c["bs"], kv)


def decode(pool, kv):
    """Codes of a pool as fp32 values, before their scale."""
    if kv == "fp8":
        return pool.view(torch.float8_e4m3fn).float()
    return torch.stack([(pool & 15).float() - 8, (pool >> 4).float() - 8], -1).flatten(-2)


def encode(x, scale, kv):
    y = torch.where(scale == 0, torch.zeros_like(x), x / scale)
    if kv == "fp8":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    return y.round().clamp(-7, 7)


def write_codes(x, pool, scale, slots, bs, kv):
    """The absmax-scaled write: a block's tokens are applied in the order of their rows (which
    is the order of the tokens); a token that raises the block's scale has the codes below it
    encoded anew.  The scale is absmax times the fp32 reciprocal of the largest code."""
    blocks, which = torch.unique(slots // bs, return_inverse=True)
    off = slots % bs
    code = decode(pool[blocks], kv)                       # [M, bs, Hkv, D]
    sc = scale[blocks]                                    # [M, Hkv]
    new = torch.zeros_like(code)
    new[which, off] = x.float()
    has = torch.zeros(len(blocks), bs, dtype=torch.bool, device=x.device)
    has[which, off] = True
    cand = new.abs().amax(-1) * float(np.float32(1) / np.float32(MAX_CODE[kv]))     # [M, bs, Hkv]
    for i in range(bs):
        here = has[:, i, None]
        up = torch.where(here, cand[:, i] if i == 0 else torch.maximum(sc, cand[:, i]), sc)
        if i:
            grown = (here & (up > sc))[:, None, :, None]
            again = encode(code[:, :i] * sc[:, None, :, None], up[:, None, :, None], kv)
            code[:, :i] = torch.where(grown, again, code[:, :i])
        code[:, i] = torch.where(here[..., None], encode(new[:, i], up[..., None], kv), code[:, i])
        sc = up
    if kv == "fp8":
        pool[blocks] = code.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        u = (code + 8).to(torch.uint8)
        pool[blocks] = u[..., 0::2] | (u[..., 1::2] << 4)
    scale[blocks] = sc


def read_plain(s):
    bs = s.case["bs"]
    t = torch.arange(s.T, device=s.k.device)
    b = torch.searchsorted(s.offsets.long(), t, right=True) - 1
    at = s.starts.long()[b] + t - s.offsets.long()[b]
    block, off = s.block_tables.long()[b, at // bs], at % bs
    for out, pool, scale in ((s.k, s.k_pool, s.k_scale), (s.v, s.v_pool, s.v_scale)):
        rows = pool[block, off]
        if scale is None:
            out.copy_(rows)
        else:
            out.copy_(decode(rows, s.case["kv"]) * scale[block][..., None])


def attend_plain(s):
    c = s.case
    B, Hkv, D, bs = c["B"], c["Hkv"], c["D"], c["bs"]
    G, nb = c["Hq"] // Hkv, -(-s.L_max // bs)
    L, off = s.seq_lens.long(), s.offsets.long()
    n = off[1:] - off[:-1]
    blocks = s.block_tables[:, :nb].long()

    def rows(pool, scale):                                # [B, Hkv, keys, D]
        x = pool[blocks].float() if scale is None else decode(pool[blocks], c["kv"]) * scale[blocks][:, :, None, :, None]
        return x.reshape(B, nb * bs, Hkv, D).transpose(1, 2)

    i, j = torch.arange(s.n_max, device=L.device), torch.arange(nb * bs, device=L.device)
    real = i[None] < n[:, None]                           # [B, queries]
    take = torch.where(real, off[:-1, None] + i[None], 0)
    q = s.q[take].float().view(B, s.n_max, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * s.n_max, D)
    score = (q @ rows(s.k_pool, s.k_scale).transpose(2, 3)).view(B, Hkv, G, s.n_max, nb * bs) * s.sm_scale
    me = (L - n)[:, None] + i[None]                       # position of each query
    if c.get("cap"):
        score.div_(c["cap"]).tanh_().mul_(c["cap"])
    if s.slopes is not None:
        far = (me[..., None] - j).abs().float()           # [B, queries, keys]
        slope = s.slopes.view(Hkv, G)
        for h in range(Hkv):
            for k in range(G):
                score[:, h, k] -= slope[h, k] * far
    last = me if s.prefix is None else torch.maximum(me, s.prefix.long()[:, None] - 1)
    seen = (j <= last[..., None]) & (j < L[:, None, None])
    if c.get("window", 0):
        seen &= j > me[..., None] - c["window"]
    score = score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, G * s.n_max, nb * bs) @ rows(s.v_pool, s.v_scale)
    o = o.view(B, Hkv, G, s.n_max, D) / torch.where(total > 0, total, 1)
    s.out[take[real]] = o.permute(0, 3, 1, 2, 4).reshape(B, s.n_max, c["Hq"], D)[real].bfloat16()
    return s.out


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": exact_append, "read": exact_read}.get(case["op"], exact_attend)(s)


def exact_append(s):
    c, half = s.case, s.case["D"] // 2
    table = s.cos_sin.double()
    turn = torch.empty(s.T, 1, half, dtype=torch.complex128, device="cuda")
    for pair, axis in enumerate(s.axis):
        row = table[s.positions[axis].long()]
        turn[:, 0, pair] = torch.complex(row[:, pair], row[:, half + pair])

    def rotated(x):
        x = x.double()
        pair = x.reshape(*x.shape[:-1], half, 2) if s.interleaved else \
            x.reshape(*x.shape[:-1], 2, half).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        return z.flatten(-2) if s.interleaved else z.transpose(-1, -2).flatten(-2)

    out = {"q": rotated(s.q), "k": None, "v": None}
    if c["kv"] == "bf16":
        for x, val in (("k", rotated(s.k)), ("v", s.v.double())):
            pool = s[x + "_pool"].double().flatten(0, 1)
            pool[s.slots] = val
            out[x] = pool.view(s[x + "_pool"].shape)
    else:                            # codes have no value in 64 bits, nor has the scale of rounded keys
        out["k_scale"] = out["v_scale"] = None
    return out


def values(pool, scale, kv):
    """Pool rows [blocks, bs, Hkv, D] in 64 bits."""
    if kv == "int4":
        x = torch.stack([pool % 16, pool // 16], -1).flatten(-2).double() - 8
    else:
        x = pool.view(torch.float8_e4m3fn).double() if kv == "fp8" else pool.double()
    return x if scale is None else x * scale.double()[:, None, :, None]


def exact_read(s):
    c = s.case
    n, L = lengths(c)
    out = {"k": [], "v": []}
    for b in range(c["B"]):
        table = s.block_tables[b, :-(-L[b] // c["bs"])].long()
        for x in "kv":
            scale = s[x + "_scale"]
            rows = values(s[x + "_pool"][table], None if scale is None else scale[table], c["kv"])
            out[x].append(rows.flatten(0, 1)[L[b] - n[b]:L[b]])
    return {x: torch.cat(y) for x, y in out.items()}


def exact_attend(s):
    c = s.case
    n, L = lengths(c)
    Hq, Hkv, D, bs, W, cap = c["Hq"], c["Hkv"], c["D"], c["bs"], c.get("window", 0), c.get("cap", 0.0)
    P = prefixes(c) if c.get("prefix") else [0] * c["B"]
    G = Hq // Hkv
    out = torch.empty(s.T, Hq, D, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(c["B"]):
        table = s.block_tables[b, :-(-L[b] // bs)].long()
        keys = [values(pool[table], None if scale is None else scale[table], c["kv"]).flatten(0, 1)[:L[b]]
                for pool, scale in ((s.k_pool, s.k_scale), (s.v_pool, s.v_scale))]
        pos = torch.arange(L[b], device="cuda")
        for i0 in range(0, n[b], 256):
            i1 = min(n[b], i0 + 256)
            me = torch.arange(i0, i1, device="cuda")[:, None] + (L[b] - n[b])
            hide = (pos > me) & (pos >= P[b])
            if W:
                hide |= pos <= me - W
            far = (me - pos).abs().double()
            for h in range(Hkv):
                q = s.q[at + i0:at + i1, h * G:(h + 1) * G].double().transpose(0, 1)
                w = q @ keys[0][:, h].T * s.sm_scale
                if cap:
                    w = cap * torch.tanh(w / cap)
                if s.slopes is not None:
                    w = w - s.slopes[h * G:(h + 1) * G].double()[:, None, None] * far
                w = w.masked_fill(hide, float("-inf")).softmax(-1)
                out[at + i0:at + i1, h * G:(h + 1) * G] = (w @ keys[1][:, h]).transpose(0, 1)
        at += n[b]
    return out
