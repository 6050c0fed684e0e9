"""What is timed of the appending and multi-token attention operators, and their plain forms.

Three operators around the paged cache of this package:

  append   pa_rope_and_cache: the position rotation of a call's queries and keys, and the
           slot-mapped write of the rotated keys and the values (bf16, E4M3, 4-bit pools)
  extend   pa_extend: attention of the query tokens that a call appends (a prompt, a chunk
           of one, a few speculated tokens) over the paged cache, causal, with a window
  cross    pa_cross_attend: attention of ragged decoder tokens to an encoder's states of
           another length, held in the same paged pools, without a causal mask

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


def listed():
    # the layer shape of the 70B-class workloads of this repository
    big = {"Hq": 64, "Hkv": 8, "D": 128, "bs": 16}
    tiny = {"Hq": 8, "Hkv": 2, "D": 64, "bs": 16}
    enc = {"Hq": 16, "Hkv": 16, "D": 64, "bs": 16}
    return [
        # one decode step of a batch of 64: its new tokens, each in a block of its own
        case("append step", "append", "bf16", big, B=64, n=(1, 1), L=(1, 32768), lens=1),
        # a long prompt's tokens at once, from a fused QKV projection
        case("append prompt", "append", "bf16", big, B=1, n=(16384, 16384), L=(16384, 16384), lens=2,
             fused=True),
        # ragged chunks of prompts into an E4M3 cache, starting inside blocks
        case("append chunks fp8", "append", "fp8", big, B=7, n=(400, 2011), L=(2100, 18000), lens=3),
        # a few tokens of each sequence into a 4-bit cache, pairs of neighbouring channels
        case("append int4", "append", "int4", big, B=96, n=(1, 9), L=(10, 4000), lens=4,
             interleaved=True, rotary=64),
        # the smallest call: four speculated tokens of one short sequence, little heads
        case("extend tiny", "extend", "bf16", tiny, B=1, n=(4, 4), L=(100, 100), lens=5),
        # whole prompts around the median length, with the system prompt's 900 tokens cached
        case("extend prompts", "extend", "bf16", big, B=4, n=(1210, 2400), L=(2110, 3300), lens=6),
        # one chunk of a long prompt
        case("extend chunk", "extend", "bf16", big, B=1, n=(2048, 2048), L=(18000, 18000), lens=7),
        # verification of speculated tokens for a batch, E4M3 cache
        case("extend verify fp8", "extend", "fp8", big, B=64, n=(2, 8), L=(150, 8000), lens=8),
        # a few tokens after very long contexts: few rows, a long axis
        case("extend long", "extend", "bf16", dict(big, bs=32), B=2, n=(9, 16), L=(120001, 131072),
             lens=9),
        # a sliding-window layer over a 4-bit cache
        case("extend window int4", "extend", "int4", big, B=2, n=(600, 1501), L=(6000, 9000), lens=10,
             window=4096),
        # decoder prompts against encoder states of another length, one KV head per query head
        case("cross prompts", "cross", "bf16", enc, B=16, n=(60, 448), L=(700, 1500), lens=11),
        # one decoder token per request against its encoder states
        case("cross step", "cross", "bf16", enc, B=32, n=(1, 1), L=(1, 1500), lens=12),
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

    op = rng.choice(["append", "extend", "extend", "cross"])
    kv = rng.choice(["bf16", "bf16", "fp8", "int4"])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    if op == "cross" and rng.random() < 0.5:
        Hkv, G = 16, 1
    heads = {"Hq": Hkv * G, "Hkv": Hkv, "D": rng.choice([64, 128]) if kv == "bf16" else 128,
             "bs": rng.choice([16, 32])}
    lens = rng.randrange(1 << 30)
    if op == "append":
        B = log(1, 128)
        n = log(1, max(1, min(4096, 16384 // B)))
        return {k: v for k, v in case("", op, kv, heads, B=B, n=(max(1, n // 3), n), L=(n, n + log(1, 30000)),
                                      lens=lens, fused=rng.random() < 0.5,
                                      interleaved=rng.random() < 0.3,
                                      rotary=heads["D"] if rng.random() < 0.7 else 32).items() if k != "name"}
    B = log(1, 64)
    n = log(1, 2048)
    # queries x keys x heads of the padded batch, and the cache, stay below the largest listed case's
    Lmax = int(min(131072, 2.2e9 / (B * n * heads["Hq"]), 3e8 / (B * Hkv * heads["D"])))
    if op == "cross":
        Lmax = min(Lmax, 4096)
    else:
        n = min(n, max(1, Lmax // 2))
    L = log(max(n, 16), max(n + 1, Lmax)) if op == "extend" else log(1, max(2, Lmax))
    c = case("", op, kv, heads, B=B, n=(max(1, n // 4), n),
             L=(max(n, L // 3), max(n, L)) if op == "extend" else (max(1, L // 3), L), lens=lens)
    if op == "extend" and rng.random() < 0.3:
        c["window"] = log(1, 2 * c["L_max"])
    return {k: v for k, v in c.items() if k != "name"}


def lengths(case):
    """Query tokens and cached tokens of each sequence, from the case alone; the first
    sequence has the longest of both."""
    r = random.Random(case["lens"])
    n = [case["n_max"]] + [r.randint(case["n_min"], case["n_max"]) for _ in range(case["B"] - 1)]
    lo, hi = case["L_min"], case["L_max"]
    L = [hi] + [int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))) for _ in range(case["B"] - 1)]
    if case["op"] != "cross":        # the query tokens are the last of the cached ones
        L = [max(a, b) for a, b in zip(n, L)]
    return n, L


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
        r = case.get("rotary", D)
        pairs = T * (Hq + Hkv) * r // 2
        nbytes = 2 * T * Hq * D * 2 + 2 * T * Hkv * D * 2 + 2 * T * row_bytes(case) + T * (r * 4 + 12)
        if quant:                    # the scales of the blocks written, read and written
            nbytes += 2 * 2 * 4 * Hkv * sum(blocks_touched(a, b, bs) for a, b in zip(n, L))
        return {"bytes": nbytes, "flops": 6 * pairs}
    W = case.get("window", 0)
    keys = pairs = blocks = 0
    for a, b in zip(n, L):
        if case["op"] == "cross":
            keys, pairs, blocks = keys + b, pairs + a * b, blocks + -(-b // bs)
            continue
        first = b - a                # position of the first query token
        lo = max(0, first - W + 1) if W else 0
        keys, blocks = keys + b - lo, blocks + -(-b // bs) - lo // bs
        full = a * first + a * (a + 1) // 2
        if W:                        # keys before each token's window
            full -= sum(max(0, first + i + 1 - W) for i in range(a))
        pairs += full
    nbytes = 2 * keys * row_bytes(case) + 2 * T * Hq * D * 2 + 4 * blocks + 8 * case["B"]
    if quant:
        nbytes += 2 * 4 * Hkv * blocks
    return {"bytes": nbytes, "flops": 4 * D * Hq * pairs}


class State(dict):
    __getattr__ = dict.__getitem__


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    n, L = lengths(case)
    B, Hq, Hkv, D, bs, kv = (case[k] for k in ("B", "Hq", "Hkv", "D", "bs", "kv"))
    T = sum(n)
    s = State(case=case, T=T, n_max=max(n), L_max=max(L))
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device=dev)  # noqa: E731
    s["offsets"] = ints(np.concatenate([[0], np.cumsum(n)]).tolist())
    s["seq_lens"] = ints(L)
    normal = lambda *sh: torch.randn(*sh, generator=g, device=dev, dtype=torch.float32).bfloat16()  # noqa: E731
    if case["op"] == "append":
        # only the blocks that the call touches are held: block j of sequence b is the j-th of
        # them, at a random place of the pool
        first = [(b - a) // bs for a, b in zip(n, L)]
        count = [blocks_touched(a, b, bs) for a, b in zip(n, L)]
        nblocks = sum(count) + 3
        place = torch.randperm(nblocks, generator=g, device=dev)
        base = np.concatenate([[0], np.cumsum(count)])
        pos = np.concatenate([np.arange(b - a, b) for a, b in zip(n, L)])
        blk = np.concatenate([base[i] + np.arange(b - a, b) // bs - first[i]
                              for i, (a, b) in enumerate(zip(n, L))])
        s["positions"] = ints(pos.tolist())
        s["slots"] = place[ints(blk.tolist(), torch.int64)] * bs + s.positions.long() % bs
        qkv = normal(T, Hq + 2 * Hkv, D)
        parts = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["q"], s["k"], s["v"] = parts if case.get("fused") else (p.contiguous() for p in parts)
        r = case.get("rotary", D)
        s["rotary"], s["interleaved"] = r, bool(case.get("interleaved"))
        # the table that a program builds once: cos, then sin, of every position (base 500000)
        f = torch.arange(0, r, 2, device=dev, dtype=torch.float64) / r
        angle = torch.arange(max(L), device=dev, dtype=torch.float64)[:, None] * 500000.0 ** -f
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        B = T                        # the cache write's shape counts tokens
        max_blocks = 1
    else:
        count = [-(-b // bs) for b in L]
        max_blocks = max(max(count), 1)
        nblocks = sum(count) + 5
        place = torch.randperm(nblocks, generator=g, device=dev, dtype=torch.int32)
        base = torch.tensor(np.concatenate([[0], np.cumsum(count)[:-1]]), device=dev)
        j = torch.arange(max_blocks, device=dev)
        held = j[None, :] < ints(count, torch.int64)[:, None]
        s["block_tables"] = torch.where(held, place[(base[:, None] + j).clamp(max=nblocks - 1)], 0).contiguous()
        s["q"] = normal(T, Hq, D)
        s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        s["sm_scale"] = D ** -0.5
    s["nblocks"], s["max_blocks"] = nblocks, max_blocks
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
        if case["op"] != "append":
            sms = torch.cuda.get_device_properties(0).multi_processor_count
            s["workspace"] = torch.empty(pa.pa_attend_workspace_bytes(s.shape, T, sms),
                                         dtype=torch.uint8, device=dev)
    return s


def run(s):
    op = s.case["op"]
    if op == "append":
        if own:
            import paged_kv_cache_28_gb300 as pa
            pa.pa_rope_and_cache(s.shape, s.cos_sin, s.positions, s.q_out, s.q, s.k, s.v, s.k_pool,
                                 s.v_pool, s.k_scale, s.v_scale, s.slots, s.err,
                                 interleaved=s.interleaved)
        else:
            append_plain(s)
        if s.case["kv"] == "fp8":    # the codes as the E4M3 numbers that they are, and the scales
            return {"q": s.q_out, "k": s.k_pool.view(torch.float8_e4m3fn),
                    "v": s.v_pool.view(torch.float8_e4m3fn), "k_scale": s.k_scale, "v_scale": s.v_scale}
        if s.case["kv"] == "int4":
            return {"q": s.q_out, "k": s.k_pool, "v": s.v_pool, "k_scale": s.k_scale, "v_scale": s.v_scale}
        return {"q": s.q_out, "k": s.k_pool, "v": s.v_pool}
    if own:
        import paged_kv_cache_28_gb300 as pa
        if op == "extend":
            pa.pa_extend(s.shape, s.out, s.q, s.offsets, s.k_pool, s.v_pool, s.k_scale, s.v_scale,
                         s.block_tables, s.seq_lens, s.sm_scale, s.workspace, s.err,
                         window=s.case.get("window", 0))
        else:
            pa.pa_cross_attend(s.shape, s.out, s.q, s.offsets, s.k_pool, s.v_pool, s.k_scale,
                               s.v_scale, s.block_tables, s.seq_lens, s.sm_scale, s.workspace, s.err)
        return s.out
    return attend_plain(s)


# ------------------------------------------------------------------ plain forms

def rotate(x, c, sn, r, interleaved):
    """x [T, H, D] fp32 rotated in its first r channels by the angles of c, sn [T, 1, r/2]."""
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    ya, yb = a * c - b * sn, b * c + a * sn
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = ya, yb
    else:
        y[..., :r // 2], y[..., r // 2:r] = ya, yb
    return y


def append_plain(s):
    c, r, kv = s.case, s.rotary, s.case["kv"]
    cs = s.cos_sin[s.positions.long()][:, None, :]
    cos, sin = cs[..., :r // 2], cs[..., r // 2:]
    s.q_out.copy_(rotate(s.q.float(), cos, sin, r, s.interleaved))
    k = rotate(s.k.float(), cos, sin, r, s.interleaved).bfloat16()
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
    encoded anew."""
    blocks, which = torch.unique(slots // bs, return_inverse=True)
    off = slots % bs
    code = decode(pool[blocks], kv)                       # [M, bs, Hkv, D]
    sc = scale[blocks]                                    # [M, Hkv]
    new = torch.zeros_like(code)
    new[which, off] = x.float()
    has = torch.zeros(len(blocks), bs, dtype=torch.bool, device=x.device)
    has[which, off] = True
    cand = new.abs().amax(-1) / MAX_CODE[kv]              # [M, bs, Hkv]
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
    last = L[:, None] - 1 if c["op"] == "cross" else (L - n)[:, None] + i[None]      # of each query
    seen = (j <= last.expand(B, s.n_max)[..., None]) & (j < L[:, None, None])
    if c.get("window", 0):
        seen &= j > last[..., None] - c["window"]
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
    return exact_append(s) if case["op"] == "append" else exact_attend(s)


def exact_append(s):
    c, half = s.case, s.rotary // 2
    angle = s.cos_sin.double()[s.positions.long()]
    turn = torch.complex(angle[:, :half], angle[:, half:])[:, None]

    def rotated(x):
        x = x.double()
        head, rest = x[..., :2 * half], x[..., 2 * half:]
        pair = head.reshape(*head.shape[:-1], half, 2) if s.interleaved else \
            head.reshape(*head.shape[:-1], 2, half).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z.flatten(-2) if s.interleaved else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, rest], -1)

    out = {"q": rotated(s.q), "k": None, "v": None}
    if c["kv"] == "bf16":
        for x, val in (("k", rotated(s.k)), ("v", s.v.double())):
            pool = s[x + "_pool"].double().flatten(0, 1)
            pool[s.slots] = val
            out[x] = pool.view(s[x + "_pool"].shape)
    else:                            # codes have no value in 64 bits, nor has the scale of rounded keys
        out["k_scale"] = out["v_scale"] = None
    return out


def exact_attend(s):
    c = s.case
    n, L = lengths(c)
    Hq, Hkv, D, bs, W = c["Hq"], c["Hkv"], c["D"], c["bs"], c.get("window", 0)
    out = torch.empty(s.T, Hq, D, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(c["B"]):
        table = s.block_tables[b, :-(-L[b] // bs)].long()
        keys = []
        for pool, scale in ((s.k_pool, s.k_scale), (s.v_pool, s.v_scale)):
            x = pool[table]
            if c["kv"] == "int4":
                x = torch.stack([x % 16, x // 16], -1).flatten(-2).double() - 8
            x = x.view(torch.float8_e4m3fn).double() if c["kv"] == "fp8" else x.double()
            if scale is not None:
                x = x * scale[table].double()[:, None, :, None]
            keys.append(x.flatten(0, 1)[:L[b]])
        pos = torch.arange(L[b], device="cuda")
        for i0 in range(0, n[b], 256):
            i1 = min(n[b], i0 + 256)
            me = torch.arange(i0, i1, device="cuda")[:, None] + (L[b] - n[b])
            hide = torch.zeros(i1 - i0, L[b], dtype=torch.bool, device="cuda")
            if c["op"] == "extend":
                hide = pos > me
                if W:
                    hide |= pos <= me - W
            for h in range(Hkv):
                G = Hq // Hkv
                q = s.q[at + i0:at + i1, h * G:(h + 1) * G].double().transpose(0, 1)
                w = (q @ keys[0][:, h].T * s.sm_scale).masked_fill(hide, float("-inf")).softmax(-1)
                out[at + i0:at + i1, h * G:(h + 1) * G] = (w @ keys[1][:, h]).transpose(0, 1)
        at += n[b]
    return out
