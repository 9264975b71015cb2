"""The 8-bit KV cache and what feeds it: what is measured, and the plain forms.

Three operators, as a decode server of this package uses them together:

* ``rope``   the RMS norm of every query and key head and the rotation by
             position, in one pass over the projections' output;
* ``write``  new tokens' K/V quantised into the paged 8-bit cache as they are
             written (one float32 scale for each block of 16 tokens, KV head
             and K or V), and the blocks they touched read back;
  ``read``   a stretch of the 8-bit cache read back (as a prefix is, when it
             is moved to another cache);
* ``attn``   one query token per row over the row's whole paged history, or
             over one region of it, held in 8 bits.

Formulas (positions 1-indexed, position p in block column (p-1)//16, slot (p-1)%16):

  rope   y = x * rsqrt(mean(x^2) + eps) * w  for each head; pairs (a, b) of y
         become (a cos - b sin, b cos + a sin), angle = position * inv_freq.
  write  a = max |x| over a block's new tokens and dims, for each head and for
         K and V apart; scale = max(a / top, the scale the block had for the
         tokens it held before), 0 where that is below 2^-107;
         code = round(x * (1 / scale)), ties to even, to whole numbers within
         +-127 (int8, top = 127) or to e4m3 numbers (top = 448); where the scale
         grew, the codes held before become round(code * (old scale * (1 / scale))).
         scale, 1 / scale and the products are float32 numbers.
  read   code * scale.
  attn   softmax_j(q . (kcode_j kscale) / sqrt(d)) over the row's positions,
         times (vcode_j vscale); lse = log sum_j exp(score_j).
"""

import math
import random

import numpy as np
import torch

own = False

TOKENS = 16                                     # tokens of a block of the paged cache
SINK, WINDOW = 4, 2048                          # ring of the local window
KIND = {"bf16": torch.bfloat16, "f32": torch.float32}
TOP = {"int8": 127.0, "e4m3": 448.0}
LEAST = 2.0 ** -107


# --------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest decode attention: two short rows, one KV head, float32
        dict(name="attn_tiny_f32", op="attn", fmt="int8", dtype="f32", hq=2, hkv=1, d=64, rows=2,
             ctx_lo=40, ctx_hi=64, rate=1.0, region=False),
        # a batch of eight at 16K, all rows attend over the whole history
        dict(name="attn_16k_b8", op="attn", fmt="e4m3", dtype="bf16", hq=16, hkv=8, d=128, rows=8,
             ctx_lo=16384, ctx_hi=16384, rate=1.0, region=False),
        # one long request
        dict(name="attn_128k_b1", op="attn", fmt="int8", dtype="bf16", hq=16, hkv=8, d=128, rows=1,
             ctx_lo=131072, ctx_hi=131072, rate=1.0, region=False),
        # a serving batch of mixed lengths of which 41 % recompute over everything
        dict(name="attn_mixed_b32", op="attn", fmt="e4m3", dtype="bf16", hq=16, hkv=8, d=128,
             rows=32, ctx_lo=4096, ctx_hi=65536, rate=0.41, region=False),
        # regions with odd ends, four query heads to a KV head
        dict(name="attn_region_g4", op="attn", fmt="int8", dtype="bf16", hq=8, hkv=2, d=128, rows=5,
             ctx_lo=3000, ctx_hi=20011, rate=1.0, region=True),
        # a decode step's queries and keys, out of one fused projection
        dict(name="rope_decode_b16", op="rope", dtype="bf16", hq=16, hkv=8, d=128, rot=128, n=16,
             first=-1, pairs="halves", fused=True),
        # a prefill chunk far into a document
        dict(name="rope_prefill_16k", op="rope", dtype="bf16", hq=16, hkv=8, d=128, rot=128,
             n=16384, first=114688, pairs="halves", fused=True),
        # odd count, part of each head rotated, neighbouring pairs, float32
        dict(name="rope_part_f32", op="rope", dtype="f32", hq=4, hkv=2, d=64, rot=32, n=1537,
             first=77, pairs="neighbours", fused=False),
        # a decode step of a batch: one token a row, all layers in one call
        dict(name="write_decode_l28_b32", op="write", fmt="int8", dtype="bf16", hkv=8, d=128,
             layers=28, rows=32, new_lo=1, new_hi=1, past_lo=30, past_hi=700, ring=False),
        # a prefill chunk of one request, into the cache and the ring
        dict(name="write_prefill_16k", op="write", fmt="e4m3", dtype="bf16", hkv=8, d=128, layers=1,
             rows=1, new_lo=16384, new_hi=16384, past_lo=0, past_hi=0, ring=True),
        # ragged chunks that start and end inside blocks, some of them empty
        dict(name="write_ragged_f32", op="write", fmt="int8", dtype="f32", hkv=2, d=64, layers=3,
             rows=9, new_lo=0, new_hi=300, past_lo=0, past_hi=90, ring=False),
        # cached prefixes of a batch read back at 16K
        dict(name="read_16k_b8", op="read", fmt="e4m3", dtype="bf16", hkv=8, d=128, layers=1,
             rows=8, len_lo=16384, len_hi=16384),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "write", "read"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    fmt = rng.choice(["int8", "e4m3"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "attn":
        rows = _spread(rng, 1, 40)
        # at most 600 thousand tokens of 8 KV heads in all
        most = min(262144, 600000 * 8 // (rows * hkv))
        hi = _spread(rng, 1, most)
        lo = rng.choice([hi, max(1, hi // rng.choice([2, 7, 50]))])
        return dict(op="attn", fmt=fmt, dtype=dtype, hq=hkv * rng.choice([1, 2, 2, 4]), hkv=hkv, d=d,
                    rows=rows, ctx_lo=lo, ctx_hi=hi, rate=rng.choice([1.0, 1.0, 0.41, 0.125]),
                    region=rng.random() < 0.25)
    if op == "rope":
        n = _spread(rng, 1, 20000)
        rot = rng.choice([d, d, d // 2, d // 4, 16 * rng.randint(1, d // 16)])
        return dict(op="rope", dtype=dtype, hq=hkv * rng.choice([1, 2, 4]), hkv=hkv, d=d, rot=rot,
                    n=n, first=rng.choice([-1, rng.randrange(1 << 20)]),
                    pairs=rng.choice(["halves", "neighbours"]), fused=rng.random() < 0.5)
    layers = rng.choice([1, 1, 2, 5, 28])
    rows = _spread(rng, 1, 40)
    most = max(1, 16384 * 8 // (layers * rows * hkv))
    hi = rng.choice([1, _spread(rng, 1, most), _spread(rng, 1, most)])
    lo = rng.choice([hi, 0 if op == "write" else 1, max(1, hi // 3)])
    lo = min(lo, hi)
    if op == "write":
        past = rng.choice([0, _spread(rng, 1, 1000)])
        return dict(op="write", fmt=fmt, dtype=dtype, hkv=hkv, d=d, layers=layers, rows=rows,
                    new_lo=lo, new_hi=hi, past_lo=past // 2, past_hi=past, ring=rng.random() < 0.4)
    return dict(op="read", fmt=fmt, dtype=dtype, hkv=hkv, d=d, layers=layers, rows=rows,
                len_lo=max(lo, 1), len_hi=hi)


def _lengths(case):
    """The rows' lengths: part of the case, not of the values that the seed makes.
    attn: (t, lo, hi, listed rows); write: (past, new); read: (t, n)."""
    r = random.Random("lengths %s" % sorted((k, v) for k, v in case.items() if k != "name"))
    rows = case["rows"]
    if case["op"] == "attn":
        t = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(rows)]
        t[0], t[-1] = case["ctx_lo"], case["ctx_hi"]
        lo, hi = [1] * rows, [x + 1 for x in t]
        if case["region"]:
            lo = [r.randint(1, x) for x in t]
            hi = [r.randint(a + 1, x + 1) for a, x in zip(lo, t)]
        rate = case["rate"]
        flagged = [b for b in range(rows) if rate >= 1.0 or r.random() < rate] or [rows - 1]
        return t, lo, hi, flagged
    if case["op"] == "write":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(rows)]
        new[-1] = max(1, case["new_hi"])
        return [r.randint(case["past_lo"], case["past_hi"]) for _ in range(rows)], new
    n = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(rows)]
    return [x + r.randint(0, 40) for x in n], n


def _touched(past, new):
    """Tokens from the start of the first block that a row's new tokens touch to its end."""
    return [past_b + n - past_b // TOKENS * TOKENS if n else 0 for past_b, n in zip(past, new)]


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] == "rope":
        rows = case["n"] * (case["hq"] + case["hkv"])
        return {"bytes": 2.0 * rows * d * size + 4.0 * case["n"] + 2.0 * d * size + 2.0 * case["rot"],
                "flops": rows * (4.0 * d + 3.0 * case["rot"])}
    hkv = case["hkv"]
    if case["op"] == "attn":
        t, lo, hi, flagged = _lengths(case)
        tokens = sum(hi[b] - lo[b] for b in flagged)
        blocks = sum((hi[b] - 2) // TOKENS - (lo[b] - 1) // TOKENS + 1 for b in flagged)
        return {"bytes": tokens * hkv * 2.0 * d + blocks * (hkv * 8.0 + 4.0) +
                len(flagged) * case["hq"] * (2.0 * d * size + 4.0) + 16.0 * case["rows"],
                "flops": 4.0 * tokens * case["hq"] * d}
    layers = case["layers"]
    if case["op"] == "write":
        past, new = _lengths(case)
        n, back = sum(new), sum(_touched(past, new))
        # new K/V read, codes written; the touched blocks' codes read, their values written
        each = n * (size + 1.0) + (back - n) * 1.0 + back * size
        blocks = sum(-(-x // TOKENS) for x in _touched(past, new))
        kept = sum(min(m, WINDOW) + min(SINK, m) for m in new) * size if case["ring"] else 0.0
        return {"bytes": layers * hkv * 2.0 * (d * (each + kept) + 4.0 * blocks) + 12.0 * case["rows"],
                "flops": layers * hkv * 2.0 * d * (3.0 * n + back)}
    t, n = _lengths(case)
    blocks = sum((a - 1) // TOKENS - (a - x) // TOKENS + 1 for a, x in zip(t, n))
    return {"bytes": layers * hkv * 2.0 * (d * sum(n) * (1.0 + size) + 4.0 * blocks) + 12.0 * case["rows"],
            "flops": layers * hkv * 2.0 * d * sum(n)}


# ------------------------------------------------------------------- prepare

def _to_codes(y, fmt):
    """Values in units of the scale -> the 8-bit codes nearest to them, as bytes."""
    if fmt == "int8":
        return y.round().clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _from_codes(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def _cache(case, blocks, g):
    """A paged cache with quantised values in it: keys with a few strong channels, values normal."""
    hkv, d = case["hkv"], case["d"]
    layers = case.get("layers", 1)
    codes = torch.empty((layers, blocks, hkv, 2, TOKENS, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((layers, blocks, hkv, 2), dtype=torch.float32, device="cuda")
    channel = torch.exp(0.8 * torch.randn((layers, 1, hkv, 2, 1, d), generator=g, device="cuda"))
    channel[:, :, :, 1] = 1.0
    step = max(1, (1 << 28) // (hkv * 2 * TOKENS * d))
    for l in range(layers):
        for a in range(0, blocks, step):
            m = min(step, blocks - a)
            x = torch.randn((m, hkv, 2, TOKENS, d), generator=g, device="cuda").mul_(0.5).mul_(channel[l])
            s = x.abs().amax((3, 4)) / TOP[case["fmt"]]
            scales[l, a:a + m] = s
            codes[l, a:a + m] = _to_codes(x.mul_((1.0 / s)[..., None, None]), case["fmt"])
    return codes, scales


def _table(lengths, g, spare=3):
    """Block table of rows of these lengths over shuffled blocks; -1 behind a row's last."""
    need = [max(1, -(-t // TOKENS)) for t in lengths]
    blocks = sum(need) + spare
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, blocks


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    return _ints(np.concatenate([[0], np.cumsum(counts)]).tolist())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    dtype, d = KIND[case["dtype"]], case["d"]
    s = {"case": case}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    if case["op"] == "rope":
        n, hq, hkv = case["n"], case["hq"], case["hkv"]
        if case["fused"]:                       # views of one projection's output, V behind them
            qkv = normal(n, hq + 2 * hkv, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            s["q"], s["k"] = normal(n, hq, d), normal(n, hkv, d)
        s["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)
        s["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)
        s["inv_freq"] = 10000.0 ** (-torch.arange(case["rot"] // 2, device="cuda").float() * 2.0 / case["rot"])
        if case["first"] < 0:                   # a decode batch: every row at a position of its own
            s["positions"] = torch.randint(1, 131072, (n,), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["positions"] = case["first"] + torch.arange(1, n + 1, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.empty((n, hq, d), dtype=dtype, device="cuda")
        s["k_out"] = torch.empty((n, hkv, d), dtype=dtype, device="cuda")
        return s

    rows, hkv = case["rows"], case["hkv"]
    if case["op"] == "attn":
        t, lo, hi, flagged = _lengths(case)
        s["table"], s["blocks"] = _table(t, g)
        s["codes"], s["scales"] = _cache(case, s["blocks"], g)
        s["q"] = normal(rows, case["hq"], d)
        s["t"], s["lo"], s["hi"] = _ints(t), _ints(lo), _ints(hi)
        s["idx"], s["count"] = _ints(flagged + [-1] * (rows - len(flagged))), _ints([len(flagged)])
        s["listed"] = len(flagged)              # known to the program, as the batch is
        s["out"] = normal(rows, case["hq"], d) * 0.005  # rows that are not listed keep what they hold
        s["lse"] = torch.zeros((rows, case["hq"]), dtype=torch.float32, device="cuda")
        return s

    if case["op"] == "write":
        past, n = _lengths(case)
        t, back = [a + b for a, b in zip(past, n)], _touched(past, n)
        s["start"], s["total"] = _starts(n), sum(n)
        s["k"], s["v"] = (0.5 * torch.randn((case["layers"], sum(n), hkv, d), generator=g, device="cuda")
                          .to(dtype) for _ in "kv")
        s["ring"] = None
        if case["ring"]:
            tiles = -(-(SINK + WINDOW) // TOKENS)
            s["ring"] = torch.zeros((case["layers"], rows, hkv, tiles, 2, TOKENS, d), dtype=dtype, device="cuda")
    else:
        t, back = _lengths(case)
    s["t"], s["back"], s["back_total"] = _ints(t), _starts(back), sum(back)
    s["blocks_touched"] = sum(-(-x // TOKENS) for x in back)
    s["table"], s["blocks"] = _table(t, g)
    s["codes"], s["scales"] = _cache(case, s["blocks"], g)
    s["k_out"], s["v_out"] = (torch.empty((case["layers"], sum(back), hkv, d), dtype=dtype, device="cuda")
                              for _ in "kv")
    return s


# --------------------------------------------------------------- plain forms

def _plain_rope(s):
    case = s["case"]
    half = case["rot"] // 2
    # far positions: the angle is formed and reduced in 64 bits
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        r = y[..., :case["rot"]]
        if case["pairs"] == "halves":
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out.append(torch.cat([r, y[..., case["rot"]:]], -1).to(KIND[case["dtype"]]))
    return out


def _row_of(starts, total):
    """The row of each of `total` items that `starts` divides among the rows."""
    counts = (starts[1:] - starts[:-1]).long()
    return torch.repeat_interleave(torch.arange(len(counts), device="cuda"), counts, output_size=total)


def _plain_read(s):
    case = s["case"]
    row = _row_of(s["back"], s["back_total"])
    at = torch.arange(s["back_total"], device="cuda") - s["back"].long()[row]
    p = s["t"].long()[row] - (s["back"][1:] - s["back"][:-1]).long()[row] + at      # 0-indexed position
    block = s["table"][row, p // TOKENS].long()
    out = []
    for kv in (0, 1):
        # two index tensors apart from each other: their dimension comes first
        c = _from_codes(s["codes"][:, :, :, kv][:, block, :, p % TOKENS], case["fmt"]).transpose(0, 1)
        out.append((c * s["scales"][:, :, :, kv][:, block][..., None]).to(KIND[case["dtype"]]))
    return out


def _plain_write(s):
    case = s["case"]
    fmt, layers, hkv, d = case["fmt"], case["layers"], case["hkv"], case["d"]
    n_b = (s["start"][1:] - s["start"][:-1]).long()
    t = s["t"].long()
    past = t - n_b
    first = past // TOKENS
    blocks_b = torch.where(n_b > 0, (t - 1) // TOKENS - first + 1, torch.zeros_like(t))
    block_start = torch.cat([blocks_b.new_zeros(1), blocks_b.cumsum(0)])
    nb = s["blocks_touched"]
    brow = _row_of(block_start, nb)
    column = first[brow] + torch.arange(nb, device="cuda") - block_start[brow]
    block = s["table"][brow, column].long()
    p = column[:, None] * TOKENS + torch.arange(TOKENS, device="cuda")               # [nb][16]
    old, new = p < past[brow][:, None], (p >= past[brow][:, None]) & (p < t[brow][:, None])
    token = (s["start"].long()[brow][:, None] + p - past[brow][:, None]).clamp(0, s["total"] - 1)
    had_any = old.any(1)
    for kv, x in ((0, s["k"]), (1, s["v"])):
        x = x[:, token].float().permute(0, 1, 3, 2, 4)                                # [L][nb][hkv][16][d]
        x = torch.where(new[None, :, None, :, None], x, torch.zeros_like(x))
        held = torch.where(had_any[None, :, None], s["scales"][:, :, :, kv][:, block], 0.0)
        a = x.abs().amax((3, 4))
        scale = torch.maximum(a / a.new_full((), TOP[fmt]), held)   # a tensor: by a number torch multiplies
        scale = torch.where(scale < LEAST, torch.zeros_like(scale), scale)
        inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
        had = s["codes"][:, :, :, kv][:, block]                                       # [L][nb][hkv][16][d]
        grown = (scale > held)[..., None, None]
        moved = _to_codes(_from_codes(had, fmt) * (held * inv)[..., None, None], fmt)
        code = torch.where(new[None, :, None, :, None], _to_codes(x * inv[..., None, None], fmt),
                           torch.where(old[None, :, None, :, None] & grown, moved, had))
        s["codes"][:, :, :, kv][:, block] = code
        s["scales"][:, :, :, kv][:, block] = scale
    out = _plain_read(s)
    if s["ring"] is None:
        return out
    row = _row_of(s["start"], s["total"])
    p = past[row] + torch.arange(s["total"], device="cuda") - s["start"].long()[row]  # 0-indexed
    for kv, x in ((0, s["k"]), (1, s["v"])):
        flat = s["ring"][:, :, :, :, kv].permute(1, 3, 4, 0, 2, 5)                    # [B][tile][16][L][hkv][d]
        for slot, keep in ((SINK + p % WINDOW, p >= t[row] - WINDOW), (p.clamp(max=SINK), p < SINK)):
            # what is not kept goes to a slot behind the ring's last, where the last tile has one
            slot = torch.where(keep, slot, torch.full_like(slot, SINK + WINDOW))
            flat[row, slot // TOKENS, slot % TOKENS] = x.transpose(0, 1)
        flat[:, (SINK + WINDOW) // TOKENS, (SINK + WINDOW) % TOKENS] = 0
    return out + [s["ring"]]


def _plain_attn(s):
    case = s["case"]
    hq, hkv, d, fmt = case["hq"], case["hkv"], case["d"], case["fmt"]
    rows = s["idx"][:s["listed"]].long()
    table = s["table"][rows].clamp(min=0).long()                                      # [R][mb]
    p = torch.arange(table.shape[1] * TOKENS, device="cuda") + 1
    inside = (p >= s["lo"][rows][:, None]) & (p < s["hi"][rows][:, None])             # [R][T]
    q = s["q"][rows].float().view(len(rows), hkv, hq // hkv, d)

    def values(kv):                                                                   # [R][hkv][T][d]
        x = _from_codes(s["codes"][0, :, :, kv][table], fmt)                          # [R][mb][hkv][16][d]
        x *= s["scales"][0, :, :, kv][table][..., None, None]
        return x.transpose(1, 2).reshape(len(rows), hkv, -1, d)

    k = values(0)
    score = torch.stack([(k @ q[:, :, h, :, None])[..., 0] for h in range(hq // hkv)], 2) / math.sqrt(d)
    del k
    score = score.masked_fill(~inside[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    e = (score - top).exp()
    total = e.sum(-1, keepdim=True)
    v = values(1)
    # positions outside hold nothing of the row: their values take no part
    v = v.masked_fill(~inside[:, None, :, None], 0.0)
    o = (e / total) @ v
    s["out"][rows] = o.reshape(len(rows), hq, d).to(s["out"].dtype)
    s["lse"][rows] = (top + total.log()).reshape(len(rows), hq)
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------- own form

_contexts = {}


def _context(s):
    """The library handle of this shape, which a program makes once and keeps."""
    from gated_local_full_b200 import oda
    case = s["case"]
    table = s.get("table")
    key = (case.get("layers", 1), case.get("rows", 1), case.get("hq", case["hkv"]), case["hkv"], case["d"],
           case["dtype"], 1 if table is None else table.shape[1], s.get("blocks", 1))
    if key not in _contexts:
        layers, rows, hq, hkv, d, dtype, columns, blocks = key
        _contexts[key] = oda.OdaContext(oda.make_config(
            layers=layers, max_batch=rows, hq=hq, hkv=hkv, head_dim=d, sink=SINK, window=WINDOW,
            dtype=dtype, max_blocks_per_seq=columns, num_blocks=blocks))
    return _contexts[key]


def _own(s):
    case = s["case"]
    ctx = _context(s)
    if case["op"] == "rope":
        ctx.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], 1e-6, s["inv_freq"],
                         s["positions"], s["q_out"], s["k_out"],
                         interleaved=case["pairs"] == "neighbours")
        return [s["q_out"], s["k_out"]]
    if case["op"] == "attn":
        if case["region"]:
            ctx.range_attn_kv8(case["fmt"], 0, s["q"], s["t"], s["lo"], s["hi"], s["table"], s["codes"],
                               s["scales"], s["idx"], s["count"], s["out"], s["lse"], case["rows"])
        else:
            ctx.full_attn_kv8(case["fmt"], 0, s["q"], s["t"], s["table"], s["codes"], s["scales"],
                              s["idx"], s["count"], s["out"], s["lse"], case["rows"])
        return [s["out"], s["lse"]]
    if case["op"] == "write":
        one_each = case["new_lo"] == 1 and case["new_hi"] == 1
        ctx.append_kv8(case["fmt"], 0, case["layers"], s["k"], s["v"], s["t"], s["table"], s["codes"],
                       s["scales"], s["ring"], case["rows"], tok_start=None if one_each else s["start"])
    ctx.read_kv8(case["fmt"], 0, case["layers"], s["t"], s["table"], s["codes"], s["scales"],
                 s["k_out"], s["v_out"], case["rows"], tok_start=s["back"])
    out = [s["k_out"], s["v_out"]]
    return out + [s["ring"]] if s.get("ring") is not None else out


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    if op == "write":
        return _plain_write(state)
    if op == "read":
        return _plain_read(state)
    return _plain_attn(state)


# ---------------------------------------------------------------------- exact

def _nearest(y, fmt):
    """The number of the 8-bit format nearest to each y (64 bits in and out), ties to even."""
    if fmt == "int8":
        return torch.clamp(torch.round(y), -127.0, 127.0)
    size = y.abs()
    _, exponent = torch.frexp(size)                          # size = f * 2^exponent, f in [1/2, 1)
    gap = torch.ldexp(torch.ones_like(size), torch.clamp(exponent - 1, min=-6) - 3)
    return torch.sign(y) * torch.clamp(torch.round(size / gap) * gap, max=448.0)


def _held(codes, fmt):
    """The numbers that 8-bit codes stand for, in 64 bits, from their bits."""
    c = codes.to(torch.int32)
    if fmt == "int8":
        return torch.where(c > 127, c - 256, c).double()
    e, m = (c >> 3) & 15, (c & 7).double()
    size = torch.where(e > 0, torch.ldexp(1.0 + m / 8.0, e - 7), m * 2.0 ** -9)
    return torch.where(c > 127, -size, size)


def _single(x):
    return x.float().double()


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "rope":
        angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle)
        out = []
        for x, w in ((s["q"].double(), s["q_weight"].double()), (s["k"].double(), s["k_weight"].double())):
            y = x / (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w
            r, h = y[..., :case["rot"]], case["rot"] // 2
            z = torch.complex(r[..., :h], r[..., h:]) if case["pairs"] == "halves" else \
                torch.view_as_complex(r.reshape(*r.shape[:-1], h, 2).contiguous())
            z = z * turn
            r = torch.cat([z.real, z.imag], -1) if case["pairs"] == "halves" else torch.view_as_real(z).flatten(-2)
            out.append(torch.cat([r, y[..., case["rot"]:]], -1))
        return out
    if case["op"] == "attn":
        t, lo, hi, flagged = _lengths(case)
        out, lse = s["out"].double(), s["lse"].double()
        group = case["hq"] // case["hkv"]
        for b in flagged:
            first = (lo[b] - 1) // TOKENS
            blocks = s["table"][b, first:(hi[b] - 2) // TOKENS + 1].long()
            a, e = lo[b] - 1 - first * TOKENS, hi[b] - 1 - first * TOKENS
            for h in range(case["hkv"]):
                k, v = ((_held(s["codes"][0, blocks, h, kv], case["fmt"]) *
                         s["scales"][0, blocks, h, kv].double()[:, None, None]).reshape(-1, d)[a:e] for kv in (0, 1))
                q = s["q"][b, h * group:(h + 1) * group].double()
                score = q @ k.T / math.sqrt(d)
                sums = torch.logsumexp(score, -1)
                out[b, h * group:(h + 1) * group] = torch.exp(score - sums[:, None]) @ v
                lse[b, h * group:(h + 1) * group] = sums
        return [out, lse]
    fmt, layers = case["fmt"], case["layers"]
    table = s["table"].tolist()
    if case["op"] == "write":
        past, new = _lengths(case)
        lengths, back = [a + n for a, n in zip(past, new)], _touched(past, new)
    else:
        lengths, back = _lengths(case)
    # the rows' blocks that are read back, one after another: row b's block column c is at[b] + c
    used, at_row = [], []
    for t, n, blocks in zip(lengths, back, table):
        first = (t - n) // TOKENS
        at_row.append(len(used) - first)
        used += blocks[first:(t - 1) // TOKENS + 1] if n else []
    used = torch.tensor(used, device="cuda")
    values = _held(s["codes"][:, used], fmt)                 # [L][used][hkv][2][16][d]
    scales = s["scales"][:, used].double()
    if case["op"] == "write":
        at = 0
        for b, n in enumerate(new):
            p = past[b]
            while p < past[b] + n:                           # one block after another
                end = min((p // TOKENS + 1) * TOKENS, past[b] + n)
                block, o = at_row[b] + p // TOKENS, p % TOKENS
                for kv, x in ((0, s["k"]), (1, s["v"])):
                    x = x[:, at:at + end - p].double().transpose(1, 2)                # [L][hkv][m][d]
                    before = scales[:, block, :, kv] if o else torch.zeros_like(scales[:, block, :, kv])
                    a = x.abs().amax((2, 3))
                    scale = torch.maximum(_single(a / a.new_full((), TOP[fmt])), before)
                    scale = torch.where(scale < LEAST, 0.0, scale)
                    inv = torch.where(scale > 0, _single(1.0 / scale), 0.0)
                    kept = values[:, block, :, kv, :o]
                    moved = _nearest(_single(kept * _single(before * inv)[..., None, None]), fmt)
                    values[:, block, :, kv, :o] = torch.where((scale > before)[..., None, None], moved, kept)
                    values[:, block, :, kv, o:o + end - p] = _nearest(_single(x * inv[..., None, None]), fmt)
                    scales[:, block, :, kv] = scale
                at, p = at + end - p, end
    values *= scales[..., None, None]
    out = [torch.empty(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in "kv"]
    at = 0
    for t, n, a in zip(lengths, back, at_row):
        if n:
            first = (t - n) // TOKENS
            v = values[:, a + first:a + (t - 1) // TOKENS + 1]
            v = v.permute(3, 0, 1, 4, 2, 5).flatten(2, 3)    # [2][L][tokens][hkv][d]
            o = t - n - first * TOKENS
            out[0][:, at:at + n], out[1][:, at:at + n] = v[0][:, o:o + n], v[1][:, o:o + n]
            at += n
    if s.get("ring") is None:
        return out
    ring = s["ring"].double()
    at = 0
    for b, (p0, n) in enumerate(zip(past, new)):
        for i in range(n):
            p = p0 + i + 1
            for slot in ([SINK + (p - 1) % WINDOW] if i >= n - WINDOW else []) + ([p - 1] if p <= SINK else []):
                for kv, x in ((0, s["k"]), (1, s["v"])):
                    ring[:, b, :, slot // TOKENS, kv, slot % TOKENS] = x[:, at + i].double()
        at += n
    return out + [ring]
