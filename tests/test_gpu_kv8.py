"""The 8-bit cache, its attention and the head norm with rotation on the GPU,
against the float64 oracle.

Codes, scales and values read back are equal bit for bit. The bounds of the
others are worked out at `attn_bound` and `rope_bound`.
"""

import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24                                  # half a float32 step, relative
HALF = {"bf16": 2.0 ** -8, "f32": U32}            # rounding of the output


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("needs a GPU")
    return t


class Case:
    """A context with an 8-bit cache, its oracle and shuffled blocks."""

    def __init__(self, torch, fmt="int8", dtype="bf16", hq=4, hkv=2, d=128, layers=1, rows=3,
                 columns=8, sink=4, window=32, seed=0, spare=2, num_blocks=None):
        from gated_local_full_b200 import oda
        self.t, self.oda, self.fmt, self.dtype = torch, oda, fmt, dtype
        self.hq, self.hkv, self.d, self.layers, self.rows = hq, hkv, d, layers, rows
        self.sink, self.window, self.columns = sink, window, columns
        self.blocks = num_blocks or rows * columns + spare
        self.cfg = oda.make_config(layers=layers, max_batch=rows, hq=hq, hkv=hkv, head_dim=d,
                                   sink=sink, window=window, dtype=dtype,
                                   max_blocks_per_seq=columns, num_blocks=self.blocks)
        self.ctx = oda.OdaContext(self.cfg)
        self.kind = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.r = np.random.default_rng(seed)
        order = self.r.permutation(self.blocks)[:rows * columns]
        if num_blocks:
            order[0], order[-1] = num_blocks - 1, num_blocks - 2      # the far end of the pool
        self.table_h = order.reshape(rows, columns).astype(np.int32)
        self.table = torch.from_numpy(self.table_h).cuda()
        lay = oda.kv8_layout(self.cfg)
        shape = (layers, self.blocks, hkv, 2, 16, d)
        assert layers * lay["cache_layer_bytes"] == int(np.prod(shape, dtype=np.int64))
        if num_blocks:
            self.codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
            return
        # what no token has written yet: NaN codes (e4m3) under odd scales
        self.codes_h = np.full(shape, 0x7F if fmt == "e4m3" else 0x81, np.uint8)
        self.scales_h = np.full(shape[:4], np.float32(3.25), np.float32)
        self.codes = torch.from_numpy(self.codes_h.copy()).cuda()
        self.scales = torch.from_numpy(self.scales_h.copy()).cuda()
        tiles = self.ctx.layout["ring_blocks"]
        self.ring = torch.full((layers, rows, hkv, tiles, 2, 16, d), 5.0, dtype=self.kind, device="cuda")
        self.ring_h = self.ring.double().cpu().numpy()

    def ints(self, x):
        return self.t.tensor(list(x), dtype=self.t.int32, device="cuda")

    def values(self, *shape, scale=1.0):
        """Numbers of the context's type, as (float64, device tensor)."""
        x = self.t.from_numpy(self.r.standard_normal(shape) * scale).to(self.kind)
        return x.double().numpy(), x.cuda()

    def starts(self, n):
        return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)

    def oracle_write(self, k, v, n, past, ring=True):
        at = self.starts(n)
        for b, (m, p0) in enumerate(zip(n, past)):
            for l in range(self.layers):
                for kv, x in ((0, k), (1, v)):
                    for g in range(self.hkv):
                        p = p0
                        while p < p0 + m:
                            end = min(p // 16 * 16 + 16, p0 + m)
                            blk = self.table_h[b, p // 16]
                            i = at[b] + p - p0
                            self.scales_h[l, blk, g, kv] = O.kv8_write_block(
                                self.codes_h[l, blk, g, kv], self.scales_h[l, blk, g, kv], p % 16,
                                x[l, i:i + end - p, g], self.fmt)
                            p = end
                    for i in range(m) if ring else ():
                        p = p0 + i
                        slots = [p] if p < self.sink else []
                        if p >= p0 + m - self.window:
                            slots.append(self.sink + p % self.window)
                        for s in slots:
                            self.ring_h[l, b, :, s // 16, kv, s % 16] = x[l, at[b] + i]

    def write(self, n, past, one_each=False, ring=True, scale=1.0):
        total = int(sum(n))
        (k, kd), (v, vd) = (self.values(self.layers, total, self.hkv, self.d, scale=scale) for _ in "kv")
        t = [a + b for a, b in zip(past, n)]
        self.ctx.append_kv8(self.fmt, 0, self.layers, kd, vd, self.ints(t), self.table, self.codes,
                            self.scales, self.ring if ring else None, len(n),
                            tok_start=None if one_each else self.ints(self.starts(n)))
        self.oracle_write(k, v, n, past, ring)
        return t

    def check(self):
        assert self.ctx.get_device_error() == 0
        assert np.array_equal(self.scales.cpu().numpy(), self.scales_h, equal_nan=True)
        assert np.array_equal(self.codes.cpu().numpy(), self.codes_h)
        assert np.array_equal(self.ring.double().cpu().numpy(), self.ring_h)

    def kv(self, layer, b, t):
        """K, V of a row's positions 1..t as the codes' values, float64 [hkv][t][d]."""
        out = []
        for kv in (0, 1):
            blk = self.table_h[b, :(t + 15) // 16]
            x = O.kv8_value(self.codes_h[layer, blk, :, kv], self.fmt) * \
                self.scales_h[layer, blk, :, kv].astype(np.float64)[..., None, None]
            out.append(x.transpose(1, 0, 2, 3).reshape(self.hkv, -1, self.d)[:, :t])
        return out


# ------------------------------------------------------------ write, read back

WRITES = [
    dict(fmt="int8", dtype="bf16", d=128), dict(fmt="e4m3", dtype="bf16", d=128, hkv=3, hq=3),
    dict(fmt="int8", dtype="f32", d=64, layers=2), dict(fmt="e4m3", dtype="f32", d=128),
    dict(fmt="e4m3", dtype="bf16", d=64, hkv=1, hq=4), dict(fmt="int8", dtype="f32", d=128),
    dict(fmt="int8", dtype="bf16", d=64), dict(fmt="e4m3", dtype="f32", d=64),
]


@pytest.mark.parametrize("kw", WRITES, ids=lambda k: "-".join(map(str, k.values())))
def test_codes_scales_and_ring_bit_exact(torch, kw):
    """Ragged chunks (none, one, across borders, longer than the ring), then
    single tokens, then ragged again, into the same blocks."""
    c = Case(torch, rows=5, sink=3, window=20, columns=6, **kw)
    t = c.write([0, 1, 16, 37, 5], [0, 0, 0, 0, 0])
    c.check()
    for _ in range(4):
        t = c.write([1] * 5, t, one_each=True)
    c.check()
    t = c.write([13, 0, 1, 40, 26], t, scale=2.5)
    c.check()
    # read back: all of each row, then a ragged stretch into one output only
    for n, only in ((t, None), ([1, 0, 7, 33, 20], 1)):
        total, at = sum(n), c.starts(n)
        outs = [torch.full((c.layers, total, c.hkv, c.d), 9.0, dtype=c.kind, device="cuda") for _ in "kv"]
        c.ctx.read_kv8(c.fmt, 0, c.layers, c.ints(t), c.table, c.codes, c.scales,
                       outs[0] if only is None else None, outs[1], 5, tok_start=c.ints(at))
        for l in range(c.layers):
            for b in range(5):
                for kv, x in enumerate(c.kv(l, b, t[b])):
                    if kv == 0 and only is not None:
                        continue
                    want = torch.from_numpy(x[:, t[b] - n[b]:t[b]]).float().to(c.kind)
                    got = outs[kv][l, at[b]:at[b + 1]].transpose(0, 1).cpu()
                    assert torch.equal(got, want), (l, b, kv)
    one = [torch.zeros((c.layers, 5, c.hkv, c.d), dtype=c.kind, device="cuda") for _ in "kv"]
    c.ctx.read_kv8(c.fmt, 0, c.layers, c.ints(t), c.table, c.codes, c.scales, one[0], one[1], 5)
    assert torch.equal(one[1][0, 3].cpu().double(),
                       torch.from_numpy(c.kv(0, 3, t[3])[1][:, -1]).float().to(c.kind).double())
    assert c.ctx.get_device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_zero_tiny_and_not_finite_values(torch, fmt):
    c = Case(torch, fmt=fmt, dtype="f32", hq=1, hkv=1, d=64, rows=6, columns=2)
    x = np.zeros((1, 6, 1, 64))
    x[0, 1] = 2.0 ** -101
    x[0, 2, 0, 3], x[0, 3, 0, 5], x[0, 4, 0, 7] = np.nan, np.inf, -np.inf
    x[0, 5] = 3.0e38
    xd = torch.from_numpy(x).float().cuda()
    c.ctx.append_kv8(fmt, 0, 1, xd, xd, c.ints([1] * 6), c.table, c.codes, c.scales, None, 6)
    assert c.ctx.get_device_error() == 0
    s = c.scales.cpu().numpy()[0, c.table_h[:, 0], 0]
    assert np.all(s[:2] == 0) and np.isnan(s[2:5]).all() and np.all(s[5] > 0)
    codes = c.codes.cpu().numpy()[0, c.table_h[:, 0], 0, :, 0]
    assert not codes[:2].any()
    # a later token leaves the block NaN; the block's next start clears it
    ones = torch.ones((1, 6, 1, 64), device="cuda")
    c.ctx.append_kv8(fmt, 0, 1, ones, ones, c.ints([2] * 6), c.table, c.codes, c.scales, None, 6)
    s = c.scales.cpu().numpy()[0, c.table_h[:, 0], 0]
    assert np.isnan(s[2:5]).all() and np.all(s[:2] == np.float32(1 / np.float32(O.KV8_TOP[fmt])))
    out = torch.zeros((1, 6, 1, 64), device="cuda")
    c.ctx.read_kv8(fmt, 0, 1, c.ints([2] * 6), c.table, c.codes, c.scales, out, None, 6)
    assert torch.isnan(out[0, 2:5]).all() and torch.isfinite(out[0, [0, 1, 5]]).all()
    c.ctx.append_kv8(fmt, 0, 1, ones, ones, c.ints([1] * 6), c.table, c.codes, c.scales, None, 6)
    c.ctx.read_kv8(fmt, 0, 1, c.ints([1] * 6), c.table, c.codes, c.scales, out, None, 6)
    assert torch.allclose(out, ones, rtol=2.0 ** -20, atol=0)


def test_write_errors_skip_the_row_and_are_recorded(torch):
    oda = pytest.importorskip("gated_local_full_b200.oda")
    c = Case(torch, rows=4, columns=3)
    k = torch.ones((1, 8, 2, 128), dtype=c.kind, device="cuda")

    def bad(t, at, table=None, what=None):
        before = (c.codes.clone(), c.scales.clone(), c.ring.clone())
        out = torch.full_like(k, 7.0)
        for f in (lambda: c.ctx.append_kv8("int8", 0, 1, k, k, c.ints(t), table if table is not None else c.table,
                                           c.codes, c.scales, c.ring, 4, tok_start=c.ints(at)),
                  lambda: c.ctx.read_kv8("int8", 0, 1, c.ints(t), table if table is not None else c.table,
                                         c.codes, c.scales, out, None, 4, tok_start=c.ints(at))):
            f()
            assert c.ctx.get_device_error() == oda.ERR_BOUNDS
        return before, out

    # row 1 has more new tokens than positions; row 2 too many columns; rows 0 and 3 are written
    before, out = bad([2, 2, 60, 1], [0, 2, 5, 7, 8])
    blk = c.table_h[0, 0]
    assert not torch.equal(c.codes[0, blk], before[0][0, blk])
    assert torch.equal(c.codes[0, c.table_h[1]], before[0][0, c.table_h[1]])
    assert torch.equal(c.ring[0, 1], before[2][0, 1])
    assert (out[0, 2:5] == 7).all() and (out[0, :2] != 7).all()
    table = c.table.clone()
    table[0, 0], table[3, 0] = -1, c.blocks
    before, out = bad([2, 3, 2, 1], [0, 2, 5, 7, 8], table)
    assert torch.equal(c.codes[0, c.table_h[0, 0]], before[0][0, c.table_h[0, 0]])
    for at in ([0, 9, 5, 7, 8], [0, 2, 5, 7, 9], [-1, 2, 5, 7, 8]):
        bad([3, 9, 2, 3], at)


# ---------------------------------------------------------------------- attention

def attn_bound(q, K, V, lo, hi, dtype, lse=False):
    """Largest error of out [hq][d] (or lse [hq]) over positions lo..hi-1.

    A score is a sum of d products and takes at most (d + 8) float32 roundings
    (counted as whole steps, 2^-23, for the tensor cores), each of at most
    A = max_j sum |q k| / sqrt(d); the query's f16 form adds 2^-21 A; its scaling
    2^-22 |s|. So |ds| <= e = (d + 16) 2^-23 A + 2^-21 A. Weights move by a
    factor of at most exp(2 e); exponents of 2 are rounded at magnitudes below
    64 (2^-18), approximated within 2^-21, split within 2^-22, and the sums over
    up to n weights are taken by tile and then by warp, n / 64 + 64 steps of
    2^-24 at most: together w. An output then moves by (2 e + w) sum_j p_j |v_j|,
    and its rounding adds half a step."""
    d = q.shape[1]
    n = hi - lo
    group = q.shape[0] // K.shape[0]
    bounds = []
    for h in range(q.shape[0]):
        k, v = K[h // group, lo - 1:hi - 1], V[h // group, lo - 1:hi - 1]
        s = k @ q[h] / np.sqrt(d)
        A = (np.abs(k) @ np.abs(q[h])).max() / np.sqrt(d)
        e = (d + 16) * 2.0 ** -23 * A + 2.0 ** -21 * A
        w = 2.0 ** -18 + 2.0 ** -20 + (n / 64 + 64) * U32
        p = np.exp(s - s.max())
        p /= p.sum()
        o = p @ v
        if lse:
            L = s.max() + np.log(np.exp(s - s.max()).sum())
            bounds.append(e + w + 2.0 ** -22 * abs(L))
        else:
            bounds.append((2 * e + w) * (p @ np.abs(v)) + HALF[dtype] * np.abs(o) + 1e-30)
    return np.array(bounds)


def check_rows(c, q, out, lse, rows, t, lo=None, hi=None, layer=0):
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in rows:
        a, e = (1, t[b] + 1) if lo is None else (lo[b], hi[b])
        K, V = c.kv(layer, b, t[b])
        want, wl = O.range_attention(q[b], K, V, a, e)
        assert np.all(np.abs(got[b] - want) <= attn_bound(q[b], K, V, a, e, c.dtype)), b
        assert np.all(np.abs(gl[b] - wl) <= attn_bound(q[b], K, V, a, e, c.dtype, lse=True)), b


def listed(c, rows, B):
    return c.ints(list(rows) + [-1] * (B - len(rows))), c.ints([len(rows)])


ATTN = [
    dict(fmt="int8", dtype="bf16", hq=4, hkv=2, d=128), dict(fmt="e4m3", dtype="bf16", hq=4, hkv=2, d=128),
    dict(fmt="int8", dtype="f32", hq=4, hkv=2, d=128), dict(fmt="e4m3", dtype="f32", hq=2, hkv=1, d=64),
    dict(fmt="int8", dtype="bf16", hq=8, hkv=2, d=128), dict(fmt="e4m3", dtype="bf16", hq=3, hkv=3, d=64),
    dict(fmt="e4m3", dtype="f32", hq=4, hkv=1, d=128), dict(fmt="int8", dtype="f32", hq=4, hkv=1, d=64),
    dict(fmt="int8", dtype="bf16", hq=4, hkv=1, d=64), dict(fmt="e4m3", dtype="f32", hq=1, hkv=1, d=128),
]


@pytest.mark.parametrize("kw", ATTN, ids=lambda k: "-".join(map(str, k.values())))
def test_attention_of_listed_rows(torch, kw):
    t = [1, 2, 15, 16, 17, 100, 333, 1500]
    c = Case(torch, rows=8, columns=94, **kw)
    c.write(t, [0] * 8, ring=False)
    c.check()
    q, qd = c.values(8, c.hq, c.d, scale=2.0)
    for rows in ([0, 1, 2, 3, 4, 5, 6, 7], [7], [2, 0], []):
        out = torch.full((8, c.hq, c.d), 7.0, dtype=c.kind, device="cuda")
        lse = torch.full((8, c.hq), 7.0, device="cuda")
        idx, count = listed(c, rows, 8)
        c.ctx.full_attn_kv8(c.fmt, 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 8)
        assert c.ctx.get_device_error() == 0
        check_rows(c, q, out, lse, rows, t)
        rest = [b for b in range(8) if b not in rows]
        assert (out[rest] == 7).all() and (lse[rest] == 7).all()
        again = torch.zeros_like(out)
        c.ctx.full_attn_kv8(c.fmt, 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, again, None, 8)
        torch.cuda.synchronize()
        assert not rows or torch.isfinite(again[rows]).all()


@pytest.mark.parametrize("kw", ATTN[:6], ids=lambda k: "-".join(map(str, k.values())))
def test_attention_of_regions(torch, kw):
    """Regions that start and end inside blocks, of one position, and of all."""
    t = [1, 40, 40, 40, 700, 700, 1201]
    lo = [1, 5, 40, 16, 17, 300, 2]
    hi = [2, 6, 41, 18, 701, 333, 1200]
    c = Case(torch, rows=7, columns=76, **kw)
    c.write(t, [0] * 7, ring=False)
    q, qd = c.values(7, c.hq, c.d, scale=2.0)
    out, lse = torch.zeros((7, c.hq, c.d), dtype=c.kind, device="cuda"), torch.zeros((7, c.hq), device="cuda")
    idx, count = listed(c, range(7), 7)
    c.ctx.range_attn_kv8(c.fmt, 0, qd, c.ints(t), c.ints(lo), c.ints(hi), c.table, c.codes, c.scales,
                         idx, count, out, lse, 7)
    assert c.ctx.get_device_error() == 0
    check_rows(c, q, out, lse, range(7), t, lo, hi)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_scales_far_apart(torch, fmt):
    """One block's values 2^60 above the others', another's all zero; keys too
    small to matter in one block; a query with one large element."""
    t = [200]
    c = Case(torch, fmt=fmt, dtype="f32", hq=2, hkv=1, d=64, rows=1, columns=13)
    (k, _), (v, _) = (c.values(1, 200, 1, 64) for _ in "kv")
    v[:, 32:48] *= 2.0 ** 60
    v[:, 64:80] = 0.0
    v[:, 96:112] *= 2.0 ** -60
    k[:, 112:128] *= 2.0 ** -40
    k[:, 16:32] = 0.0
    c.ctx.append_kv8(fmt, 0, 1, torch.from_numpy(k).float().cuda(), torch.from_numpy(v).float().cuda(),
                     c.ints(t), c.table, c.codes, c.scales, None, 1, tok_start=c.ints([0, 200]))
    c.oracle_write(k, v, [200], [0], ring=False)
    q, _ = c.values(1, 2, 64)
    q[0, 0, 5] = 900.0                                   # a peaked softmax
    qd = torch.from_numpy(q).float().cuda()
    out, lse = torch.zeros((1, 2, 64), device="cuda"), torch.zeros((1, 2), device="cuda")
    idx, count = listed(c, [0], 1)
    c.ctx.full_attn_kv8(fmt, 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 1)
    assert c.ctx.get_device_error() == 0
    check_rows(c, q, out, lse, [0], t)
    # regions that hold the zero block alone, the tiny one alone, the last two
    for lo, hi in ((65, 81), (97, 113), (64, 200), (81, 113)):
        c.ctx.range_attn_kv8(fmt, 0, qd, c.ints(t), c.ints([lo]), c.ints([hi]), c.table, c.codes,
                             c.scales, idx, count, out, lse, 1)
        check_rows(c, q, out, lse, [0], t, [lo], [hi])


def test_not_finite_values_stay_visible(torch):
    """A NaN block poisons the rows that read it, and no other row."""
    c = Case(torch, dtype="f32", hq=2, hkv=1, d=64, rows=3, columns=3)
    t = [40, 40, 16]
    c.write(t, [0] * 3, ring=False)
    c.scales[0, c.table_h[0, 1], 0, 1] = float("nan")
    c.scales[0, c.table_h[2, 0], 0, 0] = float("nan")
    _, qd = c.values(3, 2, 64)
    out, lse = torch.zeros((3, 2, 64), device="cuda"), torch.zeros((3, 2), device="cuda")
    idx, count = listed(c, range(3), 3)
    c.ctx.full_attn_kv8("int8", 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 3)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all() and torch.isnan(out[2]).all()
    assert torch.isfinite(lse[:2]).all() and torch.isnan(lse[2]).all()
    qd[1] = float("inf")
    c.ctx.full_attn_kv8("int8", 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 3)
    assert torch.isnan(out[1]).all()


def test_attention_errors(torch):
    oda = pytest.importorskip("gated_local_full_b200.oda")
    c = Case(torch, rows=4, columns=3)
    t = [20, 30, 48, 5]
    c.write(t, [0] * 4, ring=False)
    q, qd = c.values(4, c.hq, c.d)
    out = torch.full((4, c.hq, c.d), 7.0, dtype=c.kind, device="cuda")
    lse = torch.full((4, c.hq), 7.0, device="cuda")

    def call(t2=t, rows=(0, 1, 2, 3), lo=None, hi=None, count=None):
        idx, n = listed(c, rows, 4)
        n = n if count is None else c.ints([count])
        if lo is None:
            c.ctx.full_attn_kv8("int8", 0, qd, c.ints(t2), c.table, c.codes, c.scales, idx, n, out, lse, 4)
        else:
            c.ctx.range_attn_kv8("int8", 0, qd, c.ints(t2), c.ints(lo), c.ints(hi), c.table, c.codes,
                                 c.scales, idx, n, out, lse, 4)
        return c.ctx.get_device_error()

    assert call(t2=[20, 0, 49, 5]) == oda.ERR_BOUNDS              # no position; too many columns
    assert (out[1:3] == 7).all()
    check_rows(c, q, out, lse, [0, 3], t)
    assert call(rows=(0, 4, -1)) == oda.ERR_BOUNDS
    assert call(count=9) == oda.ERR_BOUNDS and call(count=-2) == oda.ERR_BOUNDS
    for lo, hi in (([0, 1, 1, 1], [5, 5, 5, 5]), ([1, 9, 1, 1], [5, 9, 5, 5]), ([1] * 4, [5, 5, 5, 7])):
        assert call(lo=lo, hi=hi) == oda.ERR_BOUNDS
    # a block id out of range: its tokens are left out, nothing else is touched
    keep = c.table.clone()
    c.table[2, 1] = c.blocks + 5
    assert call(rows=(2,)) == oda.ERR_BOUNDS
    K, V = c.kv(0, 2, 48)
    s = list(range(1, 17)) + list(range(33, 49))
    want, _ = O.attend(q[2], K, V, s)
    assert np.abs(out[2].double().cpu().numpy() - want).max() < 2e-2
    c.table.copy_(keep)
    assert call() == 0
    check_rows(c, q, out, lse, range(4), t)


def test_refusals(torch):
    oda = pytest.importorskip("gated_local_full_b200.oda")
    c = Case(torch, layers=2, rows=2, columns=2)
    L, h = oda.lib(), c.ctx.handle
    p = c.codes.data_ptr()
    odd = p + 8
    s = torch.cuda.current_stream().cuda_stream

    def append(fmt=1, lb=0, le=2, k=p, v=p, ts=None, n=2, sl=p, bt=p, co=p, sc=p, ring=None, B=2):
        return L.oda_append_kv8(h, fmt, lb, le, k, v, ts, n, sl, bt, co, sc, ring, B, s)

    def read(fmt=1, lb=0, le=2, ts=None, n=2, sl=p, bt=p, co=p, sc=p, k=p, v=p, B=2):
        return L.oda_read_kv8(h, fmt, lb, le, ts, n, sl, bt, co, sc, k, v, B, s)

    def full(fmt=1, layer=0, q=p, sl=p, bt=p, co=p, sc=p, idx=p, cnt=p, out=p, B=2, flags=0):
        return L.oda_full_attn_kv8(h, fmt, layer, q, sl, bt, co, sc, idx, cnt, out, None, B, flags, s)

    for f in (append, read):
        assert f(fmt=0) == oda.ERR_DTYPE and f(fmt=3) == oda.ERR_DTYPE
        assert f(lb=-1) == oda.ERR_ARG and f(le=3) == oda.ERR_ARG and f(lb=2, le=1) == oda.ERR_ARG
        assert f(B=3, n=3) == oda.ERR_SHAPE and f(B=-1, n=-1) == oda.ERR_ARG
        assert f(n=3) == oda.ERR_ARG and f(ts=p, n=-1) == oda.ERR_ARG
        assert f(ts=p, n=2 ** 31) == oda.ERR_SHAPE
        for a in ("sl", "bt", "co", "sc"):
            assert f(**{a: None}) == oda.ERR_ARG, a
        assert f(co=odd) == oda.ERR_ARG and f(sc=p + 4) == oda.ERR_ARG and f(k=odd) == oda.ERR_ARG
        assert f(B=0, n=0) == oda.OK and f(lb=1, le=1) == oda.OK and f(ts=p, n=0) == oda.OK
    assert append(k=None) == oda.ERR_ARG and append(ring=odd) == oda.ERR_ARG
    assert read(k=None, v=None) == oda.OK
    assert full(fmt=7) == oda.ERR_DTYPE and full(layer=2) == oda.ERR_ARG and full(layer=-1) == oda.ERR_ARG
    assert full(flags=2) == oda.ERR_ARG and full(B=3) == oda.ERR_SHAPE and full(B=0) == oda.OK
    for a in ("q", "sl", "bt", "co", "sc", "idx", "cnt", "out"):
        assert full(**{a: None}) == oda.ERR_ARG, a
    for a in ("q", "co", "out"):
        assert full(**{a: odd}) == oda.ERR_ARG, a
    assert L.oda_range_attn_kv8(h, 1, 0, p, p, None, p, p, p, p, p, p, p, None, 2, 0, s) == oda.ERR_ARG

    def rope(q=p, qs=512, k=p, ks=256, w=None, eps=1e-6, f=p, rot=128, pos=p, n=2, qo=p, qos=512, ko=p,
             kos=256, flags=0):
        return L.oda_qk_norm_rope(h, q, qs, k, ks, w, w, eps, f, rot, pos, 0, n, qo, qos, ko, kos, flags, s)

    assert rope(eps=-1.0) == oda.ERR_ARG and rope(eps=float("nan")) == oda.ERR_ARG
    for r in (-16, 8, 24, 144):
        assert rope(rot=r) == oda.ERR_SHAPE, r
    assert rope(qs=511) == oda.ERR_SHAPE and rope(qs=516) == oda.ERR_SHAPE and rope(kos=200) == oda.ERR_SHAPE
    assert rope(q=None) == oda.ERR_ARG and rope(qo=None) == oda.ERR_ARG and rope(pos=None) == oda.ERR_ARG
    assert rope(f=None) == oda.ERR_ARG and rope(ko=None) == oda.ERR_ARG and rope(k=None) == oda.ERR_ARG
    assert rope(q=odd) == oda.ERR_ARG and rope(w=odd) == oda.ERR_ARG and rope(flags=2) == oda.ERR_ARG
    assert rope(n=-1) == oda.ERR_ARG and rope(n=2 ** 31) == oda.ERR_SHAPE and rope(n=0) == oda.OK
    torch.cuda.synchronize()
    assert c.ctx.get_device_error() == 0


# ------------------------------------------------------------------ norm, rotation

def rope_bound(x, w, eps, pos, f, neighbours, dtype):
    """The norm's sum takes d roundings, its root halves them, rsqrt and the two
    products add 4 steps: (d / 2 + 6) 2^-24 relative. The fraction of a turn is
    within 2^-25 turns (2 pi 2^-25 < 2^-22 in the angle) and what float64 loses of the
    turns; sine and cosine are within 2^-22: 2^-21 of |a| + |b|, and 3 roundings."""
    d = x.shape[-1]
    y = np.abs(O.norm_rotate(x, w, eps, pos, None))
    size = y.copy()
    far = 0.0
    if f is not None:
        half = len(f)
        i = np.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
        size[..., ia] = size[..., ib] = y[..., ia] + y[..., ib]
        far = 2.0 ** -50 * np.abs(np.asarray(pos, np.float64)).max()
    ref = np.abs(O.norm_rotate(x, w, eps, pos, f, neighbours))
    return size * ((d / 2 + 10) * U32 + 2.0 ** -21 + far) + HALF[dtype] * ref + 1e-30


ROPE = [
    dict(dtype="bf16", d=128, rot=128), dict(dtype="bf16", d=128, rot=80, neighbours=True),
    dict(dtype="bf16", d=64, rot=64, hq=3, hkv=3), dict(dtype="f32", d=64, rot=32, neighbours=True),
    dict(dtype="f32", d=128, rot=128, hq=8), dict(dtype="f32", d=128, rot=48), dict(dtype="bf16", d=64, rot=16),
    dict(dtype="bf16", d=128, rot=0), dict(dtype="f32", d=64, rot=64, neighbours=True),
]


@pytest.mark.parametrize("kw", ROPE, ids=lambda k: "-".join(map(str, k.values())))
@pytest.mark.parametrize("n", [1, 2, 7, 130])
def test_norm_and_rotation(torch, kw, n):
    kw = dict(kw)
    rot, nb = kw.pop("rot"), kw.pop("neighbours", False)
    c = Case(torch, rows=2, columns=2, seed=n, **kw)
    f = (10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))).astype(np.float32) if rot else None
    pos = c.r.integers(0, 1 << 20, n)
    pos[0], pos[-1] = 0, (1 << 31) - 5
    fd = torch.from_numpy(f).cuda() if rot else None
    pd = c.ints(pos) if rot else None
    (q, _), (k, _) = c.values(n, c.hq, c.d, scale=3.0), c.values(n, c.hkv, c.d)
    q[0, 0] = 0.0                                        # a head of zeros
    (qw, qwd), (kw_, kwd) = c.values(c.d), c.values(c.d)
    # the heads inside a wider row, V behind them; outputs with a stride of their own
    fused = torch.zeros((n, c.hq + 2 * c.hkv, c.d), dtype=c.kind, device="cuda")
    fused[:, :c.hq] = torch.from_numpy(q)
    fused[:, c.hq:c.hq + c.hkv] = torch.from_numpy(k)
    qv, kv = fused[:, :c.hq], fused[:, c.hq:c.hq + c.hkv]
    wide = torch.full((n, c.hq + c.hkv + 1, c.d), 7.0, dtype=c.kind, device="cuda")
    qo, ko = wide[:, :c.hq], wide[:, c.hq:c.hq + c.hkv]
    for weights in ((qw, kw_), (None, kw_), (None, None)):
        wd = [None if w is None else x for w, x in zip(weights, (qwd, kwd))]
        c.ctx.qk_norm_rope(qv, kv, wd[0], wd[1], 1e-5, fd, pd, qo, ko, interleaved=nb)
        for x, w, o in ((q, weights[0], qo), (k, weights[1], ko)):
            want = O.norm_rotate(x, w, 1e-5, pos, f, nb)
            err = np.abs(o.double().cpu().numpy() - want)
            assert np.all(err <= rope_bound(x, w, 1e-5, pos, f, nb, c.dtype))
        assert (wide[:, -1] == 7).all()
    # in place, positions shifted, queries alone
    want = O.norm_rotate(q, qw, 1e-5, pos - 1, f, nb)
    c.ctx.qk_norm_rope(qv, None, qwd, None, 1e-5, fd, pd, qv, None, pos_offset=-1, interleaved=nb)
    err = np.abs(qv.double().cpu().numpy() - want)
    assert np.all(err <= rope_bound(q, qw, 1e-5, pos - 1, f, nb, c.dtype))
    assert torch.equal(kv.double().cpu(), torch.from_numpy(k))
    assert c.ctx.get_device_error() == 0


# --------------------------------------------------------------- used together

def steps(c, torch, out, lse, q, k, v, pos, at, f, w, buf):
    """One decode step: norm and rotation, the write, attention over everything."""
    qr, kr = buf
    c.ctx.qk_norm_rope(q, k, w, w, 1e-6, f, pos, qr, kr, pos_offset=-1)
    c.ctx.append_kv8(c.fmt, 0, 1, kr[None], v[None], pos, c.table, c.codes, c.scales, c.ring, c.rows)
    idx, count = at
    c.ctx.full_attn_kv8(c.fmt, 0, qr, pos, c.table, c.codes, c.scales, idx, count, out, lse, c.rows)


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("how", ["plain", "stream", "graph"])
def test_decode_loop(torch, fmt, dtype, how):
    """Twenty steps from a prefilled cache: plain calls, calls on another stream,
    and one captured graph replayed with new inputs in the same buffers."""
    c = Case(torch, fmt=fmt, dtype=dtype, rows=3, columns=6, sink=2, window=16)
    t = c.write([30, 1, 47], [0] * 3)
    f = torch.from_numpy((10000.0 ** (-np.arange(64) / 64.0)).astype(np.float32)).cuda()
    _, w = c.values(c.d)
    q, k, v = (torch.zeros((3, h, c.d), dtype=c.kind, device="cuda") for h in (c.hq, c.hkv, c.hkv))
    pos = c.ints([0, 0, 0])
    out, lse = torch.zeros((3, c.hq, c.d), dtype=c.kind, device="cuda"), torch.zeros((3, c.hq), device="cuda")
    buf = torch.zeros_like(q), torch.zeros_like(k)
    at = listed(c, [0, 2, 1], 3)
    stream = torch.cuda.Stream() if how != "plain" else torch.cuda.current_stream()
    graph = None
    torch.cuda.synchronize()
    if how == "graph":
        pos.copy_(c.ints([x + 1 for x in t]))
        saved = c.codes.clone(), c.scales.clone(), c.ring.clone()
        with torch.cuda.stream(stream):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                steps(c, torch, out, lse, q, k, v, pos, at, f, w, buf)
        torch.cuda.synchronize()
        for a, b in zip((c.codes, c.scales, c.ring), saved):
            assert torch.equal(a, b)                       # capturing ran nothing
    for step in range(20):
        t = [x + 1 for x in t]
        with torch.cuda.stream(stream):
            for x in (q, k, v):
                x.copy_(c.values(*x.shape)[1])
            pos.copy_(c.ints(t))
            if graph is not None:
                graph.replay()
            else:
                steps(c, torch, out, lse, q, k, v, pos, at, f, w, buf)
        torch.cuda.synchronize()
        kr = buf[1].double().cpu().numpy()                 # what the cache was given
        want = O.norm_rotate(k.double().cpu().numpy(), w.double().cpu().numpy(), 1e-6,
                             np.array(t) - 1, f.double().cpu().numpy())
        assert np.all(np.abs(kr - want) <= rope_bound(k.double().cpu().numpy(), w.double().cpu().numpy(), 1e-6,
                                                      np.array(t) - 1, f.double().cpu().numpy(), False, c.dtype))
        c.oracle_write(kr[None], v.double().cpu().numpy()[None], [1] * 3, [x - 1 for x in t])
        c.check()
        check_rows(c, buf[0].double().cpu().numpy(), out, lse, range(3), t)


def test_a_long_cache_past_32_bits(torch):
    """Blocks whose codes lie behind 4 GB of one layer, in the second layer."""
    c = Case(torch, fmt="e4m3", hq=2, hkv=1, d=128, layers=2, rows=1, columns=3, num_blocks=(1 << 20) + 300)
    c.scales = torch.zeros((2, c.blocks, 1, 2), device="cuda")
    (k, kd), (v, vd) = (c.values(1, 40, 1, 128) for _ in "kv")
    c.ctx.append_kv8("e4m3", 1, 2, kd, vd, c.ints([40]), c.table, c.codes, c.scales, None, 1,
                     tok_start=c.ints([0, 40]))
    codes, scales = np.zeros((3, 2, 16, 128), np.uint8), np.zeros((3, 2), np.float32)
    for j in range(3):
        for kv, x in enumerate((k, v)):
            scales[j, kv] = O.kv8_write_block(codes[j, kv], 0.0, 0, x[0, 16 * j:min(40, 16 * j + 16), 0], "e4m3")
    where = torch.from_numpy(c.table_h[0].astype(np.int64)).cuda()
    got = c.codes[1, where, 0].cpu().numpy()
    assert np.array_equal(got[:2], codes[:2]) and np.array_equal(got[2, :, :8], codes[2, :, :8])
    assert np.array_equal(c.scales[1, where, 0].cpu().numpy(), scales)
    q, qd = c.values(1, 2, 128)
    out, lse = torch.zeros((1, 2, 128), dtype=c.kind, device="cuda"), torch.zeros((1, 2), device="cuda")
    idx, count = listed(c, [0], 1)
    c.ctx.full_attn_kv8("e4m3", 1, qd, c.ints([40]), c.table, c.codes, c.scales, idx, count, out, lse, 1)
    assert c.ctx.get_device_error() == 0
    K, V = ((O.kv8_value(codes[:, kv], "e4m3") * scales[:, kv, None, None].astype(np.float64)).reshape(1, 48, 128)[:, :40]
            for kv in (0, 1))
    want, wl = O.full_attention(q[0], K, V, 40)
    assert np.all(np.abs(out[0].double().cpu().numpy() - want) <= attn_bound(q[0], K, V, 1, 41, "bf16"))
    back = torch.zeros((1, 40, 1, 128), dtype=c.kind, device="cuda")
    c.ctx.read_kv8("e4m3", 1, 2, c.ints([40]), c.table, c.codes, c.scales, None, back, 1, tok_start=c.ints([0, 40]))
    assert torch.equal(back[0, :, 0].cpu(), torch.from_numpy(V[0]).float().to(c.kind))


def test_long_rows_and_many_rows(torch):
    """A row long enough to be split over the whole grid beside short ones, and
    more rows than the grid has CTAs; the result does not depend on the split."""
    c = Case(torch, fmt="int8", hq=2, hkv=1, d=128, rows=2, columns=1260, window=32)
    t = [20137, 3]
    c.write(t, [0, 0], ring=False)
    q, qd = c.values(2, 2, 128, scale=2.0)
    out, lse = torch.zeros((2, 2, 128), dtype=c.kind, device="cuda"), torch.zeros((2, 2), device="cuda")
    idx, count = listed(c, [1, 0], 2)
    c.ctx.full_attn_kv8("int8", 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 2)
    check_rows(c, q, out, lse, [0, 1], t)
    many = Case(torch, fmt="e4m3", hq=4, hkv=4, d=64, rows=400, columns=3, seed=3)
    t = [int(x) for x in many.r.integers(1, 49, 400)]
    many.write(t, [0] * 400, ring=False)
    q, qd = many.values(400, 4, 64)
    out, lse = torch.zeros((400, 4, 64), dtype=many.kind, device="cuda"), torch.zeros((400, 4), device="cuda")
    idx, count = listed(many, range(400), 400)
    many.ctx.full_attn_kv8("e4m3", 0, qd, many.ints(t), many.table, many.codes, many.scales, idx, count,
                           out, lse, 400)
    assert many.ctx.get_device_error() == 0
    check_rows(many, q, out, lse, range(0, 400, 7), t)


# ------------------------------------------------- calls beside each other, repeated

def same_everywhere(torch, c, t, **more):
    """Buffers and a call of the rows of `t` in any order; returns (call, out, lse)."""
    q, qd = c.values(len(t), c.hq, c.d, scale=2.0)
    out = torch.zeros((len(t), c.hq, c.d), dtype=c.kind, device="cuda")
    lse = torch.zeros((len(t), c.hq), device="cuda")
    idx, count = listed(c, range(len(t)), len(t))
    td = c.ints(t)
    ctx = more.get("ctx", c.ctx)

    def call():
        ctx.full_attn_kv8(c.fmt, 0, qd, td, c.table, c.codes, c.scales, idx, count, out, lse, len(t))
    return call, out, lse, q


@pytest.mark.parametrize("hq,hkv,d,dtype,fmt", [(4, 1, 128, "bf16", "int8"), (4, 2, 128, "f32", "e4m3"),
                                                (4, 1, 64, "bf16", "e4m3"), (2, 2, 128, "bf16", "e4m3")])
def test_a_context_for_large_batches(torch, hq, hkv, d, dtype, fmt):
    """A batch of three in a context for 1024 rows, whose row arrays leave room for fewer stages."""
    c = Case(torch, fmt=fmt, dtype=dtype, hq=hq, hkv=hkv, d=d, rows=3, columns=70)
    t = [1111, 1, 640]
    c.write(t, [0] * 3, ring=False)
    big = c.oda.OdaContext(c.oda.make_config(layers=1, max_batch=1024, hq=hq, hkv=hkv, head_dim=d, sink=4,
                                             window=32, dtype=dtype, max_blocks_per_seq=70,
                                             num_blocks=c.blocks))
    call, out, lse, q = same_everywhere(torch, c, t, ctx=big)
    call()
    assert big.get_device_error() == 0
    check_rows(c, q, out, lse, range(3), t)


@pytest.mark.parametrize("fmt,dtype,hq,hkv", [("int8", "bf16", 8, 2), ("e4m3", "f32", 2, 1)])
def test_equal_calls_give_equal_bits(torch, fmt, dtype, hq, hkv):
    """Plain, behind other work, from two graphs that share the context's scratch, and while
    another context works on another stream."""
    c = Case(torch, fmt=fmt, dtype=dtype, hq=hq, hkv=hkv, rows=4, columns=320)
    t = [5003, 17, 2048, 901]
    c.write(t, [0] * 4, ring=False)
    call, out, lse, q = same_everywhere(torch, c, t)
    call()
    check_rows(c, q, out, lse, range(4), t)
    want = out.clone(), lse.clone()
    other = Case(torch, fmt=fmt, dtype=dtype, hq=hq, hkv=hkv, rows=2, columns=200, seed=5)
    t2 = [3001, 3200]
    other.write(t2, [0, 0], ring=False)
    call2, out2, lse2, _ = same_everywhere(torch, other, t2)
    call2()
    torch.cuda.synchronize()
    want2 = out2.clone(), lse2.clone()
    side = torch.cuda.Stream()
    for _ in range(20):
        out.zero_()
        out2.zero_()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            call()
            with torch.cuda.stream(side):
                call2()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(out2, want2[0]) and torch.equal(lse2, want2[1])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            call()
            call()
        graphs.append(g)
    for _ in range(5):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for g in graphs + graphs[::-1]:
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert c.ctx.get_device_error() == 0 and other.ctx.get_device_error() == 0


def test_a_row_listed_twice_and_shared_blocks(torch):
    """A row twice in the list, and two rows over the same physical blocks (a shared prefix)."""
    c = Case(torch, fmt="int8", hq=4, hkv=2, rows=3, columns=40)
    t = [600, 600, 33]
    c.write(t, [0] * 3, ring=False)
    c.table[1] = c.table[0]
    c.table_h[1] = c.table_h[0]
    q, qd = c.values(3, c.hq, c.d)
    qd[1] = qd[0]
    q[1] = q[0]
    out, lse = torch.zeros((3, c.hq, c.d), dtype=c.kind, device="cuda"), torch.zeros((3, c.hq), device="cuda")
    idx, count = listed(c, [0, 2, 0], 3)
    c.ctx.full_attn_kv8("int8", 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 3)
    assert c.ctx.get_device_error() == 0
    check_rows(c, q, out, lse, [0, 2], t)
    idx, count = listed(c, [1, 0], 3)
    c.ctx.full_attn_kv8("int8", 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 3)
    check_rows(c, q, out, lse, [0, 1], t)


def test_lists_that_change_between_calls(torch):
    """Lengths, rows and the block table written by the launch just before, in the same stream:
    what was worked out ahead of the wait must not be used."""
    c = Case(torch, fmt="int8", hq=4, hkv=2, rows=4, columns=60)
    c.write([900, 900, 900, 900], [0] * 4, ring=False)
    q, qd = c.values(4, c.hq, c.d)
    out, lse = torch.zeros((4, c.hq, c.d), dtype=c.kind, device="cuda"), torch.zeros((4, c.hq), device="cuda")
    td, (idx, count) = c.ints([900] * 4), listed(c, range(4), 4)
    table = c.table.clone()
    lists = []
    for _ in range(12):
        n = int(c.r.integers(1, 5))
        rows = [int(x) for x in c.r.permutation(4)[:n]]
        t = [int(x) for x in c.r.integers(1, 901, 4)]
        perm = c.r.permutation(4)
        lists.append((rows, t, perm, c.ints(t), *listed(c, rows, 4), c.table[torch.from_numpy(perm).cuda()].contiguous()))
    got = []
    for rows, t, perm, t2, i2, n2, tab in lists:               # no wait in between
        td.copy_(t2)
        idx.copy_(i2)
        count.copy_(n2)
        table.copy_(tab)
        c.ctx.full_attn_kv8("int8", 0, qd, td, table, c.codes, c.scales, idx, count, out, lse, 4)
        got.append((out.clone(), lse.clone()))
    keep = c.table_h.copy()
    for (rows, t, perm, *_), (o, l) in zip(lists, got):
        c.table_h = keep[perm]
        check_rows(c, q, o, l, rows, t)
    assert c.ctx.get_device_error() == 0


def test_refusals_of_the_compiled_calls(torch):
    """What the binding itself refuses, and what it hands on: nothing is launched."""
    c = Case(torch, rows=2, columns=2)
    oda = c.oda
    t, idx = c.ints([3, 4]), listed(c, [0, 1], 2)
    (_, kd), (_, vd) = c.values(1, 2, c.hkv, c.d), c.values(1, 2, c.hkv, c.d)
    _, qd = c.values(2, c.hq, c.d)
    out = torch.zeros_like(qd)

    def append(format="int8", k=kd, v=vd, sl=t, B=2, stream=None):
        c.ctx.append_kv8(format, 0, 1, k, v, sl, c.table, c.codes, c.scales, None, B, stream=stream)

    def attn(ctx=c.ctx, format="int8", q=qd, table=c.table, out=out, stream=None):
        ctx.full_attn_kv8(format, 0, q, t, table, c.codes, c.scales, *idx, out, None, 2, stream=stream)

    for f in (append, attn):
        for name in ("int3", 0, 9):
            with pytest.raises(oda.OdaError) as e:
                f(format=name)
            assert e.value.status == oda.ERR_DTYPE
        with pytest.raises(TypeError):
            f(format=None)
        with pytest.raises((AttributeError, TypeError, ValueError)):
            f(stream="s")
    with pytest.raises(ValueError, match="tensor"):
        append(k=[1.0])
    with pytest.raises(ValueError, match="tensor"):
        append(k=None)
    with pytest.raises(ValueError, match="contiguous"):
        append(k=kd.expand(1, 2, c.hkv, c.d).transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="GPU"):
        append(sl=t.cpu())
    with pytest.raises(ValueError, match="contiguous"):
        attn(table=c.table.t())
    with pytest.raises(oda.OdaError) as e:
        attn(q=None)
    assert e.value.status == oda.ERR_ARG
    with pytest.raises(TypeError):
        append(B="two")
    gone = oda.OdaContext(c.cfg)
    attn(ctx=gone)
    torch.cuda.synchronize()
    gone.close()
    with pytest.raises(oda.OdaError) as e:
        attn(ctx=gone)
    assert e.value.status == oda.ERR_ARG
    # addresses in tensors' place, and streams as objects and numbers
    s = torch.cuda.Stream()
    for x in (s, s.cuda_stream, None):
        c.ctx.full_attn_kv8(oda.KV8_INT8, 0, qd.data_ptr(), t.data_ptr(), c.table, c.codes, c.scales, *idx,
                            out.data_ptr(), 0, 2, stream=x)
    torch.cuda.synchronize()
    assert c.ctx.get_device_error() == 0


@pytest.mark.parametrize("fmt,dtype,hq,hkv,d", [("int8", "bf16", 4, 2, 128), ("e4m3", "bf16", 4, 1, 128),
                                                ("int8", "f32", 4, 1, 64), ("e4m3", "f32", 2, 2, 128)])
def test_inputs_ready(torch, fmt, dtype, hq, hkv, d):
    """The first tiles staged before the dependency wait: the same bits, with new queries written
    by the launch just before, for rows of all lengths, regions, and no rows."""
    c = Case(torch, fmt=fmt, dtype=dtype, hq=hq, hkv=hkv, d=d, rows=5, columns=130)
    t = [2077, 1, 16, 515, 1300]
    c.write(t, [0] * 5, ring=False)
    lo, hi = [3, 1, 2, 200, 1000], [2078, 2, 17, 201, 1299]
    qs = [c.values(5, hq, d, scale=2.0) for _ in range(4)]
    qd = torch.zeros_like(qs[0][1])
    td, ld, hd = c.ints(t), c.ints(lo), c.ints(hi)

    def run(ready, region, rows):
        idx, count = listed(c, rows, 5)
        got = []
        torch.cuda.synchronize()
        for _, q in qs:
            out = torch.full_like(qd, 7.0)
            lse = torch.full((5, hq), 7.0, device="cuda")
            qd.copy_(q)
            if region:
                c.ctx.range_attn_kv8(fmt, 0, qd, td, ld, hd, c.table, c.codes, c.scales, idx, count, out, lse,
                                     5, inputs_ready=ready)
            else:
                c.ctx.full_attn_kv8(fmt, 0, qd, td, c.table, c.codes, c.scales, idx, count, out, lse, 5,
                                    inputs_ready=ready)
            got.append((out, lse))
        torch.cuda.synchronize()
        assert c.ctx.get_device_error() == 0
        return got

    for region in (False, True):
        for rows in ([0, 1, 2, 3, 4], [4, 1], [2], []):
            plain, early = run(False, region, rows), run(True, region, rows)
            for (o, l), (o2, l2) in zip(plain, early):
                assert torch.equal(o, o2) and torch.equal(l, l2)
            for (q, _), (o, l) in zip(qs, early):
                check_rows(c, q, o, l, rows, t, *((lo, hi) if region else ()))


# ------------------------------------------------- lists written late by the launch before

@pytest.fixture(scope="module")
def late_store(tmp_path_factory):
    """late_store(dst, src): a launch that releases the next one before it stores dst."""
    import ctypes
    import os
    import subprocess

    from gated_local_full_b200 import build
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "late_store.cu")
    lib = str(tmp_path_factory.mktemp("late") / "late_store.so")
    r = subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", src,
                        "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    f = ctypes.CDLL(lib).late_store
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p]

    def store(dst, new):
        import torch
        assert dst.numel() == new.numel() and dst.dtype == new.dtype == torch.int32
        assert f(dst.data_ptr(), new.data_ptr(), new.numel(), 60000,
                 torch.cuda.current_stream().cuda_stream) == 0
    return store


@pytest.mark.parametrize("late,region", [(k, False) for k in ("t", "idx", "count", "table")] +
                         [(k, True) for k in ("t", "idx", "count", "lo", "hi", "table")])
@pytest.mark.parametrize("B,columns", [(5, 130), (40, 13)])
def test_a_list_written_late_by_the_launch_before(torch, late_store, late, region, B, columns):
    """The launch before lets the attention start, and only then stores one of the lists: lengths
    that a region's end outgrows or that are refused as they were, ids and blocks out of range, counts
    of none and of too many, bounds of nothing. What was worked out from the old list must not be used, and
    the call after it, with nothing changed, gives the same bits (no ticket is left over)."""
    c = Case(torch, fmt="int8", hq=4, hkv=2, rows=B, columns=columns)
    full_t = [min(16 * columns, x) for x in ([2077, 900, 16, 515, 1300] * 8)[:B]]
    c.write(full_t, [0] * B, ring=False)
    q, qd = c.values(B, c.hq, c.d)
    held = {k: c.ints([0] * (1 if k == "count" else B)) for k in ("t", "idx", "count", "lo", "hi")}
    held["table"] = c.table.flatten()
    blocks = c.table_h.reshape(-1).tolist()
    for step in range(10):
        t = [int(c.r.integers(x // 2 + 1, x + 1)) for x in full_t]
        rows = [int(x) for x in c.r.permutation(B)[:1 + step % 5 * (B // 5)]]
        hi = [x + 1 for x in t]                            # regions that end at the row's last position
        lo = [int(c.r.integers(1, h)) for h in hi]
        new = dict(t=t, idx=rows + [-1] * (B - len(rows)), count=[len(rows)], lo=lo, hi=hi, table=blocks)
        old = dict(t=[[1] * B, [x - 1 for x in t], [0] * B, [x // 3 + 1 for x in t], [2 ** 31 - 1] * B],
                   idx=[[-1] * B, list(range(B))[::-1], [B + 2] * B, [0] * B, [2 ** 31 - 1] * B],
                   count=[[0], [B], [B + 4], [-3], [1]],
                   lo=[[0] * B, [x + 1 for x in t], [1] * B, [-5] * B, [x // 2 for x in hi]],
                   hi=[[0] * B, [x + 1 for x in lo], [x + 2 for x in t], [-2 ** 31] * B, [x // 2 + 1 for x in hi]],
                   table=[blocks[::-1], [-1] * len(blocks), [c.blocks] * len(blocks), [0] * len(blocks),
                          blocks[columns:] + blocks[:columns]])
        before = old[late][step % 5]
        device = {k: c.ints(v) for k, v in new.items()}
        for k in held:
            held[k].copy_(c.ints(before) if k == late else device[k])
        out = torch.full((B, c.hq, c.d), 7.0, dtype=c.kind, device="cuda")
        lse = torch.full((B, c.hq), 7.0, device="cuda")
        again, lse2 = out.clone(), lse.clone()
        torch.cuda.synchronize()
        late_store(held[late], device[late])
        for o, l in ((out, lse), (again, lse2)):
            table = held["table"].view(B, columns)
            if region:
                c.ctx.range_attn_kv8(c.fmt, 0, qd, held["t"], held["lo"], held["hi"], table, c.codes, c.scales,
                                     held["idx"], held["count"], o, l, B)
            else:
                c.ctx.full_attn_kv8(c.fmt, 0, qd, held["t"], table, c.codes, c.scales, held["idx"],
                                    held["count"], o, l, B)
        assert c.ctx.get_device_error() == 0, step
        check_rows(c, q, out, lse, rows, t, *((lo, hi) if region else ()))
        assert torch.equal(out, again) and torch.equal(lse, lse2), (step, before)
        rest = [b for b in range(B) if b not in rows]
        assert (out[rest] == 7).all()


# ------------------------------------------------------- stretches that are not in order

@pytest.mark.parametrize("starts,first", [
    ([0, 48, 16, 64], 1),                         # rows 1 and 2 would start at the same item
    ([0, 40, 20, 64], 1), ([0, 0, 64, 10, 64], 2), ([64, 0, 64], 0), ([0, 16, 65], 1), ([0, 65, 64], 0),
    ([0, 20, -1, 64], 1), ([-64, 20, 64], 0), ([80, 90, 90], 0), ([0, -2 ** 31, 2 ** 31 - 1, 64], 0),
    (list(range(0, 37)) + [35, 64, 64], 36),      # behind the first 32 rows
    ([0] * 33 + [64, 63] + [64] * 5, 33), ([0] * 39 + [65], 38), ([0] * 64 + [-3], 63),
])
def test_token_starts_out_of_order(torch, starts, first):
    """Rows before the first spoilt stretch are written and read, that one and those behind are
    not, and the error is raised however far behind it lies."""
    oda = pytest.importorskip("gated_local_full_b200.oda")
    B = len(starts) - 1
    c = Case(torch, dtype="f32", hq=1, hkv=1, d=64, rows=B, columns=5, sink=2, window=12)
    (k, kd), (v, vd) = (c.values(1, 64, 1, 64) for _ in "kv")
    n = [starts[b + 1] - starts[b] for b in range(first)]
    past = [int(x) for x in c.r.integers(0, 14, B)]
    t = [p + m for p, m in zip(past, n)] + [64] * (B - first)
    c.ctx.append_kv8("int8", 0, 1, kd, vd, c.ints(t), c.table, c.codes, c.scales, c.ring, B,
                     tok_start=c.ints(starts))
    assert c.ctx.get_device_error() == oda.ERR_BOUNDS
    if first:
        assert starts[0] == 0
        c.oracle_write(k, v, n, past[:first])
    c.check()
    out = torch.full((1, 64, 1, 64), 9.0, device="cuda")
    c.ctx.read_kv8("int8", 0, 1, c.ints(t), c.table, c.codes, c.scales, out, None, B, tok_start=c.ints(starts))
    assert c.ctx.get_device_error() == oda.ERR_BOUNDS
    got = out[0, :, 0].cpu().numpy()
    for b in range(first):
        want = c.kv(0, b, t[b])[0][0, t[b] - n[b]:].astype(np.float32)
        assert np.array_equal(got[starts[b]:starts[b + 1]], want), b
    assert np.all(got[starts[first] if first else 0:] == 9)


# ------------------------------------------------------------ what is held in fewer bits

def held_bound(q, K, V, fmt, dtype, scales):
    """attn_bound, and what the forms of queries and weights lose below their range: a query element is
    held to 2^-22 of itself (counted there) or to 2^-36 (int8: 2^-30) of its head's largest, which
    moves a score by D = 2^-36 max|q| sum|k| / sqrt(d) and weights by a factor within exp(2 D); a weight
    times its block's scale to 2^-22 of itself (counted there) or to 2^-47 of the row's largest."""
    d, n = q.shape[1], K.shape[1]
    group = q.shape[0] // K.shape[0]
    more = []
    for h in range(q.shape[0]):
        k, v = K[h // group], V[h // group]
        s = k @ q[h] / np.sqrt(d)
        p = np.exp(s - s.max())
        p /= p.sum()
        D = (2.0 ** -30 if fmt == "int8" else 2.0 ** -36) * np.abs(q[h]).max() * np.abs(k).sum(1).max() / np.sqrt(d)
        if dtype == "bf16" and np.abs(q[h]).max() <= 2.0 ** 22 * np.abs(q[h])[q[h] != 0].min():
            D = 0.0                                          # bf16 has 8 bits: held whole
        scale = scales[h // group].repeat(16)[:n]
        codes = np.abs(v) / np.where(scale > 0, scale, 1.0)[:, None]
        more.append(2 * np.expm1(2 * D) * (p @ np.abs(v)) + 2.0 ** -47 * (p * scale).max() * codes.sum(0))
    return attn_bound(q, K, V, 1, n + 1, dtype) + np.array(more)


def v_scales(c, b, t):
    return c.scales_h[0, c.table_h[b, :(t + 15) // 16], :, 1].astype(np.float64).T


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_block_with_one_large_dim(torch, fmt, dtype):
    """A block whose V is far above the others' in one dim and zero in the rest, early, late and in the
    middle of the rows: the other dims are those of the other blocks' tokens."""
    up = [0, 12, 24, 40]
    t = [700, 650, 300, 200]
    c = Case(torch, fmt=fmt, dtype=dtype, hq=2, hkv=1, d=64, rows=4, columns=44)
    (k, kd), (v, _) = (c.values(1, sum(t), 1, 64) for _ in "kv")
    at = c.starts(t)
    for b, e in enumerate(up):
        for block in (1, 3, (t[b] // 16) // 2, t[b] // 16 - 1):
            s = slice(at[b] + 16 * block, at[b] + 16 * block + 16)
            v[:, s, :, 1:] = 0.0
            v[:, s, :, 0] = (2.0 ** e) * (1 + (v[:, s, :, 0] > 0))
    c.ctx.append_kv8(fmt, 0, 1, kd, torch.from_numpy(v).to(c.kind).cuda(), c.ints(t), c.table, c.codes, c.scales,
                     None, 4, tok_start=c.ints(at))
    c.oracle_write(k, v, t, [0] * 4, ring=False)
    c.check()
    q, qd = c.values(4, 2, 64)
    out, lse = torch.zeros((4, 2, 64), dtype=c.kind, device="cuda"), torch.zeros((4, 2), device="cuda")
    idx, count = listed(c, range(4), 4)
    c.ctx.full_attn_kv8(fmt, 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 4)
    assert c.ctx.get_device_error() == 0
    got = out.double().cpu().numpy()
    for b in range(4):
        K, V = c.kv(0, b, t[b])
        want, _ = O.full_attention(q[b], K, V, t[b])
        err, bound = np.abs(got[b] - want), held_bound(q[b], K, V, fmt, dtype, v_scales(c, b, t[b]))
        assert np.all(err <= bound), (b, (err / bound).max())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_query_with_one_large_element(torch, fmt, dtype):
    """A query element 2^12 to 2^26 above the others, where the keys are zero: the scores are the others'."""
    up = [12, 18, 21, 26]
    t = [90, 200, 33, 400]
    c = Case(torch, fmt=fmt, dtype=dtype, hq=2, hkv=1, d=64, rows=4, columns=25)
    (k, _), (v, vd) = (c.values(1, sum(t), 1, 64) for _ in "kv")
    k[..., 7] = 0.0
    c.ctx.append_kv8(fmt, 0, 1, torch.from_numpy(k).to(c.kind).cuda(), vd, c.ints(t), c.table, c.codes, c.scales,
                     None, 4, tok_start=c.ints(c.starts(t)))
    c.oracle_write(k, v, t, [0] * 4, ring=False)
    q, _ = c.values(4, 2, 64)
    q = np.where(np.abs(q) < 0.5, np.where(q < 0, -0.5, 0.5), q)   # no element far below the others
    for b, e in enumerate(up):
        q[b, :, 7] = 2.0 ** e
    qd = torch.from_numpy(q).to(c.kind).cuda()
    out, lse = torch.zeros((4, 2, 64), dtype=c.kind, device="cuda"), torch.zeros((4, 2), device="cuda")
    idx, count = listed(c, range(4), 4)
    c.ctx.full_attn_kv8(fmt, 0, qd, c.ints(t), c.table, c.codes, c.scales, idx, count, out, lse, 4)
    assert c.ctx.get_device_error() == 0
    got = out.double().cpu().numpy()
    for b in range(4):
        K, V = c.kv(0, b, t[b])
        want, _ = O.full_attention(q[b], K, V, t[b])
        err, bound = np.abs(got[b] - want), held_bound(q[b], K, V, fmt, dtype, v_scales(c, b, t[b]))
        assert np.all(err <= bound), (b, (err / bound).max())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("apart", [10, 30, 60, 90])
def test_small_values_far_below_the_largest_weight(torch, fmt, apart):
    """Tokens whose V is zero have the largest weights by 2^20; the others' V is 2^-(6 + apart) and less:
    the output is theirs alone, however small (no smaller than float32's normal numbers)."""
    t = 30 * 16
    c = Case(torch, fmt=fmt, dtype="f32", hq=2, hkv=1, d=64, rows=1, columns=30)
    (k, _), (v, _) = (c.values(1, t, 1, 64) for _ in "kv")
    high = np.zeros(t, bool)
    for block in (0, 7, 20):
        high[16 * block:16 * block + 16] = True
    q = np.zeros((1, 2, 64))
    q[0, :, 0] = 1.0
    k[0, :, 0, 0] = np.where(high, 20 * np.log(2) * 8, 0.0)      # a score of 20 ln 2 where high, else 0
    k = k.astype(np.float32).astype(np.float64)
    v = np.where(high[None, :, None, None], 0.0, v * 2.0 ** -apart / 64)
    v = v.astype(np.float32).astype(np.float64)
    kd, vd = torch.from_numpy(k).float().cuda(), torch.from_numpy(v).float().cuda()
    c.ctx.append_kv8(fmt, 0, 1, kd, vd, c.ints([t]), c.table, c.codes, c.scales, None, 1, tok_start=c.ints([0, t]))
    c.oracle_write(k, v, [t], [0], ring=False)
    c.check()
    out, lse = torch.zeros((1, 2, 64), device="cuda"), torch.zeros((1, 2), device="cuda")
    idx, count = listed(c, [0], 1)
    c.ctx.full_attn_kv8(fmt, 0, torch.from_numpy(q).float().cuda(), c.ints([t]), c.table, c.codes, c.scales, idx, count,
                        out, lse, 1)
    assert c.ctx.get_device_error() == 0
    K, V = c.kv(0, 0, t)
    want, _ = O.full_attention(q[0], K, V, t)
    # numbers relative to the values' size, so that no bound rests on a fixed smallest one
    unit = 2.0 ** -apart
    bound = held_bound(q[0], K, V / unit, fmt, "f32", v_scales(c, 0, t) / unit) * unit
    assert np.abs(want).max() > 2.0 ** -126
    err = np.abs(out[0].double().cpu().numpy() - want)
    assert np.all(err <= bound + 2.0 ** -148), (err / bound).max()


# ------------------------------------------------------- the gated step over the 8-bit cache

@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("how", ["plain", "graph"])
def test_local_gate_and_full_over_8_bits(torch, fmt, dtype, how):
    """A decode step as a server composes it: the write into cache and ring, Local from the ring (the
    model's type), the gate, Full over the 8-bit cache for the rows that the gate lists; from no row
    to all of them, with the context's scratch shared by Local and Full."""
    from tests._harness import BF16_ATOL, BF16_RTOL, F32_ATOL, F32_RTOL
    B, t = 4, [70, 17, 33, 200]
    c = Case(torch, fmt=fmt, dtype=dtype, rows=B, columns=14, sink=3, window=21)
    atol, rtol = (BF16_ATOL, BF16_RTOL) if dtype == "bf16" else (F32_ATOL, F32_RTOL)
    kept = [[np.zeros((c.hkv, 224, c.d)) for _ in range(B)] for _ in "kv"]    # the model's values
    past = t
    starts = c.starts(past)
    new = [c.values(1, sum(past), c.hkv, c.d) for _ in "kv"]
    c.ctx.append_kv8(fmt, 0, 1, new[0][1], new[1][1], c.ints(past), c.table, c.codes, c.scales, c.ring, B,
                     tok_start=c.ints(starts))
    c.oracle_write(new[0][0], new[1][0], past, [0] * B)
    for b in range(B):
        for kv in (0, 1):
            kept[kv][b][:, :past[b]] = new[kv][0][0, starts[b]:starts[b + 1]].transpose(1, 0, 2)
    q, k, v = (torch.zeros((B, h, c.d), dtype=c.kind, device="cuda") for h in (c.hq, c.hkv, c.hkv))
    pos, scores = c.ints([0] * B), torch.zeros(B, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros((B, c.hq), device="cuda")
    flags = torch.zeros(B, dtype=torch.uint8, device="cuda")
    idx, count = c.ints([0] * B), c.ints([0])

    def step():
        c.ctx.append_kv8(fmt, 0, 1, k[None], v[None], pos, c.table, c.codes, c.scales, c.ring, B)
        c.ctx.local_attn(0, q, pos, c.ring, out, lse, B)
        c.ctx.gate(scores, 0.0, B, flags, idx, count)
        c.ctx.full_attn_kv8(fmt, 0, q, pos, c.table, c.codes, c.scales, idx, count, out, lse, B)

    graph = None
    if how == "graph":
        pos.copy_(c.ints([x + 1 for x in t]))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for flagged in ([], [2], [0, 1, 2, 3], [3, 0], [1], []):
        t = [x + 1 for x in t]
        fresh = [c.values(*x.shape) for x in (q, k, v)]
        for x, (_, y) in zip((q, k, v), fresh):
            x.copy_(y)
        pos.copy_(c.ints(t))
        scores.copy_(torch.tensor([0.5 if b in flagged else -0.5 for b in range(B)]))
        if graph is not None:
            graph.replay()
        else:
            step()
        assert c.ctx.get_device_error() == 0
        c.oracle_write(fresh[1][0][None], fresh[2][0][None], [1] * B, [x - 1 for x in t])
        c.check()
        assert int(count.item()) == len(flagged) and idx.tolist()[:len(flagged)] == sorted(flagged)
        qh = fresh[0][0]
        check_rows(c, qh, out, lse, flagged, t)
        for b in range(B):
            for kv in (0, 1):
                kept[kv][b][:, t[b] - 1] = fresh[1 + kv][0][b]
            if b in flagged:
                continue
            want, wl = O.local_attention(qh[b], kept[0][b][:, :t[b]], kept[1][b][:, :t[b]], t[b], c.sink, c.window)
            assert np.all(np.abs(out[b].double().cpu().numpy() - want) <= atol + rtol * np.abs(want)), b
            assert np.all(np.abs(lse[b].double().cpu().numpy() - wl) <= atol + rtol * np.abs(wl)), b


@pytest.mark.parametrize("late,one_each", [(k, False) for k in ("seq_lens", "block_table", "tok_start", "k_new")] +
                         [(k, True) for k in ("seq_lens", "block_table", "k_new")])
def test_a_write_and_a_read_of_what_the_launch_before_stores_late(torch, late_store, late, one_each):
    """The write and the read are released early by the launch that stores one of their inputs: they
    use it as it was stored, not as it was."""
    B, new = 5, [1] * 5 if one_each else [3, 40, 0, 17, 1]
    c = Case(torch, fmt="int8", dtype="f32", hq=1, hkv=1, d=64, rows=B, columns=6, sink=3, window=20)
    past = [0, 9, 30, 16, 50]
    c.write(past, [0] * B)
    c.check()
    t = [a + n for a, n in zip(past, new)]
    total = sum(new)
    (k, kd), (v, vd) = (c.values(1, total, 1, 64) for _ in "kv")
    right = dict(seq_lens=c.ints(t), block_table=c.table.clone().flatten(), tok_start=c.ints(c.starts(new)),
                 k_new=kd.clone().flatten().view(torch.int32))
    wrong = dict(seq_lens=c.ints([5, 1, 96, 20, 7] if one_each else [40, 44, 0, 50, 96]),
                 block_table=right["block_table"].flip(0).contiguous(),
                 tok_start=c.ints([0, total, total, total, total, total]), k_new=torch.zeros_like(right["k_new"]))
    held = {n: (wrong if n == late else right)[n].clone() for n in right}
    out = [torch.full((1, total, 1, 64), 9.0, device="cuda") for _ in "kv"]
    table = held["block_table"].view(B, 6)
    starts = None if one_each else held["tok_start"]
    torch.cuda.synchronize()
    late_store(held[late], right[late])
    c.ctx.append_kv8("int8", 0, 1, held["k_new"].view(torch.float32).view(1, total, 1, 64), vd, held["seq_lens"], table,
                     c.codes, c.scales, c.ring, B, tok_start=starts)
    c.oracle_write(k, v, new, past)
    c.check()
    if late != "k_new":
        held[late].copy_(wrong[late])
        torch.cuda.synchronize()
        late_store(held[late], right[late])
    c.ctx.read_kv8("int8", 0, 1, held["seq_lens"], table, c.codes, c.scales, out[0], out[1], B, tok_start=starts)
    assert c.ctx.get_device_error() == 0
    at = c.starts(new)
    for b in range(B):
        for o, x in zip(out, c.kv(0, b, t[b])):
            want = x[0, t[b] - new[b]:].astype(np.float32)
            assert np.array_equal(o[0, at[b]:at[b + 1], 0].cpu().numpy(), want), b


@pytest.mark.parametrize("late", ["positions", "q", "inv_freq", "weight"])
def test_a_rotation_of_what_the_launch_before_stores_late(torch, late_store, late):
    c = Case(torch, dtype="f32", hq=2, hkv=1, d=64, rows=1, columns=1)
    n = 40
    f = (10000.0 ** (-np.arange(32) / 32.0)).astype(np.float32)
    pos = c.r.integers(0, 1 << 17, n)
    (q, qd), (w, wd) = c.values(n, 2, 64), c.values(64)
    bits = lambda x: x.clone().flatten().view(torch.int32)  # noqa: E731
    right = dict(positions=c.ints(pos), q=bits(qd), inv_freq=bits(torch.from_numpy(f).cuda()), weight=bits(wd))
    held = {k: torch.zeros_like(x) if k == late else x.clone() for k, x in right.items()}
    out = torch.full((n, 2, 64), 9.0, device="cuda")
    torch.cuda.synchronize()
    late_store(held[late], right[late])
    c.ctx.qk_norm_rope(held["q"].view(torch.float32).view(n, 2, 64), None, held["weight"].view(torch.float32), None, 1e-5,
                       held["inv_freq"].view(torch.float32), held["positions"], out, None)
    want = O.norm_rotate(q, w, 1e-5, pos, f)
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= rope_bound(q, w, 1e-5, pos, f, False, "f32"))
    assert c.ctx.get_device_error() == 0
