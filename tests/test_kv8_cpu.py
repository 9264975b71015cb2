"""The 8-bit cache on the CPU: the oracle's own pins, the sizes and refusals
that need no GPU, and the numbering of the write's work items."""

import ctypes

import numpy as np
import pytest

import oracle as O
from tests.test_boundary import _cfg, _ensure_built


# ------------------------------------------------------------------ the oracle

def test_e4m3_bytes_round_trip():
    b = np.arange(256, dtype=np.uint8)
    v = O.kv8_value(b, "e4m3")
    fine = ~np.isnan(v)
    assert fine.sum() == 254
    n, byte = O.kv8_round(v[fine], "e4m3")
    assert np.array_equal(n, v[fine]) and np.array_equal(byte, b[fine])
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1.0


def test_rounding_is_to_nearest_with_ties_to_even():
    grid = np.unique(O.kv8_value(np.arange(127, dtype=np.uint8), "e4m3"))
    mid = (grid[1:] + grid[:-1]) / 2
    got = O.kv8_round(mid, "e4m3")[1]
    assert np.all(got % 2 == 0)                            # the even neighbour
    y = np.random.default_rng(1).uniform(-500, 500, 4000)
    n, _ = O.kv8_round(y, "e4m3")
    near = grid[np.abs(np.abs(y)[:, None] - grid).argmin(1)]
    assert np.array_equal(np.abs(n), near)
    assert np.array_equal(O.kv8_round([0.5, 1.5, -2.5, 127.4, 300], "int8")[0], [0, 2, -2, 127, 127])


def test_oracle_matches_torch_rounding():
    torch = pytest.importorskip("torch")
    y = torch.randn(20000, generator=torch.Generator().manual_seed(3)) * 60
    want = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.kv8_round(y.numpy().astype(np.float64), "e4m3")[1], want)


@pytest.mark.parametrize("fmt,step", [("int8", 0.5 / 127), ("e4m3", 2.0 ** -4)])
def test_a_block_written_at_once_and_token_by_token(fmt, step):
    """At once every element is within half a step of the format; token by token
    each growth of the scale may add half a step of the scale it grew to."""
    r = np.random.default_rng(5)
    x = r.standard_normal((16, 64)).astype(np.float32).astype(np.float64)
    one = np.zeros((16, 64), np.uint8)
    s1 = O.kv8_write_block(one, 0.0, 0, x, fmt)
    top = np.abs(x).max()
    e = np.abs(O.kv8_value(one, fmt) * s1 - x)
    unit = np.full_like(x, top) if fmt == "int8" else np.maximum(np.abs(x), top * 2.0 ** -14)
    assert np.all(e <= step * unit * (1 + 1e-6))
    many, s, scales = np.zeros((16, 64), np.uint8), 0.0, []
    for i in range(16):
        s = O.kv8_write_block(many, s, i, x[i:i + 1], fmt)
        scales.append(s)
    assert s == s1 and sorted(scales) == scales
    growths = len(set(scales)) + 1
    e = np.abs(O.kv8_value(many, fmt) * s - x)
    assert np.all(e <= growths * step * unit * (1 + 1e-6))


def test_zero_tiny_and_infinite_blocks():
    c = np.full((16, 64), 7, np.uint8)
    assert O.kv8_write_block(c, 0.0, 0, np.zeros((16, 64)), "int8") == 0.0 and not c.any()
    assert O.kv8_write_block(c, 0.0, 0, np.full((16, 64), 2.0 ** -101), "e4m3") == 0.0
    x = np.ones((3, 64))
    x[1, 5] = np.inf
    assert np.isnan(O.kv8_write_block(c, 0.0, 0, x, "int8"))
    assert np.isnan(O.kv8_write_block(c, np.nan, 3, np.ones((1, 64)), "int8"))
    assert O.kv8_write_block(c, np.nan, 0, np.ones((1, 64)), "int8") == np.float32(1 / 127)


def test_norm_rotate_special_cases():
    r = np.random.default_rng(2)
    x = r.standard_normal((3, 2, 8))
    f = 1.0 / 10.0 ** np.arange(3)
    for nb in (False, True):
        y = O.norm_rotate(x, None, 0.0, [0, 0, 0], f, nb)
        assert np.array_equal(y, x)                        # position 0 turns nothing
        y = O.norm_rotate(x, None, 0.0, [5, 9, 2 ** 20], f, nb)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.array_equal(y[..., 6:], x[..., 6:])      # behind the rotated part
    # the score of a rotated pair depends on the distance of their positions only
    q, k = r.standard_normal((1, 1, 8)), r.standard_normal((1, 1, 8))
    a = [(O.norm_rotate(q, None, 0, [p], f) * O.norm_rotate(k, None, 0, [p - 3], f)).sum() for p in (3, 500)]
    assert abs(a[0] - a[1]) < 1e-12
    y = O.norm_rotate(3.0 * x, np.ones(8), 0.0, [0] * 3, f)
    assert np.allclose((y ** 2).mean(-1), 1.0)


# ------------------------------------------------------------ sizes, refusals

def test_kv8_layout():
    _ensure_built()
    from gated_local_full_b200 import oda
    lay = oda.kv8_layout(_cfg())
    assert lay == dict(tile_bytes=2 * 16 * 128, cache_layer_bytes=8257 * 8 * 4096,
                       scale_layer_elems=8257 * 8 * 2)
    assert oda.kv8_layout(_cfg(head_dim=64, dtype="f32"))["tile_bytes"] == 2048
    with pytest.raises(oda.OdaError) as e:
        oda.kv8_layout(_cfg(head_dim=96))
    assert e.value.status == oda.ERR_SHAPE


def test_null_contexts_are_refused():
    _ensure_built()
    from gated_local_full_b200 import oda
    L = oda.lib()
    n = None
    assert L.oda_kv8_layout(n, n) == oda.ERR_ARG
    assert L.oda_append_kv8(n, 1, 0, 1, n, n, n, 1, n, n, n, n, n, 1, n) == oda.ERR_ARG
    assert L.oda_read_kv8(n, 1, 0, 1, n, 1, n, n, n, n, n, n, 1, n) == oda.ERR_ARG
    assert L.oda_full_attn_kv8(n, 1, 0, n, n, n, n, n, n, n, n, n, 1, 0, n) == oda.ERR_ARG
    assert L.oda_range_attn_kv8(n, 1, 0, n, n, n, n, n, n, n, n, n, n, n, 1, 0, n) == oda.ERR_ARG
    assert L.oda_qk_norm_rope(n, n, 0, n, 0, n, n, 1e-6, n, 0, n, 0, 1, n, 0, n, 0, 0, n) == oda.ERR_ARG


def test_tensors_off_the_gpu_are_refused():
    torch = pytest.importorskip("torch")
    _ensure_built()
    from gated_local_full_b200 import oda

    class Ctx(oda.OdaContext):                             # the binding's checks alone
        def __init__(self, cfg):
            self.cfg, self.handle = cfg, None

    ctx = Ctx(_cfg())
    kv = torch.zeros((1, 2, 8, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        ctx.append_kv8("int8", 0, 1, kv, kv, i, i, kv, kv, None, 2)
    with pytest.raises(ValueError, match="dtype"):
        ctx.append_kv8("int8", 0, 1, kv.float(), kv.float(), i, i, kv, kv, None, 2)
    with pytest.raises(ValueError, match="layers"):
        ctx.append_kv8("int8", 0, 2, kv, kv, i, i, kv, kv, None, 2)
    with pytest.raises(ValueError, match="differ"):
        ctx.append_kv8("int8", 0, 1, kv, kv[:, :1], i, i, kv, kv, None, 2)
    with pytest.raises(ValueError, match="needs"):
        ctx.read_kv8("int8", 0, 1, i, i, kv, kv, None, None, 2)
    q, k = torch.zeros((2, 16, 128), dtype=torch.bfloat16), torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    f = torch.ones(64)
    with pytest.raises(ValueError, match="context's dtype"):
        ctx.qk_norm_rope(q.float(), k, None, None, 0.0, f, i, q, k)
    with pytest.raises(ValueError, match="context's dtype"):
        ctx.qk_norm_rope(q, k[:, :4], None, None, 0.0, f, i, q, k)
    with pytest.raises(ValueError, match="positions"):
        ctx.qk_norm_rope(q, k, None, None, 0.0, f, i.long(), q, k)
    with pytest.raises(ValueError, match="norm weight"):
        ctx.qk_norm_rope(q, k, f.bfloat16(), None, 0.0, f, i, q, k)
    with pytest.raises(ValueError, match="GPU"):
        ctx.qk_norm_rope(q, k, None, None, 0.0, f, i, q, k)


def test_write_items_never_meet():
    """Row b's items start at tok_start[b] // 16 + 2 b; a row of n tokens touches
    at most n // 16 + 2 blocks, wherever its first token falls."""
    r = np.random.default_rng(9)
    for _ in range(300):
        B = int(r.integers(1, 12))
        n = r.integers(0, 70, B) * r.integers(0, 2, B)
        past = r.integers(0, 100, B)
        ts = np.concatenate([[0], np.cumsum(n)])
        items, used = int(ts[-1]) // 16 + 2 * B, set()
        start = [int(ts[b]) // 16 + 2 * b for b in range(B)]
        for b in range(B):
            if n[b]:
                touched = (past[b] + n[b] - 1) // 16 - past[b] // 16 + 1
                for j in range(touched):
                    it = start[b] + j
                    assert it < items and it not in used
                    assert max(x for x in range(B) if start[x] <= it) == b
                    used.add(it)


# ------------------------------------------------------------ the compiled calls

def _bare():
    """A binding's context without a library handle: every call ends with ODA_ERR_ARG at the latest."""
    from gated_local_full_b200 import oda

    class Ctx(oda.OdaContext):
        def __init__(self, cfg):
            self.cfg, self.handle = cfg, None

    return Ctx(_cfg())


def test_numbers_past_32_bits_are_refused():
    pytest.importorskip("torch")
    _ensure_built()
    from gated_local_full_b200 import oda
    ctx = _bare()

    def full(layer=0, B=1, format="int8"):
        ctx.full_attn_kv8(format, layer, 64, 64, 64, 64, 64, 64, 64, 64, None, B, stream=0)

    def ranged(layer=0, B=1):
        ctx.range_attn_kv8("int8", layer, 64, 64, 64, 64, 64, 64, 64, 64, 64, 64, None, B, stream=0)

    for f in (full, ranged):
        with pytest.raises(oda.OdaError):
            f()
        for v in (2 ** 31, 2 ** 32, 2 ** 32 + 1, -2 ** 31 - 1, 2 ** 63, 2 ** 70):
            with pytest.raises(OverflowError):
                f(layer=v)
            with pytest.raises(OverflowError):
                f(B=v)
    torch = pytest.importorskip("torch")
    kv = torch.zeros((1, 2, 8, 128), dtype=torch.bfloat16)
    for v in (2 ** 32, 2 ** 33 + 1):
        with pytest.raises(OverflowError):
            ctx.append_kv8("int8", v, v + 1, kv, kv, 64, 64, 64, 64, None, 2, stream=0)
        with pytest.raises(OverflowError):
            ctx.read_kv8("int8", v, v + 1, 64, 64, 64, 64, kv, kv, 2, stream=0)


def test_calls_leave_the_interpreter_to_other_threads():
    """With a function that sleeps in the library's place (its first argument, the context's
    handle, is the time in us), another thread counts on while a call is under way."""
    pytest.importorskip("torch")
    _ensure_built()
    import threading
    from gated_local_full_b200 import oda
    f = oda._fastcall()
    sleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    key = (300000,) + _bare()._context()[1:]
    args = ("int8", 0) + (64,) * 8 + (None, 1, 0, 0)       # layer, ..., lse, B, flags, stream
    started, seen, stop = threading.Event(), [0], threading.Event()

    def count():
        started.set()
        while not stop.wait(0.005):
            seen[0] += 1

    other = threading.Thread(target=count)
    try:
        f.bind(oda.OdaError, *[sleep] * len(oda._FAST_CALLS))
        other.start()
        started.wait(10)
        before = seen[0]
        f.full_attn_kv8(key, *args)
        after = seen[0]
    finally:
        stop.set()
        other.join()
        oda._fast = None                                   # bound to the library again by the next call
    assert after - before >= 5
    oda._fastcall()


@pytest.mark.parametrize("region", [False, True], ids=["full", "region"])
def test_types_and_sizes_of_the_attention_calls(region):
    """A tensor in a wrong type, or shorter than what the call would read or write, is refused for that
    (before its place is looked at); a right one only for not being on a GPU."""
    torch = pytest.importorskip("torch")
    _ensure_built()
    from gated_local_full_b200 import oda
    ctx = _bare()
    ctx.cfg = _cfg(layers=2, max_blocks_per_seq=5, num_blocks=7)
    i32, f32, b16, u8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8
    right = dict(q=((3, 16, 128), b16), seq_lens=((3,), i32), block_table=((3, 5), i32),
                 codes=((2, 7, 8, 2, 16, 128), u8), scales=((2, 7, 8, 2), f32), idx=((3,), i32), count=((1,), i32),
                 out=((3, 16, 128), b16), lse=((3, 16), f32))
    if region:
        right.update(range_lo=((3,), i32), range_hi=((3,), i32))
    f = ctx.range_attn_kv8 if region else ctx.full_attn_kv8
    names = [n for n in ("q", "seq_lens", "range_lo", "range_hi", "block_table", "codes", "scales", "idx", "count", "out",
                         "lse") if n in right]

    def call(name, x, layer=1, B=3):
        f("int8", layer, *[x if n == name else 64 for n in names], B, stream=0)

    for name in names:
        shape, kind = right[name]
        with pytest.raises(ValueError, match="GPU"):
            call(name, torch.zeros(shape, dtype=kind))
        with pytest.raises(ValueError, match="GPU"):
            call(name, torch.zeros(int(np.prod(shape)) + 1, dtype=kind))
        for other in {torch.int64, f32, b16, torch.float16, i32, u8} - {kind}:
            with pytest.raises(ValueError, match=name):
                call(name, torch.zeros(shape, dtype=other))
        with pytest.raises(ValueError, match=name):
            call(name, torch.zeros(int(np.prod(shape)) - 1, dtype=kind))
        if name in ("codes", "scales"):                    # what layer 0 alone needs
            with pytest.raises(ValueError, match="GPU"):
                call(name, torch.zeros(shape[1:], dtype=kind), layer=0)
        elif name != "count":
            with pytest.raises(ValueError, match=name):
                call(name, torch.zeros(shape, dtype=kind), B=4)
    for wide in (4, 6, 15):                                # rows of another length
        with pytest.raises(ValueError, match="block_table"):
            call("block_table", torch.zeros((30, wide), dtype=i32))
    for e in (torch.int8, torch.float8_e4m3fn):            # codes seen as what they hold
        with pytest.raises(ValueError, match="GPU"):
            call("codes", torch.zeros((2, 7, 8, 2, 16, 128), dtype=torch.int8).view(e))
    with pytest.raises(oda.OdaError):                      # a layer that there is none of: the library's answer
        call("q", 64, layer=2 ** 31 - 1)


def test_types_and_sizes_of_the_lists_of_write_and_read():
    torch = pytest.importorskip("torch")
    _ensure_built()
    ctx = _bare()
    ctx.cfg = _cfg(layers=2, max_blocks_per_seq=5, num_blocks=7, window=12, max_batch=3)
    kv = torch.zeros((1, 9, 8, 128), dtype=torch.bfloat16)
    right = dict(tok_start=((4,), torch.int32), seq_lens=((3,), torch.int32), block_table=((3, 5), torch.int32),
                 codes=((2, 7, 8, 2, 16, 128), torch.uint8), scales=((2, 7, 8, 2), torch.float32),
                 ring=((2, 3, 8, 1, 2, 16, 128), torch.bfloat16))

    def append(name, x):
        a = {n: x if n == name else 64 for n in right}
        ctx.append_kv8("e4m3", 1, 2, kv, kv, a["seq_lens"], a["block_table"], a["codes"], a["scales"], a["ring"], 3,
                       tok_start=a["tok_start"], stream=0)

    def read(name, x):
        a = {n: x if n == name else 64 for n in right}
        ctx.read_kv8("e4m3", 1, 2, a["seq_lens"], a["block_table"], a["codes"], a["scales"], kv, None, 3,
                     tok_start=a["tok_start"], stream=0)

    for f in (append, read):
        for name, (shape, kind) in right.items():
            if f is read and name == "ring":
                continue
            with pytest.raises(ValueError, match="GPU"):
                f(name, torch.zeros(shape, dtype=kind))
            for other in {torch.int64, torch.float64} - {kind}:
                with pytest.raises(ValueError, match=name):
                    f(name, torch.zeros(shape, dtype=other))
            with pytest.raises(ValueError, match=name):
                f(name, torch.zeros(int(np.prod(shape)) - 1, dtype=kind))


def test_the_library_builds_without_the_binding(monkeypatch):
    """The C ABI's users need neither torch's headers nor g++: only the binding does."""
    from gated_local_full_b200 import build as b

    def absent():
        raise RuntimeError("no headers")

    monkeypatch.setattr(b, "_build_fastcall", absent)
    monkeypatch.setattr(b, "_build_lib", lambda name, *a: name)
    assert b.build(binding=False) == ["liboda.so", "libsynth.so"]
    with pytest.raises(RuntimeError, match="no headers"):
        b.build()
