"""The batch calls (rotary positions, dense attention, pages) on the host: the
frequency tables against their formulas, workspace arithmetic, and refusals
before any launch. Pointers are fakes that no check reads."""

import ctypes
import math

import pytest
import torch

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def zha():
    from hierarchical_sparse_attention_zha_b200 import zha as z
    return z


def _cfg(zha, **kw):
    base = dict(n_kv_heads=4, n_q_heads=32, head_dim=128, chunk=64, levels=1, n_ref=1,
                kv_dtype=torch.bfloat16, max_tokens=1 << 20)
    base.update(kw)
    return zha.make_config(**base)


def _thetas(d, pairs, base, scaling, f, L, low, high, freq):
    D = freq or 2 * pairs
    out = []
    for i in range(pairs):
        t = base ** (-2 * i / D)
        if scaling == "linear":
            t /= f
        elif scaling == "ntk":
            t = (base * f ** (D / (D - 2))) ** (-2 * i / D) if D > 2 else t / f
        elif scaling == "yarn":
            lo, hi = (D * math.log(L / (2 * math.pi * n)) / (2 * math.log(base)) for n in (high, low))
            lo, hi = max(0, math.floor(lo)), min(pairs - 1, math.ceil(hi))
            w = min(1, max(0, (i - lo) / max(hi - lo, 0.001)))
            t = t * (1 - w) + t / f * w
        elif scaling == "bands":
            w = min(1, max(0, (L * t / (2 * math.pi) - low) / (high - low)))
            t = w * t + (1 - w) * t / f
        out.append(t)
    return out


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "bands"])
@pytest.mark.parametrize("d,pairs,freq,base", [(128, 64, 0, 10000.0), (64, 1, 0, 500.0), (64, 13, 64, 1e6),
                                               (128, 33, 0, 1.5)])
def test_rope_table_holds_the_formulas_frequencies(zha, scaling, d, pairs, freq, base):
    r = zha.Rope(d, pairs, "half", base, scaling, 8.0, 4096.0, 1.0, 32.0, freq).table
    want = _thetas(d, pairs, base, scaling, 8.0, 4096.0, 1.0, 32.0, freq)
    assert (r.head_dim, r.pairs, r.layout) == (d, pairs, 1)
    for i, t in enumerate(want):
        # both sides round a power, a quotient and a few products in 64 bits
        assert abs(r.turn[i] / 2.0 ** 64 - t / (2 * math.pi)) <= 2.0 ** -48 * t
    assert list(r.turn[pairs:]) == [0] * (64 - pairs)
    amp = 0.1 * math.log(8.0) + 1 if scaling == "yarn" else 1.0
    assert abs(r.amplitude - amp) <= 2.0 ** -24 * amp


def test_rope_init_refuses_bad_rotations(zha):
    ok = dict(head_dim=128, pairs=64)
    zha.Rope(**ok)
    for bad in (dict(head_dim=96), dict(pairs=0), dict(pairs=65), dict(base=1.0), dict(base=float("nan")),
                dict(base=float("inf")), dict(freq_dim=1), dict(freq_dim=-2), dict(scaling="linear", factor=0.5),
                dict(scaling="ntk", factor=float("inf")), dict(scaling="yarn", factor=2.0),
                dict(scaling="yarn", factor=2.0, original_tokens=100.0, low=4.0, high=4.0),
                dict(scaling="bands", factor=2.0, original_tokens=100.0, low=0.0, high=4.0),
                dict(amplitude=-1.0), dict(amplitude=float("nan"))):
        with pytest.raises(zha.ZhaError):
            zha.Rope(**{**ok, **bad})
    for bad in (dict(layout="third"), dict(scaling="other")):
        with pytest.raises(ValueError):
            zha.Rope(**{**ok, **bad})
    spec = zha.RopeSpec(128, 64, 2, 0, 0, 0, 1e4)
    out = zha.RopeTable()
    assert zha.lib.zha_rope_init(ctypes.byref(spec), ctypes.byref(out)) == zha.ZHA_ERR_INVALID
    spec.layout, spec.reserved = 0, 1
    assert zha.lib.zha_rope_init(ctypes.byref(spec), ctypes.byref(out)) == zha.ZHA_ERR_INVALID
    spec.reserved = 0
    assert zha.lib.zha_rope_init(ctypes.byref(spec), ctypes.byref(out)) == zha.ZHA_OK
    assert zha.lib.zha_rope_init(None, ctypes.byref(out)) == zha.ZHA_ERR_INVALID
    assert zha.lib.zha_rope_init(ctypes.byref(spec), None) == zha.ZHA_ERR_INVALID


def _kv(zha, ld=1000, blocks=0):
    return zha.KvCache(1 << 40, 1 << 41, ld, (1 << 42) if blocks else None, blocks)


def test_attend_batch_refusals(zha):
    cfg = _cfg(zha)
    before = zha.launch_count()
    ws = zha.attend_batch_workspace_bytes(cfg, 4, 1000)
    assert ws > 0

    def call(cfg=cfg, q=1 << 43, qt=0, kv=None, n=4, tokens=1 << 44, most=1000, o=1 << 45, w=1 << 46, size=ws):
        kv = _kv(zha) if kv is None else kv
        return zha.lib.zha_attend_batch_kv(ctypes.byref(cfg), q, qt, ctypes.byref(kv), n, tokens, most, o, None, w,
                                           size, None, None)

    inv, cap, uns = zha.ZHA_ERR_INVALID, zha.ZHA_ERR_CAPACITY, zha.ZHA_ERR_UNSUPPORTED
    assert call(cfg=_cfg(zha, n_q_heads=30)) == inv
    assert call(q=None) == inv and call(q=(1 << 43) + 8) == inv and call(o=None) == inv
    assert call(qt=2) == inv and call(tokens=None) == inv and call(n=0) == inv and call(n=65536) == inv
    assert call(most=-1) == inv
    assert call(most=1001) == inv and "max_tokens" in zha.last_error()
    assert call(kv=_kv(zha, 1000, 15), most=961) == inv              # 15 pages of 64
    assert call(kv=zha.KvCache(None, 1 << 41, 1000, None, 0)) == inv
    assert call(kv=zha.KvCache(1 << 40, (1 << 41) + 2, 1000, None, 0)) == inv
    assert call(kv=_kv(zha, 0)) == inv
    assert call(kv=_kv(zha, 1 << 28)) == uns                         # 4 * 4 * 2^28 rows
    assert call(kv=_kv(zha, 1 << 26, 16)) == uns                     # 2^32 rows in the pool
    assert call(w=None) == cap and call(w=(1 << 46) + 128) == cap and call(size=ws - 1) == cap
    huge = _cfg(zha, n_kv_heads=1 << 12, n_q_heads=1 << 12)
    assert call(cfg=huge, n=2000, most=0, kv=_kv(zha, 1)) == uns
    assert zha.attend_batch_workspace_bytes(huge, 2000, 0) == 0
    for bad in ((0, 10), (65536, 10), (4, -1)):
        assert zha.attend_batch_workspace_bytes(cfg, *bad) == 0
    assert zha.lib.zha_attend_batch_kv(ctypes.byref(cfg), 1 << 43, 0, None, 4, 1 << 44, 10, 1 << 45, None, 1 << 46, ws,
                                       None, None) == inv
    assert zha.launch_count() == before


def test_rope_refusals(zha):
    cfg = _cfg(zha)
    rope = zha.Rope(128)
    before = zha.launch_count()
    rows = lambda *a: ctypes.byref(zha.Rows(*a))
    good = (1 << 40, 512, 128)

    def turn(r=rope.table, x=good, xt=1, pos=1 << 41, n=5, h=4, y=(1 << 42, 512, 128), yt=1):
        return zha.lib.zha_rope_apply(None if r is None else ctypes.byref(r), rows(*x), xt, pos, n, h, 0, rows(*y), yt,
                                      None)

    inv = zha.ZHA_ERR_INVALID
    assert turn(r=None) == inv and turn(r=zha.RopeTable()) == inv
    assert turn(xt=2) == inv and turn(yt=-1) == inv and turn(n=-1) == inv and turn(h=0) == inv and turn(pos=None) == inv
    assert turn(x=(None, 512, 128)) == inv and turn(x=((1 << 40) + 8, 512, 128)) == inv
    assert turn(x=(1 << 40, 516, 128)) == inv and turn(y=(1 << 42, 512, 132)) == inv   # 16-byte pieces of 8 bf16
    assert turn(y=(1 << 40, 512, 128), yt=0) == inv                                    # in place, another type
    assert turn(y=(1 << 40, 1024, 128)) == inv                                         # in place, other strides
    assert turn(y=(1 << 42, 0, 128)) == inv and turn(y=(1 << 42, 512, 0)) == inv       # rows that lie on one another
    assert turn(y=(1 << 42, 128, 64)) == inv and turn(y=(1 << 42, 256, 128)) == inv
    assert turn(n=0, x=(None, 0, 0), pos=None) == zha.ZHA_OK

    def append(cfg=cfg, r=rope.table, q=good, k=good, v=good, st=1, n=3, kv=None, seqs=2, seq=1 << 43, index=1 << 44,
               out=1 << 45, qt=0):
        kv = _kv(zha) if kv is None else kv
        return zha.lib.zha_rope_append_kv(
            ctypes.byref(cfg), None if r is None else ctypes.byref(r), None if q is None else rows(*q), rows(*k),
            rows(*v), st, n, ctypes.byref(kv), seqs, seq, index, None, out, qt, None, None)

    assert append(r=zha.Rope(64).table) == inv and append(r=zha.RopeTable()) == inv
    assert append(cfg=_cfg(zha, chunk=1)) == zha.ZHA_ERR_UNSUPPORTED
    assert append(st=3) == inv and append(qt=2) == inv and append(n=-1) == inv and append(seqs=0) == inv
    assert append(k=(None, 0, 0)) == inv and append(v=((1 << 40) + 4, 512, 128)) == inv
    assert append(q=(1 << 40, 12, 128)) == inv and append(out=None) == inv and append(out=(1 << 45) + 8) == inv
    assert append(seq=None) == inv and append(index=None) == inv
    assert append(kv=_kv(zha, 0)) == inv and append(kv=_kv(zha, 1 << 28), seqs=4) == zha.ZHA_ERR_UNSUPPORTED
    assert append(n=0, k=(None, 0, 0), seq=None) == zha.ZHA_OK
    assert zha.launch_count() == before


def test_pages_refusals(zha):
    cfg = _cfg(zha)
    before = zha.launch_count()

    def pool(**kw):
        a = dict(k=1 << 40, v=1 << 41, n_pages=500, block_table=1 << 42, max_blocks=16, refs=1 << 43, n_seqs=8,
                 reserved=0)
        a.update(kw)
        return zha.PagePool(**a)

    ws = zha.pages_workspace_bytes(cfg, pool(), 8)
    assert ws > 0
    L, b = zha.lib, ctypes.byref
    inv, cap = zha.ZHA_ERR_INVALID, zha.ZHA_ERR_CAPACITY

    def calls(c=cfg, p=None, n=8, w=1 << 46, size=ws, seqs=1 << 44, tok=1 << 45):
        p = pool() if p is None else p
        return (L.zha_pages_extend(b(c), b(p), seqs, tok, n, w, size, None, None),
                L.zha_pages_fork(b(c), b(p), seqs, seqs, tok, n, w, size, None, None),
                L.zha_pages_free(b(c), b(p), seqs, tok, n, None, None) if w and size == ws and tok else inv,
                L.zha_pages_compact(b(c), b(p), None, None, w, size, None, None) if n == 8 and seqs and tok else inv)

    for bad in (dict(k=None), dict(v=(1 << 41) + 8), dict(n_pages=0), dict(block_table=None), dict(max_blocks=0),
                dict(refs=None), dict(refs=(1 << 43) + 2), dict(n_seqs=0), dict(n_seqs=65536), dict(reserved=1)):
        assert set(calls(p=pool(**bad))) == {inv}, bad
        assert zha.pages_workspace_bytes(cfg, pool(**bad), 8) == 0
    assert set(calls(p=pool(n_pages=1 << 26))) == {zha.ZHA_ERR_UNSUPPORTED}
    assert set(calls(c=_cfg(zha, head_dim=96))) == {zha.ZHA_ERR_UNSUPPORTED}
    assert set(calls(n=-1)) == {inv} and set(calls(n=65536)) == {inv}
    assert set(calls(seqs=None)) == {inv} and set(calls(tok=None)) == {inv}
    for w, size in ((None, ws), ((1 << 46) + 64, ws), (1 << 46, 16)):
        assert L.zha_pages_extend(b(cfg), b(pool()), 1 << 44, 1 << 45, 8, w, size, None, None) == cap
        assert L.zha_pages_fork(b(cfg), b(pool()), 1 << 44, 1 << 44, 1 << 45, 8, w, size, None, None) == cap
        assert L.zha_pages_compact(b(cfg), b(pool()), None, None, w, size, None, None) == cap
    assert L.zha_pages_extend(b(cfg), b(pool()), None, None, 0, None, 0, None, None) == zha.ZHA_OK
    assert L.zha_pages_fork(b(cfg), b(pool()), None, None, None, 0, None, 0, None, None) == zha.ZHA_OK
    assert L.zha_pages_free(b(cfg), b(pool()), None, None, 0, None, None) == zha.ZHA_OK
    assert zha.pages_workspace_bytes(cfg, pool(), 65536) == 0 and zha.pages_workspace_bytes(cfg, pool(), -1) == 0
    assert L.zha_pages_free(b(cfg), None, 1 << 44, None, 1, None, None) == inv
    assert zha.launch_count() == before


def test_binding_refuses_what_the_c_calls_cannot_see(zha):
    """Tensors of a wrong kind are refused before a pointer is taken."""
    with pytest.raises(ValueError):
        zha.kv_batch(torch.zeros(2, 4, 10, 64), torch.zeros(2, 4, 10, 64))            # not on a GPU
    with pytest.raises(ValueError):
        zha.rope_apply(zha.Rope(64), torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        zha.rope_apply(zha.Rope(64), torch.zeros(3, 2, 128), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        zha.rope_apply(zha.Rope(64), torch.zeros(3, 2, 64, dtype=torch.float64), torch.zeros(3, dtype=torch.int64))


def _described(c, index=0):
    """What kv_batch() and page_pool() note beside the C struct, for _cfg()'s cache."""
    c.shape, c.dtype, c.heads, c.seqs, c.index, c.device = (500, 64, 128), 1, 4, 8, index, None
    return c


def test_page_calls_take_pools_and_the_others_caches(zha):
    """A zha_kv_cache is shorter than a zha_page_pool: a page call that took one would read its
    counts from behind it. Both are refused for each other before any pointer is taken."""
    cfg = _cfg(zha)
    kv = _described(_kv(zha, 500, 16))
    pool = _described(zha.PagePool(1 << 40, 1 << 41, 500, 1 << 42, 16, 1 << 43, 8, 0))
    assert ctypes.sizeof(kv) < ctypes.sizeof(pool)
    ints = torch.zeros(2, dtype=torch.int32)
    longs = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: zha.pages_workspace_bytes(cfg, kv, 2), lambda: zha.pages_extend(cfg, kv, ints, longs),
                 lambda: zha.pages_fork(cfg, kv, ints, ints, longs), lambda: zha.pages_free(cfg, kv, ints),
                 lambda: zha.pages_compact(cfg, kv)):
        with pytest.raises(ValueError, match=r"page_pool\(\)"):
            call()
    x = torch.zeros(2, 4, 128)
    for call in (lambda: zha.attend_batch_kv(cfg, torch.zeros(8, 32, 128), pool, 8, longs, 10),
                 lambda: zha.rope_append_kv(cfg, None, None, x, x, pool, 8, ints, longs)):
        with pytest.raises(ValueError, match=r"kv_batch\(\)$"):
            call()
    assert zha.pages_workspace_bytes(cfg, pool, 2) > 0


class _OnGpu:
    """A CPU tensor that passes for one on a GPU where only a handle is made of it."""
    is_cuda = True

    def __init__(self, x):
        self._x = x

    def __getattr__(self, name):
        return getattr(self._x, name)


@pytest.mark.parametrize("shape", [(8, 4, 0), (0, 4, 16), (8, 0, 16)])
def test_caches_refuse_a_block_table_without_entries(zha, shape):
    """Its address is NULL, with which the C calls would take the pool for contiguous caches
    of n_pages rows, and read behind it where sequences times heads are more than the chunk."""
    pool = _OnGpu(torch.zeros(6, 64, 128, dtype=torch.bfloat16))
    assert zha.kv_batch(pool, pool, _OnGpu(torch.zeros(8, 4, 16, dtype=torch.int32))).block_table
    empty = torch.zeros(shape, dtype=torch.int32)
    assert empty.data_ptr() == 0
    with pytest.raises(ValueError, match="at least one entry"):
        zha.kv_batch(pool, pool, _OnGpu(empty))
    with pytest.raises(ValueError, match="at least one entry"):
        zha.kv_cache(pool, pool, _OnGpu(empty[0] if shape[0] else torch.zeros(0, 16, dtype=torch.int32)))
    with pytest.raises(ValueError, match="at least one entry"):
        zha.page_pool(pool, pool, _OnGpu(empty), _OnGpu(torch.zeros(6, dtype=torch.int32)))


@pytest.mark.parametrize("args,kept", [
    # x(32) = 128 ln(4096 / 64 pi) / (2 ln 10000) = 20.9 and x(1) = 45.03: the ramp is 20..46, beyond
    # the 32 pairs that turn; pair 31 turns 7.5 times over the original length
    (dict(head_dim=128, pairs=32, freq_dim=128, factor=8.0, original_tokens=4096.0, high=32.0),
     {0: 0, 20: 0, 21: 1 / 26, 30: 10 / 26, 31: 11 / 26}),
    # x(32) = 45.03, x(1) = 69.1: 45..70
    (dict(head_dim=128, pairs=64, factor=4.0, original_tokens=131072.0, high=32.0),
     {45: 0, 46: 1 / 25, 62: 17 / 25, 63: 18 / 25}),
    # x(32) = 2.87, x(1) = 5.12: 2..6
    (dict(head_dim=64, pairs=6, factor=8.0, original_tokens=16384.0, high=32.0),
     {1: 0, 2: 0, 3: 1 / 4, 4: 2 / 4, 5: 3 / 4}),
    # x(10000) = 8 ln(100 / 2 pi) / (2 ln 100) = 2.4, x(1) = 10.4: cut to freq_dim - 1 = 7, 2..7
    (dict(head_dim=64, pairs=4, base=100.0, factor=8.0, original_tokens=1e6, high=10000.0), {2: 0, 3: 1 / 5}),
    # a ramp inside the pairs: x(32) = 20.9, x(1) = 45.03 of 64
    (dict(head_dim=128, pairs=64, factor=8.0, original_tokens=4096.0, high=32.0), {20: 0, 33: 13 / 26, 46: 1, 63: 1}),
])
def test_yarn_ramp_ends_where_the_method_ends_it(zha, args, kept):
    """The published ramp runs from floor(x(high)) to ceil(x(low)), cut to [0, freq_dim - 1] and
    not to the pairs that there are. `kept`: pair -> its interpolated part, worked out by hand."""
    base, f, D = args.get("base", 10000.0), args["factor"], args.get("freq_dim") or 2 * args["pairs"]
    r = zha.Rope(layout="half", scaling="yarn", low=1.0, **args).table
    for i, w in kept.items():
        want = base ** (-2.0 * i / D) * ((1 - w) + w / f) / (2 * math.pi)
        assert abs(r.turn[i] / 2.0 ** 64 - want) <= 2.0 ** -46 * want, i


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int8])
def test_caches_refuse_other_element_types(zha, dtype):
    """With the ValueError of the other checks."""
    x = _OnGpu(torch.zeros(6, 64, 128, dtype=dtype))
    table = _OnGpu(torch.zeros(8, 4, 16, dtype=torch.int32))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        zha.kv_batch(x, x, table)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        zha.page_pool(x, x, table, _OnGpu(torch.zeros(6, dtype=torch.int32)))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        zha.kv_batch(_OnGpu(torch.zeros(2, 4, 9, 128, dtype=dtype)), _OnGpu(torch.zeros(2, 4, 9, 128, dtype=dtype)))


def test_attend_batch_refuses_an_output_that_overlaps_the_queries(zha):
    """A unit's output would be written over queries that another unit still reads."""
    cfg = _cfg(zha)
    before = zha.launch_count()
    ws = zha.attend_batch_workspace_bytes(cfg, 4, 1000)
    kv = _kv(zha)
    for dt, elt in ((0, 4), (1, 2)):
        size = 4 * 32 * 128 * elt
        for shift in (16, size // 2, size - 16, -16, 16 - size):
            rc = zha.lib.zha_attend_batch_kv(ctypes.byref(cfg), 1 << 43, dt, ctypes.byref(kv), 4, 1 << 44, 1000,
                                             (1 << 43) + shift, None, 1 << 46, ws, None, None)
            assert rc == zha.ZHA_ERR_INVALID and "overlaps" in zha.last_error(), (dt, shift)
        for shift in (size, -size, 0):                       # beside it, or it: the next check answers
            rc = zha.lib.zha_attend_batch_kv(ctypes.byref(cfg), 1 << 43, dt, ctypes.byref(kv), 4, 1 << 44, 1000,
                                             (1 << 43) + shift, None, None, ws, None, None)
            assert rc == zha.ZHA_ERR_CAPACITY, (dt, shift)
    assert zha.launch_count() == before


@pytest.mark.parametrize("amplitude", [1e39, 1e308, 1e-60])
def test_rope_init_refuses_amplitudes_that_float32_does_not_hold(zha, amplitude):
    """They became infinity, or 0, in the table, and the turned rows with them."""
    with pytest.raises(zha.ZhaError):
        zha.Rope(64, amplitude=amplitude)
    assert zha.Rope(64, amplitude=3e38).table.amplitude > 2.9e38 and zha.Rope(64, amplitude=1e-40).table.amplitude > 0


def test_batch_calls_refuse_words_between_their_addresses(zha):
    """An access there would be an error of the GPU's; the host refuses the call. The workspace's
    answer comes after it, and shows that the same call with good addresses passes."""
    cfg, rope, before = _cfg(zha), zha.Rope(128), zha.launch_count()
    b, L, kv = ctypes.byref, zha.lib, _kv(zha)
    inv, cap = zha.ZHA_ERR_INVALID, zha.ZHA_ERR_CAPACITY
    rows = lambda at: b(zha.Rows(at, 512, 128))
    pool = zha.PagePool(1 << 40, 1 << 41, 500, 1 << 42, 16, 1 << 43, 8, 0)
    at = {k: 1 << (44 + i) for i, k in enumerate(("n", "lse", "status", "seq", "index", "pos", "dst"))}

    def attend(n, lse, status):
        return L.zha_attend_batch_kv(b(cfg), 1 << 52, 0, b(kv), 4, n, 1000, 1 << 53, lse, None, 0, status, None)

    def append(seq, index, pos, status):
        return L.zha_rope_append_kv(b(cfg), b(rope.table), None, rows(1 << 52), rows(1 << 53), 1, 3, b(kv), 2, seq, index,
                                    pos, None, 0, status, None)

    def extend(seq, n, status):
        return L.zha_pages_extend(b(cfg), b(pool), seq, n, 8, None, 0, status, None)

    def fork(seq, dst, n, status):
        return L.zha_pages_fork(b(cfg), b(pool), seq, dst, n, 8, None, 0, status, None)

    def free(seq, n, status):
        return L.zha_pages_free(b(cfg), b(pool), seq, n, 8, status, None)

    def compact(dst, n, status):
        return L.zha_pages_compact(b(cfg), b(pool), dst, n, None, 0, status, None)

    def turn(pos):
        return L.zha_rope_apply(b(rope.table), rows(1 << 52), 1, pos, 5, 4, 0, rows(1 << 53), 1, None)

    for call, names, answer in ((attend, ("n", "lse", "status"), cap), (append, ("seq", "index", "pos", "status"), None),
                                (extend, ("seq", "n", "status"), cap), (fork, ("seq", "dst", "n", "status"), cap),
                                (free, ("seq", "n", "status"), None), (compact, ("dst", "n", "status"), cap),
                                (turn, ("pos",), None)):
        good = [at[k] for k in names]
        if answer is not None:
            assert call(*good) == answer, call.__name__
        for i, k in enumerate(names):
            for shift in (1, 2, 4) if k in ("index", "pos") or (k == "n" and call is not compact) else (1, 2, 3):
                assert call(*good[:i], good[i] + shift, *good[i + 1:]) == inv, (call.__name__, k, shift)
    assert zha.launch_count() == before
