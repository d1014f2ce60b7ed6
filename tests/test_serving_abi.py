"""Refusals of the serving-step entry points, decided on the host before anything is enqueued."""
import ctypes

import numpy as np
import pytest

OUT = ctypes.c_void_p


@pytest.fixture(scope="module")
def gear():
    from kv_cache_compression_gear_b200 import build
    build.build()
    import kv_cache_compression_gear_b200 as g
    return g


class Pair:
    """A paged K and V cache laid out over addresses that nothing reads, rows 0 and 1 encoded (100 and 40 tokens),
    row 2 empty; buffers of 20 holding 3 and 20 tokens."""

    def __init__(self, gear, dtype=0, pages=12, **kw):
        L = gear.lib
        p = gear.make_params(**kw)
        self.B, self.H, self.P, self.NP, self.ppr, self.nblk = 3, 2, 32, pages, 6, 4
        nb = L.gear_paged_cache_bytes(ctypes.byref(p), 3, 2, 128, 32, pages, 6, 4, dtype)
        nh = L.gear_paged_host_ints(3, 6, pages)
        self.c, self.host = [], []
        for i in range(2):
            c, host = gear.GearCacheStruct(), np.zeros(nh, np.int32)
            # laid out by hand where there is no device to clear the tables on
            L.gear_paged_cache_init(ctypes.byref(c), ctypes.byref(p), 3, 2, 128, 32, pages, 6, 4, dtype,
                                    ctypes.c_void_p((1 << 40) + (i << 36)), nb, ctypes.c_void_p(host.ctypes.data), nh,
                                    None)
            host[:9] = [100, 40, 0, 1, 1, 0, 3, 20, 0]
            table = np.full((3, 6), -1, np.int32)
            table[0, :4], table[1, :2] = range(4), [4, 5]
            host[9:27] = table.reshape(-1)
            host[-1] = pages - 6
            c.n_comp, c.n_buf, c.n_blk = 100, 20, 1
            self.c.append(c)
            self.host.append(host)

    def refs(self):
        return ctypes.byref(self.c[0]), ctypes.byref(self.c[1])


def ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


A = 1 << 42   # a 16-byte aligned address


def test_norm_rope_refusals(gear):
    L, E = gear.lib, gear.gear
    good = dict(q=A, qs=256, Hq=2, k=A, ks=128, Hk=1, T=4, d=128, dt=0, qw=A, kw=None, eps=1e-6, pos=A, table=A,
                max_pos=8, rot=128, inter=0, qo=A + 4096, qos=256, ko=A + 8192, kos=128)

    def call(**kw):
        a = {**good, **kw}
        return L.gear_qk_norm_rope(*[a[n] for n in good], None)

    inv, uns = E.GEAR_ERR_INVALID_ARG, E.GEAR_ERR_UNSUPPORTED
    for bad in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(q=A + 2), dict(qo=A + 8), dict(qs=255),
                dict(qs=130), dict(ks=64), dict(qos=128), dict(T=-1), dict(Hq=-1), dict(Hq=0, Hk=0), dict(dt=3),
                dict(eps=-1.0), dict(eps=float("nan")), dict(pos=None), dict(table=None), dict(table=A + 4),
                dict(max_pos=0), dict(inter=2), dict(qw=A + 2), dict(kw=A + 8), dict(pos=A + 1),
                dict(qo=A, qos=512)):
        assert call(**bad) == inv, bad
    for bad in (dict(d=64), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(Hq=65535)):
        assert call(**bad) == uns, bad
    assert call(T=0, q=None, k=None, pos=None) == E.GEAR_OK


def test_append_refusals(gear):
    L, E = gear.lib, gear.gear
    pr = Pair(gear)
    before = [h.copy() for h in pr.host]
    k, v = pr.refs()
    good = dict(k=k, v=v, rows=ints(0, 1), counts=ints(2, 1), n=2, kn=A, ks=256, vn=A, vs=256, w=None, eps=1e-6, pos=A,
                table=A, max_pos=8, rot=128, inter=0, ws=A, wn=1 << 40)

    def call(**kw):
        a = {**good, **kw}
        return L.gear_append_rope_rows(*[a[n] for n in good], None)

    for bad in (dict(v=k), dict(rows=None), dict(rows=ints(0, 0)), dict(rows=ints(0, 3)), dict(rows=ints(0, 2)),
                dict(counts=None), dict(counts=ints(1, -1)), dict(n=0), dict(n=4), dict(kn=None), dict(vn=None),
                dict(kn=A + 2), dict(ks=255), dict(vs=128), dict(pos=None), dict(table=None), dict(w=A + 2),
                dict(counts=ints(2 ** 31 - 1, 2 ** 31 - 1)), dict(eps=float("inf"))):
        assert call(**bad) == E.GEAR_ERR_INVALID_ARG, bad
    assert call(rot=20) == E.GEAR_ERR_UNSUPPORTED
    assert call(ws=None, wn=0) == E.GEAR_ERR_WORKSPACE       # row 1's buffer is full: its flush needs scratch
    assert call(wn=1024) == E.GEAR_ERR_WORKSPACE
    assert call(counts=ints(100, 0)) == E.GEAR_ERR_CAPACITY  # five blocks, three are left
    assert call(counts=ints(0, 0), kn=None, pos=None) == E.GEAR_OK
    assert L.gear_append_rope_rows_workspace_bytes(k, ints(0), ints(17), 1) == 0     # fills the buffer exactly
    assert L.gear_append_rope_rows_workspace_bytes(k, ints(0), ints(18), 1) > 0
    assert L.gear_append_rope_rows_workspace_bytes(k, ints(3), ints(1), 1) == 0
    small = Pair(gear, pages=6)   # no free page: row 1 (2 pages, 64 tokens) takes one block of 20, not two
    ks, vs = small.refs()
    assert call(k=ks, v=vs, rows=ints(1), counts=ints(21), n=1) == E.GEAR_ERR_CAPACITY
    pr.host[1][6] += 1            # K and V no longer agree
    assert call() == E.GEAR_ERR_INVALID_ARG
    pr.host[1][6] -= 1
    assert all(np.array_equal(a, b) for a, b in zip(before, pr.host))


def test_truncate_refusals(gear):
    L, E = gear.lib, gear.gear
    pr = Pair(gear)
    before = [h.copy() for h in pr.host]
    k, v = pr.refs()
    for rows, counts, n in ((ints(0), ints(4), 1), (ints(1, 0), ints(20, 4), 2), (ints(2), ints(1), 1),
                            (ints(0), ints(-1), 1), (ints(0, 0), ints(1, 1), 2), (ints(5), ints(0), 1),
                            (None, ints(1), 1), (ints(0), None, 1)):
        assert L.gear_truncate_rows(k, v, rows, counts, n, None) == E.GEAR_ERR_INVALID_ARG
    assert L.gear_truncate_rows(k, k, ints(0), ints(1), 1, None) == E.GEAR_ERR_INVALID_ARG
    assert all(np.array_equal(a, b) for a, b in zip(before, pr.host))


def test_chunk_refusals(gear):
    L, E = gear.lib, gear.gear
    pr = Pair(gear)
    k, v = pr.refs()
    good = dict(k=k, v=v, rows=ints(0, 2), counts=ints(3, 2), n=2, q=A, qs=512, kn=A, ks=256, vn=A, vs=256, Hq=4,
                scale=0.1, plen=None, out=A, od=0, ws=A, wn=1 << 40)

    def call(**kw):
        a = {**good, **kw}
        return L.gear_chunk_attn(*[a[n] for n in good], None)

    for bad in (dict(rows=None), dict(rows=ints(0, 0)), dict(rows=ints(0, 3)), dict(counts=None),
                dict(counts=ints(1, -2)), dict(n=0), dict(q=None), dict(q=A + 2), dict(qs=511), dict(qs=256),
                dict(kn=None), dict(vn=None), dict(kn=A + 4), dict(vs=64), dict(Hq=0), dict(Hq=3),
                dict(scale=float("nan")), dict(out=None), dict(out=A + 2), dict(od=1), dict(plen=A + 2)):
        assert call(**bad) == E.GEAR_ERR_INVALID_ARG, bad
    assert call(Hq=2 * 129, qs=2 * 129 * 128) == E.GEAR_ERR_UNSUPPORTED
    need = L.gear_chunk_workspace_bytes(k, v, ints(0, 2), ints(3, 2), 2, 4, 1)
    assert need > 0
    for bad in (dict(ws=None), dict(ws=A + 16), dict(wn=need - 1)):
        assert call(**bad) == E.GEAR_ERR_WORKSPACE, bad
    assert call(counts=ints(0, 0), q=None, kn=None, vn=None, out=None) == E.GEAR_OK
    assert L.gear_chunk_workspace_bytes(k, v, ints(0, 0), ints(3, 2), 2, 4, 1) == 0
    # caches that do not belong together
    other = Pair(gear, bits=8)
    assert call(v=other.refs()[1]) == E.GEAR_ERR_INVALID_ARG
    p, c = gear.make_params(), gear.GearCacheStruct()
    nb = L.gear_cache_bytes(ctypes.byref(p), 3, 2, 128, 192, 4, 0)
    assert L.gear_cache_init(ctypes.byref(c), ctypes.byref(p), 3, 2, 128, 192, 4, 0, OUT(1 << 43), nb) == E.GEAR_OK
    assert call(v=ctypes.byref(c)) == E.GEAR_ERR_INVALID_ARG


def test_chunk_plan_covers_every_size(gear):
    """The scratch of a call grows with what it splits, and never needs 2^31 rows."""
    L = gear.lib
    pr = Pair(gear)
    k, v = pr.refs()
    sizes = [L.gear_chunk_workspace_bytes(k, v, ints(0), ints(n), 1, 4, 1) for n in (1, 2, 63, 64, 65, 1000, 5000)]
    assert all(s > 0 for s in sizes)
    assert L.gear_chunk_workspace_bytes(k, v, ints(0), ints(2 ** 29), 1, 4, 1) == 0


def test_chunk_too_many_tiles_is_refused(gear):
    """Millions of new tokens: units of row blocks times tiles of keys that 32 bits do not number."""
    L, E = gear.lib, gear.gear
    for dtype, n in ((0, 10_000_000), (2, 3_000_000)):
        pr = Pair(gear, dtype=dtype)
        k, v = pr.refs()
        assert L.gear_chunk_workspace_bytes(k, v, ints(0), ints(n), 1, 2, 1) == 0
        assert L.gear_chunk_workspace_bytes(k, v, ints(0), ints(n // 100), 1, 2, 1) > 0
        assert L.gear_chunk_attn(k, v, ints(0), ints(n), 1, A, 256, A, 256, A, 256, 2, 0.1, None, A, dtype, A, 1 << 62,
                                 None) == E.GEAR_ERR_UNSUPPORTED


def test_chunk_scratch_beside_short_rows(gear):
    """One long chunk, whose tiles are rebuilt ahead, in a call with many single tokens over long contexts: the
    scratch holds the tiles of 4096 x 96 tokens and heads at most, wherever in the call the long chunk comes."""
    L = gear.lib
    B, H, P, ppr = 96, 8, 256, 100
    p = gear.make_params()
    nb = L.gear_paged_cache_bytes(ctypes.byref(p), B, H, 128, P, B * ppr, ppr, 4, 0)
    nh = L.gear_paged_host_ints(B, ppr, B * ppr)
    caches, hosts = [], []
    for i in range(2):
        c, host = gear.GearCacheStruct(), np.zeros(nh, np.int32)
        L.gear_paged_cache_init(ctypes.byref(c), ctypes.byref(p), B, H, 128, P, B * ppr, ppr, 4, 0,
                                ctypes.c_void_p((1 << 40) + (i << 38)), nb, ctypes.c_void_p(host.ctypes.data), nh, None)
        host[:B], host[B:2 * B] = 21500, 1
        host[0] = 8192
        c.n_comp, c.n_buf, c.n_blk = 21500, 0, 1
        caches.append(c)
        hosts.append(host)
    k, v = (ctypes.byref(c) for c in caches)
    tile, parts = 64640, 148 * (2 * 256 * 132 * 4 + 32) + 512
    for at in (0, 50, 95):
        rows = [b for b in range(1, B)]
        rows.insert(at, 0)
        counts = [16384 if b == 0 else 1 for b in rows]
        got = L.gear_chunk_workspace_bytes(k, v, ints(*rows), ints(*counts), B, 8 * H, 1)
        assert 2048 * tile < got <= 4096 * tile + parts, (at, got)
    # one sequence alone may need more
    assert L.gear_chunk_workspace_bytes(k, v, ints(1), ints(40000), 1, 8 * H, 1) > 4096 * tile


def test_append_counts_near_2_31(gear):
    """A buffer's fill and a count that pass 2^31 together are too much for the row, like any other large count."""
    L, E = gear.lib, gear.gear
    for dtype in (0, 2):
        pr = Pair(gear, dtype=dtype)
        before = [h.copy() for h in pr.host]
        k, v = pr.refs()
        for rows, counts in ((ints(0), ints(2 ** 31 - 1)), (ints(1, 0), ints(0, 2 ** 31 - 2)), (ints(1), ints(2 ** 31 - 19))):
            st = L.gear_append_rope_rows(k, v, rows, counts, len(rows), A, 256, A, 256, None, 1e-6, None, None, 0, 0, 0, A,
                                         1 << 40, None)
            assert st == E.GEAR_ERR_CAPACITY
        assert all(np.array_equal(a, b) for a, b in zip(before, pr.host))
