"""Arguments of the paged cache path's calls that are taken or refused on the host (no GPU needed: the pointers are never
dereferenced)."""
import ctypes

import dflash_draft_selection_gb300 as d2

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
P = ctypes.c_void_p(4096)
CACHE = dict(k=4096, v=4096, weight=4096, pos=4096, num_pages=4, page_stride=2 * 16 * 64, head_stride=16 * 64,
             slot_stride=64, Hkv=2, page_size=16, d=64, dt=1)


def library():
    from dflash_draft_selection_gb300 import build
    build.build()
    return d2.load_library()


def record(**kw):
    from dflash_draft_selection_gb300.binding import _CacheRecord
    return _CacheRecord(**{**CACHE, **kw})


def append(cache=None, **kw):
    r = record(**(cache or {}))
    a = dict(cache=ctypes.byref(r), table=P, max_pages=4, kv_len=P, q_len=ctypes.c_void_p(8192),
             seq_pos=ctypes.c_void_p(12288), q=P, k=P, v=P, qs=256, ks=128, vs=128, B=2, T=2, Hq=4, cos_sin=P, n_pos=10,
             rot=64, pos_ids=P, axes=1, pair_axis=None, interleaved=0, q_norm=P, k_norm=P, eps=1e-6,
             q_out=ctypes.c_void_p(16384), kv_len_out=ctypes.c_void_p(512), stream=None)
    a.update(kw)
    return library().dflash2_rope_append(*a.values())


def attend(cache=None, **kw):
    r = record(**(cache or {}))
    a = dict(cache=ctypes.byref(r), table=P, max_pages=4, kv_len=P, q_len=P, seq_pos=P, q=P, B=2, T=2, Hq=4,
             scale=0.125, window=0, flags=1, out=ctypes.c_void_p(1024), lse=P, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return library().dflash2_paged_attn(*a.values())


def evict(cache=None, **kw):
    r = record(**(cache or {}))
    a = dict(cache=ctypes.byref(r), table=P, max_pages=4, kv_len=P, seq_len=P, B=2, budget=8, recent=0, sink=0, out=P,
             ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return library().dflash2_kv_evict(*a.values())


def test_an_empty_batch_has_no_table():
    for call in (append, attend, evict):
        assert call(B=0) == call(B=0, table=None) == call(B=0, max_pages=0) == call(B=0, table=None, max_pages=0) == OK
        assert call(B=0, max_pages=-1) == call(B=-1) == INVALID
        assert call(table=None) == call(max_pages=0) == INVALID
    for no in (dict(B=0), dict(T=0)):
        assert attend(q=None, out=None, lse=None, flags=3, **no) == OK
    assert attend(lse=None, flags=3) == INVALID


def test_a_call_of_more_places_than_31_bits_is_refused():
    """An item takes at most cap / 32 + 5 places of a call's line (a tile of 128 keys that is not full, and 4 beside)."""
    small = dict(Hkv=1, page_size=8)
    per = 8 / 32 + 5
    for dt in (0, 1):
        assert attend(dict(small, dt=dt), B=480_000_000, T=1, Hq=1, max_pages=1) == UNSUPPORTED
        assert attend(dict(small, dt=dt), B=int(2 ** 31 / per) + 1, T=1, Hq=1, max_pages=1) == UNSUPPORTED
        # one request less passes the guard, and is stopped by the next check
        assert attend(dict(small, dt=dt), B=int(2 ** 31 / per), T=1, Hq=1, max_pages=1, ws_bytes=0) == WORKSPACE


def test_appended_lengths_over_an_array_that_tokens_read_are_refused():
    for T in (0, 2):
        for n in ("kv_len", "q_len", "seq_pos"):
            p = ctypes.c_void_p(65536)
            assert append(T=T, kv_len_out=p, **{n: p}) == INVALID, n


def test_queries_turned_in_place_have_to_be_contiguous():
    p, q = ctypes.c_void_p(65536), ctypes.c_void_p(131072)
    assert append(q=p, q_out=p, qs=512) == INVALID           # slices of a fused projection
    assert append(k=q, q_out=q) == append(v=q, q_out=q) == INVALID


def test_more_heads_than_a_block_can_count_are_refused():
    big = dict(Hkv=1 << 24, page_size=1)
    assert attend(big, T=4, Hq=1 << 24, B=1, max_pages=1, ws_bytes=0) == UNSUPPORTED
    assert attend(dict(big, Hkv=(1 << 24) - 1), T=4, Hq=(1 << 24) - 1, B=1, max_pages=1, ws_bytes=0) == WORKSPACE


def test_appends_of_more_heads_than_31_bits_are_refused():
    for Hq, Hkv in ((2 ** 31 - 1, 1), (2, 2 ** 30)):
        assert append(dict(Hkv=Hkv, d=8, slot_stride=8), B=1, T=1, rot=8, Hq=Hq, qs=2 ** 40, ks=2 ** 40,
                      vs=2 ** 40) == UNSUPPORTED
