"""Host-side checks of the 8-bit cache's calls (no GPU)."""
from test_abi import _run_without_devices
from test_cache_oracle import _CACHE


def test_workspace_of_page_weights_follows_the_rows_and_pages_that_exist():
    _run_without_devices(_CACHE + """
    def size(w, T, R, pages, total, Nq, max_q, Hq=32):
        n = ctypes.c_size_t(0)
        c = cache(P_phys=total, T=T, R=R, total_pages=total, max_pages=pages)
        assert lib.qup_cache_attn_workspace(ctypes.byref(c), Nq, max_q, Hq, w, ctypes.byref(n)) == 0
        return n.value
    def extra(*a, w=2, **k):
        return size(w, *a, **k) - size(0, *a, **k)
    rows = lambda Nq, Hq=32: 4 * Nq * Hq + 1024  # the rows' lse, and rounding
    # one chunk of 1,024 queries behind 16K tokens: a sum for each row and page
    assert 8 * 1024 * 32 * 273 <= extra(64, 1, 273, 273, 1024, 1024) <= 8 * 1024 * 32 * 273 + rows(1024)
    # a chunk beside 63 single queries of 32K tokens: no request pays for the chunk's rows but itself
    got = extra(64, 64, 512, 64 * 512, 1087, 1024)
    assert got <= 8 * 1087 * 32 * 512 + 8 * 16 * 8 * 64 * 512 * 4 + rows(1087), got
    # six ragged prompts
    assert extra(128, 6, 129, 6 * 110, 83000, 16384) <= 8 * 83000 * 32 * 129 + 8 * 16 * 8 * 6 * 110 * 8 + rows(83000)
    # single queries: every 16 tokens of every page, whichever way it is asked for
    assert extra(64, 32, 128, 32 * 100, 32, 1) <= 8 * 32 * 4 * 32 * 100 + rows(32)
    # TopK calls fit what is reported for any call
    assert size(1, 64, 1, 273, 273, 1024, 1024) >= 4 * 8 * 1024 * 32 * 273
    for w in (-1, 3):  # any truth value but 2 asks for both kinds of call
        assert size(w, 64, 1, 273, 273, 1024, 1024) == size(1, 64, 1, 273, 273, 1024, 1024)
    # sizes whose product passes 64 bits
    assert size(1, 128, 1, 1 << 23, 1 << 30, 1 << 30, 1 << 27) >= 1 << 62
""")


def test_eviction_limit_is_the_headers():
    import os
    import re

    import query_union_paged_b200 as qup
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "query_union_paged.h")).read()
    assert int(re.search(r"#define QUP_CACHE_EVICT_PAGES (\d+)", text).group(1)) == qup.EVICT_PAGES


def test_outputs_over_inputs_or_each_other_are_refused():
    _run_without_devices(_CACHE + """
    V = ctypes.c_void_p
    ws = ctypes.c_size_t(0)
    c = cache(total_pages=30, R=3)
    lib.qup_cache_attn_workspace(ctypes.byref(c), 5, 3, 32, 0, ctypes.byref(ws))
    def attn(q, o, stride=4096, Nq=5):
        return lib.qup_cache_attn(ctypes.byref(c), V(q), stride, A[1], Nq, min(3, Nq), 32, 128, None, 0, 0.1, V(o), None,
                                  None, A[3], ws.value, None)
    q, row = 0x400000, 8192
    for o in (q, q + row, q + 4 * row, q + 5 * row - 16, q - row, q - 5 * row + 16, q + 16):
        assert attn(q, o) == ARG, o - q
    for o in (q + 5 * row, q - 5 * row):
        assert attn(q, o) == NODEV, o - q
    # Q as columns of a wider buffer of three rows' width: O may lie between two rows only where it fits
    wide = 3 * 4096
    for o in (q + 16, q + 2 * 3 * row, q + 4 * 3 * row, q + row, q - 5 * row + 16, q + 4 * 3 * row + row - 16):
        assert attn(q, o, wide) == ARG, o - q
    assert attn(q, q + row, wide, Nq=1) == NODEV and attn(q, q + 2 * row, wide, Nq=1) == NODEV
    assert attn(q, q + row, wide, Nq=2) == NODEV and attn(q, q + 2 * row, wide, Nq=2) == ARG
    assert attn(q, q + 4 * 3 * row + row, wide) == NODEV

    own = dict(table=c.page_table, acc=0x600000, lens=c.kv_len, src=0x700000, ptr=c.page_ptr, w=0x800000)
    def evict(table=0x610000, acc=0x620000, lens=0x630000, src=0x700000):
        return lib.qup_cache_evict(ctypes.byref(c), V(own["w"]), V(own["acc"]), 0.9, 8, 1, 1, V(table), V(acc), V(lens),
                                   V(src), None)
    assert evict() == NODEV
    assert evict(own["table"], own["acc"], own["lens"]) == NODEV  # in place
    for kw in (dict(table=own["acc"]), dict(acc=own["table"]), dict(src=own["table"]), dict(lens=own["ptr"]),
               dict(src=own["w"] + 956), dict(acc=own["w"]), dict(lens=own["table"]), dict(acc=own["acc"] + 4),
               dict(table=own["table"] + 8), dict(lens=own["lens"] - 8), dict(src=own["lens"]), dict(table=own["ptr"]),
               dict(table=0x700000), dict(acc=0x610000), dict(lens=0x700000 + 116), dict(acc=0x700000 - 116)):
        assert evict(**kw) == ARG, kw
    assert evict(src=own["w"] + 960) == NODEV and evict(acc=0x700000 - 120) == NODEV
    for kw in (dict(V=0x1000000), dict(v_scale=0x1020000)):
        bad = cache(**kw)
        assert bad.K == bad.V or bad.k_scale == bad.v_scale
        assert lib.qup_cache_append(ctypes.byref(bad), A[0], A[1], 1, 1024, 1024, A[2], 5, 128, None) == ARG, kw
""")
