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
    n = ctypes.c_size_t(0)
    for w in (-1, 3):
        assert lib.qup_cache_attn_workspace(ctypes.byref(cache()), 5, 3, 32, w, ctypes.byref(n)) == ARG
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
