"""Calls of the 8-bit cache that its documentation allows beside those of test_gpu_cache.py: other streams
with buffers of the call's own, odd scales, requests that contradict themselves, waits that run out."""
import math

import numpy as np
import pytest

import oracle.cache as oc
import query_union_paged_b200 as qup
from test_gpu_cache import Case, _bf16, _check_attn, _ptr, _run_attn, _topk

pytestmark = pytest.mark.gpu


def _t():
    import torch
    return torch


# ------------------------------------------------------------------ buffers that the call makes

@pytest.mark.parametrize("n", [1, 20])  # the small kernel, and the chunk kernel
def test_buffers_of_a_call_on_another_stream_belong_to_it(monkeypatch, n):
    """A workspace or an output that cache_attn or cache_evict makes for a call on another stream is not memory
    that the current stream has in use or is handed next."""
    torch = _t()
    c = Case(91, [400, 300], T=64)
    cache, ptr = c.cache(), torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    _, q = _bf16(c.rng.standard_normal((2 * n, 8, 128)))
    want = qup.cache_attn(cache, q, ptr, n)
    w, acc = torch.rand(len(c.table), 2, device="cuda"), torch.rand(len(c.table), device="cuda")
    kept = qup.cache_evict(cache, w, acc, 3)
    torch.cuda.synchronize()
    made = []
    real = qup.cache_attn_workspace

    def recorded(*args, **kw):
        made.append(real(*args, **kw))
        return made[-1]
    monkeypatch.setattr(qup, "cache_attn_workspace", recorded)
    s = torch.cuda.Stream()
    free = [torch.empty_like(t) for t in (want, *kept)]  # blocks that the current stream may still have in use
    used = {t.data_ptr() for t in free}
    del free
    o = qup.cache_attn(cache, q, ptr, n, stream=s)
    assert o.data_ptr() not in used
    size, at = made[0].numel(), made[0].data_ptr()
    made.clear()
    assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != at
    out = qup.cache_evict(cache, w, acc, 3, stream=s)
    assert not used & {t.data_ptr() for t in out}
    torch.cuda.synchronize()
    assert torch.equal(o, want) and all(torch.equal(a, b) for a, b in zip(out, kept)) and qup.get_error() == 0


def test_two_streams_at_once_without_buffers_of_their_own():
    torch = _t()
    rng = np.random.default_rng(92)
    c = Case(92, [int(x) for x in rng.integers(1500, 3000, 12)], T=64)
    cache, ptr = c.cache(), torch.arange(13, dtype=torch.int32, device="cuda")
    q = [_bf16(rng.standard_normal((12, 8, 128)))[1] for _ in range(2)]
    want = [qup.cache_attn(cache, x, ptr, 1) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [qup.cache_attn(cache, x, ptr, 1, stream=s) for s, x in zip(streams, q)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert qup.get_error() == 0


# ------------------------------------------------------------------ scales

def test_zero_and_tiny_query_rows_over_negative_scales():
    """Rows of zeros (padding) and of tiny elements, whose score factor is next to nothing, where pages with a
    negative, a -0 and a subnormal negative K scale hold tokens that they do not see."""
    c = Case(93, [200, 90, 130], T=32)
    p0, p1, p2 = (c.table[a:] for a in c.page_ptr[:3])
    c.ks[p0[5]] *= -1          # request 0's queries are at 160 .. 199
    c.ks[p0[6]] = -0.0
    c.ks[p1[1]] = -1e-40       # request 1's at 50 .. 89
    c.ks[p1[2]] *= -1
    c.ks[p2[4]] *= -1e-20      # request 2's at 90 .. 129
    q = 1.5 * c.rng.standard_normal((120, 8, 128))
    q[[0, 5, 39, 40, 50, 79, 90, 119]] = 0
    q[7, 3], q[44, 6] = 0, 0
    q[[3, 60, 100]] *= 2.0 ** -112
    o, lse, w, ref = _run_attn(c, [40, 40, 40], 4, q=q)
    _check_attn(o, lse, w, ref, 200, "zero rows")


@pytest.mark.parametrize("n", [2, 20])
def test_v_scales_to_the_ends_of_their_range_and_past_them(n):
    """V scales of 2^-80 and 2^80 are read as they are; past them a page is reported and not seen."""
    torch = _t()
    for k in (-80, 80):
        c = Case(94 + k, [300, 70], T=64)
        c.vs[:] = 2.0 ** k
        o, lse, w, ref = _run_attn(c, [n, n], 4)
        _check_attn(o, lse, w, ref, 300, k)
    for bad in (2.0 ** -81, 1e-40, 2.0 ** 81, 3e38):
        c = Case(95, [300, 70], T=64)
        page = int(c.table[1])
        good = c.vs[page].copy()
        c.vs[page, 1] = bad
        _, qt = _bf16(q := _bf16(c.rng.standard_normal((2 * n, 8, 128)))[0])
        ptr = _ptr([n, n])
        lse = torch.empty(2 * n, 8, device="cuda")
        o = qup.cache_attn(c.cache(), qt, torch.from_numpy(ptr).cuda(), n, lse=lse)
        assert qup.get_error() == qup.ERR["SCALE"], bad
        c.vs[page] = good
        topk = np.broadcast_to(np.arange(5, dtype=np.int32), (8, 2 * n, 5)).copy()
        topk[4:, :n, 1] = -1  # request 0, KV head 1
        ref = oc.attn(q, c.K, c.V, c.ks, c.vs, c.table, c.page_ptr, c.lens, ptr, 1 / math.sqrt(128), topk)
        _check_attn(o.double().cpu().numpy(), lse.double().cpu().numpy(), None, ref, 300, bad)


@pytest.mark.parametrize("n", [2, 30])
@pytest.mark.parametrize("octaves", [16, 24, 30])
def test_a_page_whose_scale_an_unseen_token_made_large(n, octaves):
    """The header's bound where one page's V scale is far above the values that the row sees of it: each
    token may be off by 2^-33 * 448 * the largest V scale of the row's pages."""
    c = Case(96, [200, 150], T=64)
    for r in range(2):
        last = c.table[c.page_ptr[r] + (c.lens[r] - 1) // 64]
        c.vs[last] *= 2.0 ** octaves
        c.V[last, :, :(c.lens[r] - 1) % 64] = 0x01  # 2^-9 but for the last token, which the last query alone sees
    o, lse, w, ref = _run_attn(c, [n, n], 4)
    for r in range(2):
        top = c.vs[c.table[c.page_ptr[r]:c.page_ptr[r] + (c.lens[r] + 63) // 64]].max(axis=0)
        ref["vtop"][r * n:(r + 1) * n] = 448.0 * np.repeat(top, 4)
    _check_attn(o, lse, w, ref, 200, (n, octaves))


# ------------------------------------------------------------------ requests that contradict themselves

def _faulty(c, ns, max_q, bad, g=4, lens=None, cut=0, topk=None, max_pages=None, code="GROUP"):
    """Rows of the requests `bad` get O = 0 and lse = -inf, rows of no request are left alone, the others'
    results are the oracle's.  lens: kv_len on the device; cut: rows that Q has fewer than q_ptr says."""
    torch = _t()
    ptr = _ptr(ns)
    N = int(ptr[-1]) - cut
    qv, qt = _bf16(c.rng.standard_normal((int(ptr[-1]) + 2, 2 * g, 128)))
    rows = N + (0 if cut else 2)  # two rows of no request
    qt = qt[:rows].contiguous()
    kw = {} if max_pages is None else dict(max_pages=max_pages)
    cache = c.cache(**kw)
    if lens is not None:
        cache.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    o = torch.full((rows, 2 * g, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, 2 * g), 5.0, device="cuda")
    w = torch.full((len(c.table), 2), 5.0, device="cuda")
    tk = None
    if topk:
        tk = torch.arange(topk, dtype=torch.int32, device="cuda").expand(2 * g, rows, topk).contiguous()
    qup.cache_attn(cache, qt, torch.from_numpy(ptr).cuda(), max_q, topk=tk, out=o, lse=lse, page_weight=w)
    assert qup.get_error() == qup.ERR[code]
    sel = None if tk is None else tk.cpu().numpy()
    full = oc.attn(np.concatenate([qv, qv])[:int(ptr[-1])], c.K, c.V, c.ks, c.vs, c.table, c.page_ptr, c.lens, ptr,
                   1 / math.sqrt(128), None if sel is None else np.resize(sel[:, :1], (2 * g, int(ptr[-1]), topk)))
    og, lg, wg = o.double().cpu().numpy(), lse.double().cpu().numpy(), w.cpu().numpy()
    for r in range(len(ns)):
        a, b = int(ptr[r]), min(int(ptr[r + 1]), rows)
        pages = slice(int(c.page_ptr[r]), int(c.page_ptr[r + 1]))
        if r in bad:
            assert np.all(og[a:b] == 0) and np.all(np.isneginf(lg[a:b])), r
            assert np.all(wg[pages] == 0), r
        else:
            ref = {k: v[a:b] for k, v in full.items() if k != "weight"}
            _check_attn(og[a:b], lg[a:b], None, ref, int(c.lens[r]), r)
    if not cut:
        assert np.all(og[N:] == 5) and np.all(lg[N:] == 5)


@pytest.mark.parametrize("n,topk", [(1, None), (4, None), (40, None), (2, 3)])
def test_every_row_of_a_faulty_request_is_zero(n, topk):
    lens = [300, 200, 250, 190]
    case = lambda: Case(97, lens, T=64)
    _faulty(case(), [n, 3 * n + 1, n, n], n, [1], topk=topk)                   # more queries than max_q
    _faulty(case(), [n, n, n, n], n, [2], lens=[300, 200, 10 ** 6, 190], topk=topk)  # more tokens than pages
    _faulty(case(), [n, n, n, n + 1], n + 1, [3], cut=1, topk=topk)            # rows past the batch
    _faulty(Case(98, [300, 200, 700, 190], T=64), [n] * 4, n, [2], max_pages=6, topk=topk, code="CAPACITY")


def test_faulty_requests_among_small_and_large_ones():
    c = Case(99, [300, 400, 250, 190, 60, 600], T=64)
    _faulty(c, [2, 70, 30, 3, 1, 40], 40, [1, 4], lens=[300, 400, 250, 190, 10 ** 6, 600])
    c = Case(99, [300, 400, 250, 190, 60, 600], T=64)
    _faulty(c, [40, 3, 41, 4, 40, 2], 40, [2, 3], lens=[300, 400, 250, 10 ** 6, 60, 600])


def test_no_queries_of_any_request():
    """max_q = 0: a batch of nothing but padding rows; a request that has rows all the same is faulty."""
    torch = _t()
    c = Case(100, [100, 40], T=16)
    _, qt = _bf16(c.rng.standard_normal((3, 8, 128)))
    for topk in (None, torch.zeros(8, 3, 2, dtype=torch.int32, device="cuda")):
        o = torch.full((3, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        lse, w = torch.full((3, 8), 5.0, device="cuda"), torch.full((len(c.table), 2), 5.0, device="cuda")
        qup.cache_attn(c.cache(), qt, torch.zeros(3, dtype=torch.int32, device="cuda"), 0, topk=topk, out=o, lse=lse,
                       page_weight=w)
        assert qup.get_error() == 0 and torch.all(o == 5) and torch.all(lse == 5) and torch.all(w == 0)
        qup.cache_attn(c.cache(), qt, torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda"), 0, topk=topk, out=o,
                       lse=lse, page_weight=w)
        assert qup.get_error() == qup.ERR["GROUP"] and torch.all(o[:2] == 0) and torch.all(lse[:2] == -math.inf)
        assert torch.all(o[2] == 5) and torch.all(w == 0)


# ------------------------------------------------------------------ arguments

def test_a_long_page_table_of_short_requests_is_evicted():
    """Without max_pages a table longer than one request's limit is no error; a request past the limit is."""
    torch = _t()
    rng = np.random.default_rng(101)
    lens, pages = np.array([150, 90, 24600 * 16], np.int32), [12, 9, 24610]
    ptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    n = 30000
    table = rng.permutation(n).astype(np.int32)
    dev = lambda a: torch.from_numpy(a).cuda()
    kv = torch.zeros(1, 1, 16, 128, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, 1, device="cuda")
    make = lambda **kw: qup.KVCache(kv, kv, one, one, dev(table), dev(ptr), dev(lens), **kw)
    acc, w = rng.random(n).astype(np.float32), rng.random((n, 1)).astype(np.float32)
    got = qup.cache_evict(make(), dev(w), dev(acc), 4)
    assert qup.get_error() == qup.ERR["CAPACITY"]
    want = oc.evict(table, acc, w, ptr[:3], lens[:2], 16, 4, 1, 1, 1.0)
    m = int(ptr[2])
    for a, b in zip((got[0][:m], got[1][:m], got[2][:2], got[3][:m]), (want[0][:m], want[1][:m], want[2], want[3][:m])):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(got[0][m:ptr[3]].cpu().numpy(), table[m:ptr[3]]) and int(got[2][2]) == lens[2]
    with pytest.raises(qup.QupError):  # a limit that the caller gives is taken at its word
        qup.cache_evict(make(max_pages=n), dev(w), dev(acc), 4)


def test_numbers_past_32_bits_are_refused():
    torch = _t()
    c = Case(102, [100, 40], T=16)
    cache, n = c.cache(), len(c.table)
    _, qt = _bf16(c.rng.standard_normal((2, 8, 128)))
    ptr = torch.arange(3, dtype=torch.int32, device="cuda")
    w, acc = torch.rand(n, 2, device="cuda"), torch.rand(n, device="cuda")
    for big in (1 << 31, 1 << 32, (1 << 32) + 1, 1 << 63, -(1 << 32) + 1):
        for kw in (dict(budget=big), dict(sink=big), dict(recent=big)):
            with pytest.raises(ValueError):
                qup.cache_evict(cache, w, acc, **{**dict(budget=3), **kw})
        with pytest.raises(ValueError):
            qup.cache_attn(cache, qt, ptr, big)
        for sizes in ((big, 8, 1), (2, big, 1), (2, 8, big)):
            with pytest.raises(ValueError):
                qup.cache_attn_workspace(cache, *sizes)
    assert qup.get_error() == 0


# ------------------------------------------------------------------ waits that run out

@pytest.mark.parametrize("ns,topk", [([1, 1, 1], None), ([4, 4, 2], None), ([40, 40, 40], None), ([70, 1, 3], None),
                                     ([1, 1, 1], 6), ([2, 1, 1], 40)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(ns, topk):
    """One stage of every CTA is not loaded: the waits end at their limit, QUP_ERR_TIMEOUT is raised, the
    kernels leave and the next call gives the bits of an undisturbed one."""
    torch = _t()
    c = Case(103, [20000, 9000, 900], T=64)
    cache, ptr = c.cache(), torch.from_numpy(_ptr(ns)).cuda()
    _, q = _bf16(c.rng.standard_normal((sum(ns), 8, 128)))
    tk = None
    if topk:
        tk = torch.arange(topk, dtype=torch.int32, device="cuda").remainder(11).expand(8, sum(ns), topk).contiguous()
    w = [torch.empty(len(c.table), 2, device="cuda") for _ in range(2)]
    want = qup.cache_attn(cache, q, ptr, max(ns), topk=tk, page_weight=w[0])
    assert qup.get_error() == 0
    for stage in (0, 1) if topk is None else (0,):  # a CTA of these TopK calls has one stage
        try:
            qup.set_debug(wait_limit_ms=50, skip_stage=stage)
            qup.cache_attn(cache, q, ptr, max(ns), topk=tk, page_weight=w[1])
            code = qup.get_error()
        finally:
            qup.set_debug(0, -1)
        assert code == qup.ERR["TIMEOUT"], (stage, code)
        got = qup.cache_attn(cache, q, ptr, max(ns), topk=tk, page_weight=w[1])
        assert qup.get_error() == 0 and torch.equal(got, want) and torch.equal(w[0], w[1]), stage


# ------------------------------------------------------------------ page weights

@pytest.mark.parametrize("lens,ns,topk", [
    ([100, 900, 500], [40, 40, 40], False),                       # sums placed by pages, chunk kernel
    ([300, 300, 290], [90, 33, 20], False),                       # by rows
    ([500, 500, 500, 480], [1, 4, 1, 1], False),                  # by rows, small kernel
    ([1500, 90, 200, 40], [1, 1, 1, 1], False),                   # by pages
    ([1500, 90, 600, 1400, 33], [1, 70, 20, 2, 1], False),        # both kernels
    ([500, 490, 500], [1, 6, 1], True),                           # TopK: by rows
    ([700, 40, 500], [2, 2, 2], True),                            # and by pages
])
@pytest.mark.parametrize("T", [16, 64, 128])
def test_page_weights_stay_in_their_workspace(T, lens, ns, topk):
    """The smallest workspace that is reported, full of NaN, with a guard behind it: weights within their bound,
    the guard untouched, the same bits with a workspace for any call."""
    torch = _t()
    c = Case(110 + T, lens, T=T)
    g, N = 4, sum(ns)
    tk = _topk(c, ns, g, 5, c.rng) if topk else None
    o, lse, w, ref = _run_attn(c, ns, g, topk=tk, q=(q := 1.5 * c.rng.standard_normal((N, 8, 128))))
    _check_attn(o, lse, w, ref, max(lens), (T, ns))
    cache, ptr, qt = c.cache(), torch.from_numpy(_ptr(ns)).cuda(), _bf16(q)[1]
    for kind in (topk, True):
        size = qup.cache_attn_workspace(cache, N, 8, max(ns), page_weight=True, topk=kind).numel()
        buf = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
        again = torch.empty(len(c.table), 2, device="cuda")
        got = qup.cache_attn(cache, qt, ptr, max(ns), topk=None if tk is None else torch.from_numpy(tk).cuda(),
                             page_weight=again, workspace=buf[:size])
        assert qup.get_error() == 0 and torch.all(buf[size:] == 255)
        assert np.array_equal(again.double().cpu().numpy(), w) and np.array_equal(got.double().cpu().numpy(), o)
    small = qup.cache_attn_workspace(cache, N, 8, max(ns), page_weight=True, topk=topk)
    with pytest.raises(qup.QupError):
        qup.cache_attn(cache, qt, ptr, max(ns), topk=None if tk is None else torch.from_numpy(tk).cuda(),
                       page_weight=again, workspace=small[:4 << 20])  # less than the smallest of all


@pytest.mark.parametrize("n", [1, 20])
def test_small_weights_of_pages_of_zero_scale(n):
    """A page of zeros (V scale 0) whose softmax weight is next to nothing, before and behind the pages that carry the
    row: its weight is there down to what its exponentials can hold."""
    c = Case(130, [300, 290], T=32)
    for r in range(2):
        p = c.table[c.page_ptr[r]:]
        for x in (0, 4):
            c.vs[p[x]], c.V[p[x]], c.ks[p[x]] = 0.0, 0, 0.0  # scores of 0: a weight of 32 e^-lse
    o, lse, w, ref = _run_attn(c, [n, n], 4, qstd=14.0 if n == 1 else 17.0)
    small = ref["weight"][c.page_ptr[:2]]
    assert 2.0 ** -66 < small.min() < 2.0 ** -57 and small.max() < 2.0 ** -45
    _check_attn(o, lse, w, ref, 300, n)
