"""The 8-bit page-scaled cache on the GPU against the fp64 oracle: append and eviction bit for bit,
attention within bounds derived from its roundings, and the three in a serving loop.

Attention bounds (per element, E = 2^-24 the fp32 half step):
  scores  128 products summed in fp32 in some order, truncated sums counted as a whole step each:
          |ds| <= 2 * 128 * E * sum|q||k| = 2^-16 smag  (smag: the largest such sum of the row, scaled)
  weights a factor 1 + d with |d| <= 2^-11 (P rounded to fp16) + 2^-18 (exponentials, the running sum's
          rescalings, log2 of the V scale) + 2 |ds|, and below fp16's normal range at most 2^-25 where the
          row's largest is at least 2^8: 2^-33 of the largest |v| for each token
  O       those against sum p|v|, and bf16's half step 2^-8 of |O|
  scores of requests with more than 16 rows: Q's low part is within 2^-17 of the row's largest element
          where that is coarser than its last bit, so |ds| grows by 2^-17 max|q| sum|k|, which is at most
          2^-17 * (sum|q||k| max|q| sum|k| / sum|q||k|); the oracle returns qk = max|q| sum|k| (scaled)
  lse     |ds| + 2^-18 + E |lse| + E * tokens (the sum of weights, in order)
  page weights  a relative 2 |ds| + 2^-17 + 2 E * tokens, and what is flushed: a token's exponential is
          p = 2^(x - m + 8), x = log2(e) s + log2 vs (a scale of 0 counts as 2^-64), and lost below 2^-126.  Its
          weight is p / vs * 2^(m - 8 - lse'), with lse' the row's lse in base 2.  m is at most the largest x,
          so at most lse' + log2 of the head's largest scale: a token loses less than
          2^-134 vs_max / vs, a page that for each of its tokens and the request's rows
"""
import math

import numpy as np
import pytest

import oracle.cache as oc
import query_union_paged_b200 as qup

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def _t():
    import torch
    return torch


def _bf16(x):
    """float64 -> (the bf16 values, their tensor on the GPU)"""
    torch = _t()
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


class Case:
    """A seeded cache of requests with these lengths; pages shuffled over a larger physical cache, slots
    past each sequence's end filled with NaN bytes."""

    def __init__(self, seed, lens, Hkv=2, T=64, spare=1, spread=2.0, fill_tail=0x7F):
        rng = self.rng = np.random.default_rng(seed)
        self.T, self.Hkv, self.lens = T, Hkv, np.array(lens, np.int32)
        pages = [-(-n // T) + spare for n in lens]
        self.page_ptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        total = max(int(self.page_ptr[-1]), 1)
        P = total + 3
        self.table = rng.permutation(P)[:total].astype(np.int32)
        self.K, self.ks = self._values(P, spread)
        self.V, self.vs = self._values(P, spread)
        self.max_pages = max(max(pages, default=1), 1)
        for r, n in enumerate(lens):
            if n % T and fill_tail is not None:
                p = self.table[self.page_ptr[r] + n // T]
                self.K[p, :, n % T:] = fill_tail
                self.V[p, :, n % T:] = fill_tail

    def _values(self, P, spread):
        x = self.rng.standard_normal((P, self.Hkv, self.T, 128)) * np.exp2(
            spread * (self.rng.random((P, self.Hkv, 1, 1)) - 0.5))
        s = np.exp2(np.ceil(np.log2(np.abs(x).max(axis=(2, 3)) / 448)))
        return oc.encode(x / s[:, :, None, None]), s.astype(np.float32)

    def cache(self, **kw):
        torch = _t()
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        return qup.KVCache(dev(self.K), dev(self.V), dev(self.ks), dev(self.vs), dev(self.table), dev(self.page_ptr),
                           dev(self.lens), max_pages=kw.pop("max_pages", self.max_pages))


def _same(got, want, what=""):
    """Equal bit for bit (NaN equal to NaN); a failure names the first differences only."""
    got = got.cpu().numpy() if hasattr(got, "cpu") else got
    diff = ~((got == want) | ((got != got) & (want != want)))
    n = int(diff.sum())
    first = [(tuple(int(x) for x in i), got[tuple(i)].item(), want[tuple(i)].item()) for i in np.argwhere(diff)[:4]]
    assert n == 0, (what, n, first)


def _ptr(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def _check_attn(got, lse, weight, ref, tokens, what, p_round=2.0 ** -11):
    ds = 2.0 ** -16 * ref["smag"] + 2.0 ** -17 * ref["qk"]
    rel = p_round + 2.0 ** -18 + 2 * ds
    tol = 2.0 ** -8 * np.abs(ref["o"]) + rel[..., None] * ref["vmag"] + (tokens * 2.0 ** -33 * ref["vtop"])[..., None]
    err = np.abs(got - ref["o"])
    assert np.all(err <= tol * (1 + 2.0 ** -8)), (what, float((err - tol).max()), np.argwhere(err > tol)[:4])
    if lse is not None:
        fin = np.isfinite(ref["lse"])
        assert np.array_equal(np.isneginf(lse), np.isneginf(ref["lse"])), what
        lt = ds + 2.0 ** -18 + E * np.abs(np.where(fin, ref["lse"], 0)) + E * tokens
        le = np.abs(np.where(fin, lse, 0) - np.where(fin, ref["lse"], 0))
        assert np.all(le <= lt), (what, float((le - lt).max()))
    if weight is not None:
        wt = ref["weight"] * (2 * ds.max() + 2.0 ** -17 + 2 * E * tokens) + ref.get("flushed", 0.0) + 1e-30
        we = np.abs(weight - ref["weight"])
        assert np.all(we <= wt), (what, float((we - wt).max()))


def _run_attn(c, ns, g, topk=None, weights=True, scale=None, qstd=1.5, max_q=None, cache=None, q=None):
    torch = _t()
    ns = np.asarray(ns)
    ptr = _ptr(ns)
    Hq = c.Hkv * g
    N = int(ptr[-1])
    if q is None:
        q = qstd * c.rng.standard_normal((N, Hq, 128))
    qv, qt = _bf16(q)
    scale = 1 / math.sqrt(128) if scale is None else scale
    cache = c.cache() if cache is None else cache
    lse = torch.full((N, Hq), 7.0, device="cuda")
    w = torch.full((len(c.table), c.Hkv), 7.0, device="cuda") if weights else None
    tk = None if topk is None else torch.from_numpy(topk).cuda()
    o = qup.cache_attn(cache, qt, torch.from_numpy(ptr).cuda(), int(max_q or max(ns)), topk=tk, softmax_scale=scale,
                       lse=lse, page_weight=w)
    torch.cuda.synchronize()
    assert qup.get_error() == 0
    ref = oc.attn(qv, c.K, c.V, c.ks, c.vs, c.table, c.page_ptr, c.lens, ptr, scale, topk)
    vs = np.maximum(np.abs(c.vs[c.table].astype(np.float64)), 2.0 ** -64)
    ref["flushed"] = 2.0 ** -134 * c.T * max(ns) * g * vs.max(axis=0) / vs
    return (o.double().cpu().numpy(), lse.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), ref)


def _topk(c, ns, g, K, rng, dup=False):
    """Random pages for each query head and query, -1 padded; the query's own page among them."""
    N, Hq = int(sum(ns)), c.Hkv * g
    t = np.full((Hq, N, K), -1, np.int32)
    row = 0
    for r, n in enumerate(ns):
        for i in range(n):
            pos = c.lens[r] - n + i
            for h in range(Hq):
                have = max(pos // c.T + 1, 1)
                k = min(int(rng.integers(1, K + 1)), have)
                s = rng.permutation(have)[:k]
                t[h, row, :k] = s
                if dup and k < K:
                    t[h, row, k] = s[0]
            row += 1
    return t


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_matches_the_oracle_bit_for_bit(T, dtype):
    torch = _t()
    rng = np.random.default_rng(T)
    lens, ns = [1, 5, 64, 200, 333, T, T + 1, 2 * T, 130], [1, 3, 64, 137, 0, T, 1, T, 1]
    c = Case(T + 1, lens, Hkv=3, T=T)
    ptr = _ptr(ns)
    N = int(ptr[-1]) + 2  # rows behind the last request's
    new = [rng.standard_normal((N, 3, 128)) * np.exp2(rng.uniform(-8, 8, (N, 3, 1))) for _ in range(2)]
    new[0][3] = 0.0
    new[1][4, 1, 5], new[1][4, 2, 6], new[0][7, 0, 0] = np.inf, np.nan, -np.inf
    tt = torch.bfloat16 if dtype == "bf16" else torch.float32
    dev = [torch.from_numpy(x.astype(np.float32)).to(tt).cuda() for x in new]
    vals = [d.double().cpu().numpy() for d in dev]
    if T == 32:  # one projection's rows: K and V side by side
        both = torch.cat([d.reshape(N, -1) for d in dev], dim=1)
        dev = [both[:, :384].unflatten(1, (3, 128)), both[:, 384:].unflatten(1, (3, 128))]
    cache = c.cache()
    qup.cache_append(cache, dev[0], dev[1], torch.from_numpy(ptr).cuda())
    torch.cuda.synchronize()
    assert qup.get_error() == 0
    for got, gs, old, os_, x in ((cache.K, cache.k_scale, c.K, c.ks, vals[0]), (cache.V, cache.v_scale, c.V, c.vs, vals[1])):
        want, ws = oc.append(old, os_, x, c.table, c.page_ptr, c.lens, ptr)
        _same(gs, ws)
        _same(got, want)


def test_append_one_token_at_a_time_fills_pages():
    torch = _t()
    rng = np.random.default_rng(5)
    c = Case(6, [40, 40], Hkv=2, T=16, fill_tail=None)
    cache = c.cache()
    x = rng.standard_normal((40, 2, 2, 128)) * np.exp2(rng.uniform(-3, 3, (40, 2, 1, 1)))
    K, ks = c.K, c.ks
    ptr = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for t in range(40):
        vals, dev = _bf16(x[t])
        lens = np.array([t + 1, t + 1], np.int32)
        cache.kv_len.copy_(torch.from_numpy(lens))
        qup.cache_append(cache, dev, dev, ptr)
        K, ks = oc.append(K, ks, vals, c.table, c.page_ptr, lens, np.array([0, 1, 2]))
    torch.cuda.synchronize()
    assert qup.get_error() == 0
    _same(cache.K, K)
    _same(cache.k_scale, ks)


def test_append_reports_bad_requests_and_pages_and_writes_the_rest():
    torch = _t()
    c = Case(8, [20, 30, 40, 52], Hkv=1, T=16)
    c.table[c.page_ptr[1] + 1] = 999          # request 1's second page is out of range
    c.ks[c.table[c.page_ptr[3] + 3], 0] = -1  # request 3's last page, which holds older tokens
    c.lens[2] = 1                             # fewer tokens than are appended
    cache = c.cache()
    vals, dev = _bf16(np.random.default_rng(1).standard_normal((4 * 2, 1, 128)))
    ptr = np.array([0, 2, 4, 6, 8], np.int32)
    qup.cache_append(cache, dev, dev, torch.from_numpy(ptr).cuda())
    code = qup.get_error()
    assert code == qup.ERR["PHYS_PAGE"] | qup.ERR["GROUP"] | qup.ERR["SCALE"]
    only = np.array([0, 2, 2, 2, 2])
    want, ws = oc.append(c.K, c.ks, vals, c.table, c.page_ptr, c.lens, only)
    _same(cache.K, want)
    _same(cache.k_scale, ws)


# ------------------------------------------------------------------ attention over all pages

@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("g", [1, 4, 7, 16])
def test_decode_matches_the_oracle(T, g):
    c = Case(100 * T + g, [1, 2, 63, 64, 65, 300, T, T + 1, 700], T=T)
    o, lse, w, ref = _run_attn(c, [1] * 9, g)
    _check_attn(o, lse, w, ref, 700, (T, g))


@pytest.mark.parametrize("T,g,n", [(16, 7, 5), (64, 4, 4), (32, 8, 3), (128, 5, 13), (64, 32, 1), (16, 40, 2)])
def test_short_runs_match_the_oracle(T, g, n):
    c = Case(7 * T + g, [n, n + 1, 63, 64 + n, 500], T=T)
    o, lse, w, ref = _run_attn(c, [n, n, 1, n, max(1, n - 1)], g)
    _check_attn(o, lse, w, ref, 500, (T, g, n))


@pytest.mark.parametrize("T,g,n,L", [(64, 4, 100, 400), (16, 3, 77, 77), (32, 8, 65, 1000), (128, 1, 200, 260),
                                     (64, 40, 30, 190), (16, 8, 33, 900)])
def test_chunks_match_the_oracle(T, g, n, L):
    c = Case(T + n, [L, L - 3, n // 2], T=T)
    o, lse, w, ref = _run_attn(c, [n, n - 5, n // 2], g, weights=False)
    _check_attn(o, lse, None, ref, L, (T, g, n))


def test_page_weights_of_a_chunk():
    c = Case(77, [300, 180], T=32)
    o, lse, w, ref = _run_attn(c, [90, 33], 4)
    _check_attn(o, lse, w, ref, 300, "chunk weights")


def test_many_requests_and_long_ones_share_the_grid():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 200, 70)] + [9000, 3, 5001]
    c = Case(9, lens, Hkv=1, T=64)
    o, lse, w, ref = _run_attn(c, [1] * len(lens), 4)
    _check_attn(o, lse, w, ref, 9000, "mixed lengths")


def test_requests_without_tokens_or_rows_and_rows_of_no_request():
    torch = _t()
    c = Case(12, [0, 40, 0, 100, 17], T=16)
    ns = [0, 1, 2, 0, 1]  # request 2 has rows and no tokens: they see nothing
    ptr = _ptr(ns)
    N = int(ptr[-1])
    qv, qt = _bf16(c.rng.standard_normal((N + 3, 4, 128)))
    o = torch.full((N + 3, 4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N + 3, 4), 5.0, device="cuda")
    w = torch.full((len(c.table), 2), 5.0, device="cuda")
    qup.cache_attn(c.cache(), qt, torch.from_numpy(ptr).cuda(), 2, out=o, lse=lse, page_weight=w)
    assert qup.get_error() == 0
    ref = oc.attn(qv[:N], c.K, c.V, c.ks, c.vs, c.table, c.page_ptr, c.lens, ptr, 1 / math.sqrt(128))
    assert torch.all(o[N:] == 5) and torch.all(lse[N:] == 5)
    _check_attn(o[:N].double().cpu().numpy(), lse[:N].double().cpu().numpy(), w.double().cpu().numpy(), ref, 100, "empty")
    assert np.all(o[1:3].float().cpu().numpy() == 0) and np.all(np.isneginf(lse[1:3].cpu().numpy()))


def test_more_queries_than_tokens_see_nothing():
    c = Case(13, [3, 20], T=16)
    o, lse, w, ref = _run_attn(c, [5, 5], 2)
    _check_attn(o, lse, w, ref, 20, "n > len")
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:2]))


@pytest.mark.parametrize("qstd,scale", [(40.0, None), (1e-3, None), (3.0, 1.0), (1.5, 1e-6)])
def test_peaked_and_flat_softmax(qstd, scale):
    c = Case(14, [513, 64], T=64, spread=6.0)
    o, lse, w, ref = _run_attn(c, [3, 1], 4, qstd=qstd, scale=scale)
    _check_attn(o, lse, w, ref, 513, (qstd, scale))


@pytest.mark.parametrize("T", [16, 64, 128])
@pytest.mark.parametrize("g,n", [(8, 5), (8, 20), (8, 40)])
def test_rows_of_every_width_peaked_and_with_odd_scales(T, g, n):
    """40, 160 and 320 rows: one row tile split over both warpgroups (pages of up to 64), one, and two."""
    c = Case(T + n, [700, 129 + n, n + 3], T=T, spread=6.0)
    p = c.table[:c.page_ptr[1]]
    c.vs[p[1]], c.V[p[1]], c.ks[p[2]] = 0.0, 0, 0.0
    c.ks[p[3]] = -c.ks[p[3]]
    c.vs[p[4]] *= 1.37 * 2.0 ** 12
    o, lse, w, ref = _run_attn(c, [n, n, n], g, qstd=12.0)
    _check_attn(o, lse, w, ref, 700, (T, g, n))


def test_pages_of_zero_scale_and_of_far_apart_scales():
    c = Case(15, [300], T=16)
    p = c.table[:19]
    c.vs[p[2]], c.V[p[2]] = 0.0, 0
    c.ks[p[3]] = 0.0
    c.vs[p[4]] *= 2.0 ** 20
    c.vs[p[5]] *= 2.0 ** -20
    c.ks[p[6]] = -c.ks[p[6]]
    c.ks[p[7]] *= 1.37  # a scale need not be a power of two
    c.vs[p[8]] *= 1.37
    o, lse, w, ref = _run_attn(c, [2], 4)
    # fp16 weights below 2^-14 of the offset range: 2^-33 of the largest value times the token count
    _check_attn(o, lse, w, ref, 300, "scales")


def test_nan_tokens_reach_only_the_rows_that_see_them():
    c = Case(16, [100, 100], T=16)
    c.V[c.table[c.page_ptr[0] + 6], 0, 1, 9] = 0x7F  # request 0, token 97: seen by its last three queries
    c.K[c.table[c.page_ptr[1] + 6], 1, 2, 0] = 0xFF  # request 1, token 98
    o, lse, w, ref = _run_attn(c, [5, 5], 4, weights=False)
    nan_o, want = np.isnan(o), np.isnan(ref["o"])
    assert np.array_equal(nan_o, want) and want.any()
    assert np.array_equal(np.isnan(lse), np.isnan(ref["lse"]))
    ok = ~want.any(axis=2)
    for k in ("o", "lse", "smag", "vmag", "vtop", "qk"):
        ref[k] = ref[k][ok]
    _check_attn(o[ok], lse[ok], None, ref, 100, "beside NaN")


def test_nan_tokens_of_a_chunk_reach_only_the_rows_that_see_them():
    c = Case(18, [300, 200, 260], T=32)
    c.V[c.table[c.page_ptr[0] + 7], 0, 5, 9] = 0x7F   # request 0, token 229
    c.V[c.table[c.page_ptr[0] + 8], 0, 0, 70] = 0xFF  # and 256, another column
    c.K[c.table[c.page_ptr[1] + 5], 1, 2, 0] = 0xFF   # request 1, token 162
    o, lse, w, ref = _run_attn(c, [90, 60, 40], 4, weights=False)
    want = np.isnan(ref["o"])
    assert np.array_equal(np.isnan(o), want) and want.any()
    assert np.array_equal(np.isnan(lse), np.isnan(ref["lse"]))
    ok = ~want.any(axis=2)
    for k in ("o", "lse", "smag", "vmag", "vtop", "qk"):
        ref[k] = ref[k][ok]
    _check_attn(o[ok], lse[ok], None, ref, 300, "beside NaN")


def test_small_and_large_requests_in_one_batch():
    c = Case(19, [500, 90, 700, 0, 33, 1200, 256], T=64)
    ns = [1, 90, 40, 0, 3, 1, 256]
    o, lse, w, ref = _run_attn(c, ns, 4)
    _check_attn(o, lse, w, ref, 1200, "mixed rows")


def test_many_requests_of_a_few_rows_share_the_grid():
    rng = np.random.default_rng(21)
    lens = [int(x) for x in rng.integers(5, 260, 170)] + [2000]
    c = Case(21, lens, T=32)
    o, lse, w, ref = _run_attn(c, [5] * len(lens), 5)
    _check_attn(o, lse, w, ref, 2000, "few rows")
    # and a few of more than one row tile between them
    ns = [40 if r % 9 == 4 and lens[r] > 40 else 4 for r in range(len(lens))]
    o, lse, w, ref = _run_attn(c, ns, 5)
    _check_attn(o, lse, w, ref, 2000, "few and more rows")


def test_bad_pages_scales_and_lengths_in_chunks():
    torch = _t()
    c = Case(20, [300, 300, 300, 300], T=64)
    p = [c.table[c.page_ptr[r]:c.page_ptr[r + 1]] for r in range(4)]
    bad = [int(c.page_ptr[0]) + 1, int(p[1][2]), int(c.page_ptr[3])]
    ns = [40, 40, 40, 40]
    ptr = _ptr(ns)
    qv, qt = _bf16(c.rng.standard_normal((160, 8, 128)))
    good = oc.attn(qv, c.K, c.V, c.ks, c.vs, c.table, c.page_ptr, c.lens, ptr, 1 / math.sqrt(128))
    c.table[bad[0]] = -7
    c.vs[bad[1]] = np.nan
    c.lens[3] = 10 ** 7
    o = qup.cache_attn(c.cache(), qt, torch.from_numpy(ptr).cuda(), 40)
    assert qup.get_error() == qup.ERR["PHYS_PAGE"] | qup.ERR["SCALE"] | qup.ERR["GROUP"]
    assert torch.isfinite(o).all() and torch.all(o[120:] == 0)
    ref = {k: v[80:120] for k, v in good.items() if k != "weight"}
    _check_attn(o[80:120].double().cpu().numpy(), None, None, ref, 300, "the good request")
    # the pages that are not seen: the oracle over the others
    c.lens[3] = 300
    sel = np.array([[0, 2, 3, 4], [0, 1, 3, 4], [0, 1, 2, 3], [-1, -1, -1, -1]])
    topk = np.broadcast_to(np.repeat(sel, 40, axis=0), (8, 160, 4)).astype(np.int32)
    c.table[bad[0]] = 0
    c.vs[bad[1]] = 1
    part = oc.attn(qv, c.K, c.V, c.ks, c.vs, c.table, c.page_ptr, c.lens, ptr, 1 / math.sqrt(128), topk)
    ref = {k: v[:80] for k, v in part.items() if k != "weight"}
    _check_attn(o[:80].double().cpu().numpy(), None, None, ref, 300, "pages not seen")


def test_query_with_infinite_elements_gives_nan_and_leaves_others():
    c = Case(17, [90], T=32)
    q = c.rng.standard_normal((2, 8, 128))
    q[0, 3, 5] = np.inf
    q[1, 1, 7] = np.nan
    o, lse, w, ref = _run_attn(c, [2], 4, weights=False, q=q)
    bad = np.zeros((2, 8), bool)
    bad[0, 3] = bad[1, 1] = True
    assert np.isnan(o[bad]).all()
    for k in ("o", "lse", "smag", "vmag", "vtop", "qk"):
        ref[k] = ref[k][~bad]
    _check_attn(o[~bad], lse[~bad], None, ref, 90, "beside inf")


# ------------------------------------------------------------------ attention over TopK pages

@pytest.mark.parametrize("T,g,K,ns", [(16, 4, 9, [1, 1, 1]), (64, 8, 5, [1, 2, 1]), (128, 3, 3, [2, 1, 3]),
                                      (32, 16, 12, [1, 1, 1]), (64, 32, 4, [1, 1, 2]), (64, 1, 1, [1, 1, 1])])
def test_topk_pages_match_the_oracle(T, g, K, ns):
    c = Case(T + g + K, [5, 700, 1500], T=T)
    topk = _topk(c, ns, g, K, c.rng, dup=True)
    topk[0, 0, :] = -1  # a row that selects nothing
    o, lse, w, ref = _run_attn(c, ns, g, topk=topk)
    _check_attn(o, lse, w, ref, 1500, (T, g, K))


def test_topk_of_no_entries_sees_nothing_and_output_in_place_of_q_is_refused():
    torch = _t()
    c = Case(32, [40, 300], T=16)
    _, qt = _bf16(c.rng.standard_normal((2, 8, 128)))
    ptr = torch.arange(3, dtype=torch.int32, device="cuda")
    lse = torch.zeros(2, 8, device="cuda")
    w = torch.full((len(c.table), 2), 3.0, device="cuda")
    o = qup.cache_attn(c.cache(), qt, ptr, 1, topk=torch.empty(8, 2, 0, dtype=torch.int32, device="cuda"), lse=lse,
                       page_weight=w)
    assert torch.all(o == 0) and torch.all(lse == -math.inf) and torch.all(w == 0) and qup.get_error() == 0
    with pytest.raises(qup.QupError):
        qup.cache_attn(c.cache(), qt, ptr, 1, out=qt)


def test_topk_of_many_queries_and_pages_behind_the_query():
    c = Case(31, [400, 300], T=16)
    ns = [60, 45]
    topk = _topk(c, ns, 4, 6, c.rng)
    topk[:, :5, 1] = 24  # request 0's last page: invisible to its first queries
    o, lse, w, ref = _run_attn(c, ns, 4, topk=topk)
    _check_attn(o, lse, w, ref, 400, "chunk topk")


def test_bad_pages_lengths_and_ids_are_reported_and_not_seen():
    torch = _t()
    c = Case(41, [100, 100, 100, 100], T=16)
    good = c.table.copy()
    c.table[c.page_ptr[0] + 2] = 10 ** 6
    c.table[c.page_ptr[1] + 3] = -1
    cache = c.cache()
    q, qt = _bf16(c.rng.standard_normal((4, 4, 128)))
    ptr = torch.arange(5, dtype=torch.int32, device="cuda")
    o = qup.cache_attn(cache, qt, ptr, 1)
    assert qup.get_error() == qup.ERR["PHYS_PAGE"]
    full = oc.attn(q, c.K, c.V, c.ks, c.vs, good, c.page_ptr, c.lens, np.arange(5), 1 / math.sqrt(128))
    _check_attn(o[2:].double().cpu().numpy(), None, None, {k: v[2:] for k, v in full.items() if k != "weight"}, 100, "others")
    assert torch.isfinite(o).all()
    # page IDs outside the request
    c.table[:] = good
    cache = c.cache()
    topk = torch.tensor([0, 3, 7, 8], dtype=torch.int32, device="cuda").expand(4, 4, 4).contiguous()
    topk[:, 1, 2] = -5
    o = qup.cache_attn(cache, qt, ptr, 1, topk=topk)
    assert qup.get_error() == qup.ERR["PAGE_ID"]
    sel = topk.cpu().numpy().copy()
    sel[(sel > 7) | (sel < 0)] = -1
    ref = oc.attn(q, c.K, c.V, c.ks, c.vs, good, c.page_ptr, c.lens, np.arange(5), 1 / math.sqrt(128), sel)
    _check_attn(o.double().cpu().numpy(), None, None, ref, 100, "ids")
    # a length past the request's pages, rows past the batch, more queries and more pages than declared
    cache.kv_len[1] = 10 ** 6
    o = qup.cache_attn(cache, qt, ptr, 1)
    assert qup.get_error() == qup.ERR["GROUP"] and torch.all(o[1] == 0)
    cache.kv_len[1] = 100
    o = qup.cache_attn(cache, qt, torch.tensor([0, 2, 3, 3, 4], dtype=torch.int32, device="cuda"), 1)
    assert qup.get_error() == qup.ERR["GROUP"]
    qup.cache_attn(cache, qt, torch.tensor([0, 1, 2, 3, 9], dtype=torch.int32, device="cuda"), 1)
    assert qup.get_error() == qup.ERR["GROUP"]
    o = qup.cache_attn(c.cache(max_pages=7), qt, ptr, 1)
    assert qup.get_error() == qup.ERR["CAPACITY"] and torch.all(o == 0)
    # scales
    cache.v_scale[int(good[c.page_ptr[2]]), 0] = -1
    cache.k_scale[int(good[c.page_ptr[3]]), 1] = math.inf
    o = qup.cache_attn(cache, qt, ptr, 1)
    assert qup.get_error() == qup.ERR["SCALE"] and torch.isfinite(o).all()


def test_strided_queries_and_given_outputs():
    torch = _t()
    c = Case(51, [130, 77], T=64)
    q = c.rng.standard_normal((2, 8, 128))
    qv, qt = _bf16(q)
    wide = torch.zeros(2, 3 * 8 * 128, dtype=torch.bfloat16, device="cuda")
    wide[:, :1024] = qt.reshape(2, -1)
    view = wide[:, :1024].unflatten(1, (8, 128))
    ptr = torch.arange(3, dtype=torch.int32, device="cuda")
    cache = c.cache()
    a = qup.cache_attn(cache, view, ptr, 1)
    b = qup.cache_attn(cache, qt, ptr, 1, out=torch.empty_like(qt), workspace=qup.cache_attn_workspace(cache, 2, 8, 1))
    assert torch.equal(a, b)
    for bad in (dict(out=torch.empty(2, 8, 128, device="cuda")), dict(lse=torch.empty(2, 4, device="cuda")),
                dict(page_weight=torch.empty(3, 2, device="cuda")), dict(topk=torch.zeros(8, 2, 4, device="cuda")),
                dict(workspace=torch.empty(64, device="cuda"))):
        with pytest.raises(ValueError):
            qup.cache_attn(cache, qt, ptr, 1, **bad)
    with pytest.raises(ValueError):
        qup.cache_attn(cache, qt.float(), ptr, 1)
    with pytest.raises(ValueError):
        qup.cache_attn(cache, qt.cpu(), ptr, 1)
    with pytest.raises(qup.QupError):
        qup.cache_attn(cache, qt, ptr, 1, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_same_bits_every_run_on_two_streams_at_once_and_in_graphs():
    torch = _t()
    rng = np.random.default_rng(61)
    lens = [int(x) for x in rng.integers(100, 3000, 12)]
    c = Case(61, lens, T=64)
    cache = c.cache()
    q = [_bf16(rng.standard_normal((12, 8, 128)))[1] for _ in range(2)]
    ptr = torch.arange(13, dtype=torch.int32, device="cuda")
    first = [qup.cache_attn(cache, x, ptr, 1) for x in q]
    torch.cuda.synchronize()
    streams, ws = [torch.cuda.Stream() for _ in q], [qup.cache_attn_workspace(cache, 12, 8, 1) for _ in q]
    outs = [torch.empty_like(x) for x in q]
    for _ in range(20):
        for s, x, o, w in zip(streams, q, outs, ws):
            qup.cache_attn(cache, x, ptr, 1, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    graphs = []
    for s, x, o, w in zip(streams, q, outs, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qup.cache_attn(cache, x, ptr, 1, out=o, workspace=w)
        graphs.append(g)
    # lengths and contents change between replays: the graph reads them on the device
    cache.kv_len.copy_(cache.kv_len // 2)
    want = [qup.cache_attn(cache, x, ptr, 1) for x in q]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs)) and qup.get_error() == 0


def test_a_step_of_all_calls_in_one_graph_and_chunks_on_two_streams():
    """Append, chunk attention with page weights and eviction captured together and replayed on changed
    contents; two chunk calls at the same time give the bits of one alone."""
    torch = _t()
    c = Case(62, [300, 150, 220], T=32, Hkv=2, fill_tail=None)
    ns, g = [70, 30, 3], 4
    ptr = torch.from_numpy(_ptr(ns)).cuda()
    cache, ref = c.cache(), c.cache()
    N = sum(ns)
    k, v = (torch.empty(N, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.empty(N, 8, 128, dtype=torch.bfloat16, device="cuda")
    n = len(c.table)

    def step(cache, o, w, acc, out, ws):
        qup.cache_append(cache, k, v, ptr)
        qup.cache_attn(cache, q, ptr, 70, out=o, page_weight=w, workspace=ws)
        qup.cache_evict(cache, w, acc, 4, decay=0.5, out=out)

    def buffers(cache):
        return (torch.empty_like(q), torch.empty(n, 2, device="cuda"), torch.zeros(n, device="cuda"),
                (torch.empty_like(cache.page_table), torch.empty(n, device="cuda"), torch.empty_like(cache.kv_len),
                 torch.empty_like(cache.page_table)), qup.cache_attn_workspace(cache, N, 8, 70, page_weight=True))

    gen = torch.Generator("cuda").manual_seed(5)
    fill = lambda: [t.copy_(torch.randn(t.shape, generator=gen, device="cuda")) for t in (k, v, q)]
    fill()
    a, b = buffers(cache), buffers(ref)
    step(cache, *a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, *a)
    for _ in range(2):
        fill()
        cache.K.copy_(ref.K), cache.V.copy_(ref.V), cache.k_scale.copy_(ref.k_scale), cache.v_scale.copy_(ref.v_scale)
        graph.replay()
        step(ref, *b)
        torch.cuda.synchronize()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(x, y) for x, y in zip(a[3], b[3]))
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    ws = [qup.cache_attn_workspace(ref, N, 8, 70) for _ in range(2)]
    want = qup.cache_attn(ref, q, ptr, 70)
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, x in zip(streams, outs, ws):
            qup.cache_attn(ref, q, ptr, 70, out=o, workspace=x, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and qup.get_error() == 0


# ------------------------------------------------------------------ eviction

@pytest.mark.parametrize("budget,sink,recent,decay", [(5, 1, 2, 0.9), (1, 0, 1, 1.0), (3, 4, 4, 0.0), (100, 1, 1, 0.5),
                                                      (20, 0, 3, -1.0)])
def test_eviction_matches_the_oracle_bit_for_bit(budget, sink, recent, decay):
    torch = _t()
    rng = np.random.default_rng(budget)
    lens = [0, 1, 16, 17, 100, 333, 16 * 600, 16 * 45 + 3]
    c = Case(71, lens, Hkv=3, T=16, spare=2)
    n = len(c.table)
    acc, w = rng.random(n).astype(np.float32), np.exp(rng.standard_normal((n, 3))).astype(np.float32)
    acc[::7] = 0.25
    w[::7] = 0.5  # ties
    acc[30], w[31, 1], acc[32] = np.nan, np.inf, 1e-42
    at, wt = torch.from_numpy(acc).cuda(), torch.from_numpy(w).cuda()
    cache = c.cache()
    got = qup.cache_evict(cache, wt, at, budget, sink=sink, recent=recent, decay=decay)
    d32 = float(np.float32(decay))
    want = oc.evict(c.table, acc, w, c.page_ptr, c.lens, 16, budget, sink, recent, d32)
    again = (cache.page_table, at, cache.kv_len, torch.empty_like(cache.page_table))
    qup.cache_evict(cache, wt, at, budget, sink=sink, recent=recent, decay=decay, out=again)  # in place
    assert qup.get_error() == 0
    for res in (got, again):
        for a, b in zip(res, want):
            _same(a, b)


def test_eviction_leaves_bad_requests_unchanged():
    torch = _t()
    c = Case(72, [100, 200, 150], Hkv=1, T=16)
    c.lens[1] = 10 ** 6
    n = len(c.table)
    acc, w = torch.rand(n, device="cuda"), torch.rand(n, 1, device="cuda")
    out = qup.cache_evict(c.cache(), w, acc, 2)
    assert qup.get_error() == qup.ERR["GROUP"]
    a, b = int(c.page_ptr[1]), int(c.page_ptr[2])
    _same(out[0][a:b], c.table[a:b])
    assert torch.equal(out[1][a:b], acc[a:b])
    assert out[2].tolist() == [100 - 5 * 16, 10 ** 6, 150 - 8 * 16]


# ------------------------------------------------------------------ the three together

def test_serving_loop_append_attend_evict():
    """Prompts are appended as a chunk and attended, then tokens one at a time with page weights; every
    eight steps the cache is evicted in place.  Every step's cache, outputs and tables match the oracle."""
    torch = _t()
    rng = np.random.default_rng(81)
    T, Hkv, g, R = 16, 2, 4, 3
    prompts = [70, 33, 101]
    c = Case(81, [p + 40 for p in prompts], Hkv=Hkv, T=T, fill_tail=None)
    cache = c.cache()
    K, V, ks, vs, table = c.K, c.V, c.ks, c.vs, c.table.copy()
    lens = np.array(prompts, np.int32)
    n_pages = len(table)
    acc, acc_ref = torch.zeros(n_pages, device="cuda"), np.zeros(n_pages, np.float32)
    w = torch.empty(n_pages, Hkv, device="cuda")
    src = torch.empty(n_pages, dtype=torch.int32, device="cuda")
    for step in range(25):
        ns = np.array(prompts if step == 0 else [1] * R)
        if step:
            lens = lens + 1
        ptr = _ptr(ns)
        kv, kt = _bf16(rng.standard_normal((ptr[-1], Hkv, 128)) * np.exp2(rng.uniform(-2, 2)))
        vv, vt = _bf16(rng.standard_normal((ptr[-1], Hkv, 128)))
        qv, qt = _bf16(rng.standard_normal((ptr[-1], Hkv * g, 128)))
        cache.kv_len.copy_(torch.from_numpy(lens))
        ptr_t = torch.from_numpy(ptr).cuda()
        qup.cache_append(cache, kt, vt, ptr_t)
        lse = torch.empty(int(ptr[-1]), Hkv * g, device="cuda")
        o = qup.cache_attn(cache, qt, ptr_t, int(ns.max()), lse=lse, page_weight=w)
        K, ks = oc.append(K, ks, kv, table, c.page_ptr, lens, ptr)
        V, vs = oc.append(V, vs, vv, table, c.page_ptr, lens, ptr)
        _same(cache.K, K)
        _same(cache.V, V)
        ref = oc.attn(qv, K, V, ks, vs, table, c.page_ptr, lens, ptr, 1 / math.sqrt(128))
        wd = w.cpu().numpy()
        _check_attn(o.double().cpu().numpy(), lse.double().cpu().numpy(), wd.astype(np.float64), ref, 150, step)
        if step % 8 == 7:
            qup.cache_evict(cache, w, acc, 5, recent=2, decay=0.5, out=(cache.page_table, acc, cache.kv_len, src))
            # the device's own weights decide: they are compared above
            table, acc_ref, lens, sref = oc.evict(table, acc_ref, wd, c.page_ptr, lens, T, 5, 1, 2, 0.5)
            for a, b in ((cache.page_table, table), (cache.kv_len, lens), (acc, acc_ref), (src, sref)):
                _same(a, b)
    assert qup.get_error() == 0
