"""The cache oracle pinned against torch's E4M3 conversion and hand-worked cases, and the host-side
refusals of the cache calls (no GPU)."""
import math

import numpy as np
import pytest

import oracle.cache as oc

from test_abi import _run_without_devices


def test_e4m3_table_and_rounding_match_torch():
    import torch
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oc.TABLE, want, equal_nan=True)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(4096) * np.exp2(rng.uniform(-12, 8, 4096)), want[np.isfinite(want)],
                        (want[:126] + want[1:127]) / 2, [0.0, -0.0, 448.0, -448.0]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    got = oc.encode(x)
    assert np.array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(oc.encode(np.array([np.inf, -np.inf, np.nan]))) == [127, 127, 127]


def test_page_scale_is_the_smallest_power_of_two():
    for a in (1e-30, 0.1, 447.9, 448.0, 448.1, 500.0, 896.0, 896.5, 3e38):
        s = oc.page_scale(a)
        assert a <= 448 * s and (s == 2.0 ** -64 or a > 448 * s / 2) and math.frexp(s)[0] == 0.5
    assert oc.page_scale(0.0) == 2.0 ** -64


def test_append_grows_the_scale_and_keeps_older_values():
    cache, scale = np.zeros((2, 1, 16, 128), np.uint8), np.zeros((2, 1), np.float32)
    small, big = np.full((1, 1, 128), 3.0), np.full((1, 1, 128), 900.0)
    table, pp = np.array([1]), np.array([0, 1])
    cache, scale = oc.append(cache, scale, small, table, pp, np.array([1]), np.array([0, 1]))
    assert scale[1, 0] == 2.0 ** -7 and np.all(oc.TABLE[cache[1, 0, 0]] == 384.0)
    cache, scale = oc.append(cache, scale, big, table, pp, np.array([2]), np.array([0, 1]))
    assert scale[1, 0] == 4.0 and np.all(oc.TABLE[cache[1, 0, 0]] == 0.75) and np.all(oc.TABLE[cache[1, 0, 1]] == 224.0)


def test_attention_of_one_and_of_equal_tokens():
    rng = np.random.default_rng(2)
    K, V = rng.integers(0, 100, (2, 1, 16, 128)).astype(np.uint8), rng.integers(0, 100, (2, 1, 16, 128)).astype(np.uint8)
    K[:] = K[0, 0, 0]  # equal keys: the mean of the values, lse = s + log n
    one = np.ones((2, 1), np.float32)
    q = rng.standard_normal((2, 1, 128))
    r = oc.attn(q, K, V, one, one, np.array([1, 0]), np.array([0, 2]), np.array([18]), np.array([0, 2]), 0.1)
    v = oc.TABLE[V[[1, 0], 0]].reshape(-1, 128)
    assert np.allclose(r["o"][0, 0], v[:17].mean(axis=0)) and np.allclose(r["o"][1, 0], v[:18].mean(axis=0))
    s = oc.TABLE[K[0, 0, 0]] @ q[0, 0] * 0.1
    assert np.isclose(r["lse"][0, 0], s + math.log(17))
    assert np.allclose(r["weight"][:, 0], [16 / 17 + 16 / 18, 1 / 17 + 2 / 18])


def test_eviction_by_hand():
    table = np.array([7, 3, 9, 4, 8, 1], np.int32)
    acc = np.array([0, 5, 1, 1, 2, 6], np.float32)
    w = np.zeros((6, 2), np.float32)
    w[4] = 0.25
    got = oc.evict(table, acc, w, np.array([0, 6]), np.array([70], np.int32), 16, 3, 1, 1, 1.0)
    # five used pages, budget 3: pages 2 and 3 (score 1, ties to the lower first) go; 0 and 4 are kept whatever
    assert list(got[3]) == [0, 1, 4, 2, 3, 5] and list(got[0]) == [7, 3, 8, 9, 4, 1]
    assert list(got[1]) == [0, 5, 2.5, 0, 0, 6] and got[2][0] == 70 - 32


_CACHE = """
    import ctypes
    import query_union_paged_b200 as qup
    qup.load()
    lib = qup._lib
    A = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(24)]
    def cache(**kw):
        f = dict(P_phys=40, Hkv=8, T=64, R=3, total_pages=30, max_pages=12)
        ptr = {k: 0x1000000 + 0x10000 * i for i, k in enumerate(("K", "V", "k_scale", "v_scale", "page_table",
                                                                   "page_ptr", "kv_len"))}
        f.update({k: v for k, v in kw.items() if k in f})
        ptr.update({k: v for k, v in kw.items() if k in ptr})
        return qup._CacheStruct(*[ptr[k] for k in ("K", "V", "k_scale", "v_scale", "page_table", "page_ptr", "kv_len")],
                                *[f[k] for k in ("P_phys", "Hkv", "T", "R", "total_pages", "max_pages")])
    BAD_CACHE = (dict(P_phys=0), dict(Hkv=0), dict(T=48), dict(T=256), dict(R=-1), dict(total_pages=0),
                 dict(max_pages=0), dict(max_pages=31), dict(total_pages=1 << 30, max_pages=1 << 25, T=128))
    ARG, CAP, NODEV = qup.ERR["ARG"], qup.ERR["CAPACITY"], qup.ERR["CUDA"]
"""


def test_append_refusals_before_any_device_work():
    _run_without_devices(_CACHE + """
    def call(ck={}, k=A[0], v=A[1], dtype=1, ks=1024, vs=1024, ptr=A[2], N=5, d=128):
        return lib.qup_cache_append(ctypes.byref(cache(**ck)), k, v, dtype, ks, vs, ptr, N, d, None)
    assert call() == NODEV
    for ck in BAD_CACHE + (dict(K=0), dict(v_scale=0), dict(page_table=0), dict(kv_len=0), dict(V=0x1000008)):
        assert call(ck) == ARG, ck
    for kw in (dict(k=None), dict(ptr=None), dict(dtype=2), dict(ks=1016), dict(vs=1028), dict(N=-1), dict(d=64),
               dict(k=ctypes.c_void_p(0x10008))):
        assert call(**kw) == ARG, kw
    assert call(dtype=0, ks=1028) == NODEV  # 16 bytes of fp32
    assert call(N=0) == 0 and call(dict(R=0)) == 0
    assert lib.qup_cache_append(None, A[0], A[1], 1, 1024, 1024, A[2], 5, 128, None) == ARG
""")


def test_attention_refusals_before_any_device_work():
    _run_without_devices(_CACHE + """
    ws = ctypes.c_size_t(0)
    def size(ck={}, Nq=5, max_q=3, Hq=32, w=0):
        return lib.qup_cache_attn_workspace(ctypes.byref(cache(**ck)), Nq, max_q, Hq, w, ctypes.byref(ws))
    assert size() == 0 and ws.value > 0
    plain = ws.value
    assert size(w=1) == 0 and ws.value > plain
    weighted = ws.value
    def call(ck={}, q=A[0], qs=4096, ptr=A[1], Nq=5, max_q=3, Hq=32, d=128, topk=None, K=0, sc=0.1, o=A[2], lse=None,
             w=None, wsp=A[3], n=plain):
        return lib.qup_cache_attn(ctypes.byref(cache(**ck)), q, qs, ptr, Nq, max_q, Hq, d, topk, K, sc, o, lse, w, wsp, n,
                                  None)
    assert call() == NODEV and call(topk=A[5], K=9) == NODEV
    for ck in BAD_CACHE:
        assert call(ck) == ARG and size(ck) == ARG, ck
    for kw in (dict(q=None), dict(qs=4088), dict(qs=4100), dict(ptr=None), dict(Nq=-1), dict(max_q=6), dict(Hq=30),
               dict(Hq=0), dict(d=64), dict(K=3), dict(topk=A[5], K=-1), dict(sc=0.0), dict(sc=float("nan")),
               dict(sc=float("inf")), dict(o=None), dict(wsp=None), dict(o=A[0]), dict(o=ctypes.c_void_p(0x20008)),
               dict(topk=A[5], K=9, Hq=8 * 33, qs=8 * 33 * 128), dict(ck=dict(kv_len=0))):
        assert call(**kw) == ARG, kw
    assert call(n=plain - 1) == CAP and call(w=A[6], n=plain) == CAP and call(w=A[6], n=weighted) == NODEV
    assert call(Nq=0, max_q=0) == 0
""")


def test_eviction_refusals_before_any_device_work():
    _run_without_devices(_CACHE + """
    def call(ck={}, w=A[0], acc=A[1], decay=0.9, budget=8, sink=1, recent=1, outs=A[2:6]):
        return lib.qup_cache_evict(ctypes.byref(cache(**ck)), w, acc, decay, budget, sink, recent, *outs, None)
    assert call() == NODEV
    for ck in BAD_CACHE + (dict(total_pages=30000, max_pages=24577),):
        assert call(ck) == ARG, ck
    for kw in (dict(w=None), dict(acc=None), dict(decay=float("nan")), dict(budget=0), dict(sink=-1), dict(recent=0),
               dict(outs=[None] + A[3:6]), dict(outs=A[2:5] + [None])):
        assert call(**kw) == ARG, kw
    assert call(dict(R=0)) == 0
""")


def test_python_refusals():
    import torch

    import query_union_paged_b200 as qup
    z = torch.zeros
    good = dict(K=z(4, 2, 16, 128, dtype=torch.uint8), V=z(4, 2, 16, 128, dtype=torch.uint8), k_scale=z(4, 2),
                v_scale=z(4, 2), page_table=z(6, dtype=torch.int32), page_ptr=z(3, dtype=torch.int32),
                kv_len=z(2, dtype=torch.int32))
    for bad in (dict(K=z(4, 2, 16, 64, dtype=torch.uint8)), dict(K=z(4, 2, 16, 128)), dict(V=z(4, 2, 32, 128, dtype=torch.uint8)),
                dict(k_scale=z(2)), dict(v_scale=z(4, 2, dtype=torch.float64)), dict(page_table=z(6, dtype=torch.int64)),
                dict(page_ptr=z(2, dtype=torch.int32)), dict(kv_len=z(4, dtype=torch.int32)[::2]), dict(max_pages=7),
                dict(max_pages=0), dict(V=z(4, 2, 16, 256, dtype=torch.uint8)[..., ::2]),
                dict(k_scale=z(4, 2, device="meta"))):
        with pytest.raises(ValueError):
            qup.KVCache(**{**good, **bad})
    with pytest.raises(ValueError, match="CUDA"):
        qup.KVCache(**good)


def test_quartic_exponential_is_the_fit_and_within_its_bound():
    import importlib.util
    import os
    import re

    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "query_union_paged_b200", "csrc")
    m = re.search(r"kExp2Q1 = ([0-9.]+)f, kExp2Q2 = ([0-9.]+)f, kExp2Q3 = ([0-9.]+)f, kExp2Q4 = ([0-9.]+)f",
                  open(os.path.join(csrc, "ptx.cuh")).read())
    have = [np.float32(x) for x in m.groups()]
    spec = importlib.util.spec_from_file_location("fit_exp2_poly", os.path.join(csrc, "fit_exp2_poly.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    coef, err = mod.fit(4)
    # coefficients of a nearly flat optimum move by more than their effect: compare what they evaluate to
    f = np.linspace(-0.5, 0.5, 20001)
    poly = lambda c: 1 + f * (c[0] + f * (c[1] + f * (c[2] + f * c[3])))
    assert np.abs(poly([float(x) for x in have]) / poly(coef) - 1).max() < 2e-7
    assert err < 2.9e-6 and mod.fp32_error(have) < 3.1e-6  # fp32 evaluation adds at most 3 steps of 2^-24
