"""Cases of the 8-bit page-scaled cache operators: writing tokens into the cache, attention that
reads it (single tokens, short runs, chunks, TopK pages), and eviction of its pages by accumulated
attention weight.

Cache layout: K, V [P_phys][Hkv][T][128] E4M3 bytes, k_scale and v_scale [P_phys][Hkv] fp32; request r
owns the logical pages page_table[page_ptr[r] .. page_ptr[r+1]) and holds kv_len[r] tokens, the new
ones included.  Queries (or new tokens) of request r are the batch rows ptr[r] .. ptr[r+1), at its last
positions.
"""
import math

import torch

own = False

D = 128
E4 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: every sequence writes one token into its last page
        dict(name="append 64 x 1", op="append", requests=64, n=1, ctx=8192, ragged=True, hkv=8, page=64, dtype="bf16"),
        # six prompts' tokens, 10K to 16K each, as a chunked prefill writes them
        dict(name="append 6 prompts", op="append", requests=6, n=16384, ctx=16384, ragged=True, hkv=8, page=128,
             dtype="bf16"),
        # short ragged runs behind older tokens, fp32 projections, small pages, an odd head count
        dict(name="append ragged fp32", op="append", requests=9, n=300, ctx=1201, ragged=True, hkv=5, page=16,
             dtype="fp32"),
        # one user, a short context: latency
        dict(name="decode 1 x 1000", op="attn", requests=1, n=1, ctx=1000, ragged=False, hq=32, hkv=8, page=64, topk=0,
             weights=False),
        # an ordinary decode batch, page weights kept for eviction
        dict(name="decode 32 x 8K weights", op="attn", requests=32, n=1, ctx=8192, ragged=True, hq=32, hkv=8, page=64,
             topk=0, weights=True),
        # long contexts: the largest read of the cache
        dict(name="decode 16 x 64K", op="attn", requests=16, n=1, ctx=65536, ragged=True, hq=32, hkv=8, page=128, topk=0,
             weights=False),
        # sparse decode: 32 selected pages of 64 tokens for each sequence and KV head
        dict(name="decode 32 x 32K top 32", op="attn", requests=32, n=1, ctx=32768, ragged=True, hq=32, hkv=8, page=64,
             topk=32, weights=False),
        # several drafted tokens verified at once, 7 query heads per KV head, 16-token pages, odd lengths
        dict(name="verify 24 x 5 g7", op="attn", requests=24, n=5, ctx=6001, ragged=True, hq=28, hkv=4, page=16, topk=0,
             weights=True),
        # one prompt's chunk behind a 16K prefix
        dict(name="chunk 1024 of 17K", op="attn", requests=1, n=1024, ctx=17408, ragged=False, hq=32, hkv=8, page=64,
             topk=0, weights=False),
        # ragged short prompts in one batch
        dict(name="chunks 6 ragged", op="attn", requests=6, n=700, ctx=4001, ragged=True, hq=16, hkv=2, page=32, topk=0,
             weights=False),
        # a few sequences over their budget
        dict(name="evict 8 x 130", op="evict", requests=8, ctx=130 * 64 - 5, ragged=True, hkv=8, page=64, keep=0.75),
        # a full server's batch
        dict(name="evict 256 x 1024", op="evict", requests=256, ctx=65536, ragged=True, hkv=8, page=64, keep=0.9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "evict"])
    c = dict(op=op, requests=_log(rng, 1, 64), ragged=rng.random() < 0.7, hkv=rng.choice([1, 2, 3, 4, 8]),
             page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        c.update(n=1 if rng.random() < 0.4 else _log(rng, 2, 4096), dtype=rng.choice(["bf16", "bf16", "fp32"]))
        c["requests"] = max(1, min(c["requests"], 65536 // c["n"]))
        c["ctx"] = c["n"] + _log(rng, 1, 4096)
    elif op == "evict":
        c.update(ctx=_log(rng, 200, 65536), keep=rng.choice([0.5, 0.75, 0.9, 1.0]))
    else:
        g = rng.choice([1, 2, 4, 5, 7, 8, 16])
        kind = rng.choice(["decode", "decode", "verify", "topk", "chunk"])
        n = {"decode": 1, "verify": rng.randint(2, max(2, 64 // g)), "topk": rng.choice([1, 1, 2, 3]),
             "chunk": _log(rng, 65, 1024)}[kind]
        c.update(hq=g * c["hkv"], n=n, topk=_log(rng, 4, 64) if kind == "topk" else 0,
                 weights=kind != "chunk" and n * g <= 64 and rng.random() < 0.4)
        # rows x tokens bounded by the largest listed chunk, tokens by the largest listed batch
        ctx = _log(rng, 1, 65536)
        ctx = min(ctx, 8388608 // (c["requests"] * c["hkv"]), 536870912 // (c["requests"] * n * c["hq"]))
        c["ctx"] = max(n, ctx, 1)
    return c


# ------------------------------------------------------------------ inputs

def _ns(c):
    """Queries or new tokens of each request."""
    n = c.get("n", 0)
    return [n if r == 0 or not c["ragged"] or n < 4 else n - (r * 40503) % (3 * n // 8 + 1) for r in range(c["requests"])]


def _lens(c):
    """Tokens of each request's cache, the new ones included."""
    L, ns = c["ctx"], _ns(c)
    return [max(ns[r], L if r == 0 or not c["ragged"] else L - (r * 2654435761) % (L // 2 + 1), 1)
            for r in range(c["requests"])]


def _ptr(counts, dev):
    p = [0]
    for x in counts:
        p.append(p[-1] + x)
    return torch.tensor(p, dtype=torch.int32, device=dev)


def _pages(c):
    """Page table entries of each request: its pages and one to grow into."""
    return [-(-x // c["page"]) + 1 for x in _lens(c)]


def _tables(c, gen, dev):
    pages = _pages(c)
    total = sum(pages)
    phys = total + 3
    table = torch.randperm(phys, generator=gen, device=dev)[:total].to(torch.int32)
    return dict(page_table=table, page_ptr=_ptr(pages, dev),
                kv_len=torch.tensor(_lens(c), dtype=torch.int32, device=dev), max_pages=max(pages)), total, phys


def _bytes(x):
    return x.to(E4).view(torch.uint8)


def _fill(c, phys, gen, dev, spread):
    """One cache tensor and its scales: N(0, 1) times a factor per page and head (spread octaves),
    scaled by a power of two so that the page's largest value fits E4M3."""
    hkv, T = c["hkv"], c["page"]
    out = torch.empty(phys, hkv, T, D, dtype=torch.uint8, device=dev)
    scale = torch.empty(phys, hkv, dtype=torch.float32, device=dev)
    step = max(1, (1 << 27) // (hkv * T * D))
    for p in range(0, phys, step):
        x = torch.randn(min(step, phys - p), hkv, T, D, generator=gen, device=dev)
        x *= torch.exp2(spread * (torch.rand(x.shape[0], hkv, 1, 1, generator=gen, device=dev) - 0.5))
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(2, 3)) / 448.0)))
        out[p:p + step] = _bytes(x / s[:, :, None, None])
        scale[p:p + step] = s
    return out, scale


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c = case
    s, total, phys = _tables(c, gen, dev)
    s["case"] = dict(c)
    if c["op"] == "evict":
        s["K"] = s["V"] = torch.zeros(phys, c["hkv"], c["page"], D, dtype=torch.uint8, device=dev)
        s["k_scale"] = s["v_scale"] = torch.ones(phys, c["hkv"], device=dev)
        # attention mass per page: a few heavy pages and a long tail, as softmax weights have
        s["weight"] = torch.exp(2.5 * torch.randn(total, c["hkv"], generator=gen, device=dev) - 6.0)
        s["acc"] = torch.exp(2.0 * torch.randn(total, generator=gen, device=dev) - 3.0)
        s["budget"] = max(3, int(c["keep"] * (-(-c["ctx"] // c["page"]))))
        s["sink"], s["recent"], s["decay"] = 1, 2, 0.96875
        return s
    s["K"], s["k_scale"] = _fill(c, phys, gen, dev, 2.0)
    s["V"], s["v_scale"] = _fill(c, phys, gen, dev, 3.0)
    ns = _ns(c)
    s["ptr"] = _ptr(ns, dev)
    N = sum(ns)
    if c["op"] == "append":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        # channels of different size, as projections have
        ch = torch.exp2(torch.randn(c["hkv"], D, generator=gen, device=dev))
        s["k_new"] = (torch.randn(N, c["hkv"], D, generator=gen, device=dev) * ch).to(dt)
        s["v_new"] = (torch.randn(N, c["hkv"], D, generator=gen, device=dev) * ch).to(dt)
        return s
    # bytes behind a sequence's last token are whatever the memory held: NaN among them
    lens, T = s["kv_len"].long(), c["page"]
    last = s["page_table"].long()[s["page_ptr"][:-1].long() + (lens - 1) // T]
    dead = torch.arange(T, device=dev)[None, :] > ((lens - 1) % T)[:, None]
    for name in ("K", "V"):
        tail = s[name][last]
        s[name][last] = torch.where(dead[:, None, :, None], torch.full_like(tail, 0x7F), tail)
    s["q"] = (1.5 * torch.randn(N, c["hq"], D, generator=gen, device=dev)).to(torch.bfloat16)
    s["max_q"] = max(ns)
    s["scale"] = 1.0 / math.sqrt(D)
    s["topk"] = None
    if c["topk"]:
        # the own page and distinct earlier ones for each KV head, the same for its query heads;
        # -1 where a sequence has fewer pages
        req = torch.repeat_interleave(torch.arange(c["requests"], device=dev), torch.tensor(ns, device=dev))
        pos = (lens - (s["ptr"][1:] - s["ptr"][:-1]).long())[req] + torch.arange(N, device=dev) - s["ptr"].long()[req]
        mp = s["max_pages"]
        key = torch.rand(c["hkv"], N, mp, generator=gen, device=dev)
        page = torch.arange(mp, device=dev)
        key = torch.where(page == (pos // T)[:, None], torch.full_like(key, 2.0), key)
        key = torch.where(page > (pos // T)[:, None], torch.full_like(key, -1.0), key)
        k = min(c["topk"], mp)
        val, idx = key.topk(k, dim=2)
        sel = torch.where(val >= 0, idx, torch.full_like(idx, -1)).to(torch.int32)
        if k < c["topk"]:
            sel = torch.nn.functional.pad(sel, (0, c["topk"] - k), value=-1)
        s["topk"] = sel.repeat_interleave(c["hq"] // c["hkv"], dim=0).contiguous()
    return s


# ------------------------------------------------------------------ the plain forms

def _positions(s, N):
    """Request and position of each batch row."""
    i = torch.arange(N, device=s["ptr"].device)
    ptr = s["ptr"].long()
    req = torch.searchsorted(ptr, i, right=True) - 1
    n = ptr[1:] - ptr[:-1]
    return req, s["kv_len"].long()[req] - n[req] + i - ptr[req]


def _pow2_scale(amax):
    """The smallest 2^k (k >= -64) with amax <= 448 * 2^k."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [1/2, 1)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    k = torch.where(amax > 0, k, torch.full_like(k, -64)).clamp(min=-64)
    return torch.ldexp(torch.ones_like(amax), k)


def _append_one(cache, scale, new, phys, slot, first_phys, first_slot):
    x = new.float()
    P, hkv, T, _ = cache.shape
    amax = torch.zeros(P, hkv, device=x.device)
    amax.scatter_reduce_(0, phys[:, None].expand(-1, hkv), x.abs().amax(dim=2), "amax")
    touched = torch.zeros(P, dtype=torch.bool, device=x.device)
    touched[phys] = True
    older = torch.zeros(P, dtype=torch.int64, device=x.device)
    older[first_phys] = first_slot
    s_new = _pow2_scale(amax)
    s_new = torch.where(older[:, None] > 0, torch.maximum(s_new, scale), s_new)
    s_new = torch.where(touched[:, None], s_new, scale)
    old = cache[first_phys]
    again = _bytes(old.view(E4).float() * (scale / s_new)[first_phys][:, :, None, None])
    keep = torch.arange(T, device=x.device) < first_slot[:, None]
    grown = (s_new != scale)[first_phys]
    cache[first_phys] = torch.where(keep[:, None, :, None] & grown[:, :, None, None], again, old)
    cache[phys, :, slot] = _bytes(x / s_new[phys][:, :, None])
    scale.copy_(s_new)


def _append_plain(s):
    req, pos = _positions(s, s["k_new"].shape[0])
    T = s["K"].shape[2]
    phys = s["page_table"].long()[s["page_ptr"].long()[req] + pos // T]
    first = s["ptr"].long()[:-1]
    for cache, scale, new in ((s["K"], s["k_scale"], s["k_new"]), (s["V"], s["v_scale"], s["v_new"])):
        _append_one(cache, scale, new, phys, pos % T, phys[first], (pos % T)[first])


def _values(cache, scale, phys):
    """The values of whole pages, fp32."""
    return cache[phys].view(E4).float() * scale[phys][..., None, None]


def _attn_dense(s):
    c, q = s["case"], s["q"]
    R, hkv, T, mp, n = c["requests"], c["hkv"], c["page"], s["max_pages"], s["max_q"]
    g = c["hq"] // hkv
    dev = q.device
    lens, ptr, pptr = s["kv_len"].long(), s["ptr"].long(), s["page_ptr"].long()
    at = torch.minimum(pptr[:-1, None] + torch.arange(mp, device=dev), pptr[1:, None] - 1)
    phys = s["page_table"].long()[at]
    tok = torch.arange(mp * T, device=dev)
    here = tok < lens[:, None]                                                       # [R, L]
    k = _values(s["K"], s["k_scale"], phys).permute(0, 2, 1, 3, 4).reshape(R, hkv, mp * T, D)
    counts = ptr[1:] - ptr[:-1]
    rows = torch.minimum(ptr[:-1, None] + torch.arange(n, device=dev), ptr[1:, None] - 1)
    qq = q[rows].float().reshape(R, n, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(R, hkv, n * g, D)
    p = torch.matmul(qq, k.transpose(2, 3)) * s["scale"]
    del k
    pos = lens[:, None] - counts[:, None] + torch.arange(n, device=dev)              # [R, n]
    seen = (tok <= pos[:, :, None]) & here[:, None]                                  # [R, n, L]
    p = p.view(R, hkv, n, g, mp * T).masked_fill_(~seen[:, None, :, None], -math.inf)
    m = p.amax(dim=-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp_(p.sub_(m))
    total = p.sum(dim=-1, keepdim=True)
    lse = (m + torch.log(total))[..., 0]                                             # [R, hkv, n, g]
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    v = _values(s["V"], s["v_scale"], phys).permute(0, 2, 1, 3, 4).reshape(R, hkv, mp * T, D)
    v = v.masked_fill_(~here[:, None, :, None], 0.0)
    o = torch.matmul(p.view(R, hkv, n * g, mp * T), v).view(R, hkv, n, g, D)
    real = torch.arange(n, device=dev) < counts[:, None]                             # [R, n]
    weight = None
    if c["weights"]:
        w = (p * real[:, None, :, None, None]).sum(dim=(2, 3)).view(R, hkv, mp, T).sum(dim=3)  # [R, hkv, mp]
        mine = torch.arange(mp, device=dev) < (pptr[1:] - pptr[:-1])[:, None]
        weight = w.transpose(1, 2)[mine]
    o = o.permute(0, 2, 1, 3, 4).reshape(R, n, c["hq"], D)[real].to(q.dtype)
    lse = lse.permute(0, 2, 1, 3).reshape(R, n, c["hq"])[real]
    return o, lse, weight


def _attn_topk(s):
    c, q = s["case"], s["q"]
    hkv, T = c["hkv"], c["page"]
    g, N = c["hq"] // hkv, q.shape[0]
    dev = q.device
    req, pos = _positions(s, N)
    base = s["page_ptr"].long()[req]
    sel = s["topk"].long().permute(1, 0, 2)                                          # [N, hq, K]
    kk = sel.shape[2]
    head = (torch.arange(c["hq"], device=dev) // g)[:, None]
    at = base[:, None, None] + sel.clamp(min=0)
    phys = s["page_table"].long()[at]
    tok = sel[..., None] * T + torch.arange(T, device=dev)                           # [N, hq, K, T]
    seen = (sel >= 0)[..., None] & (tok <= pos[:, None, None, None])
    k = s["K"][phys, head].view(E4).float() * s["k_scale"][phys, head][..., None, None]
    p = torch.matmul(k.view(N, c["hq"], kk * T, D), q.float()[..., None])[..., 0] * s["scale"]
    del k
    p = p.masked_fill_(~seen.view(N, c["hq"], kk * T), -math.inf)
    m = p.amax(dim=-1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(p - m)
    total = p.sum(dim=-1, keepdim=True)
    lse = (m + torch.log(total))[..., 0]
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    v = s["V"][phys, head].view(E4).float() * s["v_scale"][phys, head][..., None, None]
    v = v.masked_fill_(~seen[..., None], 0.0)
    o = torch.matmul(p[:, :, None], v.view(N, c["hq"], kk * T, D))[:, :, 0].to(q.dtype)
    weight = None
    if c["weights"]:
        weight = torch.zeros(s["page_table"].numel(), hkv, device=dev)
        where = at * hkv + head
        weight.view(-1).scatter_add_(0, where.reshape(-1), p.view(N, c["hq"], kk, T).sum(dim=3).reshape(-1))
    return o, lse, weight


def _evict_plain(s):
    pptr, lens, T = s["page_ptr"].long(), s["kv_len"].long(), s["K"].shape[2]
    R, mp = lens.numel(), s["max_pages"]
    dev = lens.device
    have = pptr[1:] - pptr[:-1]
    at = torch.arange(mp, device=dev).expand(R, mp)
    mine = at < have[:, None]
    idx = torch.minimum(pptr[:-1, None] + at, pptr[1:, None] - 1)
    score = (s["decay"] * s["acc"].double() + s["weight"].double().sum(dim=1)).float()
    used = (lens + T - 1) // T
    score = torch.where(at < used[:, None], score[idx], s["acc"][idx])
    free = (at >= s["sink"]) & (at < (used - s["recent"])[:, None])
    drop = torch.minimum((used - s["budget"]).clamp(min=0), free.sum(dim=1))
    order = torch.where(free, score, torch.full_like(score, math.inf)).sort(dim=1, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, at.contiguous())
    out = free & (rank < drop[:, None])
    # kept pages in order, then the dropped ones in order, then the unused entries
    group = torch.where(out, 1, torch.where(at < used[:, None], 0, 2))
    src = group.sort(dim=1, stable=True).indices
    table = s["page_table"][idx].gather(1, src)
    acc = torch.where(out, torch.zeros_like(score), score).gather(1, src)
    return table[mine], acc[mine], (lens - drop * T).to(torch.int32), src.to(torch.int32)[mine]


# ------------------------------------------------------------------ one pass

def _cache(s):
    """The framework's handle over the state's tensors, made once."""
    if "handle" not in s:
        import query_union_paged_b200 as qup
        s["handle"] = qup.KVCache(s["K"], s["V"], s["k_scale"], s["v_scale"], s["page_table"], s["page_ptr"],
                                  s["kv_len"], max_pages=s["max_pages"])
        if s["case"]["op"] == "attn":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
            s["weight"] = None
            if s["case"]["weights"]:
                s["weight"] = torch.empty(s["page_table"].numel(), s["case"]["hkv"], device=s["q"].device)
            s["ws"] = qup.cache_attn_workspace(s["handle"], s["q"].shape[0], s["case"]["hq"], s["max_q"],
                                               page_weight=s["case"]["weights"])
        s["evicted"] = None
    return s["handle"]


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "append":
        if own:
            import query_union_paged_b200 as qup
            qup.cache_append(_cache(s), s["k_new"], s["v_new"], s["ptr"])
        else:
            _append_plain(s)
        return {"K": s["K"].view(E4), "V": s["V"].view(E4), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if op == "attn":
        if own:
            import query_union_paged_b200 as qup
            cache = _cache(s)
            qup.cache_attn(cache, s["q"], s["ptr"], s["max_q"], topk=s["topk"], softmax_scale=s["scale"], out=s["out"],
                           lse=s["lse"], page_weight=s["weight"], workspace=s["ws"])
            o, lse, w = s["out"], s["lse"], s["weight"]
        else:
            o, lse, w = _attn_topk(s) if s["topk"] is not None else _attn_dense(s)
        return {"o": o, "lse": lse} if w is None else {"o": o, "lse": lse, "weight": w}
    if own:
        import query_union_paged_b200 as qup
        s["evicted"] = qup.cache_evict(_cache(s), s["weight"], s["acc"], s["budget"], sink=s["sink"],
                                       recent=s["recent"], decay=s["decay"], out=s.get("evicted"))
        table, acc, lens, src = s["evicted"]
    else:
        table, acc, lens, src = _evict_plain(s)
    return {"page_table": table, "acc": acc, "kv_len": lens, "page_src": src}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    hkv, T = c["hkv"], c["page"]
    ns, lens = _ns(c), _lens(c)
    N = sum(ns)
    if c["op"] == "append":
        esz = 2 if c["dtype"] == "bf16" else 4
        pages = sum((le - 1) // T - (le - n) // T + 1 for n, le in zip(ns, lens))
        return {"bytes": 2 * N * hkv * D * (esz + 1) + 2 * pages * hkv * 4, "flops": 4 * N * hkv * D}
    if c["op"] == "evict":
        total = sum(_pages(c))
        return {"bytes": total * (hkv * 4 + 4 + 4 + 4 + 4 + 4) + c["requests"] * 16, "flops": total * (hkv + 2)}
    if c["topk"]:
        # tokens of the selected pages a query sees: the own page up to itself, the others whole
        toks, cut = 0, 0
        for n, le in zip(ns, lens):
            for i in range(n):
                pos = le - n + i
                toks += min(c["topk"] - 1, pos // T) * T + pos % T + 1
                cut += min(c["topk"], pos // T + 1)
        kv, pairs = toks * hkv * D * 2 + cut * hkv * 8, toks
    else:
        kv = sum(lens) * hkv * D * 2 + sum(-(-x // T) for x in lens) * hkv * 8
        pairs = sum(n * le - n * (n - 1) // 2 for n, le in zip(ns, lens))
    out = N * c["hq"] * (2 * D * 2 + 4) + (sum(_pages(c)) * hkv * 4 if c["weights"] else 0)
    return {"bytes": kv + out, "flops": 4 * pairs * c["hq"] * D}


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3_table(dev):
    """The 256 values of E4M3 by its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if b & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=dev)


def _exact_round(x):
    """Bytes of the E4M3 values nearest to x (ties to the even one); |x| <= 448."""
    table = _e4m3_table(x.device)[:127]  # 0 .. 448, ascending; the byte is the index
    a = x.abs().contiguous()
    hi = torch.searchsorted(table, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    down, up = a - table[lo], table[hi] - a
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (pick + 128 * torch.signbit(x)).to(torch.uint8)


def _exact_append(s):
    T, hkv = s["K"].shape[2], s["K"].shape[1]
    dev = s["K"].device
    table = _e4m3_table(dev)
    ptr, pptr, lens = s["ptr"].tolist(), s["page_ptr"].tolist(), s["kv_len"].tolist()
    pt = s["page_table"].tolist()
    out = {}
    for name, new in (("K", s["k_new"]), ("V", s["v_new"])):
        cache, scale = s[name].clone(), s[name.lower() + "_scale"].double()
        for r in range(len(lens)):
            n = ptr[r + 1] - ptr[r]
            at = lens[r] - n
            while at < lens[r]:
                end = min(lens[r], (at // T + 1) * T)
                p = pt[pptr[r] + at // T]
                i = ptr[r] + at - (lens[r] - n)
                x = new[i:i + end - at].double().transpose(0, 1)                    # [hkv, tokens, d]
                top = x.abs().amax(dim=(1, 2)).tolist()
                need = torch.tensor([2.0 ** max(-64, math.ceil(math.log2(t / 448.0)) if t > 0 else -64) for t in top],
                                    dtype=torch.float64, device=dev)
                if at % T:
                    need = torch.maximum(need, scale[p])
                    old = table[cache[p, :, :at % T].long()] * (scale[p] / need)[:, None, None]
                    cache[p, :, :at % T] = _exact_round(old)
                cache[p, :, at % T:at % T + end - at] = _exact_round(x / need[:, None, None])
                scale[p] = need
                at = end
        out[name], out[name.lower() + "_scale"] = cache.view(E4), scale
    return out


def _exact_attn(s):
    c = s["case"]
    hkv, hq, T = c["hkv"], c["hq"], c["page"]
    g = hq // hkv
    dev = s["q"].device
    table = _e4m3_table(dev)
    ptr, pptr, lens = s["ptr"].tolist(), s["page_ptr"].tolist(), s["kv_len"].tolist()
    N = s["q"].shape[0]
    o = torch.zeros(N, hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((N, hq), -math.inf, dtype=torch.float64, device=dev)
    weight = torch.zeros(pptr[-1], hkv, dtype=torch.float64, device=dev)
    for r in range(len(lens)):
        n, L = ptr[r + 1] - ptr[r], lens[r]
        np_ = -(-L // T)
        phys = s["page_table"][pptr[r]:pptr[r] + np_].long()
        for h in range(hkv):
            k = (table[s["K"][phys, h].long()] * s["k_scale"][phys, h].double()[:, None, None]).view(-1, D)[:L]
            v = (table[s["V"][phys, h].long()] * s["v_scale"][phys, h].double()[:, None, None]).view(-1, D)[:L]
            q = s["q"][ptr[r]:ptr[r + 1], h * g:(h + 1) * g].double().reshape(n * g, D)
            x = (q @ k.T).view(n, g, L) / math.sqrt(D)
            see = torch.arange(L, device=dev) <= (L - n + torch.arange(n, device=dev))[:, None]
            see = see[:, None].expand(n, g, L)
            if s["topk"] is not None:
                sel = s["topk"][h * g:(h + 1) * g, ptr[r]:ptr[r + 1]].long().transpose(0, 1)  # [n, g, K]
                chosen = torch.zeros(n, g, np_ + 1, dtype=torch.bool, device=dev)
                chosen.scatter_(2, torch.where(sel >= 0, sel, np_), True)
                see = see & chosen[..., :np_].repeat_interleave(T, dim=2)[..., :L]
            x = torch.where(see, x, -math.inf)
            lse_h = torch.logsumexp(x, dim=2)
            p = torch.exp(x - lse_h[..., None])
            o[ptr[r]:ptr[r + 1], h * g:(h + 1) * g] = (p.view(n * g, L) @ v).view(n, g, D)
            lse[ptr[r]:ptr[r + 1], h * g:(h + 1) * g] = lse_h
            w = torch.nn.functional.pad(p.sum(dim=(0, 1)), (0, np_ * T - L)).view(np_, T).sum(dim=1)
            weight[pptr[r]:pptr[r] + np_, h] = w
    return {"o": o, "lse": lse, "weight": weight} if c["weights"] else {"o": o, "lse": lse}


def _exact_evict(s):
    pptr, lens, T = s["page_ptr"].tolist(), s["kv_len"].tolist(), s["K"].shape[2]
    w, a = s["weight"].double().cpu().numpy(), s["acc"].double().cpu().numpy()
    table = s["page_table"].tolist()
    out_t, out_a, out_l, out_s = [], [], [], []
    for r in range(len(lens)):
        b, e = pptr[r], pptr[r + 1]
        used = -(-lens[r] // T)
        score = [s["decay"] * a[b + p] + float(w[b + p].sum()) if p < used else float(a[b + p]) for p in range(e - b)]
        free = range(s["sink"], used - s["recent"])
        drop = sorted(free, key=lambda p: (score[p], p))[:max(0, used - s["budget"])]
        gone = set(drop)
        src = [p for p in range(used) if p not in gone] + sorted(gone) + list(range(used, e - b))
        out_t += [table[b + p] for p in src]
        out_a += [0.0 if p in gone else score[p] for p in src]
        out_s += src
        out_l.append(lens[r] - len(gone) * T)
    dev = s["acc"].device
    return {"page_table": torch.tensor(out_t, dtype=torch.int32, device=dev),
            "acc": torch.tensor(out_a, dtype=torch.float64, device=dev),
            "kv_len": torch.tensor(out_l, dtype=torch.int32, device=dev),
            "page_src": torch.tensor(out_s, dtype=torch.int32, device=dev)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "evict": _exact_evict}[case["op"]](s)
