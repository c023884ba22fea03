// cache_attn.cu -- attention over the 8-bit page-scaled cache: single tokens and short runs of
// queries, over all pages of a request or over each query's TopK pages.
//
// Per row (query i, query head j of KV head h) and visible token t of page p:
//   s_t = softmax_scale * (q . k_t) * ks[p][h],  O = sum e^{s_t} vs[p][h] v_t / sum e^{s_t},
// with k_t, v_t the E4M3 values.  One pass with a running maximum over x_t = log2e s_t + log2 vs:
//   p'_t = 2^{x_t - m + 8},  O += p'_t v_t,  l += p'_t / vs,
// so the V scale costs nothing per element and P has one range whatever the scales are.
//
// Numbers: E4M3 is exact in fp16; Q (bf16) is brought to fp16 by a power of two per row (its largest
// element in [2^14, 2^15): what rounds lies 2^-31 below it), P is rounded to fp16 (2^-11; the
// offset 8 keeps weights down to 2^-32 of the largest).  Products accumulate in fp32.
//
// Layout: a work unit is 64 tokens of one KV head: 8 KB of K and 8 KB of V, streamed by one
// producer warp with TMA (128-byte swizzle) through a ring of stages.  Each of the four consumer
// warps takes 16 tokens of every unit, two units at a time, with its own running maximum, sum and output
// (no exchange inside the loop).  Tokens are the rows of the products and query rows their columns:
// S^T = K Q^T and O^T = V^T P^T as mma.m16n8k16, so 8 rows cost no more than one and the cache's bytes are
// operands as they lie: the order of d inside K's fragments and of d over the output rows is free, every
// lane reads 16 consecutive bytes of a token (conflict-free under the swizzle) and converts two
// values at a time; P^T is turned by movmatrix.  (With query rows as the products' rows a tile is 16 high:
// twice the products and exponentials for 4 heads, 437 instructions for 16 tokens.)  The warps merge
// in shared memory at the end of a segment.
//
// Work split: all pages: the units of all (request, KV head, row tile) items are laid end to end and
// cut into equal runs, one per CTA, so ragged lengths balance; an item cut across CTAs leaves one
// partial result in each, which a second kernel merges in a fixed order.  TopK pages: one item per
// (query, KV head), its distinct pages cut into an equal share per CTA.
//
// Bound by DRAM: 2 * 128 bytes per token and KV head.  16 requests of 33K to 64K tokens, 8 KV heads, 32
// heads: 258 to 280 us, 5.7 to 6.1 TB/s (0.86 to 0.94 of a copy); a TopK call of 32 pages of 64 tokens 35 us,
// 3.8 TB/s (finding a query's pages costs a CTA about 5 us before its first load).
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "cache.h"
#include "cache_attn.h"
#include "internal.h"
#include "ptx.cuh"
#include "query_union_paged.h"

namespace qup {
namespace {

constexpr int kUnit = kCacheUnit;               // tokens of a work unit
constexpr int kTile = kUnit * kHeadDim;         // bytes of one K or V tile
constexpr int kConsumers = 4;                   // consumer warps: kUnit / 16 tokens
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kMaxBoxes = kUnit / 16;           // pages in a unit at T = 16
constexpr float kOffset = 8.f;                  // log2 offset of P
constexpr float kLazy = 7.f;                    // the maximum moves once a score passes it by this
constexpr float kZeroScaleLog2 = -64.f;         // a V scale of 0 (a page of zeros) counts as 2^-64
constexpr float kNegInf = -INFINITY;

// A page of a stage, as the consumers need it.
struct PageMeta {
    float ks;        // softmax_scale * log2e is in the row's factor
    float vs_log2;
    float vs_inv;
    uint32_t mask;   // bit per row of the tile's first 32 (TopK: the query heads); all ones otherwise
    int pos;         // position of the page's first token in the unit
    int pad[3];
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {  // an 8 x 8 matrix of 16-bit elements over the warp
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
// Work units of one row tile of a request, and its row tiles.
__device__ __forceinline__ int units_of(int len) { return (len + kUnit - 1) / kUnit; }
__device__ __forceinline__ int tiles_of(int n, int g, int RT) { return (n * g + RT - 1) / RT; }

// A thread's own consecutive requests: their unit counts are added up, and the sums over the CTA.
struct Span {
    int r0, r1;
};
__device__ __forceinline__ Span my_span(int R) {
    const int per = (R + kThreads - 1) / kThreads;
    const int a = min(R, (int)threadIdx.x * per);
    return Span{a, min(R, a + per)};
}
__device__ __forceinline__ int request_units(const CacheAttnParams& p, int r, int RT, unsigned* bad) {
    const Request q = load_request(p.q_ptr, p.Nq, p.c.kv_len, p.c.page_ptr, p.c.total_pages, p.c.T, r);
    if ((long long)q.n * p.g >= p.big_rows) return 0;  // the chunk kernel's
    const unsigned f = request_fault(p, q);
    *bad |= f;
    return f ? 0 : tiles_of(q.n, p.g, RT) * p.c.Hkv * units_of(q.len);
}

// Exclusive prefix over the CTA's threads of v (kThreads of them), and the total; `part` holds one entry per
// warp.
__device__ __forceinline__ long long cta_prefix(long long v, long long* part, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    if (lane == 31) part[warp] = run;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? part[w] : 0;
        all += part[w];
    }
    *total = all;
    return before + run - v;
}

// Units of one CTA's run: an equal share of all of them.
__device__ __forceinline__ int units_per_cta(long long all, int grid) {
    return max(1, (int)((all + grid - 1) / grid));
}

// Where a CTA's run of units begins, and how long it is.
struct Start {
    int r, off, count;
};

// One item's view of the cache while it is walked: a segment [b0, b1) of its units.
struct Seg {
    int r, q0, n, len, p0, np;
    int h, tile, b0, b1, nvis;  // nvis: units that the tile's last row sees any token of
};

// Walks the units [off, ...) of requests r, r + 1, ... in (KV head, row tile, unit) order.
struct Cursor {
    int r, off, left;
    Request q;
    int nb, nt;
    __device__ __forceinline__ void begin(const Start& s) {
        r = s.r;
        off = s.off;
        left = s.count;
        nb = -1;
    }
    __device__ __forceinline__ bool next(const CacheAttnParams& p, int RT, Seg& s) {
        while (left > 0) {
            if (nb < 0) {
                if (r >= p.c.R) return false;
                q = load_request(p.q_ptr, p.Nq, p.c.kv_len, p.c.page_ptr, p.c.total_pages, p.c.T, r);
                const bool ok = request_fault(p, q) == 0u && (long long)q.n * p.g < p.big_rows;
                nb = ok ? units_of(q.len) : 0;
                nt = ok ? tiles_of(q.n, p.g, RT) : 0;
            }
            const int total = nt * p.c.Hkv * nb;
            if (off >= total) {
                off -= total;
                ++r;
                nb = -1;
                continue;
            }
            const int it = off / nb;
            s.r = r;
            s.q0 = q.q0;
            s.n = q.n;
            s.len = q.len;
            s.p0 = q.p0;
            s.np = q.np;
            s.h = it / nt;
            s.tile = it - s.h * nt;
            s.b0 = off - it * nb;
            s.b1 = min(nb, s.b0 + left);
            off += s.b1 - s.b0;
            left -= s.b1 - s.b0;
            const int last = (min((s.tile + 1) * RT, s.n * p.g) - 1) / p.g;  // the tile's last query
            const int vis = s.len - s.n + last + 1;
            s.nvis = vis <= 0 ? 0 : units_of(vis);
            return true;
        }
        return false;
    }
};

// Shared memory, from a 1024-byte boundary: the ring, then what follows.
// NT: row tiles of 8 rows.  Up to 8 rows leave registers for three CTAs on an SM (four stages each).
template <int NT>
struct Smem {
    static constexpr int RT = 8 * NT;
    static constexpr int kStages = NT == 1 ? 4 : 6;
    static constexpr uint32_t ring = 0;
    static constexpr uint32_t out = ring + kStages * 2 * kTile;             // [RT][128] fp32
    static constexpr uint32_t qfrag = out + RT * kHeadDim * 4;  // NT = 4: [NT][8][32] uint2
    static constexpr uint32_t meta = qfrag + (NT == 4 ? RT * kHeadDim * 2 : 0);  // [kStages][kMaxBoxes]
    static constexpr uint32_t ml = meta + kStages * kMaxBoxes * sizeof(PageMeta);  // [kConsumers][RT] float2
    static constexpr uint32_t bars = ml + kConsumers * RT * 8;
    static constexpr uint32_t misc = bars + 2 * kStages * 8;  // abort flag, start, scan
    static constexpr uint32_t list = misc + 64 + 64;  // TopK: bitmap, prefix, pages, masks
};

template <int NT, bool SPARSE, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, cache_attn_ctas(NT))
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CacheAttnParams p) {
    using L = Smem<NT>;
    constexpr bool kQRegs = NT < 4;  // Q stays in registers
    constexpr int RT = L::RT, NS = L::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full0 = sbase + L::bars, empty0 = full0 + 8 * NS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::misc);
    int* s_start = reinterpret_cast<int*>(smem + L::misc + 16);  // r, off, count
    long long* scan = reinterpret_cast<long long*>(smem + L::misc + 64);
    PageMeta* meta = reinterpret_cast<PageMeta*>(smem + L::meta);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int T = p.c.T, g = p.g;
    const int box = min(T, kUnit), nbox = kUnit / box;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, kConsumers);
        }
        *abort_flag = 0;
        s_start[0] = p.c.R;
        s_start[1] = 0;
        s_start[2] = 0;
        fence_mbar_init();
    }
    if (warp == kConsumers && lane == 0) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    grid_dep_wait();
    __syncthreads();

    // ---------------------------------------------------------------- this CTA's work
    Seg sg;                  // TopK: the one segment
    float2* mass = nullptr;  // page weights: of the segment's rows
    int list_lo = 0, list_n = 0;
    uint32_t *bits = nullptr, *masks = nullptr;
    int *before = nullptr, *pages = nullptr;
    if constexpr (!SPARSE) {
        const Span sp = my_span(p.c.R);
        long long sum = 0;
        unsigned bad = 0;
        for (int r = sp.r0; r < sp.r1; ++r) sum += request_units(p, r, RT, &bad);
        if (bad) atomicOr(p.err, bad);
        long long all = 0;
        const long long mine = cta_prefix(sum, scan, &all);
        const int per = units_per_cta(all, (int)gridDim.x);
        const long long u0 = (long long)blockIdx.x * per;
        if (u0 < all) {
            if (u0 >= mine && u0 < mine + sum) {
                long long at = mine;
                for (int r = sp.r0; r < sp.r1; ++r) {
                    const int u = request_units(p, r, RT, &bad);
                    if (u0 < at + u) {
                        s_start[0] = r;
                        s_start[1] = (int)(u0 - at);
                        s_start[2] = (int)min((long long)per, all - u0);
                        break;
                    }
                    at += u;
                }
            }
        }
        if (__syncthreads_or(bad != 0u)) clear_faulty(p, false);
        if (s_start[2] == 0) return;
    } else {
        // the item's query and request
        const int item = blockIdx.x / p.nsplit, split = blockIdx.x - item * p.nsplit;
        const int qi = item / p.c.Hkv, h = item - qi * p.c.Hkv;
        for (int r = tid; r < p.c.R; r += kThreads)
            if (p.q_ptr[r] <= qi && qi < p.q_ptr[r + 1]) s_start[0] = r;
        __syncthreads();
        const int r = s_start[0];
        if (r >= p.c.R) return;  // a row of no request: left as it is
        const Request q = load_request(p.q_ptr, p.Nq, p.c.kv_len, p.c.page_ptr, p.c.total_pages, T, r);
        const unsigned fault = request_fault(p, q);
        const bool ok = fault == 0u;
        if (!ok && tid == 0) atomicOr(p.err, fault);
        const int vis = ok ? q.len - q.n + (qi - q.q0) + 1 : 0;  // tokens the query sees
        const int words = ok ? (q.np + 31) / 32 : 0;
        bits = reinterpret_cast<uint32_t*>(smem + L::list);
        before = reinterpret_cast<int*>(bits + (p.max_pages + 31) / 32);
        pages = before + (p.max_pages + 31) / 32;
        masks = reinterpret_cast<uint32_t*>(pages + p.list_cap);
        for (int w = tid; w < words; w += kThreads) bits[w] = 0u;
        __syncthreads();
        const int entries = g * p.Ksel;
        for (int e = tid; e < entries; e += kThreads) {
            const int j = e / p.Ksel, k = e - j * p.Ksel;
            const int pg = __ldg(p.topk + ((size_t)(h * g + j) * p.Nq + qi) * p.Ksel + k);
            if (pg == -1) continue;
            if (pg < 0 || (ok && pg >= q.np)) {
                atomicOr(p.err, QUP_ERR_PAGE_ID);
                continue;
            }
            if ((long long)pg * T < vis) atomicOr(&bits[pg >> 5], 1u << (pg & 31));
        }
        __syncthreads();
        {  // pages before each bitmap word
            const int per = (words + kThreads - 1) / kThreads, w0 = min(words, tid * per), w1 = min(words, w0 + per);
            int sum = 0;
            for (int w = w0; w < w1; ++w) {
                before[w] = sum;
                sum += __popc(bits[w]);
            }
            long long total = 0;
            const int mine = (int)cta_prefix(sum, scan, &total), all = (int)total;
            for (int w = w0; w < w1; ++w) before[w] += mine;
            const int share = (all + p.nsplit - 1) / p.nsplit;
            list_lo = min(all, split * share);
            list_n = min(all, list_lo + share) - list_lo;
            for (int x = tid; x < list_n; x += kThreads) masks[x] = 0u;
            if (WEIGHTS && split == 0 && ok) {  // which pages this query reads, for the page weights
                uint32_t* dst = p.ws_bits + ((size_t)(q.p0 / 32 + r) * p.max_q * p.c.Hkv) +
                                ((size_t)(qi - q.q0) * p.c.Hkv + h) * ((q.np + 31) / 32);
                for (int w = tid; w < (q.np + 31) / 32; w += kThreads) dst[w] = bits[w];
            }
        }
        __syncthreads();
        for (int e = tid; e < entries; e += kThreads) {
            const int j = e / p.Ksel, k = e - j * p.Ksel;
            const int pg = __ldg(p.topk + ((size_t)(h * g + j) * p.Nq + qi) * p.Ksel + k);
            if (pg < 0 || pg >= q.np || (long long)pg * T >= vis) continue;
            const int at = before[pg >> 5] + __popc(bits[pg >> 5] & ((1u << (pg & 31)) - 1u)) - list_lo;
            if (at < 0 || at >= list_n) continue;
            pages[at] = pg;
            atomicOr(&masks[at], 1u << j);
        }
        __syncthreads();
        if constexpr (WEIGHTS) {
            mass = mass_of_query(p, q, h, qi - q.q0);
        }
        sg.r = r;
        sg.q0 = qi;
        sg.n = 1;
        sg.len = vis;  // the query is the last of its visible tokens
        sg.p0 = q.p0;
        sg.np = q.np;
        sg.h = h;
        sg.tile = split;
        sg.b0 = 0;
        sg.b1 = sg.nvis = T > kUnit ? list_n * (T / kUnit) : (list_n + nbox - 1) / nbox;
    }

    Cursor cur;
    if constexpr (!SPARSE) cur.begin(Start{s_start[0], s_start[1], s_start[2]});
    bool more = SPARSE;
    uint32_t it = 0;  // stages used so far: slot it % NS, parity (it / NS) & 1
    // A wait was given up.  The lanes of a warp agree on it: one whose own limit had run out would leave the others
    // in shuffles, votes and products of the whole warp.
    bool dead = false;

    if (warp == kConsumers) {
        // ============================================================ producer
        while (SPARSE ? more : cur.next(p, RT, sg)) {
            more = false;
            const int e0 = sg.b0, e1 = min(sg.b1, sg.nvis);  // units that are read
            // 32 pages at a time: each lane looks one up
            const int upp = T > kUnit ? T / kUnit : 1;  // units per page, or pages per unit
            const int ppu = T > kUnit ? 1 : nbox;
            int have0 = 0, have1 = 0;  // page entries the lanes hold
            int phys = -1, lpos = 0;
            float ks = 0.f, vl = 0.f, vi = 0.f;
            uint32_t msk = 0;
            for (int b = e0; b < e1 && !dead; ++b) {
                const int pe = b / upp * ppu;  // the unit's first page entry
                if (pe + ppu > have1) {
                    have0 = pe;
                    have1 = pe + 32;
                    const int e = pe + lane;
                    const int last = SPARSE ? list_n : (sg.len + T - 1) / T;
                    phys = -1;
                    msk = 0;
                    lpos = 0x40000000;  // no page: past every row's visible tokens
                    if (e < last) {
                        const int pg = SPARSE ? pages[e] : e;
                        msk = SPARSE ? masks[e] : 0xffffffffu;
                        lpos = pg * T;
                        phys = p.c.page_table[sg.p0 + pg];
                        if (phys < 0 || phys >= p.c.P_phys) {
                            atomicOr(p.err, QUP_ERR_PHYS_PAGE);
                            phys = -1;
                        } else {
                            ks = __ldg(p.c.k_scale + (size_t)phys * p.c.Hkv + sg.h);
                            const float vs = __ldg(p.c.v_scale + (size_t)phys * p.c.Hkv + sg.h);
                            if (!(fabsf(ks) < INFINITY) || !v_scale_ok(vs)) {
                                atomicOr(p.err, QUP_ERR_SCALE);
                                phys = -1;
                            }
                            vl = vs > 0.f ? lg2(vs) : kZeroScaleLog2;
                            vi = vs > 0.f ? __frcp_rn(vs) : 18446744073709551616.f;
                        }
                    }
                    if (phys < 0) msk = 0;
                }
                const uint32_t slot = it % NS, par = (it / NS) & 1;
                dead = !__all_sync(0xffffffffu, mbar_wait(empty0 + 8 * slot, par ^ 1, abort_flag, p.err, QUP_ERR_TIMEOUT,
                                                          p.wait_limit_ns));
                if (dead) break;
                const int src = pe - have0;
                uint32_t bytes = 0;
                for (int x = 0; x < nbox; ++x) {
                    const int ph = __shfl_sync(0xffffffffu, phys, src + x);
                    bytes += ph >= 0 ? 2u * box * kHeadDim : 0u;
                    if (lane == src + x) {
                        PageMeta m;
                        m.ks = ks;
                        m.vs_log2 = vl;
                        m.vs_inv = vi;
                        m.mask = msk;
                        m.pos = lpos + (b % upp) * kUnit;
                        meta[slot * kMaxBoxes + x] = m;
                    }
                }
                __syncwarp();
                const bool load = it != (uint32_t)p.dbg_skip_stage;
                if (lane == 0 && load) {
                    if (bytes) mbar_arrive_expect_tx(full0 + 8 * slot, bytes);
                    else mbar_arrive(full0 + 8 * slot);
                }
                __syncwarp();
                for (int x = 0; x < nbox; ++x) {
                    const int ph = __shfl_sync(0xffffffffu, phys, src + x);
                    if (ph >= 0 && lane == 0 && load) {
                        const uint32_t dst = sbase + L::ring + slot * 2 * kTile + x * box * kHeadDim;
                        tma_load_4d(dst, &tmK, full0 + 8 * slot, 0, (b % upp) * kUnit, sg.h, ph);
                        tma_load_4d(dst + kTile, &tmV, full0 + 8 * slot, 0, (b % upp) * kUnit, sg.h, ph);
                    }
                }
                ++it;
            }
        }
        // a run that was given up: what is in flight lands before the CTA leaves
        if (*abort_flag) {
            for (uint32_t k = it > NS ? it - NS : 0; k < it; ++k)
                mbar_wait_drain(full0 + 8 * (k % NS), (k / NS) & 1, p.wait_limit_ns);
        }
        return;
    }

    // ================================================================ consumers
    const int i = lane >> 2, q4 = lane & 3;
    float* s_out = reinterpret_cast<float*>(smem + L::out);
    float2* s_ml = reinterpret_cast<float2*>(smem + L::ml);
    uint2* s_q = reinterpret_cast<uint2*>(smem + L::qfrag);
    bool first_seg = true;
    while (SPARSE ? more : cur.next(p, RT, sg)) {
        more = false;
        const int rows = SPARSE ? g : min(RT, sg.n * g - sg.tile * RT);  // rows of the tile
        const int row0 = SPARSE ? 0 : sg.tile * RT;                     // in (query, head) order
        const int e0 = sg.b0, e1 = min(sg.b1, sg.nvis);
        // ---- Q as B operand: lane (i, q4) holds d = 32 q4 + 4 ks .. + 3 of row 8 t + i
        uint32_t qb[kQRegs ? NT : 1][8][2];
        float rs[NT][2];  // of rows 8 t + 2 q4, + 1: score factor, tokens they see, maximum, sum
        int vis[NT][2];
        float m[NT][2], l[NT][2], o[NT][8][4];
        if (!kQRegs) bar_sync(1, 32 * kConsumers);  // the last segment's are done with
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int rr = 8 * t + i;
            const bool on = rr < rows;
            const int x = row0 + (on ? rr : 0), qi = SPARSE ? 0 : x / g, j = x - qi * g;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.Q) +
                                                              (size_t)(sg.q0 + qi) * p.q_stride +
                                                              (size_t)(sg.h * g + j) * kHeadDim + 32 * q4);
            uint4 raw[4];
            uint32_t top = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                raw[u] = on ? __ldg(src + u) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7f800000u, w[e] & 0x7f800000u));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the row's largest element is in [2^e, 2^(e+1)): times 2^(14 - e)
            const int ex = max((int)(top >> 23) - 127, -100);
            const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
            const float row_rs = p.scale_log2 * __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
            const int row_vis = on ? (SPARSE ? sg.len : sg.len - sg.n + qi + 1) : 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int e = 0; e < 4; e += 2) {  // words 4 u + e, + 1: k-step 2 u + e / 2
                    const uint32_t b0 = pack_f16x2(__uint_as_float(w[e] << 16) * up,
                                                   __uint_as_float(w[e] & 0xffff0000u) * up);
                    const uint32_t b1 = pack_f16x2(__uint_as_float(w[e + 1] << 16) * up,
                                                   __uint_as_float(w[e + 1] & 0xffff0000u) * up);
                    if constexpr (kQRegs) {
                        qb[t][2 * u + e / 2][0] = b0;
                        qb[t][2 * u + e / 2][1] = b1;
                    } else if (warp == t) {
                        s_q[(t * 8 + 2 * u + e / 2) * 32 + lane] = make_uint2(b0, b1);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // lane 4 y holds row 8 t + y
                rs[t][e] = __shfl_sync(0xffffffffu, row_rs, 4 * (2 * q4 + e));
                vis[t][e] = __shfl_sync(0xffffffffu, row_vis, 4 * (2 * q4 + e));
                m[t][e] = kNegInf;
                l[t][e] = 0.f;
            }
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][d][e] = 0.f;
        }
        if (!kQRegs) bar_sync(1, 32 * kConsumers);
        // tokens that every row of the tile sees, and that any row sees
        const int vis_all = SPARSE ? sg.len : sg.len - sg.n + row0 / g + 1;
        const int vis_any = SPARSE ? sg.len : sg.len - sg.n + (row0 + rows - 1) / g + 1;
        const uint32_t all_rows = SPARSE ? (rows == 32 ? 0xffffffffu : (1u << rows) - 1u) : 0xffffffffu;

        // page weights: this tile's rows, mass_rows apart for every 16 tokens
        const int mass_rows = SPARSE ? g : sg.n * g;
        if constexpr (WEIGHTS && !SPARSE) {
            Request q{};
            q.q0 = sg.q0;
            q.n = sg.n;
            q.p0 = sg.p0;
            q.np = sg.np;
            mass = mass_of(p, q, sg.h, false) + row0;
        }
        // One turn: NG units, 16 tokens of each.  Two at a time hide each other's latencies (products in a
        // chain, conversions, the row maximum's shuffles): one warp alone keeps its scheduler a third busy.
        const auto turn = [&](auto groups) {
            constexpr int NG = decltype(groups)::value;
            bool here = true;  // tried once, all together; waited for only where that fails
#pragma unroll
            for (int n = 0; n < NG; ++n) here &= mbar_try_wait(full0 + 8 * ((it + n) % NS), ((it + n) / NS) & 1);
            if (!__all_sync(0xffffffffu, here)) {
                here = true;
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    here = here && mbar_wait(full0 + 8 * ((it + n) % NS), ((it + n) / NS) & 1, abort_flag, p.err,
                                             QUP_ERR_TIMEOUT, p.wait_limit_ns);
                dead = !__all_sync(0xffffffffu, here);
                if (dead) return;
            }
            PageMeta pm[NG];
            int pos[NG];  // of the warp's first token of each
            bool live[NG], mixed[NG], any = false;
            uint32_t tile[NG];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const uint32_t slot = (it + n) % NS;
                pm[n] = meta[slot * kMaxBoxes + 16 * warp / box];
                pos[n] = pm[n].pos + (16 * warp) % box;
                live[n] = pm[n].mask != 0u && pos[n] < vis_any;
                mixed[n] = !live[n] || pos[n] + 16 > vis_all || (pm[n].mask & all_rows) != all_rows;
                any = any || live[n];
                tile[n] = sbase + L::ring + slot * 2 * kTile;
            }
            if (any) {
                // ---- S^T = K Q^T: tokens i and i + 8 of the warp, d = 32 q4 .. + 31 of each in two loads
                float c[NG][NT][4];
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[n][t][e] = 0.f;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    uint4 k[NG][2];
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            k[n][y] = lds128(tile[n] + (16 * warp + 8 * y + i) * kHeadDim + (((2 * q4 + s) ^ i) << 4));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t b[NT][2];
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if constexpr (kQRegs) {
                                b[t][0] = qb[t][4 * s + e][0];
                                b[t][1] = qb[t][4 * s + e][1];
                            } else {
                                const uint2 v = s_q[(t * 8 + 4 * s + e) * 32 + lane];
                                b[t][0] = v.x;
                                b[t][1] = v.y;
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            uint32_t a[4];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t w = e < 2 ? (e == 0 ? k[n][y].x : k[n][y].y)
                                                         : (e == 2 ? k[n][y].z : k[n][y].w);
                                cvt_e4m3x4(w, a[y], a[y + 2]);
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) mma16816(c[n][t], a, b[t][0], b[t][1]);
                        }
                    }
                }
                uint32_t pb[NG][NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float x[NG][4], bm[2] = {kNegInf, kNegInf};
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        // c: token i of rows 2 q4, + 1, then token i + 8 of them
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[n][e] = fmaf(c[n][t][e], rs[t][e & 1] * pm[n].ks, pm[n].vs_log2);
                        if (mixed[n]) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const bool on = live[n] && (!SPARSE || ((pm[n].mask >> (8 * t + 2 * q4 + (e & 1))) & 1u));
                                if (!on || pos[n] + i + 8 * (e >> 1) >= vis[t][e & 1]) x[n][e] = kNegInf;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) bm[e] = fmaxf(bm[e], fmaxf(x[n][e], x[n][e + 2]));
                    }
#pragma unroll
                    for (int o2 = 4; o2 < 32; o2 *= 2)
#pragma unroll
                        for (int e = 0; e < 2; ++e) bm[e] = fmaxf(bm[e], __shfl_xor_sync(0xffffffffu, bm[e], o2));
                    if (__any_sync(0xffffffffu, bm[0] > m[t][0] + kLazy || bm[1] > m[t][1] + kLazy)) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const bool mv = bm[e] > m[t][e] + kLazy;  // -inf + kLazy = -inf
                            const float a = mv ? ex2(m[t][e] - bm[e]) : 1.f;
                            if (mv) m[t][e] = bm[e];
                            l[t][e] *= a;
#pragma unroll
                            for (int d = 0; d < 8; ++d) {
                                o[t][d][e] *= a;
                                o[t][d][e + 2] *= a;
                            }
                        }
                    }
                    float sub[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) sub[e] = m[t][e] == kNegInf ? 0.f : m[t][e] - kOffset;
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[n][e] = ex2(x[n][e] - sub[e & 1]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float sum = (x[n][e] + x[n][e + 2]) * pm[n].vs_inv;
                            l[t][e] += sum;
                            if constexpr (WEIGHTS) {
#pragma unroll
                                for (int o2 = 4; o2 < 32; o2 *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
                                const int rr = 8 * t + 2 * q4 + e;
                                if (i == 0 && rr < rows && pos[n] < vis_any)
                                    mass[(size_t)(pos[n] / 16) * mass_rows + rr] = make_float2(sum, m[t][e]);
                            }
                        }
                        // P^T as B operand: rows to lanes, tokens to registers
                        pb[n][t][0] = transpose8(pack_f16x2(x[n][0], x[n][1]));
                        pb[n][t][1] = transpose8(pack_f16x2(x[n][2], x[n][3]));
                    }
                }
                // ---- O^T += V^T P^T: tokens 2 q4, + 1, + 8, + 9 of the warp, d = 16 i .. + 15 of each; product
                // 2 w + hi takes d = 16 i + 4 w + 2 hi and the one after it
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    uint32_t v[4][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = 2 * q4 + (e & 1) + 8 * (e >> 1);
                        const uint4 w = lds128(tile[n] + kTile + (16 * warp + t) * kHeadDim + ((i ^ (t & 7)) << 4));
                        v[e][0] = w.x;
                        v[e][1] = w.y;
                        v[e][2] = w.z;
                        v[e][3] = w.w;
                    }
                    bool slow = false;
                    if (mixed[n]) {
                        // bytes behind the last visible token may be anything; a NaN that some rows see and
                        // others do not must not reach the others as 0 * NaN
                        bool nan = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (!live[n] || pos[n] + 2 * q4 + (e & 1) + 8 * (e >> 1) >= vis_any)
                                v[e][0] = v[e][1] = v[e][2] = v[e][3] = 0u;
                            nan = nan || (nan_bytes(v[e][0]) | nan_bytes(v[e][1]) | nan_bytes(v[e][2]) | nan_bytes(v[e][3])) != 0u;
                        }
                        slow = __any_sync(0xffffffffu, nan);
                    }
                    const auto operand = [](const uint32_t (&v)[4][4], int w, int hi, uint32_t (&a)[4]) {
                        const uint32_t x0 = __byte_perm(v[0][w], v[1][w], hi ? 0x7362 : 0x5140);
                        const uint32_t x1 = __byte_perm(v[2][w], v[3][w], hi ? 0x7362 : 0x5140);
                        cvt_e4m3x4(x0, a[0], a[1]);
                        cvt_e4m3x4(x1, a[2], a[3]);
                    };
                    if (!slow) {
#pragma unroll
                        for (int w = 0; w < 4; ++w)
#pragma unroll
                            for (int hi = 0; hi < 2; ++hi) {
                                uint32_t a[4];
                                operand(v, w, hi, a);
#pragma unroll
                                for (int t = 0; t < NT; ++t) mma16816(o[t][2 * w + hi], a, pb[n][t][0], pb[n][t][1]);
                            }
                    } else {
                        // row by row: the other rows' weights and the tokens the row does not see are zero
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll 1
                            for (int y = 0; y < 8 && 8 * t + y < rows; ++y) {
                                const int rr = 8 * t + y, rv = SPARSE ? sg.len : sg.len - sg.n + (row0 + rr) / g + 1;
                                const bool on = !SPARSE || ((pm[n].mask >> rr) & 1u);
                                uint32_t z[4][4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
#pragma unroll
                                    for (int w = 0; w < 4; ++w)
                                        z[e][w] = on && pos[n] + 2 * q4 + (e & 1) + 8 * (e >> 1) < rv ? v[e][w] : 0u;
                                const uint32_t b0 = y == i ? pb[n][t][0] : 0u, b1 = y == i ? pb[n][t][1] : 0u;
#pragma unroll
                                for (int w = 0; w < 4; ++w)
#pragma unroll
                                    for (int hi = 0; hi < 2; ++hi) {
                                        uint32_t a[4];
                                        operand(z, w, hi, a);
                                        float r4[4] = {0.f, 0.f, 0.f, 0.f};
                                        mma16816(r4, a, b0, b1);
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (2 * q4 + (e & 1) == y) o[t][2 * w + hi][e] += r4[e];
                                    }
                            }
                    }
                }
            } else if (WEIGHTS) {
                // pages that no row reads (bad pages): zero mass
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    for (int rr = lane; rr < rows && pos[n] < vis_any; rr += 32)
                        mass[(size_t)(pos[n] / 16) * mass_rows + rr] = make_float2(0.f, 0.f);
            }
            __syncwarp();
            if (lane == 0)
#pragma unroll
                for (int n = 0; n < NG; ++n) mbar_arrive(empty0 + 8 * ((it + n) % NS));
            it += NG;
        };
        int b = e0;
        if (NT < 4)
            for (; b + 1 < e1 && !dead; b += 2) turn(std::integral_constant<int, 2>());
        for (; b < e1 && !dead; ++b) turn(std::integral_constant<int, 1>());

        // ---- the four warps' results, joined
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o2 = 4; o2 < 32; o2 *= 2) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], o2);
                if (i == 0) s_ml[warp * RT + 8 * t + 2 * q4 + e] = make_float2(m[t][e], l[t][e]);
            }
        bar_sync(1, 32 * kConsumers);
#pragma unroll 1
        for (int w = 0; w < kConsumers; ++w) {
            if (warp == w) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int rr = 8 * t + 2 * q4 + e;
                        float M = kNegInf;
#pragma unroll
                        for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, s_ml[x * RT + rr].x);
                        const float f = m[t][e] == kNegInf ? 0.f : ex2(m[t][e] - M);
                        // d = 16 i + 4 j .. + 3
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float4* dst = reinterpret_cast<float4*>(s_out + rr * kHeadDim + 16 * i) + j;
                            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (w > 0) x = *dst;
                            // a warp that saw nothing adds nothing (its factor 0 times 0)
                            *dst = make_float4(x.x + o[t][2 * j][e] * f, x.y + o[t][2 * j][e + 2] * f,
                                               x.z + o[t][2 * j + 1][e] * f, x.w + o[t][2 * j + 1][e + 2] * f);
                        }
                    }
            }
            bar_sync(1, 32 * kConsumers);
        }
        if (!dead) {
            // complete: this CTA saw all of the item's units; else a partial result
            const bool complete = SPARSE ? p.nsplit == 1 : (sg.b0 == 0 && sg.b1 >= sg.nvis);
            const size_t part = SPARSE ? (size_t)blockIdx.x : (size_t)2 * blockIdx.x + (first_seg ? 0 : 1);
            for (int rr = warp; rr < rows; rr += kConsumers) {
                float M = kNegInf, Ls = 0.f;
#pragma unroll
                for (int x = 0; x < kConsumers; ++x) M = fmaxf(M, s_ml[x * RT + rr].x);
#pragma unroll
                for (int x = 0; x < kConsumers; ++x) {
                    const float2 a = s_ml[x * RT + rr];
                    Ls += a.x == kNegInf ? a.y : a.y * ex2(a.x - M);
                }
                float4 v = *reinterpret_cast<const float4*>(s_out + rr * kHeadDim + 4 * lane);
                if (complete) {
                    const float inv = Ls == 0.f ? 0.f : __fdividef(1.f, Ls);
                    const int x = row0 + rr, qi = SPARSE ? 0 : x / g, j = x - qi * g;
                    const size_t at = (size_t)(sg.q0 + qi) * p.Hq + sg.h * g + j;
                    uint2 w;
                    w.x = pack_bf16x2(v.x * inv, v.y * inv);
                    w.y = pack_bf16x2(v.z * inv, v.w * inv);
                    reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + at * kHeadDim)[lane] = w;
                    const float l2 = Ls == 0.f ? kNegInf : M - kOffset + lg2(Ls);
                    if (lane == 0 && p.lse) p.lse[at] = l2 * 0.69314718055994531f;
                    if (WEIGHTS && lane == 0) p.ws_lse[at] = l2;
                } else if (!SPARSE ? e0 < e1 : true) {
                    float* dst = p.part_o + (part * RT + rr) * kHeadDim;
                    reinterpret_cast<float4*>(dst)[lane] = v;
                    if (lane == 0) p.part_ml[part * RT + rr] = make_float2(M, Ls);
                }
            }
        }
        bar_sync(1, 32 * kConsumers);  // s_out and s_ml are free again
        first_seg = false;
    }
}

// ------------------------------------------------------------------ merge
__device__ __forceinline__ void merge_write(const CacheAttnParams& p, int q0, int h, int x, float M, float Ls, float4 v,
                                            int lane) {
    const int qi = x / p.g, j = x - qi * p.g;
    const size_t at = (size_t)(q0 + qi) * p.Hq + h * p.g + j;
    const float inv = Ls == 0.f ? 0.f : __fdividef(1.f, Ls);
    uint2 w;
    w.x = pack_bf16x2(v.x * inv, v.y * inv);
    w.y = pack_bf16x2(v.z * inv, v.w * inv);
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + at * kHeadDim)[lane] = w;
    if (lane == 0) {
        const float l2 = Ls == 0.f ? kNegInf : M - kOffset + lg2(Ls);
        if (p.lse) p.lse[at] = l2 * 0.69314718055994531f;
        if (p.weight) p.ws_lse[at] = l2;
    }
}

// Row x of query q0's tile from nc partial results, at(c) their places: 32 maxima and sums at a time, a lane
// each, and the outputs added in order.
template <class At>
__device__ __forceinline__ void merge_row(const CacheAttnParams& p, int q0, int h, int x, int nc, int lane, At at) {
    float M = kNegInf, Ls = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b < nc; b += 32) {
        float2 ml = make_float2(kNegInf, 0.f);
        if (b + lane < nc) ml = p.part_ml[at(b + lane)];
        float top = ml.x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        if (top > M) {  // what was added so far is relative to M
            const float f = ex2(M - top);
            Ls *= f;
            acc.x *= f;
            acc.y *= f;
            acc.z *= f;
            acc.w *= f;
            M = top;
        }
        // a part that saw nothing holds zeros; NaN goes through
        const float f = ml.x == kNegInf ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - M);
        const float lf = ml.y * f;
#pragma unroll 4
        for (int c = 0; c < min(32, nc - b); ++c) {
            const float fc = __shfl_sync(0xffffffffu, f, c);
            const float4 v = reinterpret_cast<const float4*>(p.part_o + at(b + c) * kHeadDim)[lane];
            Ls += __shfl_sync(0xffffffffu, lf, c);
            acc.x += v.x * fc;
            acc.y += v.y * fc;
            acc.z += v.z * fc;
            acc.w += v.w * fc;
        }
    }
    merge_write(p, q0, h, x, M, Ls, acc, lane);
}

// One CTA per item: the partial results of its rows, in the order of the CTAs that left them.  Rows
// of an item that one CTA finished are left alone, as are those of faulty requests; rows that see nothing get
// O = 0, lse = -inf.
template <int RT, bool SPARSE>
__global__ void __launch_bounds__(kHeadDim) cache_merge_kernel(const __grid_constant__ CacheAttnParams p, int grid_x) {
    __shared__ long long red[2][kHeadDim / 32];
    grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = p.g;
    int q0, rows, row0, h, c0, nc;
    if constexpr (SPARSE) {
        const int item = blockIdx.x;
        q0 = item / p.c.Hkv;
        h = item - q0 * p.c.Hkv;
        row0 = 0;
        rows = g;
        c0 = item * p.nsplit;
        nc = p.nsplit;
        bool in = false;
        for (int r = tid; r < p.c.R; r += kHeadDim) in = in || (p.q_ptr[r] <= q0 && q0 < p.q_ptr[r + 1]);
        if (!__syncthreads_or(in)) return;
    } else {
        const int per_r = p.c.Hkv * p.max_tiles, r = blockIdx.x / per_r, x = blockIdx.x - r * per_r;
        const Request q = load_request(p.q_ptr, p.Nq, p.c.kv_len, p.c.page_ptr, p.c.total_pages, p.c.T, r);
        const bool mine = request_fault(p, q) == 0u && (long long)q.n * g < p.big_rows;
        const int nt = mine ? tiles_of(q.n, g, RT) : 0;
        h = x / p.max_tiles;
        const int tile = x - h * p.max_tiles;
        if (tile >= nt) return;
        q0 = q.q0;
        row0 = tile * RT;
        rows = min(RT, q.n * g - row0);
        const int nb = units_of(q.len);
        const int vis = q.len - q.n + (row0 + rows - 1) / g + 1;
        const int nvis = vis <= 0 ? 0 : units_of(vis);
        c0 = 0;
        nc = 0;
        if (nvis > 0) {
            long long sum = 0, upto = 0;
            unsigned bad = 0;
            for (int y = tid; y < p.c.R; y += kHeadDim) {
                const int u = request_units(p, y, RT, &bad);
                sum += u;
                if (y < r) upto += u;
            }
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, s);
                upto += __shfl_xor_sync(0xffffffffu, upto, s);
            }
            if (lane == 0) {
                red[0][warp] = sum;
                red[1][warp] = upto;
            }
            __syncthreads();
            sum = upto = 0;
            for (int y = 0; y < kHeadDim / 32; ++y) {
                sum += red[0][y];
                upto += red[1][y];
            }
            const int per = units_per_cta(sum, grid_x);
            const long long a = upto + (h * nt + tile) * nb;  // the item's first unit
            c0 = (int)(a / per);
            nc = (int)((a + nvis - 1) / per) - c0 + 1;
            if (nc == 1) return;
            // CTA c's partial is its first segment's unless the item begins inside its run
            for (int rr = warp; rr < rows; rr += kHeadDim / 32)
                merge_row(p, q0, h, row0 + rr, nc, lane, [&](int c) {
                    return ((size_t)2 * (c0 + c) + ((long long)(c0 + c) * per >= a ? 0 : 1)) * RT + rr;
                });
            return;
        }
    }
    for (int rr = warp; rr < rows; rr += kHeadDim / 32)
        merge_row(p, q0, h, row0 + rr, nc, lane, [&](int c) { return (size_t)(c0 + c) * RT + rr; });
}

// ------------------------------------------------------------------ page weights
// weight[page][h] = sum over the request's rows of the softmax weight on the page's tokens, from the
// sums that the attention kernel kept for every 16 tokens and row (and the maximum each was
// relative to).  One warp per KV head and a few pages, 32 / S pages at a time with S lanes on each; added
// in a fixed order.  Bound by the latency of its dependent loads.
constexpr int kWeightWarps = 8, kWeightTurns = 2;
template <bool SPARSE>
__global__ void __launch_bounds__(32 * kWeightWarps) cache_weight_kernel(const __grid_constant__ CacheAttnParams p,
                                                                         int S) {
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const long long x = (long long)blockIdx.x * kWeightWarps + (threadIdx.x >> 5);
    const int run = (int)(x / p.c.Hkv), h = (int)(x - (long long)run * p.c.Hkv);
    const int u0 = run * kWeightTurns * (32 / S), u1 = min(p.c.total_pages, u0 + kWeightTurns * (32 / S));
    if (u0 >= p.c.total_pages) return;
    const int T = p.c.T, g = p.g, sub = lane & (S - 1);
    // the lane's page and its request, looked up again only past the request's end
    int r = -1, end = -1;
    Request q{};
    bool ok = false;
    for (int u = u0 + lane / S; u - lane / S < u1; u += 32 / S) {
        if (u < u1 && u >= end) {
            int lo = 0, hi = p.c.R;  // the last request that begins at or before the page
            while (lo + 1 < hi) {
                const int mid = (lo + hi) / 2;
                if (p.c.page_ptr[mid] <= u) lo = mid;
                else hi = mid;
            }
            r = p.c.page_ptr[lo] <= u && u < p.c.page_ptr[lo + 1] ? lo : -1;
            if (r >= 0) {
                q = load_request(p.q_ptr, p.Nq, p.c.kv_len, p.c.page_ptr, p.c.total_pages, T, r);
                ok = request_fault(p, q) == 0u;
                end = p.c.page_ptr[r + 1];
            }
        }
        const bool on = u < u1 && r >= 0;  // a page of no request is left as it is
        float sum = 0.f;
        if (on && ok) {
            const int pg = u - q.p0;
            // the chunk kernel keeps one sum for each page and row, the other one for every 16 tokens
            const int rows = q.n * g;
            const bool big = !SPARSE && rows >= p.big_rows;
            const int total = rows * (big ? 1 : T / 16);
            const float2* src = SPARSE ? nullptr : mass_of(p, q, h, big) + (size_t)pg * total;
            const uint32_t* bits = SPARSE ? p.ws_bits + (size_t)(q.p0 / 32 + r) * p.max_q * p.c.Hkv : nullptr;
            for (int e = pg * T < q.len ? sub : total; e < total; e += S) {
                const int grp = e / rows, row = e - grp * rows, qi = row / g, j = row - qi * g;
                float2 a = make_float2(0.f, 0.f);
                float l2 = 0.f;
                const auto lse = [&] { return p.ws_lse[(size_t)(q.q0 + qi) * p.Hq + h * g + j]; };
                if (!SPARSE) {  // loaded whether the row sees the page or not, so that the loads wait for no test
                    a = src[e];
                    l2 = lse();
                }
                const int pos = pg * T + 16 * grp;
                // the attention kernel reads whole tiles: what a row does not see it has as zero, but
                // 16 tokens that no row of its tile sees it leaves out
                if (pos >= q.len - q.n + qi + 1) continue;
                if (SPARSE) {
                    if (!((bits[((size_t)qi * p.c.Hkv + h) * ((q.np + 31) / 32) + (pg >> 5)] >> (pg & 31)) & 1u)) continue;
                    a = mass_of_query(p, q, h, qi)[((size_t)pg * (T / 16) + grp) * g + j];
                    l2 = lse();
                }
                // a row whose running maximum was still -inf has 0 here; NaN stays NaN
                // the factor in two halves: a.x is large where the page's V scale is small, and the whole factor
                // would be lost below 2^-126 where their product is not
                const float half = ex2(0.5f * ((a.y == kNegInf ? 0.f : a.y - kOffset) - l2));
                sum += a.x == 0.f ? 0.f : a.x * half * half;
            }
        }
        for (int s = S / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        if (on && sub == 0) p.weight[(size_t)u * p.c.Hkv + h] = sum;
    }
}

template <int NT, bool SPARSE, bool WEIGHTS>
cudaError_t launch_main(const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p, int grid,
                        cudaStream_t stream) {
    const size_t smem = cache_attn_smem(NT, SPARSE, p.max_pages, p.list_cap);
    const cudaError_t e = ensure_smem_attr((const void*)cache_attn_kernel<NT, SPARSE, WEIGHTS>, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_attn_kernel<NT, SPARSE, WEIGHTS>, dim3(grid), dim3(kThreads), smem, stream, tmK, tmV, p);
}

template <int NT>
cudaError_t launch_sparse(const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p, int grid, int items,
                          cudaStream_t stream) {
    const cudaError_t e = p.weight ? launch_main<NT, true, true>(tmK, tmV, p, grid, stream)
                                   : launch_main<NT, true, false>(tmK, tmV, p, grid, stream);
    if (e != cudaSuccess || p.nsplit == 1) return e;
    return launch_pdl(cache_merge_kernel<8 * NT, true>, dim3(items), dim3(kHeadDim), 0, stream, p, grid);
}

template <int NT>
cudaError_t launch_dense(const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p, int grid, int items,
                         cudaStream_t stream) {
    const cudaError_t e = p.weight ? launch_main<NT, false, true>(tmK, tmV, p, grid, stream)
                                   : launch_main<NT, false, false>(tmK, tmV, p, grid, stream);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_merge_kernel<8 * NT, false>, dim3(items), dim3(kHeadDim), 0, stream, p, grid);
}

}  // namespace

size_t cache_attn_smem(int nt, bool sparse, int max_pages, int list_cap) {
    size_t s = nt == 1 ? Smem<1>::list : (nt == 2 ? Smem<2>::list : Smem<4>::list);
    if (sparse) s += (size_t)((max_pages + 31) / 32) * 8 + (size_t)list_cap * 8;
    return s + 1024;
}

cudaError_t launch_cache_attn(int nt, const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p,
                              int grid, int items, cudaStream_t stream) {
    if (!p.topk)  // up to 16 rows: more are the chunk kernel's
        return nt == 1 ? launch_dense<1>(tmK, tmV, p, grid, items, stream)
                       : launch_dense<2>(tmK, tmV, p, grid, items, stream);
    return nt == 1   ? launch_sparse<1>(tmK, tmV, p, grid, items, stream)
           : nt == 2 ? launch_sparse<2>(tmK, tmV, p, grid, items, stream)
                     : launch_sparse<4>(tmK, tmV, p, grid, items, stream);
}

cudaError_t launch_cache_weights(const CacheAttnParams& p, cudaStream_t stream) {
    // lanes on a page: as many as it has sums, up to a warp
    const long long sums = (long long)p.max_q * p.g * (p.max_q * p.g >= p.big_rows ? 1 : p.c.T / 16);
    int S = 2;
    while (S < 32 && S < sums) S *= 2;
    const int pages = kWeightTurns * (32 / S);
    const long long warps = (long long)((p.c.total_pages + pages - 1) / pages) * p.c.Hkv;
    const dim3 grid((unsigned)((warps + kWeightWarps - 1) / kWeightWarps));
    return p.topk ? launch_pdl(cache_weight_kernel<true>, grid, dim3(32 * kWeightWarps), 0, stream, p, S)
                  : launch_pdl(cache_weight_kernel<false>, grid, dim3(32 * kWeightWarps), 0, stream, p, S);
}

}  // namespace qup
