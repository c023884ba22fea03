// cache_chunk.cu -- attention over the 8-bit page-scaled cache for requests with many query rows
// (chunks of a prompt, drafted tokens): tcgen05 with the accumulators in TMEM.
//
// The mathematics is cache_attn.cu's: per row x_t = f q.k_t + log2 vs, with f = softmax_scale * log2e *
// ks of the token's page, p_t = 2^(x_t - m + 8), O = sum p_t v_t / sum (p_t / vs).
//
// Numbers.  S = Q K^T runs in kind::f8f6f4 straight on the cache's bytes: a bf16 row of Q is the sum of
// two E4M3 rows.  With the row scaled by a power of two so that its largest element lies in [128, 256),
// the high part is that element rounded to E4M3 (4 significant bits) and the low part the rest (at
// most 4 bits): exact for elements down to 2^-9 of the largest, within 2^-17 of the largest below.
// Two products of 8-bit operands cost what one of 16-bit operands does, and K needs no conversion.
// fp32 sums of E4M3 products on this part were measured against fp64: within 2^-21 of sum |q||k|.
// P is rounded to fp16 (half step 2^-11), V converted to fp16 (exact), O and the row sums are fp32.
//
// A work item is a tile of 256 rows (query, head of the KV head's group) of one KV head: two row tiles
// of 128, each with a softmax warpgroup, an S buffer and an O accumulator (512 TMEM columns).  While one
// warpgroup computes exponentials the tensor cores work for the other.  Steps of 128 tokens: all items'
// visible steps are laid end to end and cut into one equal run per CTA (one per SM); an item cut by a
// run's end leaves partial results, which a second kernel joins in a fixed order.
//
// Warps (384 threads): 0-3 and 4-7 softmax of row tile 0 and 1 (thread = row); 8 issues S and O += P V,
// 9 loads K and V bytes by TMA and the pages' constants; 10 and 11 convert V tiles to fp16 in the
// 128-byte-swizzled MN-major operand layout.  P goes over S in TMEM.
//
// NaN: a NaN byte of V that a row does not see must not reach it as 0 * NaN.  The converters store 0 for
// it and remember its column's first such token; the epilogue gives NaN to the rows that see it.
//
// Bound: a step of 256 rows takes about 4,600 cycles.  The two warpgroups' softmax takes 2,500 to 3,200 of
// them together (their exponentials alone 1,800 to 2,100, of which the MUFU unit 1,790), the tensor
// cores 2,050; what does not overlap is the way from P to the next S (O update, S, two completions of
// 200 to 400 cycles each).  1,024 queries x 32 heads behind 16K tokens: 316 to 328 us, 0.88 PFLOP/s.
// Measured and left out: loops unrolled over a step (instruction fetch: +23 %), the warpgroups taking
// turns (+57 %: one alone is hardly faster than both together), half steps with S, P and O update of their
// own (+14 %: products of 64 columns take as long to issue as of 128), a step's tokens split over both
// warpgroups for items of few rows (-6 % for 35 rows, +3 % for chunks), four converting warps of 128
// registers (+3 %), an E4M3 pair for P as for Q (three conversions of 6 cycles a pair instead of one of 2).
#include <algorithm>
#include <cstdint>

#include "cache.h"
#include "cache_attn.h"
#include "internal.h"
#include "ptx.cuh"
#include "query_union_paged.h"

namespace qup {
namespace {

constexpr int kThreads = 384;
constexpr int kStep = 128;                  // tokens of a step
constexpr int kCols = 32;                   // scores that a softmax thread works on at a time
constexpr int kTileRows = 128;              // rows of a warpgroup
constexpr int kItemRows = kChunkRows;       // rows of an item
constexpr int kTile = kStep * kHeadDim;     // bytes of a K or V tile
constexpr int kNK = 3, kNV = 2, kNM = 8;    // K tiles, V tiles, page constants in flight
constexpr int kConvRows = 2;                // rows of V that a converting lane has in hand
constexpr int kMarks = 5;                   // segments whose NaN marks are held
constexpr int kMaxPages = kStep / 16;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kConvWarp = 10, kConvWarps = 2;
constexpr uint32_t kColO = 0, kColS = 256;
constexpr int kPolyPairs = 1;      // of every eight pairs of exponentials, those on the FMA pipe
constexpr float kOffset = 8.f;     // log2 offset of P
constexpr float kLazy = 7.f;       // the maximum moves once a score passes it by this: P <= 2^15
constexpr float kZeroScaleLog2 = -64.f;
constexpr float kNegInf = -INFINITY;

struct __align__(16) StepMeta {  // the pages of a step
    float4 page[kMaxPages];  // ks, log2 vs, 1 / vs
    uint32_t valid, negative;  // pages that are seen, that have a negative K scale
    uint32_t pad[2];
};

struct NanMarks {  // of one segment
    int first[kHeadDim];  // token of the first NaN in each column of V
    int any;
    int pad[3];
};

struct WarpWalk;
struct Layout {
    static constexpr uint32_t q = 0;                                // [2][hi, lo][128][128]
    static constexpr uint32_t k = q + 4 * kTile;                    // [kNK]
    static constexpr uint32_t v = k + kNK * kTile;                  // [kNV]
    static constexpr uint32_t v16 = v + kNV * kTile;                // [2] fp16 tiles
    static constexpr uint32_t meta = v16 + 4 * kTile;
    static constexpr uint32_t nan = meta + kNM * sizeof(StepMeta);  // [kMarks]
    static constexpr uint32_t bars = nan + kMarks * sizeof(NanMarks);
    static constexpr uint32_t scan = bars + 8 * 40;                 // one int64 per warp
    static constexpr uint32_t misc = scan + 8 * 16;
    static constexpr uint32_t walks = misc + 64;                    // one per warp
    static constexpr uint32_t total = walks + (kThreads / 32) * 128;
};

__device__ __forceinline__ void f16x2_to_f32(uint32_t v, float& lo, float& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(v));
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {  // NaN if any is
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// sum over t in [0, n) of floor((a t + b) / m); a n + b fits 32 bits
__device__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    long long s = 0;
    while (n > 0) {
        s += (long long)((unsigned long long)(n - 1) * n / 2) * (a / m) + (long long)n * (b / m);
        a %= m;
        b %= m;
        const uint32_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const uint32_t x = m;
        m = a;
        a = x;
    }
    return s;
}

// One request's items (none of a faulty one).  Row tile t's steps: floor((g (base + 127) + last row) /
// (128 g)) with base = tokens its first query sees, which is ceil(tokens its last row sees / 128).
struct Items {
    Request q;
    int nt, rows, base;
    __device__ __forceinline__ void load(const CacheAttnParams& p, int r, unsigned* fault) {
        q = load_request(p.q_ptr, p.Nq, p.c.kv_len, p.c.page_ptr, p.c.total_pages, p.c.T, r);
        const unsigned f = request_fault(p, q);
        *fault |= f;
        rows = f ? 0 : q.n * p.g;
        if (rows < p.big_rows) rows = 0;  // the other kernel's
        nt = (rows + kItemRows - 1) / kItemRows;
        base = max(q.len - q.n, 0) + 1;
    }
    __device__ __forceinline__ int steps(const CacheAttnParams& p, int t) const {
        const int last = min((t + 1) * kItemRows, rows) - 1;
        return (int)((uint32_t)(p.g * (base + kStep - 1) + last) / (uint32_t)(kStep * p.g));
    }
    // steps of the first t < nt row tiles
    __device__ __forceinline__ long long before(const CacheAttnParams& p, int t) const {
        return floor_sum(t, kStep * p.g, kItemRows, p.g * (base + kStep - 1) + kItemRows - 1);
    }
    __device__ __forceinline__ long long total(const CacheAttnParams& p) const {
        return nt == 0 ? 0 : (before(p, nt - 1) + steps(p, nt - 1)) * p.c.Hkv;
    }
};

struct Seg {
    int r, h, tile, b0, b1, steps;
};

struct Walk {  // a CTA's run of steps, item by item
    int r, h, tile, b, left;
    bool loaded;
    Items it;
    __device__ __forceinline__ void begin(const int* start) {
        r = start[0];
        h = start[1];
        tile = start[2];
        b = start[3];
        left = start[4];
        loaded = false;
    }
    __device__ __forceinline__ bool next(const CacheAttnParams& p, Seg& s) {
        while (left > 0 && r < p.c.R) {
            if (!loaded) {
                unsigned f = 0;
                it.load(p, r, &f);
                loaded = true;
            }
            if (it.nt == 0 || h >= p.c.Hkv) {
                ++r;
                h = tile = b = 0;
                loaded = false;
                continue;
            }
            s.r = r;
            s.h = h;
            s.tile = tile;
            s.steps = it.steps(p, tile);
            s.b0 = b;
            s.b1 = min(s.steps, b + left);
            left -= s.b1 - s.b0;
            b = s.b1;
            if (b >= s.steps) {
                b = 0;
                if (++tile == it.nt) {
                    tile = 0;
                    ++h;
                }
            }
            return true;
        }
        return false;
    }
};

// A warp's walk and the segment it is in, in shared memory (kept in registers, they would be spilled
// around the softmax loop, to local memory for which little L1 is left): lane 0 moves it on.
struct WarpWalk {
    Walk wk;
    Seg sg;
    int more;
    __device__ __forceinline__ void begin(const int* start, int lane) {
        if (lane == 0) wk.begin(start);
        __syncwarp();
    }
    __device__ __forceinline__ bool next(const CacheAttnParams& p, int lane) {
        __syncwarp();
        if (lane == 0) more = wk.next(p, sg);
        __syncwarp();
        return more != 0;
    }
};

static_assert(sizeof(WarpWalk) <= 128, "a warp's walk");

struct Bars {
    uint32_t base;
    __device__ __forceinline__ uint32_t at(int i) const { return base + 8u * i; }
    __device__ __forceinline__ uint32_t kfull(int s) const { return at(s); }
    __device__ __forceinline__ uint32_t kempty(int s) const { return at(kNK + s); }
    __device__ __forceinline__ uint32_t vfull(int s) const { return at(2 * kNK + s); }
    __device__ __forceinline__ uint32_t vempty(int s) const { return at(2 * kNK + kNV + s); }
    __device__ __forceinline__ uint32_t f(int i) const { return at(2 * kNK + 2 * kNV + i); }
    __device__ __forceinline__ uint32_t cfull(int s) const { return f(s); }       // fp16 V written
    __device__ __forceinline__ uint32_t cempty(int s) const { return f(2 + s); }  // fp16 V read
    __device__ __forceinline__ uint32_t sfull(int w) const { return f(4 + w); }
    __device__ __forceinline__ uint32_t pfull(int w, int half) const { return f(15 + 2 * w + half); }
    __device__ __forceinline__ uint32_t pvdone(int w) const { return f(8 + w); }
    __device__ __forceinline__ uint32_t qfull(int w) const { return f(10 + w); }
    __device__ __forceinline__ uint32_t drain() const { return f(12); }
    __device__ __forceinline__ uint32_t sdone() const { return f(14); }  // a segment's products are done
    __device__ __forceinline__ uint32_t mfull(int s) const { return f(19 + s); }
};
static_assert(2 * kNK + 2 * kNV + 19 + kNM <= 40, "barrier block");

__device__ __forceinline__ bool warp_ok(bool ok) { return __all_sync(0xffffffffu, ok); }

template <int T, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, 1)
    cache_chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CacheAttnParams p) {
    constexpr int PPS = kStep / T, TC = T < kCols ? T : kCols;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const Bars B{sbase + Layout::bars};
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + Layout::misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Layout::misc + 4);
    int* s_start = reinterpret_cast<int*>(smem + Layout::misc + 16);  // r, h, tile, b, count
    long long* scan = reinterpret_cast<long long*>(smem + Layout::scan);
    StepMeta* meta = reinterpret_cast<StepMeta*>(smem + Layout::meta);
    NanMarks* marks = reinterpret_cast<NanMarks*>(smem + Layout::nan);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t lim = p.wait_limit_ns;
    const int g = p.g;

    if (tid == 0) {
        for (int s = 0; s < kNK; ++s) {
            mbar_init(B.kfull(s), 1);
            mbar_init(B.kempty(s), 1);
        }
        for (int s = 0; s < kNV; ++s) {
            mbar_init(B.vfull(s), 1);
            mbar_init(B.vempty(s), kConvWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(B.cfull(s), kConvWarps);
            mbar_init(B.cempty(s), 1);
            mbar_init(B.sfull(s), 1);
            mbar_init(B.pfull(s, 0), 4);
            mbar_init(B.pfull(s, 1), 4);
            mbar_init(B.pvdone(s), 1);
            mbar_init(B.qfull(s), 4);
        }
        mbar_init(B.drain(), 1);
        mbar_init(B.sdone(), 1);
        for (int s = 0; s < kNM; ++s) mbar_init(B.mfull(s), 1);
        *abort_flag = 0;
        s_start[0] = p.c.R;
        s_start[4] = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < kMarks * (int)(sizeof(NanMarks) / 4); i += kThreads)
        reinterpret_cast<int*>(marks)[i] = i % (int)(sizeof(NanMarks) / 4) < kHeadDim ? 0x7fffffff : 0;
    if (tid == kLoadWarp * 32) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32((const void*)tmem_slot), 512);
        tmem_relinquish();
    }
    grid_dep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    {  // this CTA's run: requests' steps added up, each thread over its own consecutive requests
        const int span = (p.c.R + kThreads - 1) / kThreads;
        const int r0 = min(p.c.R, tid * span), r1 = min(p.c.R, r0 + span);
        long long sum = 0;
        unsigned fault = 0;
        for (int r = r0; r < r1; ++r) {
            Items it;
            it.load(p, r, &fault);
            sum += it.total(p);
        }
        if (fault) atomicOr(p.err, fault);
        long long run = sum;  // prefix over the CTA
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += y;
        }
        if (lane == 31) scan[warp] = run;
        __syncthreads();
        long long mine = run - sum, all = 0;
#pragma unroll
        for (int t = 0; t < kThreads / 32; ++t) {
            mine += t < warp ? scan[t] : 0;
            all += scan[t];
        }
        const long long per = max((all + gridDim.x - 1) / gridDim.x, 1ll);
        const long long u0 = (long long)blockIdx.x * per;
        if (u0 < all && u0 >= mine && u0 < mine + sum) {
            long long at = mine;
            for (int r = r0; r < r1; ++r) {
                Items it;
                it.load(p, r, &fault);
                const long long u = it.total(p);
                if (u0 < at + u) {
                    const long long head = u / p.c.Hkv, off = u0 - at;
                    const long long in = off % head;
                    int lo = 0, hi = it.nt - 1;  // the last tile whose steps start at or before `in`
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) / 2;
                        if (it.before(p, mid) <= in) lo = mid;
                        else hi = mid - 1;
                    }
                    s_start[0] = r;
                    s_start[1] = (int)(off / head);
                    s_start[2] = lo;
                    s_start[3] = (int)(in - it.before(p, lo));
                    s_start[4] = (int)min(per, all - u0);
                    break;
                }
                at += u;
            }
        }
        if (__syncthreads_or(fault != 0u)) clear_faulty(p, true);
    }

    WarpWalk& ww = *reinterpret_cast<WarpWalk*>(smem + Layout::walks + warp * 128);
    const Walk& wk = ww.wk;
    const Seg& sg = ww.sg;
    ww.begin(s_start, lane);

    if (warp >= 8) {
        if (warp == kLoadWarp) {
            // ==================================================== it
            ChunkSpan info{};
            uint32_t it = 0;
            bool ok = true;
            while (ok && ww.next(p, lane)) {
                info.r = sg.r;
                info.h = sg.h;
                info.tile = sg.tile;
                info.b0 = sg.b0;
                info.ends = sg.b1 == sg.steps;
                if (info.segs == 0) info.first_ends = info.ends;
                ++info.segs;
                const int b1 = sg.b1, h = sg.h, last = (wk.it.q.len + T - 1) / T, p0 = wk.it.q.p0;
                int have0 = 0, have1 = 0, phys = -1;  // page table entries that the lanes hold
                float ks = 0.f, vl = 0.f, vi = 0.f;
                for (int b = sg.b0; b < b1 && ok; ++b, ++it) {
                    const int pe = b * PPS;
                    if (pe + PPS > have1) {
                        have0 = pe;
                        have1 = pe + 32;
                        const int e = pe + lane;
                        phys = -1;
                        if (e < last) {
                            phys = p.c.page_table[p0 + e];
                            if (phys < 0 || phys >= p.c.P_phys) {
                                atomicOr(p.err, QUP_ERR_PHYS_PAGE);
                                phys = -1;
                            } else {
                                ks = __ldg(p.c.k_scale + (size_t)phys * p.c.Hkv + h);
                                const float vs = __ldg(p.c.v_scale + (size_t)phys * p.c.Hkv + h);
                                if (!(fabsf(ks) < INFINITY) || !v_scale_ok(vs)) {
                                    atomicOr(p.err, QUP_ERR_SCALE);
                                    phys = -1;
                                }
                                vl = vs > 0.f ? lg2(vs) : kZeroScaleLog2;
                                vi = vs > 0.f ? __frcp_rn(vs) : 18446744073709551616.f;
                            }
                        }
                        if (phys < 0) ks = vl = vi = 0.f;
                        if (!(ks < 0.f)) ks = fabsf(ks);  // -0 and what is flushed to it: not a negative scale
                    }
                    const int src = pe - have0;
                    const uint32_t live = (__ballot_sync(0xffffffffu, phys >= 0) >> src) & ((1u << PPS) - 1u);
                    const uint32_t neg = (__ballot_sync(0xffffffffu, ks < 0.f) >> src) & ((1u << PPS) - 1u);
                    const uint32_t bytes = __popc(live) * T * kHeadDim;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int n = kv ? kNV : kNK;
                        const uint32_t slot = it % n, par = (it / n) & 1;
                        if (!warp_ok(mbar_wait_idle(kv ? B.vempty(slot) : B.kempty(slot), par ^ 1, abort_flag, p.err,
                                                    QUP_ERR_TIMEOUT, lim)))
                            ok = false;
                        if (!ok) break;
                        if (kv == 0) {
                            // the constants' last readers, kNM steps ago, are done: S of a later step has run
                            StepMeta& m = meta[it % kNM];
                            if (lane >= src && lane < src + PPS) m.page[lane - src] = make_float4(ks, vl, vi, 0.f);
                            if (lane == 0) {
                                m.valid = live;
                                m.negative = neg;
                            }
                            __syncwarp();
                            if (lane == 0) mbar_arrive(B.mfull(it % kNM));
                        }
                        const uint32_t full = kv ? B.vfull(slot) : B.kfull(slot);
                        const bool load = it != (uint32_t)p.dbg_skip_stage;
                        if (lane == 0 && load) {
                            if (bytes) mbar_arrive_expect_tx(full, bytes);
                            else mbar_arrive(full);
                        }
                        __syncwarp();
                        if (lane >= src && lane < src + PPS && phys >= 0 && load)
                            tma_load_4d(sbase + (kv ? Layout::v : Layout::k) + slot * kTile +
                                            (uint32_t)(lane - src) * T * kHeadDim,
                                        kv ? &tmV : &tmK, full, 0, 0, h, phys);
                        __syncwarp();
                    }
                }
            }
            if (lane == 0) {
                p.spans[blockIdx.x] = info;
                if (*abort_flag) {  // what is in flight lands before the CTA leaves
                    for (uint32_t k = it > (uint32_t)kNK ? it - kNK : 0; k <= it; ++k)
                        mbar_wait_drain(B.kfull(k % kNK), (k / kNK) & 1, lim / 16);
                    for (uint32_t k = it > (uint32_t)kNV ? it - kNV : 0; k <= it; ++k)
                        mbar_wait_drain(B.vfull(k % kNV), (k / kNV) & 1, lim / 16);
                }
            }
            __syncwarp();
        } else if (warp == kMmaWarp) {
            // ==================================================== S = Q K^T and O += P V
            constexpr uint32_t idesc_s = instr_desc(0, 0, 0, kStep, kTileRows);
            constexpr uint32_t idesc_o = instr_desc(0, 0, 1, kHeadDim, kTileRows);
            uint32_t it = 0, use[2] = {0, 0}, segs = 0;
            bool ok = true;
            const auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = ok && warp_ok(mbar_wait_idle(bar, parity & 1, abort_flag, p.err, QUP_ERR_TIMEOUT, lim));
                if (ok) tc_fence_after();
                return ok;
            };
            const auto issue_s = [&](int w, uint32_t slot, bool last) {
                const uint64_t qd = smem_desc(sbase + Layout::q + w * 2 * kTile, 16, 1024, 2);
                const uint64_t kd = smem_desc(sbase + Layout::k + slot * kTile, 16, 1024, 2);
                if (elect_one_sync()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)  // the low parts of Q first
                        tc_mma<2>(tmem + kColS + 128u * w, qd + (((kk < 4 ? kTile : 0) + (kk & 3) * 32) >> 4),
                                  kd + (((kk & 3) * 32) >> 4), idesc_s, kk > 0);
                    tc_commit(B.sfull(w));
                    if (last) tc_commit(B.kempty(slot));
                }
                __syncwarp();
            };
            while (ok && ww.next(p, lane)) {
                const int nw = min(kItemRows, wk.it.rows - sg.tile * kItemRows) > kTileRows ? 2 : 1;
                const uint32_t sp = segs++ & 1;
                const int b0 = sg.b0, b1 = sg.b1;
                // the first S: both warpgroups have come to the segment (one may have no rows in it), and
                // the O updates that last read P from the S buffers are done (at the end of a segment
                // they are waited for below)
                wait(B.qfull(0), sp);
                wait(B.qfull(1), sp);
                if (!wait(B.kfull(it % kNK), it / kNK)) break;
                for (int w = 0; w < nw; ++w) issue_s(w, it % kNK, w == nw - 1);
                for (int b = b0; b < b1 && ok; ++b, ++it) {
                    if (!wait(B.cfull(it & 1), it >> 1)) break;
                    for (int w = 0; w < nw && ok; ++w) {
                        const uint32_t k = use[w]++;
                        const uint64_t vd = smem_desc(sbase + Layout::v16 + (it & 1) * 2 * kTile, kTile, 1024, 2);
                        for (int half = 0; half < 2; ++half) {  // tokens 0 .. 63, then 64 .. 127
                            if (!wait(B.pfull(w, half), k)) break;
                            if (elect_one_sync()) {
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)  // 16 tokens each
                                    tc_mma_ts<0>(tmem + kColO + 128u * w, tmem + kColS + 128u * w + 32u * half + 8u * kk,
                                                 vd + (((4 * half + kk) * 16 * 128) >> 4), idesc_o,
                                                 b > b0 || half > 0 || kk > 0);
                                if (half == 1) tc_commit(B.pvdone(w));
                                if (half == 1 && w == nw - 1) tc_commit(B.cempty(it & 1));
                            }
                            __syncwarp();
                        }
                        // the tile's next S, over the P that this update read
                        if (b + 1 < b1) {
                            if (w == 0) wait(B.kfull((it + 1) % kNK), (it + 1) / kNK);
                            if (!wait(B.pvdone(w), k)) break;
                            issue_s(w, (it + 1) % kNK, w == nw - 1);
                        } else {
                            wait(B.pvdone(w), k);
                        }
                    }
                }
                if (lane == 0) mbar_arrive(B.sdone());
                __syncwarp();
            }
            if (elect_one_sync()) tc_commit(B.drain());
            __syncwarp();
            mbar_wait_drain(B.drain(), 0, lim);
            __syncwarp();
        } else if (warp >= kConvWarp) {
            // ==================================================== V: E4M3 bytes -> fp16 operand tiles
            const int cw = warp - kConvWarp, row8 = lane >> 3, ch = lane & 7;
            uint32_t it = 0, segs = 0;
            bool ok = true;
            while (ok && ww.next(p, lane)) {
                NanMarks& nm = marks[segs % kMarks];
                NanMarks& later = marks[(segs + 2) % kMarks];
                const int len = wk.it.q.len;
                ++segs;
                const int b0 = sg.b0, b1 = sg.b1;
                for (int b = b0; b < b1 && ok; ++b, ++it) {
                    const uint32_t vs = it % kNV, cs = it & 1;
                    ok = warp_ok(mbar_wait_idle(B.vfull(vs), (it / kNV) & 1, abort_flag, p.err, QUP_ERR_TIMEOUT, lim) &&
                                 mbar_wait_idle(B.cempty(cs), ((it >> 1) & 1) ^ 1, abort_flag, p.err, QUP_ERR_TIMEOUT,
                                                lim));
                    if (!ok) break;
                    // The marks of the segment after the next are cleared.  The other warp comes to them two
                    // steps later at the earliest, after an O update that waits for this warp's tile here.
                    // Their last readers, five segments before, are done: the O update two steps ago
                    // belongs to segment - 2 or later, whose S waited for both warpgroups to have left
                    // segment - 3.
                    if (b == b0 && cw == 0) {
                        for (int d = lane; d < kHeadDim; d += 32) later.first[d] = 0x7fffffff;
                        if (lane == 0) later.any = 0;
                        __syncwarp();
                    }
                    const uint32_t valid = meta[it % kNM].valid;
                    const int here = len - b * kStep;  // tokens of the step that exist
                    const uint8_t* src = smem + Layout::v + vs * kTile + row8 * 128;
                    uint8_t* dst = smem + Layout::v16 + cs * 2 * kTile + row8 * 128;
                    const bool whole = here >= kStep && valid == (1u << PPS) - 1u;
                    // a quarter of a warp's lanes share a row of 128 bytes: 16 each (rolled, as the softmax
                    // loops are)
#pragma unroll 1
                    for (int r0 = cw * (kStep / kConvWarps); r0 < (cw + 1) * (kStep / kConvWarps); r0 += 4 * kConvRows) {
                        uint4 raw[kConvRows];
                        uint32_t odd = 0;  // a NaN among them
#pragma unroll
                        for (int u = 0; u < kConvRows; ++u) {  // rows r0 + 4 u + row8
                            raw[u] = *reinterpret_cast<const uint4*>(src + (r0 + 4 * u) * 128 + ((ch ^ (4 * (u & 1) + row8)) << 4));
                            odd |= nan_bytes(raw[u].x) | nan_bytes(raw[u].y) | nan_bytes(raw[u].z) | nan_bytes(raw[u].w);
                        }
                        if (!whole || __any_sync(0xffffffffu, odd != 0u)) {
#pragma unroll
                            for (int u = 0; u < kConvRows; ++u) {
                                const int row = r0 + 4 * u + row8;
                                uint32_t w4[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                                if (row >= here || !((valid >> (row / T)) & 1u)) w4[0] = w4[1] = w4[2] = w4[3] = 0u;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t bad = nan_bytes(w4[e]);
                                    if (bad) {
#pragma unroll 1
                                        for (int x = 0; x < 4; ++x)
                                            if ((bad >> (8 * x)) & 0x80u)
                                                atomicMin(&nm.first[16 * ch + 4 * e + x], b * kStep + row);
                                        nm.any = 1;
                                        w4[e] &= ~((bad >> 7) * 0xffu);
                                    }
                                }
                                raw[u] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < kConvRows; ++u) {
                            uint4 o0, o1;
                            cvt_e4m3x4(raw[u].x, o0.x, o0.y);
                            cvt_e4m3x4(raw[u].y, o0.z, o0.w);
                            cvt_e4m3x4(raw[u].z, o1.x, o1.y);
                            cvt_e4m3x4(raw[u].w, o1.z, o1.w);
                            // 64 columns in each half; lanes of the two halves store their chunks in
                            // opposite order, so a quarter warp's eight stores meet different banks
                            const bool hi = ch >= 4;
                            uint8_t* line = dst + (hi ? kTile : 0) + (r0 + 4 * u) * 128;
                            const int c0 = (2 * (ch & 3) + (hi ? 1 : 0)) ^ (4 * (u & 1) + row8);
                            *reinterpret_cast<uint4*>(line + (c0 << 4)) = hi ? o1 : o0;
                            *reinterpret_cast<uint4*>(line + ((c0 ^ 1) << 4)) = hi ? o0 : o1;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(B.cfull(cs));
                        mbar_arrive(B.vempty(vs));
                    }
                }
            }
        }
    } else {
        // ======================================================== softmax, epilogue
        const int w = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + kColS + 128u * w, o_addr = tmem + lane_base + kColO + 128u * w;
        uint32_t it = 0, use = 0, segs = 0;
        bool ok = true;
        while (ok && ww.next(p, lane)) {
            const NanMarks& nm = marks[segs % kMarks];
            const bool first_seg = segs == 0;
            ++segs;
            const int row0 = sg.tile * kItemRows + w * kTileRows;  // of the warpgroup, in (query, head) order
            const int rows = min(kTileRows, wk.it.rows - row0);
            if (rows <= 0) {  // an empty row tile: the warpgroup reports its place in the walk and waits
                it += sg.b1 - sg.b0;
                if (lane == 0) mbar_arrive(B.qfull(w));
                ok = warp_ok(mbar_wait_idle(B.sdone(), (segs - 1) & 1, abort_flag, p.err, QUP_ERR_TIMEOUT, lim));
                continue;
            }
            const bool on = r < rows;
            const int x = row0 + (on ? r : rows - 1), qi = x / g, j = x - qi * g;
            // tokens this row sees, and the warpgroup's first row
            const int vis = wk.it.q.len - wk.it.q.n + qi + 1;
            const int vis_all = wk.it.q.len - wk.it.q.n + row0 / g + 1;
            // ---- Q: high and low E4M3 parts of the warp's rows, each row's score factor.  16 lanes share a
            // row: 8 elements each.  The bf16 rows come into the places that their two parts will take.
            float rs = 0.f;
            {
                const uint16_t* q0 = static_cast<const uint16_t*>(p.Q) + (size_t)wk.it.q.q0 * p.q_stride +
                                     (size_t)(sg.h * g) * kHeadDim + (lane & 15) * 8;
                uint8_t* qt = smem + Layout::q + w * 2 * kTile + wq * 32 * 128;
                const uint32_t from = (uint32_t)((lane & 8) ? kTile : 0) + (lane >> 4) * 128 + (lane & 7) * 16;
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const int row = 2 * i + (lane >> 4);
                    const int yq = __shfl_sync(0xffffffffu, qi, row), yj = __shfl_sync(0xffffffffu, j, row);
                    copy16_async(smem_u32(qt) + from + i * 256, q0 + (size_t)yq * p.q_stride + yj * kHeadDim);
                }
                copy_async_wait();
                __syncwarp();
#pragma unroll 2
                for (int i = 0; i < 16; ++i) {
                    const uint4 raw = *reinterpret_cast<const uint4*>(qt + from + i * 256);
                    const uint32_t w4[4] = {raw.x, raw.y, raw.z, raw.w};
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max((w4[e] << 16) & 0x7f800000u, w4[e] & 0x7f800000u));
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const int ex = max((int)(top >> 23) - 127, -100);  // the largest element is in [2^ex, 2^(ex+1))
                    const float up = __uint_as_float((uint32_t)(7 - ex + 127) << 23);
                    const int mine = __shfl_sync(0xffffffffu, ex, (lane & 1) << 4);  // of row 2 i + (lane & 1)
                    if ((lane >> 1) == i) {
                        rs = p.scale_log2 * __uint_as_float((uint32_t)(mine - 7 + 127) << 23);
                        if (mine == 128) rs = __uint_as_float(0x7fc00000u);  // an infinity or NaN in the row
                    }
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t a = w4[2 * e], bb = w4[2 * e + 1];
                        const float y[4] = {__uint_as_float(a << 16) * up, __uint_as_float(a & 0xffff0000u) * up,
                                            __uint_as_float(bb << 16) * up, __uint_as_float(bb & 0xffff0000u) * up};
                        hi[e] = pack_e4m3x4(y[0], y[1], y[2], y[3]);
                        float z[4];
                        uint32_t h01, h23;
                        cvt_e4m3x4(hi[e], h01, h23);
                        f16x2_to_f32(h01, z[0], z[1]);
                        f16x2_to_f32(h23, z[2], z[3]);
                        lo[e] = pack_e4m3x4(y[0] - z[0], y[1] - z[1], y[2] - z[2], y[3] - z[3]);
                    }
                    __syncwarp();  // both rows have been read
                    const int row = 2 * i + (lane >> 4), ch = (lane & 15) >> 1;
                    uint8_t* dst = qt + row * 128 + ((ch ^ (row & 7)) << 4) + (lane & 1) * 8;
                    *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2*>(dst + kTile) = make_uint2(lo[0], lo[1]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(B.qfull(w));
            }
            float m = kNegInf, l = 0.f;
            const int b0 = sg.b0, b1 = sg.b1;
            float2* mass_row = nullptr;  // page weights: this row's sums, mass_rows apart
            int mass_pages = 0, mass_rows = 0;
            if (WEIGHTS && on) {
                mass_row = mass_of(p, wk.it.q, sg.h, true) + x;
                mass_rows = wk.it.rows;
                mass_pages = (wk.it.q.len + T - 1) / T;
            }
            for (int b = b0; b < b1; ++b, ++it) {
                const uint32_t k = use++;
                ok = warp_ok(mbar_wait_idle(B.mfull(it % kNM), (it / kNM) & 1, abort_flag, p.err, QUP_ERR_TIMEOUT, lim));
                if (!ok) break;
                const StepMeta& sm = meta[it % kNM];
                const uint32_t valid = sm.valid;
                const bool plain = valid == (1u << PPS) - 1u && sm.negative == 0u && (b + 1) * kStep <= vis_all;
                ok = warp_ok(mbar_wait_idle(B.sfull(w), k & 1, abort_flag, p.err, QUP_ERR_TIMEOUT, lim));
                if (!ok) break;
                tc_fence_after();
                // The scores are read twice, 32 columns at a time with the next on their way (held in
                // registers for the whole step they would be spilled).  A step that every row sees whole,
                // without negative scales, is plain: its loops hold no branch, and they stay rolled, since
                // a loop unrolled over the step's 128 scores waits for its instructions.
                uint32_t sa[kCols], sb[kCols];
                const int seen = vis - b * kStep;  // tokens of the step that the row sees
                // scores of unseen tokens become -inf times the factor's sign; for the maximum products
                // are turned over where the scale is negative
                const auto mask = [&](uint32_t (&sv)[kCols], int c, bool turn) {
#pragma unroll
                    for (int h2 = 0; h2 < kCols / TC; ++h2) {
                        const int q2 = (c * kCols + h2 * TC) / T;
                        const bool neg = sm.page[q2].x < 0.f;
                        const int see = ((valid >> q2) & 1u) ? seen - c * kCols : 0;
                        const uint32_t unseen = __float_as_uint(neg ? -kNegInf : kNegInf);
#pragma unroll
                        for (int t = h2 * TC; t < (h2 + 1) * TC; ++t) {
                            if (t >= see) sv[t] = unseen;
                            if (turn && neg) sv[t] ^= 0x80000000u;
                        }
                    }
                };
                // a page's factor for this row, log2 of its V scale and one over it
                const auto page = [&](int q2, bool masked) {
                    float4 v = sm.page[q2];
                    v.x *= rs;
                    // one next to nothing (a scale or a row of zeros) stays away from 0 on its own side, as unseen
                    // scores, infinities of the scale's sign, times it have to be -inf
                    if (masked && fabsf(v.x) < 1e-30f) v.x = copysignf(1e-30f, v.x);
                    return v;
                };
                float bm = kNegInf;
                const auto largest = [&](const uint32_t (&sv)[kCols], int c, bool masked) {
#pragma unroll
                    for (int h2 = 0; h2 < kCols / TC; ++h2) {
                        const float4 pg = page((c * kCols + h2 * TC) / T, masked);
                        float mx[2] = {kNegInf, kNegInf};
#pragma unroll
                        for (int t = h2 * TC; t < (h2 + 1) * TC; t += 4)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                mx[e] = max3_nan(mx[e], __uint_as_float(sv[t + 2 * e]), __uint_as_float(sv[t + 2 * e + 1]));
                        bm = max3_nan(bm, fmaf(mx[0], fabsf(pg.x), pg.y), fmaf(mx[1], fabsf(pg.x), pg.y));
                    }
                };
                if (plain) {
                    tmem_ld32(s_addr, sa);
#pragma unroll 1
                    for (int c = 0; c < kStep / kCols; c += 2) {
                        tmem_wait_ld();
                        reg_fence<kCols>(sa);
                        tmem_ld32(s_addr + kCols * (c + 1), sb);
                        largest(sa, c, false);
                        tmem_wait_ld();
                        reg_fence<kCols>(sb);
                        tmem_ld32(s_addr + (c + 2) % (kStep / kCols) * kCols, sa);
                        largest(sb, c + 1, false);
                    }
                    tmem_wait_ld();
                    reg_fence<kCols>(sa);
                } else {
#pragma unroll 1
                    for (int c = 0; c < kStep / kCols; ++c) {
                        tmem_ld32_wait(s_addr + kCols * c, sa);
                        mask(sa, c, true);
                        largest(sa, c, true);
                    }
                }
                const bool mv = !(bm <= m + kLazy);  // or NaN, which then stays
                if (__any_sync(0xffffffffu, mv)) {
                    const float a = mv ? ex2(m - bm) : 1.f;
                    if (mv) m = bm;
                    l *= a;
                    // S(b) was issued after the last O update had finished: O is free to be rescaled
                    if (b > b0) {
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t ov[32];
                            tmem_ld16(o_addr + 16u * c, ov);
                            tmem_wait_ld();
                            reg_fence<16>(ov);
#pragma unroll
                            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * a);
                            tmem_st16(o_addr + 16u * c, ov);
                        }
                    }
                }
                const float sub = m == kNegInf ? 0.f : m - kOffset;
                float mass = 0.f;  // of the page so far
                // P of 16 tokens (from token t1 of the step, at sv) takes 8 columns, of scores that have
                // been read
                const auto exps = [&](const uint32_t* sv, int t1, const float4& pg) {
                    const f2 f2f{pg.x, pg.x}, off{pg.y - sub, pg.y - sub};
                    f2 e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        e[i] = fma2(f2{__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])}, f2f, off);
                        if (i < kPolyPairs) {
                            e[i] = exp2_poly2q(e[i]);
                        } else {
                            e[i].x = ex2(e[i].x);
                            e[i].y = ex2(e[i].y);
                        }
                    }
                    uint32_t ck[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) ck[i] = pack_f16x2(e[i].x, e[i].y);
                    tmem_st_x8(s_addr + (uint32_t)(t1 >> 1), ck);
                    const f2 ps = add2(add2(add2(e[0], e[1]), add2(e[2], e[3])), add2(add2(e[4], e[5]), add2(e[6], e[7])));
                    const float sum = (ps.x + ps.y) * pg.z;
                    l += sum;
                    if constexpr (WEIGHTS) {
                        mass += sum;
                        if ((t1 + 16) % T == 0) {
                            const int pg = b * PPS + t1 / T;
                            if (pg < mass_pages)
                                mass_row[(size_t)pg * mass_rows] = make_float2(mass, m);
                            mass = 0.f;
                        }
                    }
                };
                const auto signal = [&](int half) {  // half a step of P is there for the O update
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B.pfull(w, half));
                };
                if (plain) {  // the first 16 scores are there
                    float4 pa = page(0, false);
#pragma unroll 1
                    for (int t1 = 0; t1 < kStep; t1 += 32) {
                        tmem_ld16(s_addr + t1 + 16, sb);
                        const float4 pb = T < 32 ? page((t1 + 16) / T, false) : pa;
                        exps(sa, t1, pa);
                        tmem_wait_ld();
                        reg_fence<16>(sb);
                        tmem_ld16(s_addr + (t1 + 32) % kStep, sa);
                        if (T < kStep) pa = page((t1 + 32) % kStep / T, false);
                        exps(sb, t1 + 16, pb);
                        tmem_wait_ld();
                        reg_fence<16>(sa);
                        if (t1 & 32) signal(t1 >> 6);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < kStep / kCols; ++c) {
                        tmem_ld32_wait(s_addr + kCols * c, sa);
                        mask(sa, c, false);
                        exps(sa, c * kCols, page(c * kCols / T, true));
                        exps(sa + 16, c * kCols + 16, page((c * kCols + 16) / T, true));
                        if (c & 1) signal(c >> 1);
                    }
                }
            }
            if (!ok) break;
            // ---- the row's result, or its part of it
            ok = warp_ok(mbar_wait_idle(B.pvdone(w), (use - 1) & 1, abort_flag, p.err, QUP_ERR_TIMEOUT, lim));
            if (!ok) break;
            tc_fence_after();
            const bool complete = b0 == 0 && b1 == sg.steps;
            const size_t part = (size_t)2 * blockIdx.x + (first_seg ? 0 : 1);
            const size_t prow0 = part * kItemRows + w * kTileRows + wq * 32;
            const size_t q0 = (size_t)wk.it.q.q0;
            const size_t at = (q0 + qi) * p.Hq + sg.h * g + j;
            const bool nan = *reinterpret_cast<const volatile int*>(&nm.any) != 0;
            const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
            // 32 columns at a time through the warp's rows of the Q tile (every S that reads them is done),
            // so that a row's 128 (partial results) or 64 bytes leave as one piece
            uint8_t* stage = smem + Layout::q + w * 2 * kTile + wq * 32 * 128;
            const float times = complete ? inv : 1.f;
            const int place = qi * p.Hq + j;  // of the row in the request's output
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t ov[32];
                tmem_ld32_wait(o_addr + 32u * c, ov);
                __syncwarp();  // the columns before these have left
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                        make_float4(__uint_as_float(ov[4 * e]) * times, __uint_as_float(ov[4 * e + 1]) * times,
                                    __uint_as_float(ov[4 * e + 2]) * times, __uint_as_float(ov[4 * e + 3]) * times);
                if (nan) {
#pragma unroll 1
                    for (int e = 0; e < 32; ++e)
                        if (nm.first[32 * c + e] < vis)
                            *reinterpret_cast<uint32_t*>(stage + lane * 128 + (((e >> 2) ^ (lane & 7)) << 4) + (e & 3) * 4) =
                                0x7fc00000u;
                }
                __syncwarp();
#pragma unroll 2
                for (int i = 0; i < 8; ++i) {  // 4 rows, 8 lanes each
                    const int rr = 4 * i + (lane >> 3);
                    const float4 v = *reinterpret_cast<const float4*>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
                    const int to = __shfl_sync(0xffffffffu, place, rr);
                    if (wq * 32 + rr >= rows) continue;
                    const int col = 32 * c + (lane & 7) * 4;
                    if (complete)
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) +
                                                  (q0 * p.Hq + sg.h * g + (size_t)to) * kHeadDim + col) =
                            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                    else
                        *reinterpret_cast<float4*>(p.chunk_o + (prow0 + rr) * kHeadDim + col) = v;
                }
            }
            __syncwarp();
            if (on) {
                if (complete) {
                    const float l2 = l == 0.f ? kNegInf : m - kOffset + lg2(l);
                    if (p.lse) p.lse[at] = l2 * 0.69314718055994531f;
                    if (WEIGHTS) p.ws_lse[at] = l2;
                } else {
                    p.chunk_ml[prow0 + lane] = make_float2(m, l);
                }
            }
            // warpgroup 1 takes part in every phase of this barrier (see the empty row tile)
            if (w == 1) ok = warp_ok(mbar_wait_idle(B.sdone(), (segs - 1) & 1, abort_flag, p.err, QUP_ERR_TIMEOUT, lim));
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join of cut items
// CTA (c, y): if the last item of run c begins there and goes on, its rows [8 y, 8 y + 8): the parts
// of runs c, c + 1, ... in order, up to the run in which the item ends.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(kHeadDim) cache_chunk_join_kernel(const __grid_constant__ CacheAttnParams p, int runs) {
    grid_dep_wait();
    const ChunkSpan a = p.spans[blockIdx.x];
    if (a.segs == 0 || a.ends || a.b0 != 0) return;
    const Request q = load_request(p.q_ptr, p.Nq, p.c.kv_len, p.c.page_ptr, p.c.total_pages, p.c.T, a.r);
    const int rows = min(kItemRows, q.n * p.g - a.tile * kItemRows);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int last = blockIdx.x + 1;
    while (last < runs - 1 && !p.spans[last].first_ends) ++last;
    for (int rr = blockIdx.y * kJoinRows + warp; rr < min(rows, (int)(blockIdx.y + 1) * kJoinRows); rr += kHeadDim / 32) {
        float M = kNegInf, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = blockIdx.x; c <= last; ++c) {
            const size_t part = (size_t)2 * c + (c == (int)blockIdx.x && a.segs > 1 ? 1 : 0);
            M = fmaxf(M, p.chunk_ml[part * kItemRows + rr].x);
        }
        for (int c = blockIdx.x; c <= last; ++c) {
            const size_t part = (size_t)2 * c + (c == (int)blockIdx.x && a.segs > 1 ? 1 : 0);
            const size_t at = part * kItemRows + rr;
            const float2 ml = p.chunk_ml[at];
            // a part that saw nothing holds zeros; NaN goes through
            const float f = ml.x == kNegInf ? (ml.y == 0.f ? 0.f : 1.f) : ex2(ml.x - M);
            const float4 v = reinterpret_cast<const float4*>(p.chunk_o + at * kHeadDim)[lane];
            L += ml.y * f;
            acc.x += v.x * f;
            acc.y += v.y * f;
            acc.z += v.z * f;
            acc.w += v.w * f;
        }
        const int x = a.tile * kItemRows + rr, qi = x / p.g, j = x - qi * p.g;
        const size_t at = (size_t)(q.q0 + qi) * p.Hq + a.h * p.g + j;
        const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);
        uint2 o;
        o.x = pack_bf16x2(acc.x * inv, acc.y * inv);
        o.y = pack_bf16x2(acc.z * inv, acc.w * inv);
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + at * kHeadDim)[lane] = o;
        if (lane == 0) {
            const float l2 = L == 0.f ? kNegInf : M - kOffset + lg2(L);
            if (p.lse) p.lse[at] = l2 * 0.69314718055994531f;
            if (p.weight) p.ws_lse[at] = l2;
        }
    }
}

template <int T, bool WEIGHTS>
cudaError_t launch_t(const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p, int runs,
                     cudaStream_t stream) {
    const auto kernel = cache_chunk_kernel<T, WEIGHTS>;
    const size_t smem = cache_chunk_smem();
    cudaError_t e = ensure_smem_attr((const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(runs), dim3(kThreads), smem, stream, tmK, tmV, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_chunk_join_kernel, dim3(runs, kItemRows / kJoinRows), dim3(kHeadDim), 0, stream, p, runs);
}

template <int T>
cudaError_t launch_w(const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p, int runs,
                     cudaStream_t stream) {
    return p.weight ? launch_t<T, true>(tmK, tmV, p, runs, stream) : launch_t<T, false>(tmK, tmV, p, runs, stream);
}

}  // namespace

size_t cache_chunk_smem() { return Layout::total + 1024; }

cudaError_t launch_cache_chunk(const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p, int runs,
                               cudaStream_t stream) {
    switch (p.c.T) {
        case 16: return launch_w<16>(tmK, tmV, p, runs, stream);
        case 32: return launch_w<32>(tmK, tmV, p, runs, stream);
        case 64: return launch_w<64>(tmK, tmV, p, runs, stream);
        default: return launch_w<128>(tmK, tmV, p, runs, stream);
    }
}

}  // namespace qup
