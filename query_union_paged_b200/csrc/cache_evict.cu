// cache_evict.cu -- eviction of whole pages by accumulated attention weight.
//
// Per request: score(p) = decay * acc[p] + sum over KV heads of weight[p][h] for its used pages,
// computed in fp64 and rounded once to fp32, so neither the order of the heads nor a fused
// multiply decides a ranking.  Of the pages that are neither among the first `sink` nor among the
// last `recent`, the used - budget lowest are dropped (equal scores: the lower page first).  The
// kept pages move together in order, the dropped ones follow in order (their physical pages are
// the request's next ones to grow into), unused entries stay where they are.
//
// One CTA per request: scores and the request's page table in shared memory, the cut by a radix
// select over order-preserving keys (four passes of 8 bits), places by a prefix count.  Everything
// of a request is read before any of it is written, so the outputs may be the inputs' own arrays.
// Bound by latency: about 30 bytes a page (a call of 8 requests of 130 pages 7.8 us, 256 of up to 1,024 10 us).
#include <cstdint>

#include "cache.h"
#include "internal.h"
#include "ptx.cuh"
#include "query_union_paged.h"

namespace qup {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;

// fp64 conversions that keep subnormal fp32 values (the library is built with flush to zero)
__device__ __forceinline__ double to_f64(float x) {
    double d;
    asm("cvt.f64.f32 %0, %1;" : "=d"(d) : "f"(x));
    return d;
}
__device__ __forceinline__ float to_f32(double x) {
    float f;
    asm("cvt.rn.f32.f64 %0, %1;" : "=f"(f) : "d"(x));
    return f;
}

// Larger key = larger score; -0 as +0, NaN above everything (never dropped for its score).
__device__ __forceinline__ uint32_t order_key(uint32_t u) {
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    if ((u << 1) == 0u) u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of a flag over the CTA's threads, and the CTA's total; `part` holds kEvictWarps.
__device__ __forceinline__ int block_rank(bool flag, int* part, int* total) {
    const unsigned bal = __ballot_sync(0xffffffffu, flag);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) part[warp] = __popc(bal);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kEvictWarps; ++w) {
        before += w < warp ? part[w] : 0;
        all += part[w];
    }
    *total = all;
    return before + __popc(bal & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kEvictThreads) cache_evict_kernel(
    const int32_t* page_table, const int32_t* __restrict__ page_ptr, const int32_t* kv_len, int total_pages, int Hkv,
    int T, const float* __restrict__ weight, const float* acc, double decay, int budget, int sink, int recent, int cap,
    int32_t* table_out, float* acc_out, int32_t* len_out, int32_t* page_src, unsigned* err) {
    extern __shared__ uint32_t ev_sm[];
    uint32_t* score = ev_sm;                                  // [cap] fp32 bits
    int32_t* table = reinterpret_cast<int32_t*>(ev_sm + cap);  // [cap]
    __shared__ int hist[256];
    __shared__ int part[kEvictWarps];
    __shared__ uint32_t s_key;
    __shared__ int s_rem;
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    grid_dep_wait();
    const int p0 = page_ptr[r], np = page_ptr[r + 1] - p0, len = kv_len[r];
    const bool range = p0 >= 0 && np >= 0 && (long long)p0 + np <= total_pages;
    const int used = len <= 0 ? 0 : (len - 1) / T + 1;
    const bool ok = range && len >= 0 && used <= np;
    const bool fits = used <= cap;
    __syncthreads();  // every thread has read kv_len[r]: it may be len_out[r]
    if (!ok || !fits) {  // left as it is
        if (tid == 0) {
            atomicOr(err, ok ? QUP_ERR_CAPACITY : QUP_ERR_GROUP);
            len_out[r] = len;
        }
        for (int p = tid; range && p < np; p += kEvictThreads) {
            table_out[p0 + p] = page_table[p0 + p];
            acc_out[p0 + p] = acc[p0 + p];
            page_src[p0 + p] = p;
        }
        return;
    }
    for (int p = tid; p < np; p += kEvictThreads) {
        const float a = acc[p0 + p];
        const int32_t t = page_table[p0 + p];
        if (p >= used) {
            table_out[p0 + p] = t;
            acc_out[p0 + p] = a;
            page_src[p0 + p] = p;
            continue;
        }
        const float* w = weight + (size_t)(p0 + p) * Hkv;
        double sum = 0.0;
        for (int h = 0; h < Hkv; ++h) sum += to_f64(__ldg(w + h));
        score[p] = __float_as_uint(to_f32(decay * to_f64(a) + sum));
        table[p] = t;
    }
    const int lo = min(sink, used), hi = max(lo, used - recent);  // the pages that may go: [lo, hi)
    const int drop = min(max(used - budget, 0), hi - lo);
    if (tid == 0) {
        s_key = 0u;
        s_rem = drop;
    }
    __syncthreads();
    // the drop-th smallest key: after each byte the threshold's upper bytes are known, and s_rem
    // keys sharing them are still to go
    for (int byte = 3; byte >= 0 && drop > 0; --byte) {
        for (int x = tid; x < 256; x += kEvictThreads) hist[x] = 0;
        __syncthreads();
        const uint32_t pre = s_key;
        const int sh = 8 * byte;
        for (int p = lo + tid; p < hi; p += kEvictThreads) {
            const uint32_t k = order_key(score[p]);
            if (byte == 3 || (k >> (sh + 8)) == (pre >> (sh + 8))) atomicAdd(&hist[(k >> sh) & 255u], 1);
        }
        __syncthreads();
        if (tid < 32) {  // lane l holds bins 8l .. 8l + 7
            int c[8], tot = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c[e] = hist[8 * lane + e];
                tot += c[e];
            }
            int run = tot;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += y;
            }
            run -= tot;
            const int rem = s_rem;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (run < rem && run + c[e] >= rem) {
                    s_key = pre | ((uint32_t)(8 * lane + e) << sh);
                    s_rem = rem - run;
                }
                run += c[e];
            }
        }
        __syncthreads();
    }
    const uint32_t cut = s_key;
    const int ties = s_rem;  // pages whose key is the cut that go, lowest first
    const int kept = used - drop;
    int tied = 0, gone = 0;  // of the pages before this stretch
    for (int base = 0; base < used; base += kEvictThreads) {
        const int p = base + tid;
        const bool can = drop > 0 && p >= lo && p < hi;
        const uint32_t k = can ? order_key(score[p]) : 0u;
        int n = 0, m = 0;
        const int tr = tied + block_rank(can && k == cut, part, &n);
        const bool out = can && (k < cut || (k == cut && tr < ties));
        const int before = gone + block_rank(out, part, &m);
        tied += n;
        gone += m;
        if (p < used) {
            const int at = out ? kept + before : p - before;
            table_out[p0 + at] = table[p];
            acc_out[p0 + at] = out ? 0.f : __uint_as_float(score[p]);
            page_src[p0 + at] = p;
        }
    }
    if (tid == 0) len_out[r] = len - drop * T;
}

}  // namespace

size_t cache_evict_smem(int cap) { return (size_t)cap * 8; }

cudaError_t launch_cache_evict(const CacheView& c, const float* weight, const float* acc, float decay, int budget,
                               int sink, int recent, int cap, int32_t* table_out, float* acc_out, int32_t* len_out,
                               int32_t* page_src, unsigned* err, cudaStream_t stream) {
    if (c.R == 0) return cudaSuccess;
    const size_t smem = cache_evict_smem(cap);
    const cudaError_t e = ensure_smem_attr((const void*)cache_evict_kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(cache_evict_kernel, dim3(c.R), dim3(kEvictThreads), smem, stream, c.page_table, c.page_ptr,
                      c.kv_len, c.total_pages, c.Hkv, c.T, weight, acc, (double)decay, budget, sink, recent, cap,
                      table_out, acc_out, len_out, page_src, err);
}

}  // namespace qup
