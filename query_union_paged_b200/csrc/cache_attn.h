// cache_attn.h -- attention over the 8-bit page-scaled cache: parameters and launchers for the C ABI
// (cache_api.cu), and what its two kernels (cache_attn.cu, cache_chunk.cu) have in common.
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "cache.h"
#include "internal.h"
#include "query_union_paged.h"

namespace qup {

constexpr int kCacheUnit = 64;       // tokens of a work unit
constexpr int kCacheMaxSms = 148;
// CTAs of the small kernel on an SM, by its row tiles of 8 rows
__host__ __device__ constexpr int cache_attn_ctas(int nt) { return nt == 1 ? 3 : (nt == 2 ? 2 : 1); }
// rows of partial results: two tiles of every CTA (8 rows x 3 CTAs, 16 x 2 or 32 x 1 on an SM)
constexpr int kCachePartRows = 2 * 32 * kCacheMaxSms;
constexpr int kCacheSmallRows = 16;  // rows (queries x heads of a KV head) up to which a request is a small one
constexpr int kChunkRows = 256;      // rows of an item of the other kernel (cache_chunk.cu)
constexpr int kChunkMaxRuns = kCacheMaxSms;   // and its CTAs

// What a CTA of the chunk kernel worked on: its last item, from which step, whether the item ends
// with it, and the first item's end.
struct ChunkSpan {
    int r, h, tile, b0;
    int ends, first_ends, segs, pad;
};

struct CacheAttnParams {
    CacheView c;
    const void* Q;
    long long q_stride;  // elements between a row's queries
    const int32_t* q_ptr;
    const int32_t* topk;  // null: all pages
    void* O;
    float* lse;       // or null
    float* weight;    // page weights, or null
    float* part_o;    // [partial][row tile][128]: unnormalised sums, and in part_ml the log2 maximum
    float2* part_ml;  // they are relative to and the sum of weights
    float2* mass;        // page weights: per (16 tokens, row) the weights' sum and the maximum it is relative to
    float2* mass_chunk;  // and per (page, row) of the chunk kernel's requests; places by mass_of()
    float* ws_lse;    // page weights: log2-domain lse of every row
    uint32_t* ws_bits;  // page weights over TopK pages: the pages each (query, KV head) reads
    float* chunk_o;     // [2 per run][256][128], chunk_ml, spans [run]: the chunk kernel's partial results
    float2* chunk_ml;
    ChunkSpan* spans;
    unsigned* err;
    unsigned long long wait_limit_ns;
    int dbg_skip_stage;  // a stage of each CTA that is not loaded, so that its waits run out; -1: none
    float scale_log2;
    int Nq, max_q, Hq, g, Ksel;
    int max_tiles;   // all pages: row tiles of max_q queries
    int mass_per, mass_chunk_per;  // rows of one request that a page has room for, 0: places by rows
    int nsplit;      // TopK pages: CTAs of one (query, KV head)
    int max_pages;   // pages of a request, at most
    int big_rows;    // all pages: requests of this many rows or more are the chunk kernel's
    int list_cap;    // TopK pages: distinct pages of one CTA, at most
};

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// four E4M3 values to two pairs of fp16
__device__ __forceinline__ void cvt_e4m3x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {  // 0x80 at each E4M3 NaN (0x7f, 0xff)
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// V scales that can be read: 0, or 2^-80 .. 2^80.  A row's sum adds up to p / vs with p <= 2^15 for each of fewer than
// 2^31 tokens, and its largest p is at least 2^8: outside, the sum may pass fp32's range or lose what counts.
__device__ __forceinline__ bool v_scale_ok(float vs) {
    const uint32_t u = __float_as_uint(vs);
    return (u << 1) == 0u || (u >= 0x17800000u && u <= 0x67800000u);
}
// What keeps a request from being read (0: nothing), as device error bits.
__device__ __forceinline__ unsigned request_fault(const CacheAttnParams& p, const Request& q) {
    if (!q.ok || q.n > p.max_q) return QUP_ERR_GROUP;
    return q.np > p.max_pages ? QUP_ERR_CAPACITY : 0u;
}
// Page weights: where a request's sums lie.  Requests follow each other either by their pages, with room for the longest
// one's rows (per != 0), or by their rows, with room for the most pages: what takes less for the whole batch.
// All pages: the sums of request q's rows of KV head h, [page][T / 16, or 1 if big][n * g].
__device__ __forceinline__ float2* mass_of(const CacheAttnParams& p, const Request& q, int h, bool big) {
    const int per = big ? p.mass_chunk_per : p.mass_per;
    const size_t at = per ? ((size_t)q.p0 * p.c.Hkv + (size_t)h * q.np) * per
                          : ((size_t)q.q0 * p.c.Hkv + (size_t)h * q.n) * p.g * p.max_pages;
    return big ? p.mass_chunk + at : p.mass + at * (p.c.T / 16);
}
// TopK pages: those of the request's query i, [page][T / 16][g].
__device__ __forceinline__ float2* mass_of_query(const CacheAttnParams& p, const Request& q, int h, int i) {
    const size_t at = p.mass_per ? (size_t)q.p0 * p.c.Hkv * p.max_q + ((size_t)h * p.max_q + i) * q.np
                                 : ((size_t)(q.q0 + i) * p.c.Hkv + h) * p.max_pages;
    return p.mass + at * (p.c.T / 16) * p.g;
}
// Rows of faulty requests (`big`: those that would be the chunk kernel's) get O = 0 and lse = -inf: the CTAs
// take the requests in turn.
__device__ __forceinline__ void clear_faulty(const CacheAttnParams& p, bool big) {
    for (int r = blockIdx.x; r < p.c.R; r += gridDim.x) {
        const Request q = load_request(p.q_ptr, p.Nq, p.c.kv_len, p.c.page_ptr, p.c.total_pages, p.c.T, r);
        if (request_fault(p, q) == 0u || ((long long)q.n * p.g >= p.big_rows) != big) continue;
        const long long a = max(q.q0, 0), b = min((long long)q.q0 + q.n, (long long)p.Nq);
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.O) + (size_t)a * p.Hq * kHeadDim);
        for (long long x = threadIdx.x; x < (b - a) * p.Hq * (kHeadDim / 8); x += blockDim.x)
            o[x] = make_uint4(0u, 0u, 0u, 0u);
        for (long long x = threadIdx.x; p.lse && x < (b - a) * p.Hq; x += blockDim.x)
            p.lse[a * p.Hq + x] = -INFINITY;
    }
}

// nt: row tiles of 8 rows (1, 2 or 4)
size_t cache_attn_smem(int nt, bool sparse, int max_pages, int list_cap);
// items: (request, KV head, row tile) triples of max_tiles each, or (query, KV head) pairs
cudaError_t launch_cache_attn(int nt, const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p,
                              int grid, int items, cudaStream_t stream);
// the requests of big_rows or more; tensor maps with boxes of a whole page
size_t cache_chunk_smem();
cudaError_t launch_cache_chunk(const CUtensorMap& tmK, const CUtensorMap& tmV, const CacheAttnParams& p, int runs,
                               cudaStream_t stream);
// page weights from what the attention kernels left
cudaError_t launch_cache_weights(const CacheAttnParams& p, cudaStream_t stream);

}  // namespace qup
