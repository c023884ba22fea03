// cache_api.cu -- C ABI of the 8-bit page-scaled cache: argument checks, workspace layout, TMA
// tensor maps and launches.  Nothing here allocates device memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache.h"
#include "cache_attn.h"
#include "internal.h"
#include "query_union_paged.h"

namespace {

constexpr int kMaxSparseRows = 32;  // Q heads of a KV head in a TopK call: bits of a page's row mask

int check_cache(const qup_cache* c) {
    if (!c || c->P_phys <= 0 || c->Hkv <= 0 || c->Hkv > 32767 || c->R < 0 || c->total_pages <= 0) return QUP_ERR_ARG;
    if (!(c->T == 16 || c->T == 32 || c->T == 64 || c->T == 128)) return QUP_ERR_ARG;
    if (c->max_pages < 1 || c->max_pages > c->total_pages) return QUP_ERR_ARG;
    if ((int64_t)c->max_pages * c->T >= ((int64_t)1 << 31)) return QUP_ERR_ARG;  // token positions are int32
    return QUP_OK;
}

int check_cache_pointers(const qup_cache* c) {
    if (!c->K || !c->V || !c->k_scale || !c->v_scale || !c->page_table || !c->page_ptr || !c->kv_len)
        return QUP_ERR_ARG;
    return ((reinterpret_cast<uintptr_t>(c->K) | reinterpret_cast<uintptr_t>(c->V)) & 15) ? QUP_ERR_ARG : QUP_OK;
}

qup::CacheView view_of(const qup_cache* c) {
    qup::CacheView v;
    v.K = static_cast<uint8_t*>(c->K);
    v.V = static_cast<uint8_t*>(c->V);
    v.k_scale = c->k_scale;
    v.v_scale = c->v_scale;
    v.page_table = c->page_table;
    v.page_ptr = c->page_ptr;
    v.kv_len = c->kv_len;
    v.P_phys = c->P_phys;
    v.Hkv = c->Hkv;
    v.T = c->T;
    v.R = c->R;
    v.total_pages = c->total_pages;
    return v;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}
// The rows of Q (`row` bytes each, `stride` apart) against n contiguous rows of O.
bool rows_overlap(const void* Q, int64_t stride, const void* O, int64_t row, int64_t n) {
    const int64_t at = (int64_t)(reinterpret_cast<intptr_t>(O) - reinterpret_cast<intptr_t>(Q));
    const int64_t first = at < row ? 0 : (at - row) / stride + 1;  // the first row of Q that ends behind O's start
    return first < n && first * stride < at + row * n;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// All pages: requests of up to kCacheSmallRows rows (queries x heads of a KV head) go to the kernel
// of the small ones, the others to the chunk kernel.  Where every request has max_q queries or
// the batch is padded, one kernel takes them all.
struct AttnPlan {
    bool chunk, small;
    int64_t small_rows;  // rows of a request of the small kernel, at most
};
AttnPlan attn_plan(const qup_cache* c, int Nq, int max_q, int Hq, bool sparse) {
    const int g = Hq / c->Hkv;
    const int64_t big = (int64_t)max_q * g;
    AttnPlan a;
    a.chunk = !sparse && big > qup::kCacheSmallRows;
    a.small = !a.chunk || (int64_t)c->R * max_q != Nq;
    a.small_rows = a.chunk ? qup::kCacheSmallRows : big;
    return a;
}

struct AttnWs {
    size_t part_o, part_ml, chunk_o, chunk_ml, spans, mass, mass_chunk, lse, bits, total;
    int mass_per, mass_chunk_per;
};

// Bytes of the page weights' sums, `slots` for a page: by pages with room for `rows` rows of one request
// (*per), or by rows with room for max_pages pages (*per = 0), see mass_of().  Sizes past 2^62 are cut there.
size_t mass_bytes(const qup_cache* c, int Nq, int Hq, int64_t rows, int slots, int* per) {
    typedef unsigned __int128 u128;
    const u128 by_pages = (u128)c->total_pages * c->Hkv * (u128)rows, by_rows = (u128)Nq * Hq * (u128)c->max_pages;
    *per = by_pages <= by_rows ? (int)std::max<int64_t>(rows, 1) : 0;
    return (size_t)std::min<u128>(std::min(by_pages, by_rows) * slots * sizeof(float2), (u128)1 << 62);
}

// The partial results of an all-pages call: two of each CTA.  Those of a TopK call: one of each CTA
// of a (query, KV head), which is cut only while all of them fit the SMs at once.
AttnWs attn_ws_layout(const qup_cache* c, int Nq, int max_q, int Hq, bool weights, bool sparse) {
    AttnWs w;
    std::memset(&w, 0, sizeof(w));
    const AttnPlan plan = attn_plan(c, Nq, max_q, Hq, sparse);
    const size_t parts = qup::kCachePartRows;
    size_t off = 0;
    w.part_o = off;
    off = align256(off + parts * qup::kHeadDim * sizeof(float));
    w.part_ml = off;
    off = align256(off + parts * sizeof(float2));
    const size_t crows = 2 * (size_t)qup::kChunkMaxRuns * qup::kChunkRows;
    w.chunk_o = off;
    if (plan.chunk) off = align256(off + crows * qup::kHeadDim * sizeof(float));
    w.chunk_ml = off;
    if (plan.chunk) off = align256(off + crows * sizeof(float2));
    w.spans = off;
    if (plan.chunk) off = align256(off + qup::kChunkMaxRuns * sizeof(qup::ChunkSpan));
    if (weights) {
        w.mass = off;
        if (plan.small) off = align256(off + mass_bytes(c, Nq, Hq, plan.small_rows, c->T / 16, &w.mass_per));
        w.mass_chunk = off;
        if (plan.chunk)
            off = align256(off + mass_bytes(c, Nq, Hq, (int64_t)max_q * (Hq / c->Hkv), 1, &w.mass_chunk_per));
        w.lse = off;
        off = align256(off + sizeof(float) * (size_t)Nq * Hq);
        w.bits = off;
        if (sparse) off = align256(off + sizeof(uint32_t) * ((size_t)c->total_pages / 32 + c->R) * max_q * c->Hkv);
    }
    w.total = off;
    return w;
}

int check_attn_sizes(const qup_cache* c, int Nq, int max_q, int Hq) {
    const int rc = check_cache(c);
    if (rc) return rc;
    if (Nq < 0 || max_q < 0 || max_q > Nq || Hq <= 0 || Hq % c->Hkv != 0) return QUP_ERR_ARG;
    const int g = Hq / c->Hkv;
    if ((int64_t)max_q * g >= ((int64_t)1 << 30)) return QUP_ERR_ARG;
    return QUP_OK;
}

}  // namespace

extern "C" {

int qup_cache_append(const qup_cache* cache, const void* k_new, const void* v_new, int dtype, int64_t k_stride,
                     int64_t v_stride, const int32_t* tok_ptr, int N, int d, void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (N < 0 || d != qup::kHeadDim || (dtype != QUP_BF16 && dtype != QUP_F32)) return QUP_ERR_ARG;
    const int64_t unit = dtype == QUP_BF16 ? 8 : 4, least = (int64_t)cache->Hkv * d;
    if (k_stride < least || v_stride < least || k_stride % unit != 0 || v_stride % unit != 0) return QUP_ERR_ARG;
    if (N == 0 || cache->R == 0) return QUP_OK;
    if (check_cache_pointers(cache) || !k_new || !v_new || !tok_ptr) return QUP_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) return QUP_ERR_ARG;
    if (cache->K == cache->V || cache->k_scale == cache->v_scale) return QUP_ERR_ARG;  // both are written
    if (((int64_t)N / cache->T + 2 * (int64_t)cache->R) * 2 * cache->Hkv >= ((int64_t)1 << 31)) return QUP_ERR_ARG;
    qup::DeviceInfo dev;
    if ((rc = qup::device_info(&dev))) return rc;
    return qup::launch_cache_append(view_of(cache), k_new, v_new, dtype == QUP_BF16, k_stride, v_stride, tok_ptr, N,
                                    dev.sms, dev.err, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? QUP_OK
               : QUP_ERR_CUDA;
}

int qup_cache_attn_workspace(const qup_cache* cache, int Nq, int max_q, int Hq, int page_weight, size_t* ws_bytes) {
    const int rc = check_attn_sizes(cache, Nq, max_q, Hq);
    if (rc) return rc;
    if (ws_bytes) {
        *ws_bytes = attn_ws_layout(cache, Nq, max_q, Hq, page_weight != 0, false).total;
        if (page_weight != 2)  // TopK calls too
            *ws_bytes = std::max(*ws_bytes, attn_ws_layout(cache, Nq, max_q, Hq, page_weight != 0, true).total);
    }
    return QUP_OK;
}

int qup_cache_attn(const qup_cache* cache, const void* Q, int64_t q_stride, const int32_t* q_ptr, int Nq, int max_q,
                   int Hq, int d, const int32_t* topk, int Ksel, float softmax_scale, void* O, float* lse,
                   float* page_weight, void* ws, size_t ws_bytes, void* stream) {
    int rc = check_attn_sizes(cache, Nq, max_q, Hq);
    if (rc) return rc;
    const qup_cache& c = *cache;
    const int g = Hq / c.Hkv;
    if (d != qup::kHeadDim || Ksel < 0 || (Ksel > 0 && !topk)) return QUP_ERR_ARG;
    if (q_stride < (int64_t)Hq * d || q_stride % 8 != 0) return QUP_ERR_ARG;
    if (!(std::isfinite(softmax_scale) && softmax_scale > 0.f)) return QUP_ERR_ARG;
    const bool sparse = topk != nullptr;
    if (sparse && (g > kMaxSparseRows || (int64_t)g * Ksel >= ((int64_t)1 << 24))) return QUP_ERR_ARG;
    if (Nq == 0 || c.R == 0) {
        if (page_weight && c.R > 0)  // no rows: every page's weight is 0
            return cudaMemsetAsync(page_weight, 0, sizeof(float) * (size_t)c.total_pages * c.Hkv,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
                       ? QUP_OK
                       : QUP_ERR_CUDA;
        return QUP_OK;
    }
    if (check_cache_pointers(cache) || !Q || !q_ptr || !O || !ws) return QUP_ERR_ARG;
    if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(O) | reinterpret_cast<uintptr_t>(ws)) & 15)
        return QUP_ERR_ARG;
    // rows of Q are read after others of O are written
    if (rows_overlap(Q, 2 * q_stride, O, (int64_t)Hq * d * 2, Nq)) return QUP_ERR_ARG;
    const AttnWs L = attn_ws_layout(cache, Nq, max_q, Hq, page_weight != nullptr, sparse);
    if (ws_bytes < L.total) return QUP_ERR_CAPACITY;

    const AttnPlan plan = attn_plan(cache, Nq, max_q, Hq, sparse);
    const bool chunk = plan.chunk, small = plan.small;
    const int64_t small_rows = sparse ? g : plan.small_rows;  // TopK: a query's rows are a tile
    const int nt = small_rows <= 8 ? 1 : (small_rows <= 16 ? 2 : 4), rt = 8 * nt;
    qup::CacheAttnParams p;
    std::memset(&p, 0, sizeof(p));
    p.big_rows = !chunk ? 0x7fffffff : (small ? qup::kCacheSmallRows + 1 : 1);
    p.max_tiles = (int)std::max<int64_t>((small_rows + rt - 1) / rt, 1);  // max_q = 0: a request's rows are a fault
    const int64_t max_units = ((int64_t)c.max_pages * c.T + qup::kCacheUnit - 1) / qup::kCacheUnit;
    // the chunk kernel counts steps and a request's rows in 32 bits
    if (chunk && (((int64_t)c.max_pages * c.T + 256 + max_q) * g + 256 >= ((int64_t)1 << 31) ||
                  (int64_t)max_q * Hq >= ((int64_t)1 << 31)))
        return QUP_ERR_ARG;
    if (!sparse && (int64_t)p.max_tiles * c.Hkv * max_units >= ((int64_t)1 << 31)) return QUP_ERR_ARG;
    const int64_t items = sparse ? (int64_t)Nq * c.Hkv : (int64_t)c.R * c.Hkv * p.max_tiles;
    if (items >= ((int64_t)1 << 31) / 2) return QUP_ERR_ARG;

    qup::DeviceInfo dev;
    if ((rc = qup::device_info(&dev))) return rc;
    const int ctas = std::min(dev.sms, qup::kCacheMaxSms) * qup::cache_attn_ctas(nt);
    int grid = ctas;
    p.nsplit = 1;
    if (sparse) {
        const int64_t entries = std::min<int64_t>((int64_t)g * Ksel, c.max_pages);
        const int64_t units = std::max<int64_t>((entries * c.T + qup::kCacheUnit - 1) / qup::kCacheUnit, 1);
        // as many CTAs as the SMs hold at once: finding its pages costs a CTA what 8 units do, so more
        // and shorter ones lose (32 x 32K, 32 of 64-token pages: 35 us with one CTA a pair, 53 with four)
        p.nsplit = (int)std::max<int64_t>(1, std::min<int64_t>(ctas / items, units));
        p.list_cap = (int)((entries + p.nsplit - 1) / p.nsplit);
        grid = (int)(items * p.nsplit);
    }
    if (qup::cache_attn_smem(nt, sparse, c.max_pages, p.list_cap) > (size_t)dev.smem_optin ||
        qup::cache_chunk_smem() > (size_t)dev.smem_optin)
        return QUP_ERR_ARG;

    // K and V tiles: dims (d, T, Hkv, P_phys) bytes, boxes of (128, tokens, 1, 1), 128-byte swizzle
    const auto encode = [&](int box_tokens, CUtensorMap* tm) {
        const cuuint64_t row = qup::kHeadDim, page = row * c.T;
        const cuuint64_t dims[4] = {row, (cuuint64_t)c.T, (cuuint64_t)c.Hkv, (cuuint64_t)c.P_phys};
        const cuuint64_t strides[3] = {row, page, page * c.Hkv};
        const cuuint32_t box[4] = {(cuuint32_t)qup::kHeadDim, (cuuint32_t)box_tokens, 1, 1};
        const cuuint32_t estr[4] = {1, 1, 1, 1};
        void* const srcs[2] = {c.K, c.V};
        for (int i = 0; i < 2; ++i)
            if (dev.encode(&tm[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, srcs[i], dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return false;
        return true;
    };
    CUtensorMap tm[2], tmc[2];
    if ((small && !encode(std::min(c.T, qup::kCacheUnit), tm)) || (chunk && !encode(c.T, tmc))) return QUP_ERR_ARG;

    char* base = static_cast<char*>(ws);
    p.c = view_of(cache);
    p.Q = Q;
    p.q_stride = q_stride;
    p.q_ptr = q_ptr;
    p.topk = topk;
    p.O = O;
    p.lse = lse;
    p.weight = page_weight;
    p.part_o = reinterpret_cast<float*>(base + L.part_o);
    p.part_ml = reinterpret_cast<float2*>(base + L.part_ml);
    p.chunk_o = reinterpret_cast<float*>(base + L.chunk_o);
    p.chunk_ml = reinterpret_cast<float2*>(base + L.chunk_ml);
    p.spans = reinterpret_cast<qup::ChunkSpan*>(base + L.spans);
    p.mass = reinterpret_cast<float2*>(base + L.mass);
    p.mass_chunk = reinterpret_cast<float2*>(base + L.mass_chunk);
    p.mass_per = L.mass_per;
    p.mass_chunk_per = L.mass_chunk_per;
    p.ws_lse = reinterpret_cast<float*>(base + L.lse);
    p.ws_bits = reinterpret_cast<uint32_t*>(base + L.bits);
    p.err = dev.err;
    p.wait_limit_ns = qup::wait_limit_ns();
    p.dbg_skip_stage = qup::debug_skip_stage();
    p.scale_log2 = softmax_scale * 1.4426950408889634f;
    p.Nq = Nq;
    p.max_q = max_q;
    p.Hq = Hq;
    p.g = g;
    p.Ksel = Ksel;
    p.max_pages = c.max_pages;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (chunk && qup::launch_cache_chunk(tmc[0], tmc[1], p, std::min(dev.sms, qup::kChunkMaxRuns), st) != cudaSuccess)
        return QUP_ERR_CUDA;
    if (small && qup::launch_cache_attn(nt, tm[0], tm[1], p, grid, (int)items, st) != cudaSuccess) return QUP_ERR_CUDA;
    if (page_weight && qup::launch_cache_weights(p, st) != cudaSuccess) return QUP_ERR_CUDA;
    return QUP_OK;
}

int qup_cache_evict(const qup_cache* cache, const float* page_weight, const float* acc, float decay, int budget,
                    int sink, int recent, int32_t* table_out, float* acc_out, int32_t* len_out, int32_t* page_src,
                    void* stream) {
    int rc = check_cache(cache);
    if (rc) return rc;
    if (!std::isfinite(decay) || budget < 1 || sink < 0 || recent < 1) return QUP_ERR_ARG;
    if (cache->max_pages > QUP_CACHE_EVICT_PAGES) return QUP_ERR_ARG;
    if (cache->R == 0) return QUP_OK;
    if (!cache->page_table || !cache->page_ptr || !cache->kv_len || !page_weight || !acc || !table_out || !acc_out ||
        !len_out || !page_src)
        return QUP_ERR_ARG;
    // a request's entries are read before its own are written, others' perhaps after: an output may be the input of the
    // same layout and nothing else
    const size_t n = sizeof(int32_t) * (size_t)cache->total_pages, nr = sizeof(int32_t) * (size_t)cache->R;
    const struct {
        const void* p;
        size_t bytes;
        const void* same;
    } outs[4] = {{table_out, n, cache->page_table}, {acc_out, n, acc}, {len_out, nr, cache->kv_len}, {page_src, n, nullptr}},
      ins[5] = {{cache->page_table, n, nullptr},
                {acc, n, nullptr},
                {cache->kv_len, nr, nullptr},
                {cache->page_ptr, nr + sizeof(int32_t), nullptr},
                {page_weight, n * cache->Hkv, nullptr}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return QUP_ERR_ARG;
        for (const auto& in : ins)
            if (!(outs[i].p == in.p && in.p == outs[i].same) && overlap(outs[i].p, outs[i].bytes, in.p, in.bytes))
                return QUP_ERR_ARG;
    }
    qup::DeviceInfo dev;
    if ((rc = qup::device_info(&dev))) return rc;
    return qup::launch_cache_evict(view_of(cache), page_weight, acc, decay, budget, sink, recent, cache->max_pages,
                                   table_out, acc_out, len_out, page_src, dev.err,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? QUP_OK
               : QUP_ERR_CUDA;
}

}  // extern "C"
