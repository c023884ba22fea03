/*
 * query_union_paged.h -- C ABI of the B200 (sm_100a) library for token-level
 * sparse-attention prefill over a paged KV cache with page-affine query unions.
 *
 * Source of the operations: "PageWeaver: KV-Guided Query Unions for Sparse
 * Attention" (Abstract; Figure 1; Figure 2; Figure 3).  Each query attends only
 * to the tokens of its own TopK selected KV pages, causally inside a page.
 * Queries that share pages are gathered into unions of up to max_group queries,
 * so each union page is streamed once and fills tensor-core tiles, while every
 * query keeps exactly its own support and writes its output row at its
 * original query ID (no reordered Q tensor, no cross-page partial outputs).
 *
 * Conventions for every entry point
 *  - Pointers marked "device" are CUDA device pointers owned by the caller; the
 *    library never allocates or frees device memory.  Host pointers are read
 *    during the call only.
 *  - Calls are asynchronous on the given stream (cudaStream_t passed as void*;
 *    NULL = the legacy default stream) and do not synchronize.
 *  - The return value is QUP_OK or a synchronous error (bad argument, capacity,
 *    launch failure).  Errors found on the device (a page ID out of range, a
 *    bad group, a timed-out pipeline wait) are ORed into a per-device error
 *    word, read and cleared by qup_get_error().  No call aborts or traps.
 *
 * Layouts (row-major, innermost last)
 *   Q          [Nq][Hq][d]              bf16 or fp32
 *   K, V cache [P_phys][Hkv][T][d]      bf16, fp32 or FP8 E4M3 (+ fp32 scale per KV head)
 *   page_table [num_logical_pages]      int32, logical page -> physical page
 *   topk       [Hq][Nq][Ksel]           int32 logical page IDs, -1 = padding
 *   q_pos      [Nq]                     int32 token position of each query
 *   O          [Nq][Hq][d]              dtype of Q
 * Token t (logical position) lives in logical page t / T, slot t % T.  Query
 * i with position q_pos[i] attends token t iff the page of t is in its row of
 * topk, t <= q_pos[i] and t < kv_len.  KV head of Q head h' is h' / (Hq/Hkv).
 */
#ifndef QUERY_UNION_PAGED_H
#define QUERY_UNION_PAGED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* return codes and device error bits */
#define QUP_OK 0
#define QUP_ERR_ARG 1          /* null pointer, bad dimension, unsupported dtype or limit */
#define QUP_ERR_CAPACITY 2     /* workspace or union capacity too small */
#define QUP_ERR_CUDA 4         /* a CUDA runtime call or launch failed */
#define QUP_ERR_PAGE_ID 8      /* device: a TopK or union page ID outside [0, num_logical_pages) */
#define QUP_ERR_PHYS_PAGE 16   /* device: a page_table entry outside [0, P_phys) */
#define QUP_ERR_GROUP 32       /* device: a group with no members, too many rows or a bad query ID */
#define QUP_ERR_TIMEOUT 64     /* device: a pipeline wait exceeded its limit; the kernel exited cleanly */
#define QUP_ERR_SCALE 128      /* device: a cache scale that is not finite, or a negative V scale */

/* dtype codes */
#define QUP_F32 0
#define QUP_BF16 1
#define QUP_E4M3 2

/*
 * Output of qup_sparse_group (every buffer is device memory, caller-allocated;
 * sizes from qup_group_workspace).  For KV head h and group k:
 *   members  [h*Nq + group_ptr[h*(Nq+1)+k] .. h*Nq + group_ptr[h*(Nq+1)+k+1])
 *            query IDs of the group, ascending (at most max_group)
 *   union    [union_ptr[h*(Nq+1)+k] .. union_ptr[h*(Nq+1)+k+1]) indexes
 *            union_pages (sorted distinct logical pages of the group) and
 *            row_mask (bit r = rank*g + j set iff that page is in row
 *            topk[h*g+j][member of that rank]); offsets are absolute, the
 *            regions of the KV heads follow each other in head order.
 *   counters [h*4 + 0..3] = logical page visits (sum of union sizes), masked
 *            row slots, masked query slots, page edges (sum of |S(i)|).
 * (Figure 2: logical page visits and masked query-page slots.)
 *
 * Bundles (the attention kernel's work items; no counterpart on the pages,
 * which share a page between the two CTAs of one Union8 group instead):
 * the groups of one KV head are packed, inside windows of bundle_window
 * groups, into bundles of up to 128 / rows_per_group groups by a greedy on
 * group unions: seeded with the first unbundled group, grown by the group
 * with the smallest (new pages - 2 * pages already shared with the bundle
 * union), ties to the smallest index.  A bundle's query rows are
 * laid out slot by slot: row = slot*rows_per_group + rank*g + j, with
 * rows_per_group = max_group*g rounded up to a power of two (<= 32).
 *   bundle_ptr[h*(Nq+1)+b] .. [+b+1]  indexes bundle_groups[h*Nq + ...]
 *            (group indices within head h, ascending = slot order)
 *   bunion   [bunion_ptr[h*(Nq+1)+b] .. [+b+1]) indexes bunion_pages (sorted
 *            union of the bundle's groups) and bunion_mask[4*entry + w]:
 *            bit (row % 32) of word row/32 set iff the page is in that row's
 *            own TopK row.
 *   bundle_qid[(h*Nq + b)*(128/g) + row/g] = query ID of the row, -1 if the
 *            slot or rank is empty.
 *   bcounters[h*2 + 0..1] = bundle page visits (sum of bundle union sizes:
 *            the pages the attention kernel streams), number of bundles.
 *   bundle_order[0 .. total bundles) = flat bundle indices (f = bundles of
 *            earlier KV heads + b) sorted by union size, largest first, equal
 *            sizes by index: the order in which the attention kernel's CTAs
 *            claim bundles at run time.
 */
typedef struct {
    int32_t* n_groups;     /* [Hkv] */
    int32_t* group_ptr;    /* [Hkv][Nq+1] */
    int32_t* members;      /* [Hkv][Nq] */
    int32_t* union_ptr;    /* [Hkv][Nq+1] */
    int32_t* union_pages;  /* [cap_union] */
    uint64_t* row_mask;    /* [cap_union] */
    int64_t* counters;     /* [Hkv][4] */
    int64_t cap_union;     /* entries available in union_pages/row_mask and in bunion_pages */
    int32_t* n_bundles;    /* [Hkv] */
    int32_t* bundle_ptr;   /* [Hkv][Nq+1] */
    int32_t* bundle_groups;/* [Hkv][Nq] */
    int32_t* bunion_ptr;   /* [Hkv][Nq+1] */
    int32_t* bunion_pages; /* [cap_union] */
    uint32_t* bunion_mask; /* [cap_union][4] */
    int32_t* bundle_qid;   /* [Hkv][Nq][128/g] */
    int64_t* bcounters;    /* [Hkv][2] */
    int32_t* bundle_order; /* [Hkv*Nq] */
    int32_t rows_per_group;/* set by qup_sparse_group / qup_build_bundles */
    int32_t bundle_window; /* groups per bundling window: 0 (default 64) .. 256, else QUP_ERR_ARG */
} qup_groups;

/*
 * Sizes for qup_sparse_group.  Writes the scratch workspace bytes and the
 * union capacity that is always sufficient (Hkv * Nq * min(g*Ksel, pages)).
 * Returns QUP_ERR_ARG for unsupported sizes (window > 256, max_group*g > 32,
 * too many pages for the shared-memory bitsets).
 */
int qup_group_workspace(int Hq, int Hkv, int Nq, int Ksel, int num_logical_pages, int max_group,
                        int window, size_t* ws_bytes, int64_t* cap_union);

/*
 * Bounded page-affinity grouping (Abstract: a GPU search of bounded cost
 * turns selected-page affinity into query-ID lists; Figure 2).  Per KV head h, S(i) is
 * the set of distinct valid pages of the g rows topk[h*g+j][i]; inside fixed
 * windows [w*window, (w+1)*window) of query IDs a group is seeded with the
 * smallest unassigned ID and grown, up to max_group members, by the candidate
 * that adds the fewest pages to the union (ties: smallest ID).  Output as in
 * qup_groups; bit-exact with the CPU reference of the same rule.
 *   topk       device int32 [Hq][Nq][Ksel]; -1 = padding, other IDs must lie
 *              in [0, num_logical_pages) (else QUP_ERR_PAGE_ID, entry ignored)
 *   max_group  1..8 and max_group*(Hq/Hkv) <= 32; window a multiple of
 *              max_group, <= 256 (window == max_group gives fixed consecutive groups)
 *   ws         device scratch of the size qup_cache_attn_workspace reports for
 *              the same cache sizes, Nq, max_q, Hq and page_weight (0: none; 1:
 *              with page weights; 2: likewise, for calls without topk only):
 *              5 MB, or 44 where a request may have more than 16 rows (query and
 *              Q head) of a KV head.  Page weights add 8 bytes for each row and
 *              page of such requests, min(max_q * total_pages, Nq * max_pages)
 *              * Hq of them at most, and for the others and for TopK calls 8 for
 *              each row and 16 tokens of a page; many queries of long requests
 *              are better split over several calls.  Calls that
 *              may run at the same time need one each.  Its contents need no
 *              preparation and mean nothing after the call.
 * Results do not depend on the run: partial results are merged in a fixed
 * order, without atomics.  Device errors: QUP_ERR_GROUP for a contradictory
 * request or one with more than max_q queries (all of its rows in [0, Nq) get
 * O = 0, lse = -inf, its pages the weight 0), QUP_ERR_CAPACITY for a request
 * with more than max_pages pages (likewise), QUP_ERR_PAGE_ID for a TopK entry
 * outside the request's pages (ignored), QUP_ERR_PHYS_PAGE and QUP_ERR_SCALE
 * for a bad page_table entry or scale (the page is not seen), QUP_ERR_TIMEOUT
 * as elsewhere.
 */
int qup_cache_attn_workspace(const qup_cache* cache, int Nq, int max_q, int Hq, int page_weight, size_t* ws_bytes);
int qup_cache_attn(const qup_cache* cache, const void* Q, int64_t q_stride, const int32_t* q_ptr, int Nq, int max_q,
                   int Hq, int d, const int32_t* topk, int Ksel, float softmax_scale, void* O, float* lse,
                   float* page_weight, void* ws, size_t ws_bytes, void* stream);

/*
 * Eviction of whole pages by accumulated attention weight (per request; H2O-
 * style heavy hitters at page granularity).  For every page that holds tokens
 *   score[p] = decay * acc[p] + sum over heads of page_weight[p][h]
 * (in 64 bits, rounded once).  If the request holds more than `budget` such
 * pages, the lowest scores among those that are neither its first `sink` nor
 * its last `recent` pages are dropped until `budget` remain or no page may go
 * (equal scores: the lower page; NaN ranks highest); recent is at least 1, as
 * the last page may be partly filled.  Kept pages move together
 * in order, the dropped ones follow in order as pages to grow into, then the
 * entries that held no tokens.  Physical pages do not move, so positions
 * change: token t of a kept page moves with its page.
 *   page_weight device fp32 [total_pages][Hkv]; acc device fp32 [total_pages]
 *   table_out  device int32 [total_pages], the new page table; acc_out device
 *              fp32 [total_pages], the scores in the new order (0 for dropped
 *              pages, acc for unused entries); len_out device int32 [R], the
 *              new kv_len; page_src device int32 [total_pages], the old
 *              request-local place of each entry.  They are apart from each
 *              other, but may be cache's own page_table and kv_len, and acc.  Entries of no request are left
 *              as they are.
 * Device errors: QUP_ERR_GROUP (contradictory request) and QUP_ERR_CAPACITY
 * (more than max_pages pages): the request's entries are copied unchanged.
 * QUP_ERR_ARG for max_pages beyond what one CTA's shared memory holds (24576).
 */
int qup_cache_evict(const qup_cache* cache, const float* page_weight, const float* acc, float decay, int budget,
                    int sink, int recent, int32_t* table_out, float* acc_out, int32_t* len_out, int32_t* page_src,
                    void* stream);

/* Synchronizes `stream`, then reads and clears this device's error word. */
int qup_get_error(int* code, void* stream);

/* Static text for a return code or error bit. */
const char* qup_error_string(int code);

/*
 * Pipeline-wait limit and host-side fault injection (for tests of the bounded
 * waits; both reset with wait_limit_ms <= 0 and skip_stage < 0).  With
 * skip_stage >= 0 no CTA of an attention kernel (the union kernel, those of
 * the 8-bit cache) loads that stage of its K and V rings, so the consumers'
 * waits run out after wait_limit_ms, QUP_ERR_TIMEOUT is raised and every CTA
 * exits cleanly.
 */
int qup_set_debug(int wait_limit_ms, int skip_stage);

/*
 * Checked mode (process-wide, off by default; on = nonzero).  While it is on,
 * qup_sparse_prefill_attn given a non-NULL topk first runs one extra kernel on
 * the stream that checks every bundle row against its own TopK row: a mask
 * bit is set exactly for the union pages the row selected (a set: duplicates
 * and -1 dropped), every page of the row is in the bundle union, and rows of
 * empty slots carry no bits.  A mismatch raises QUP_ERR_GROUP (a TopK ID out
 * of range QUP_ERR_PAGE_ID) in the device error word; the attention call
 * still runs.  Ksel < 0 is then QUP_ERR_ARG.  Meant for groups a caller builds
 * itself; qup_sparse_group's groups satisfy it by construction.
 */
int qup_set_checked(int on);

/* Number of SMs the persistent attention kernel is sized for on the current device. */
int qup_num_sms(void);

/*
 * Test hook (no counterpart on the pages): y[i] = 2^x[i] by the polynomial
 * exponential the attention kernel uses for part of its softmax (x clamped to
 * -127, where the result is exactly +0; x must be <= 16).  x and y are device
 * float arrays of n elements; asynchronous on `stream`.  Returns QUP_ERR_ARG
 * for n < 0 or null pointers with n > 0, QUP_ERR_CUDA for a launch failure.
 */
int qup_exp2_poly(const float* x, float* y, int n, void* stream);

#ifdef __cplusplus
}
#endif
#endif
