// cache.h -- the 8-bit page-scaled cache operators (append, attention, eviction): parameter
// structs and launchers (cache_append.cu, cache_attn.cu, cache_evict.cu), for the C ABI
// (cache_api.cu).
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace qup {

// What the host layer looks up once per context (api.cu): the device error word, the SM count and
// the shared-memory limit, and the driver's tensor-map encoder.
typedef CUresult (*TensorMapEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                      const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                      CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
struct DeviceInfo {
    unsigned* err;
    int sms;
    int smem_optin;
    TensorMapEncodeFn encode;
};
int device_info(DeviceInfo* out);  // QUP_OK or QUP_ERR_CUDA
unsigned long long wait_limit_ns();  // limit of a pipeline wait (qup_set_debug)
int debug_skip_stage();              // stage that is not loaded, -1: none (likewise)

// The cache of R requests: qup_cache of the C ABI.
struct CacheView {
    uint8_t* K;
    uint8_t* V;
    float* k_scale;
    float* v_scale;
    const int32_t* page_table;
    const int32_t* page_ptr;
    const int32_t* kv_len;
    int P_phys, Hkv, T, R, total_pages;
};

// One request's rows [q0, q0 + n), cache length and pages [p0, p0 + np); ok = 0 when its entries
// contradict each other (rows outside the batch, a length past its pages, pages outside the table).
struct Request {
    int q0, n, len, p0, np, ok;
};
__device__ __forceinline__ Request load_request(const int32_t* row_ptr, int N, const int32_t* kv_len,
                                                const int32_t* page_ptr, int total_pages, int T, int r) {
    Request q;
    q.q0 = row_ptr[r];
    const int q1 = row_ptr[r + 1];
    q.len = kv_len[r];
    q.p0 = page_ptr[r];
    const int p1 = page_ptr[r + 1];
    q.n = q1 - q.q0;
    q.np = p1 - q.p0;
    q.ok = q.q0 >= 0 && q1 >= q.q0 && q1 <= N && q.p0 >= 0 && p1 >= q.p0 && p1 <= total_pages && q.len >= 0 &&
           (long long)q.len <= (long long)q.np * T;
    return q;
}

cudaError_t launch_cache_append(const CacheView& c, const void* k_new, const void* v_new, bool bf16,
                                long long k_stride, long long v_stride, const int32_t* tok_ptr, int N, int sms,
                                unsigned* err, cudaStream_t stream);

// cap: used pages of one request, at most (QUP_CACHE_EVICT_PAGES: a CTA's shared memory holds them)
size_t cache_evict_smem(int cap);
cudaError_t launch_cache_evict(const CacheView& c, const float* weight, const float* acc, float decay, int budget,
                               int sink, int recent, int cap, int32_t* table_out, float* acc_out, int32_t* len_out,
                               int32_t* page_src, unsigned* err, cudaStream_t stream);

}  // namespace qup
