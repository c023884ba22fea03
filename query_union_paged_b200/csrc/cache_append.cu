// cache_append.cu -- new tokens into the paged E4M3 cache, one scale per (page, KV head).
//
// A page's scale is a power of two: s = 2^k, the smallest k >= -64 with amax <= 448 * 2^k over the
// page's tokens (448: E4M3's largest value).  E4M3 is a floating format, so a power of two loses
// nothing against amax / 448 but the subnormal end of the range, and multiplying by it is exact:
// when a later token needs a larger scale, the page's older bytes are requantised by an exact shift
// of the exponent (only values that become subnormal are rounded again), so a page filled one token
// at a time holds the bytes of a page written at once, but for those.
//
// One CTA per run of a request's tokens inside one page, for some of its units (K or V of a KV head).  A
// unit's tokens are read once into registers (16 bytes a load), their largest finite magnitude is
// reduced over the CTA, and the registers are scaled, rounded (nearest even) and written; the next
// unit's loads are under way meanwhile.  A run without infinities and NaN takes the short way: two
// magnitudes an instruction, no test of each value (with them the kernel was bound by its instructions,
// 3.4 TB/s; now 5.3 TB/s for 83K tokens of 8 heads, and 7 us where 64 requests write one token each: a
// launch and four dependent loads).  Bound by DRAM: N * Hkv * 128 * (element + 1) bytes for each of
// K and V.
#include <algorithm>
#include <cstdint>

#include "cache.h"
#include "ptx.cuh"
#include "internal.h"
#include "query_union_paged.h"

namespace qup {
namespace {

constexpr int kChunk = 8;                        // elements of one thread's load
constexpr int kChunksPerToken = kHeadDim / kChunk;

// First item of request r: items of a request are its touched pages, at most
// min(n, n / T + 2) of them, so these starts leave every request room for its own.
__device__ __forceinline__ int item_start(int ptr, int r, int T) { return min(ptr, ptr / T + 2 * r); }

// exponent k of the smallest power of two with amax <= 448 * 2^k, at least -64; amax as fp32 bits
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23) - 127;                    // amax = 1.m * 2^e
    const int k = e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u);  // 448 = 1.75 * 2^8
    return amax_bits < 0x00800000u ? -64 : max(k, -64);
}
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}
__device__ __forceinline__ float f16_lo(uint32_t v) {
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(v));
    return f;
}
__device__ __forceinline__ float f16_hi(uint32_t v) { return f16_lo(v >> 16); }

// E4M3 bytes of four values already divided by the scale; a value that is not finite becomes NaN
// (0x7f), which the saturating conversion would turn an infinity into 448 instead of.
__device__ __forceinline__ uint32_t pack_e4m3_checked(const float* x) {
    uint32_t w = pack_e4m3x4(x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if ((__float_as_uint(x[e]) & 0x7f800000u) == 0x7f800000u) w = (w & ~(0xffu << (8 * e))) | (0x7fu << (8 * e));
    return w;
}

// The CTA's maximum; `part` holds one entry per warp.
template <int WARPS>
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t* part) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v = max(v, part[w]);
    return v;
}

template <int T>
constexpr int kAppendThreads = T == 128 ? 512 : 256;

template <int T, bool BF16>
__global__ void __launch_bounds__(kAppendThreads<T>) cache_append_kernel(CacheView c, const void* __restrict__ k_new,
                                                                           const void* __restrict__ v_new,
                                                                           long long k_stride, long long v_stride,
                                                                           const int32_t* __restrict__ tok_ptr, int N,
                                                                           int units, int groups, unsigned* err) {
    constexpr int NT = kAppendThreads<T>;
    constexpr int CH = T * kChunksPerToken / NT;  // chunks of one thread
    constexpr int W = BF16 ? 1 : 2;               // 16-byte words of a chunk
    __shared__ int s_req;
    __shared__ uint32_t s_max[2][NT / 32];
    const int tid = threadIdx.x, item = blockIdx.x / groups;
    grid_dep_wait();
    if (tid == 0) s_req = -1;
    __syncthreads();
    for (int r = tid; r < c.R; r += NT)
        if (item_start(tok_ptr[r], r, T) <= item && item < item_start(tok_ptr[r + 1], r + 1, T)) s_req = r;
    __syncthreads();
    const int r = s_req;
    if (r < 0) return;
    const Request q = load_request(tok_ptr, N, c.kv_len, c.page_ptr, c.total_pages, T, r);
    if (!q.ok || q.len < q.n) {
        if (tid == 0) atomicOr(err, QUP_ERR_GROUP);
        return;
    }
    const int start = q.len - q.n, j = item - item_start(q.q0, r, T);
    const int page = start / T + j;  // of the request
    if ((long long)page * T >= q.len || q.n == 0) return;
    const int a = j == 0 ? start % T : 0, b = min(T, q.len - page * T);  // new slots [a, b)
    const long long tok0 = (long long)q.q0 + page * T - start;           // batch row of slot 0
    const int phys = c.page_table[q.p0 + page];
    if (phys < 0 || phys >= c.P_phys) {
        if (tid == 0) atomicOr(err, QUP_ERR_PHYS_PAGE);
        return;
    }
    // units (K or V of a head) [u0, u1): the next one's tokens are on their way while one is written
    const int u0 = (blockIdx.x - item * groups) * units, u1 = min(2 * c.Hkv, u0 + units);
    const auto load = [&](int u, uint4 (&raw)[CH][W]) {
        const char* in = static_cast<const char*>((u & 1) ? v_new : k_new);
        const long long stride = (u & 1) ? v_stride : k_stride;
#pragma unroll
        for (int x = 0; x < CH; ++x) {
            const int at = tid + x * NT, slot = at / kChunksPerToken, part = at % kChunksPerToken;
#pragma unroll
            for (int v = 0; v < W; ++v) {
                raw[x][v] = make_uint4(0u, 0u, 0u, 0u);
                if (slot >= a && slot < b)
                    raw[x][v] = __ldg(reinterpret_cast<const uint4*>(
                                          in + ((tok0 + slot) * stride + (long long)(u >> 1) * kHeadDim + part * kChunk) *
                                                   (BF16 ? 2 : 4)) +
                                      v);
            }
        }
    };
    uint4 raw[CH][W], next[CH][W];
    load(u0, raw);
    for (int u = u0; u < u1; ++u) {
        const int h = u >> 1;
        const bool isv = u & 1;
        float* scale = (isv ? c.v_scale : c.k_scale) + (size_t)phys * c.Hkv + h;
        const float s_old = a > 0 ? *scale : 0.f;
        if (u + 1 < u1) load(u + 1, next);
        uint8_t* out = (isv ? c.V : c.K) + ((size_t)phys * c.Hkv + h) * T * kHeadDim;
        // the largest magnitude of the run's tokens; among finite ones only where one is not finite
        uint32_t amax = 0;
#pragma unroll
        for (int x = 0; x < CH; ++x)
#pragma unroll
            for (int v = 0; v < W; ++v) {
                const uint32_t w[4] = {raw[x][v].x, raw[x][v].y, raw[x][v].z, raw[x][v].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)  // bf16: both halves at once
                    amax = BF16 ? __vmaxu2(amax, w[e] & 0x7fff7fffu) : max(amax, w[e] & 0x7fffffffu);
            }
        if (BF16) amax = max(amax << 16, amax & 0xffff0000u);
        amax = cta_max<NT / 32>(amax, s_max[u & 1]);
        const bool finite = amax < 0x7f800000u;
        if (!finite) {
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < CH; ++x)
#pragma unroll
                for (int v = 0; v < W; ++v) {
                    const uint32_t w[4] = {raw[x][v].x, raw[x][v].y, raw[x][v].z, raw[x][v].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = BF16 ? (w[e] << 16) & 0x7fffffffu : w[e] & 0x7fffffffu, hi = w[e] & 0x7fff0000u;
                        if (lo < 0x7f800000u) top = max(top, lo);
                        if (BF16 && hi < 0x7f800000u) top = max(top, hi);
                    }
                }
            __syncthreads();  // every thread has read the first maximum
            amax = cta_max<NT / 32>(top, s_max[u & 1]);
        }
        if (!(s_old >= 0.f) || (__float_as_uint(s_old) & 0x7f800000u) == 0x7f800000u) {
            if (tid == 0) atomicOr(err, QUP_ERR_SCALE);
        } else {
            const float s = fmaxf(pow2(scale_exponent(amax)), s_old);
            // 1 / s is exact for a power of two; a caller's own scale (s_old kept) takes the division
            const bool exact = (__float_as_uint(s) & 0x7fffffu) == 0 && s < 8.5e37f;  // 2^126
            const float inv = exact ? pow2(127 - (int)(__float_as_uint(s) >> 23)) : 0.f;
            const bool plain = finite && exact;
#pragma unroll
            for (int x = 0; x < CH; ++x) {
                const int at = tid + x * NT, slot = at / kChunksPerToken, part = at % kChunksPerToken;
                uint2* dst = reinterpret_cast<uint2*>(out + (size_t)slot * kHeadDim + part * kChunk);
                float f[kChunk];
                if (slot < a) {  // an older token: requantised when the page's scale grew
                    if (s == s_old) continue;
                    const float ratio = __fdiv_rn(s_old, s);
                    const uint2 w = *dst;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t v = e4m3x2_to_f16x2((uint16_t)((e < 2 ? w.x : w.y) >> (16 * (e & 1))));
                        f[2 * e] = f16_lo(v) * ratio;
                        f[2 * e + 1] = f16_hi(v) * ratio;
                    }
                    *dst = make_uint2(pack_e4m3_checked(f), pack_e4m3_checked(f + 4));
                } else if (slot < b) {
                    if constexpr (BF16) {
                        const uint32_t w[4] = {raw[x][0].x, raw[x][0].y, raw[x][0].z, raw[x][0].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f[2 * e] = __uint_as_float(w[e] << 16);
                            f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                        }
                    } else {
#pragma unroll
                        for (int v = 0; v < W; ++v) {
                            f[4 * v] = __uint_as_float(raw[x][v].x);
                            f[4 * v + 1] = __uint_as_float(raw[x][v].y);
                            f[4 * v + 2] = __uint_as_float(raw[x][v].z);
                            f[4 * v + 3] = __uint_as_float(raw[x][v].w);
                        }
                    }
                    if (plain) {
#pragma unroll
                        for (int e = 0; e < kChunk; ++e) f[e] *= inv;
                        *dst = make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < kChunk; ++e) f[e] = exact ? f[e] * inv : __fdiv_rn(f[e], s);
                        *dst = make_uint2(pack_e4m3_checked(f), pack_e4m3_checked(f + 4));
                    }
                }
            }
            if (tid == 0 && (a == 0 || s != s_old)) *scale = s;
        }
#pragma unroll
        for (int x = 0; x < CH; ++x)
#pragma unroll
            for (int v = 0; v < W; ++v) raw[x][v] = next[x][v];
    }
}

template <int T>
cudaError_t launch_t(const CacheView& c, const void* k_new, const void* v_new, bool bf16, long long k_stride,
                     long long v_stride, const int32_t* tok_ptr, int N, int sms, unsigned* err, cudaStream_t stream) {
    const long long items = std::min<long long>(N, N / T + 2ll * c.R);
    // units of a CTA: one while the grid is small (a token for each of many requests), up to eight where
    // there are CTAs enough to fill the SMs several times
    const int all = 2 * c.Hkv;
    const int units = (int)std::max<long long>(1, std::min<long long>(std::min(8, all), items * all / (16ll * sms)));
    // a run's units are neighbours in the grid: they read the same tokens' rows at about the same time
    const int groups = (all + units - 1) / units;
    const dim3 grid((unsigned)(items * groups)), block(kAppendThreads<T>);
    return bf16 ? launch_pdl(cache_append_kernel<T, true>, grid, block, 0, stream, c, k_new, v_new, k_stride, v_stride,
                             tok_ptr, N, units, groups, err)
                : launch_pdl(cache_append_kernel<T, false>, grid, block, 0, stream, c, k_new, v_new, k_stride, v_stride,
                             tok_ptr, N, units, groups, err);
}

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, const void* k_new, const void* v_new, bool bf16,
                                long long k_stride, long long v_stride, const int32_t* tok_ptr, int N, int sms, unsigned* err,
                                cudaStream_t stream) {
    if (N == 0 || c.R == 0) return cudaSuccess;
    switch (c.T) {
        case 16: return launch_t<16>(c, k_new, v_new, bf16, k_stride, v_stride, tok_ptr, N, sms, err, stream);
        case 32: return launch_t<32>(c, k_new, v_new, bf16, k_stride, v_stride, tok_ptr, N, sms, err, stream);
        case 64: return launch_t<64>(c, k_new, v_new, bf16, k_stride, v_stride, tok_ptr, N, sms, err, stream);
        default: return launch_t<128>(c, k_new, v_new, bf16, k_stride, v_stride, tok_ptr, N, sms, err, stream);
    }
}

}  // namespace qup
