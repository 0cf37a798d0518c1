// fp4q_kv.cuh -- the paged 8-bit K/V cache and its writer.
//
// A page holds page_size tokens of one K/V head as contiguous E4M3 codes
// [page_size, D] under one power-of-two scale
//   s = 2^ceil(log2(amax / 448)),
// so that a page filled one token at a time keeps its codes when the scale
// grows: they move by a power of two, rounded again only among E4M3's
// subnormals.
#pragma once

#include "fp4q_fp8.cuh"

namespace fp4q {

struct KvCacheView {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t num_pages;
    int32_t heads, page, dim;
    const int32_t* table;
    int64_t table_stride;
};

// Smallest power of two s with amax / s <= 448 = 1.75 * 2^8, at least 2^-126
// (amax finite, >= 0; an infinity gives 2^120, whose codes saturate): amax =
// 1.f * 2^e needs 2^(e - 8), one step more where 1.f > 1.75.
__device__ __forceinline__ float kv_scale(float amax) {
    if (amax == 0.0f) return 0.0f;
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent of s
    e = e < 1 ? 1 : e;
    return __uint_as_float((uint32_t)e << 23);
}
// 1 / s, exact: s = 2^j, -126 <= j <= 120; s = 2^-126 has 2^126.
__device__ __forceinline__ float kv_inverse(float s) {
    return s == 0.0f ? 0.0f : __uint_as_float((254u << 23) - __float_as_uint(s));
}

// x / s: an exact product where s is a power of two, as this file writes it; a
// page may also carry a calibrated scale of the caller's.
__device__ __forceinline__ float kv_quot(float x, float s, float inv) {
    return (__float_as_uint(s) & 0x7fffffu) == 0 ? x * inv : __fdiv_rn(x, s);
}

struct KvAppendParams {
    KvCacheView c;
    const uint16_t *k, *v;
    int64_t ldk, ldv, tokens;
    const int32_t *cu, *lens;
    int64_t max_new;
    int64_t pages_per_seq;  // pages a sequence's new tokens may touch
};

// One CTA per (sequence, touched page, head, K or V).  Every step is a pass over
// the page's rows by all threads, eight columns each.
constexpr int kKvThreads = 128;
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvAppendParams p) {
    __shared__ float part[kKvThreads / 32];
    pdl_wait();
    pdl_trigger();
    const KvCacheView& c = p.c;
    int64_t i = blockIdx.x;
    const bool is_v = i & 1;
    i >>= 1;
    const int h = (int)(i % c.heads);
    i /= c.heads;
    const int64_t j = i % p.pages_per_seq, b = i / p.pages_per_seq;
    // the new tokens' rows and positions
    int64_t lo = p.cu[b], hi = p.cu[b + 1];
    bool bad = lo < 0 || hi < lo || hi > p.tokens || hi - lo > p.max_new;
    if (bad) hi = lo;
    const int64_t n = hi - lo, end = p.lens[b], begin = end - n;
    bad = bad || begin < 0 || end > c.table_stride * c.page;
    const int64_t pg = (begin < 0 ? 0 : begin) / c.page + j;  // page index within the sequence
    const int64_t p0 = pg * c.page;                           // its first position
    int64_t from = begin > p0 ? begin : p0, to = end < p0 + c.page ? end : p0 + c.page;
    int64_t page = -1;
    if (from < to && !bad) {
        page = c.table[b * c.table_stride + pg];
        if (page < 0 || page >= c.num_pages) bad = true;
    }
    if (bad && threadIdx.x == 0) atomicOr(&g_device_error, kErrBadIndex);
    if (bad || from >= to) return;

    const uint16_t* src = is_v ? p.v : p.k;
    const int64_t ld = is_v ? p.ldv : p.ldk;
    uint8_t* codes = (is_v ? c.v : c.k) + (page * c.heads + h) * (int64_t)c.page * c.dim;
    float* scale = (is_v ? c.v_scale : c.k_scale) + page * c.heads + h;
    const int per_row = c.dim / 8;
    const int kept = (int)(from - p0);  // rows the page has already
    const int count = (int)(to - from) * per_row;
    const uint16_t* rows = src + (lo + from - begin) * ld + (int64_t)h * c.dim;

    float amax = 0.0f;
    for (int e = threadIdx.x; e < count; e += kKvThreads) {
        const int r = e / per_row, q = e - r * per_row;
        amax = fmaxf(amax, amax8(__ldg(reinterpret_cast<const uint4*>(rows + r * ld + q * 8))));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    const float old = kept > 0 ? *scale : 0.0f;
    __syncthreads();  // every thread has the old scale before it is replaced
    for (int w = 0; w < kKvThreads / 32; ++w) amax = fmaxf(amax, part[w]);
    const float s = fmaxf(old, kv_scale(amax)), inv = kv_inverse(s);
    if (threadIdx.x == 0) *scale = s;
    if (s > old && old > 0.0f) {
        const float ratio = old * inv;
        for (int e = threadIdx.x; e < kept * per_row; e += kKvThreads) {
            uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)e * 8);
            const uint2 w = *at;
            float f[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) f[t] = e4m3_decode(((t < 4 ? w.x : w.y) >> (8 * (t & 3)))) * ratio;
            *at = make_uint2(e4m3_pack4(f[0], f[1], f[2], f[3]), e4m3_pack4(f[4], f[5], f[6], f[7]));
        }
    } else if (s > old) {  // a page of zeros so far
        for (int e = threadIdx.x; e < kept * per_row; e += kKvThreads)
            *reinterpret_cast<uint2*>(codes + (int64_t)e * 8) = make_uint2(0, 0);
    }
    for (int e = threadIdx.x; e < count; e += kKvThreads) {
        const int r = e / per_row, q = e - r * per_row;
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(rows + r * ld + q * 8));
        *reinterpret_cast<uint2*>(codes + (int64_t)(kept + r) * c.dim + q * 8) =
            make_uint2(e4m3_pack4(kv_quot(bf16lo(w.x), s, inv), kv_quot(bf16hi(w.x), s, inv),
                                  kv_quot(bf16lo(w.y), s, inv), kv_quot(bf16hi(w.y), s, inv)),
                       e4m3_pack4(kv_quot(bf16lo(w.z), s, inv), kv_quot(bf16hi(w.z), s, inv),
                                  kv_quot(bf16lo(w.w), s, inv), kv_quot(bf16hi(w.w), s, inv)));
    }
}

}  // namespace fp4q
