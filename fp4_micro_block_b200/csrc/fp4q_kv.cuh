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

// Bytes of w that are NaN codes, as 0xff; the others 0.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

struct KvAppendParams {
    KvCacheView c;
    const uint16_t *k, *v;
    int64_t ldk, ldv, tokens;
    const int32_t *cu, *lens;
    int64_t max_new;
    uint32_t pages_per_seq;  // pages a sequence's new tokens may touch
    int32_t per_row_log2;    // log2 of the eight-column pieces of a row
};

// One CTA per (sequence, touched page, head, K or V).  A thread holds up to
// kKvPieces pieces of eight columns of the page's new rows between the maximum
// and the codes, so that they are read once; the launch has threads for a whole
// page.  A CTA is one chain of dependent steps (table, rows, maximum, codes),
// with stalls on loads of 4.9 warps an issue: 4 x 2048 tokens of 8 heads of 128 10.4
// us, 0.65 of the 6458 GB/s copy rate, 64 single tokens 2.5 us.
constexpr int kKvPieces = 8, kKvMaxThreads = 512;
__global__ void __launch_bounds__(kKvMaxThreads) kv_append_kernel(const KvAppendParams p) {
    __shared__ uint32_t part[kKvMaxThreads / 32];
    pdl_wait();
    pdl_trigger();
    const KvCacheView& c = p.c;
    uint32_t i = blockIdx.x;
    const bool is_v = i & 1;
    i >>= 1;
    const int h = (int)(i % (uint32_t)c.heads);
    i /= (uint32_t)c.heads;
    const uint32_t b = i / p.pages_per_seq, j = i - b * p.pages_per_seq;
    // the new tokens' rows and positions
    int64_t lo = p.cu[b], hi = p.cu[b + 1];
    const int64_t end = p.lens[b];
    bool bad = lo < 0 || hi < lo || hi > p.tokens || hi - lo > p.max_new;
    if (bad) hi = lo;
    const int n = (int)(hi - lo);
    const int64_t begin = end - n;
    bad = bad || begin < 0 || end > c.table_stride * c.page;
    const int pg = (int)((uint32_t)(bad ? 0 : begin) / (uint32_t)c.page + j);  // page index within the sequence
    const int64_t p0 = (int64_t)pg * c.page;                                   // its first position
    const int from = (int)(begin > p0 ? begin - p0 : 0), to = (int)min64(end - p0, c.page);  // rows of the page
    int64_t page = -1;
    if (from < to && !bad) {
        page = c.table[b * c.table_stride + pg];
        if (page < 0 || page >= c.num_pages) bad = true;
    }
    if (bad && threadIdx.x == 0) atomicOr(&g_device_error, kErrBadIndex);
    if (bad || from >= to) return;

    const int64_t ld = is_v ? p.ldv : p.ldk;
    uint8_t* codes = (is_v ? c.v : c.k) + (page * c.heads + h) * (int64_t)c.page * c.dim;
    float* scale = (is_v ? c.v_scale : c.k_scale) + page * c.heads + h;
    // from: rows the page has already
    const int count = (to - from) << p.per_row_log2, mask = (1 << p.per_row_log2) - 1;
    const uint16_t* rows = (is_v ? p.v : p.k) + (lo + (p0 + from - begin)) * ld + (int64_t)h * c.dim;

    const float old = from > 0 ? *scale : 0.0f;
    uint4 w[kKvPieces];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kKvPieces; ++k) {
        const int e = threadIdx.x + k * blockDim.x;
        w[k] = make_uint4(0, 0, 0, 0);
        if (e < count) w[k] = __ldg(reinterpret_cast<const uint4*>(rows + (e >> p.per_row_log2) * ld + (e & mask) * 8));
    }
#pragma unroll
    for (int k = 0; k < kKvPieces; ++k) m = bf16x2_max(m, amax8x2(w[k]));
#pragma unroll
    for (int o = 16; o; o >>= 1) m = bf16x2_max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();  // also: every thread has the old scale before it is replaced
    for (uint32_t k = 0; k < blockDim.x / 32; ++k) m = bf16x2_max(m, part[k]);
    const float s = fmaxf(old, kv_scale(bf16x2_top(m))), inv = kv_inverse(s);
    if (threadIdx.x == 0) *scale = s;
    if (s > old && from > 0) {  // what the page has moves to the new scale (under a scale of 0: zeros and NaN, which stay)
        const float ratio = old * inv;
        for (int e = threadIdx.x; e < from << p.per_row_log2; e += blockDim.x) {
            uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)e * 8);
            const uint2 x = *at;
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = e4m3_decode(((k < 4 ? x.x : x.y) >> (8 * (k & 3)))) * ratio;
            *at = old > 0.0f ? make_uint2(e4m3_pack4(f[0], f[1], f[2], f[3]), e4m3_pack4(f[4], f[5], f[6], f[7]))
                             : make_uint2(nan_bytes(x.x) & 0x7f7f7f7fu, nan_bytes(x.y) & 0x7f7f7f7fu);
        }
    }
    uint8_t* dst = codes + ((int64_t)from << (p.per_row_log2 + 3));
    if (s != 0.0f && (__float_as_uint(s) & 0x7fffffu) == 0) {  // a power of two, as this kernel writes it: exact products
        const uint64_t inv2 = f2_both(inv);
#pragma unroll
        for (int k = 0; k < kKvPieces; ++k) {
            const int e = threadIdx.x + k * blockDim.x;
            if (e >= count) break;
            const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            uint64_t f[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) f[t] = f2_mul(f2_pack(u[t] << 16, u[t] & 0xffff0000u), inv2);
            *reinterpret_cast<uint2*>(dst + (int64_t)e * 8) =
                make_uint2(e4m3_pack4(f2_lo(f[0]), f2_hi(f[0]), f2_lo(f[1]), f2_hi(f[1])),
                           e4m3_pack4(f2_lo(f[2]), f2_hi(f[2]), f2_lo(f[3]), f2_hi(f[3])));
        }
    } else {  // a calibrated scale of the caller's, or a page without numbers
#pragma unroll 1
        for (int e = threadIdx.x; e < count; e += blockDim.x) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(rows + (e >> p.per_row_log2) * ld + (e & mask) * 8));
            *reinterpret_cast<uint2*>(dst + (int64_t)e * 8) = make_uint2(fp8_codes_ieee(x.x, x.y, s), fp8_codes_ieee(x.z, x.w, s));
        }
    }
}

}  // namespace fp4q
