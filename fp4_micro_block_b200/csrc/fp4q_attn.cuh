// fp4q_attn.cuh -- attention of bf16 queries over the paged 8-bit cache.
#pragma once

#include "fp4q_kv.cuh"

namespace fp4q {

struct AttnParams {
    KvCacheView c;
    const uint16_t* q;
    int64_t ldq, tokens;
    int32_t q_heads, group;  // query heads, query heads per K/V head
    const int32_t *cu, *lens;
    int64_t batch, max_q, max_len;
    int causal;
    float scale_log2;  // softmax_scale * log2(e)
    uint16_t* o;
    int64_t ldo;
    float* lse;
};

constexpr float kLn2 = 0.693147180559945309f;

// Rows and keys of sequence b, clamped to what exists; reports what it clamps.
struct AttnSeq {
    int64_t first, n, len;
};
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int64_t b, bool tell) {
    AttnSeq s;
    int64_t lo = p.cu[b], hi = p.cu[b + 1], len = p.lens[b];
    bool bad = lo < 0 || hi < lo || hi > p.tokens || hi - lo > p.max_q;
    if (bad) hi = lo = 0;
    const int64_t most = min64(p.c.table_stride * p.c.page, p.max_len);
    if (len < 0 || len > most) {
        bad = true;
        len = len < 0 ? 0 : most;
    }
    if (bad && tell) atomicOr(&g_device_error, kErrBadIndex);
    s.first = lo;
    s.n = hi - lo;
    s.len = len;
    return s;
}

// Page id of the sequence's page pg, clamped into the pool.
__device__ __forceinline__ int64_t attn_page(const AttnParams& p, int64_t b, int64_t pg, bool tell) {
    int64_t id = p.c.table[b * p.c.table_stride + pg];
    if (id < 0 || id >= p.c.num_pages) {
        if (tell) atomicOr(&g_device_error, kErrBadIndex);
        id = 0;
    }
    return id;
}

// One warp per (query, head); lanes share the head dimension.
template <int D>
__global__ void __launch_bounds__(128) attn_simple_kernel(const AttnParams p) {
    constexpr int N = D / 32;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int h = (int)(i % p.q_heads);
    i /= p.q_heads;
    const int64_t row = i % p.max_q, b = i / p.max_q;
    if (b >= p.batch) return;
    const AttnSeq s = attn_seq(p, b, lane == 0);
    if (row >= s.n) return;
    const int hk = h / p.group;
    const uint16_t* q = p.q + (s.first + row) * p.ldq + (int64_t)h * D + lane * N;
    float qv[N], o[N];
#pragma unroll
    for (int t = 0; t < N; ++t) {
        qv[t] = __uint_as_float((uint32_t)q[t] << 16) * p.scale_log2;
        o[t] = 0.0f;
    }
    const int64_t keys = p.causal ? s.len - s.n + row + 1 : s.len;
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = 0; j < keys; ++j) {
        const int64_t at = attn_page(p, b, j / p.c.page, lane == 0) * p.c.heads + hk;
        const int64_t off = (at * p.c.page + j % p.c.page) * D + lane * N;
        float dot = 0.0f;
#pragma unroll
        for (int t = 0; t < N; ++t) dot = fmaf(qv[t], e4m3_decode(p.c.k[off + t]), dot);
#pragma unroll
        for (int x = 16; x; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        dot *= p.c.k_scale[at];
        const float top = fmaxf(m, dot), keep = exp2f(m - top), w = exp2f(dot - top);
        const float vs = p.c.v_scale[at];
        l = l * keep + w;
#pragma unroll
        for (int t = 0; t < N; ++t) o[t] = fmaf(o[t], keep, w * vs * e4m3_decode(p.c.v[off + t]));
        m = top;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int t = 0; t < N; ++t)
        p.o[(s.first + row) * p.ldo + (int64_t)h * D + lane * N + t] = (uint16_t)bf16x2_pack(o[t] * inv, 0.0f);
    if (p.lse && lane == 0) p.lse[(s.first + row) * p.q_heads + h] = keys > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace fp4q
