// fp4q_fp8.cuh -- E4M3 codes under one FP32 scale per block of 128: the format's
// device helpers and the quantizer.
//
//   s = amax_block / 448,  code = E4M3(x / s)  (nearest even, saturating)
//
// One read of x gives the codes of x, of its transpose, or both: the blocks of
// the transpose run down the columns, so a CTA holds a whole 128 x 128 tile.
#pragma once

#include "fp4q_device.cuh"

namespace fp4q {

constexpr int kFp8Block = 128;
constexpr float kE4m3Max = 448.0f;

// Four E4M3 codes (v[0] in the low byte): nearest even, saturating, NaN -> 0x7f.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
    uint32_t w;
    asm("{ .reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h}; }"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// Four E4M3 codes as two f16 pairs (exact).
struct Half4 {
    uint32_t lo, hi;
};
__device__ __forceinline__ Half4 e4m3x4_f16(uint32_t four) {
    Half4 h;
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(h.lo), "=r"(h.hi)
        : "r"(four));
    return h;
}

// Block scale and the reciprocal that its quotients use: inv = RN(1/s) where
// div_rn's preconditions hold for every |x| <= amax, else 0 (IEEE division).
struct Fp8Scale {
    float s, inv;
};
__device__ __forceinline__ Fp8Scale fp8_scale(float amax) {
    Fp8Scale r;
    r.s = __fdiv_rn(amax, kE4m3Max);
    r.inv = div_fast_ok(r.s, amax) ? __frcp_rn(r.s) : 0.0f;
    return r;
}
__device__ __forceinline__ float fp8_quot(float x, const Fp8Scale& f) {
    if (f.inv != 0.0f) return div_rn(x, f.s, f.inv);
    return f.s == 0.0f ? 0.0f : __fdiv_rn(x, f.s);
}

struct Fp8QuantParams {
    const uint16_t* x;
    int64_t M, K, ldx;
    uint8_t* codes;
    int64_t ldc;
    float* scales;
    int64_t lds;
    uint8_t* codes_t;
    int64_t ldct;
    float* scales_t;
    int64_t ldst;
    int64_t n_kb, n_items;  // 128-column blocks of a row; work items
};

// Eight bf16 of row r, columns c .. c + 7, as four words; zeros outside [0, M) x [0, K).
__device__ __forceinline__ uint4 fp8_load8(const Fp8QuantParams& p, int64_t r, int64_t c) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (r >= p.M || c >= p.K) return w;
    const uint16_t* src = p.x + r * p.ldx + c;
    if (c + 8 <= p.K) return __ldg(reinterpret_cast<const uint4*>(src));
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = c + i < p.K ? (uint32_t)src[i] : 0u;
    w.x = e[0] | e[1] << 16;
    w.y = e[2] | e[3] << 16;
    w.z = e[4] | e[5] << 16;
    w.w = e[6] | e[7] << 16;
    return w;
}

// The first n (1..8) of eight code bytes; one 8-byte store where all are wanted
// (rows of codes start 16-byte aligned).
__device__ __forceinline__ void fp8_store8(uint8_t* dst, uint32_t lo, uint32_t hi, int64_t n) {
    if (n >= 8) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) dst[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
}

__device__ __forceinline__ float amax8(const uint4& w) {
    const float a = fmaxf(fmaxf(fabsf(bf16lo(w.x)), fabsf(bf16hi(w.x))), fmaxf(fabsf(bf16lo(w.y)), fabsf(bf16hi(w.y))));
    const float b = fmaxf(fmaxf(fabsf(bf16lo(w.z)), fabsf(bf16hi(w.z))), fmaxf(fabsf(bf16lo(w.w)), fabsf(bf16hi(w.w))));
    return fmaxf(a, b);
}

// Row blocks alone: 16 lanes hold one 1 x 128 block, eight elements each.
constexpr int kFp8RowThreads = 256;
__global__ void __launch_bounds__(kFp8RowThreads) fp8_row_kernel(const Fp8QuantParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane16 = threadIdx.x & 15;
    const int64_t step = (int64_t)gridDim.x * (kFp8RowThreads / 16);
    const int64_t first = (int64_t)blockIdx.x * (kFp8RowThreads / 16) + (threadIdx.x >> 4);
    // both halves of a warp make the same number of trips (the shuffles' lanes)
    for (int64_t base = first & ~1ll; base < p.n_items; base += step) {
        const int64_t i = base + (first & 1);
        const int64_t r = i / p.n_kb, kb = i - r * p.n_kb;
        const int64_t c = kb * kFp8Block + lane16 * 8;
        const uint4 w = i < p.n_items ? fp8_load8(p, r, c) : make_uint4(0, 0, 0, 0);
        float amax = amax8(w);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (i >= p.n_items) continue;
        const Fp8Scale f = fp8_scale(amax);
        if (c < p.K)
            fp8_store8(p.codes + r * p.ldc + c,
                       e4m3_pack4(fp8_quot(bf16lo(w.x), f), fp8_quot(bf16hi(w.x), f), fp8_quot(bf16lo(w.y), f),
                                  fp8_quot(bf16hi(w.y), f)),
                       e4m3_pack4(fp8_quot(bf16lo(w.z), f), fp8_quot(bf16hi(w.z), f), fp8_quot(bf16lo(w.w), f),
                                  fp8_quot(bf16hi(w.w), f)),
                       p.K - c);
        if (lane16 == 0) p.scales[kb * p.lds + r] = f.s;
    }
}

// One 128 x 128 tile per CTA, held in registers: thread (rg, cl) has rows
// 8 rg .. 8 rg + 7, columns 8 cl .. 8 cl + 7, so that a row's 128 columns are
// the 16 lanes of a half-warp (coalesced loads and stores, row maxima by
// shuffles) and a column's eight rows are one 8-byte piece of the transpose.
// Those pieces cross the CTA through 16 KiB of shared memory whose 8-byte units
// are swizzled by the column group, so that neither side has bank conflicts.
constexpr int kFp8TileThreads = 256;
template <bool TILE>
__global__ void __launch_bounds__(kFp8TileThreads) fp8_tile_kernel(const Fp8QuantParams p) {
    __shared__ __align__(16) uint8_t turned[kFp8Block * kFp8Block];
    __shared__ float part[8][kFp8Block];
    __shared__ Fp8Scale col_scale[kFp8Block];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cl = tid & 15, rg = tid >> 4;
    pdl_wait();
    pdl_trigger();
    const int64_t mb = blockIdx.x / p.n_kb, kb = blockIdx.x - mb * p.n_kb;
    const int64_t r0 = mb * kFp8Block + rg * 8, c = kb * kFp8Block + cl * 8;
    uint4 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = fp8_load8(p, r0 + i, c);

    Fp8Scale whole;
    if constexpr (TILE) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, amax8(w[i]));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) part[warp][0] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, part[i][0]);
        whole = fp8_scale(amax);
        if (tid == 0) {
            if (p.codes) p.scales[kb * p.lds + mb] = whole.s;
            if (p.codes_t) p.scales_t[mb * p.ldst + kb] = whole.s;
        }
    } else if (p.codes_t) {
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                m[2 * j] = fmaxf(m[2 * j], fabsf(bf16lo(u[j])));
                m[2 * j + 1] = fmaxf(m[2 * j + 1], fabsf(bf16hi(u[j])));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        if (lane < 16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) part[warp][cl * 8 + j] = m[j];
        }
        __syncthreads();
        if (tid < kFp8Block) {
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, part[i][tid]);
            const Fp8Scale f = fp8_scale(amax);
            col_scale[tid] = f;
            if (kb * kFp8Block + tid < p.K) p.scales_t[mb * p.ldst + kb * kFp8Block + tid] = f.s;
        }
        __syncthreads();
    }

    if (p.codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            Fp8Scale f;
            if constexpr (TILE) {
                f = whole;
            } else {
                float amax = amax8(w[i]);
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                f = fp8_scale(amax);
            }
            const int64_t r = r0 + i;
            if (r < p.M && c < p.K)
                fp8_store8(p.codes + r * p.ldc + c,
                           e4m3_pack4(fp8_quot(bf16lo(w[i].x), f), fp8_quot(bf16hi(w[i].x), f),
                                      fp8_quot(bf16lo(w[i].y), f), fp8_quot(bf16hi(w[i].y), f)),
                           e4m3_pack4(fp8_quot(bf16lo(w[i].z), f), fp8_quot(bf16hi(w[i].z), f),
                                      fp8_quot(bf16lo(w[i].w), f), fp8_quot(bf16hi(w[i].w), f)),
                           p.K - c);
            if (!TILE && cl == 0 && r < p.M) p.scales[kb * p.lds + r] = f.s;
        }
    }
    if (!p.codes_t) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const Fp8Scale f = TILE ? whole : col_scale[cl * 8 + j];
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = j < 2 ? w[i].x : j < 4 ? w[i].y : j < 6 ? w[i].z : w[i].w;
            q[i] = fp8_quot((j & 1) ? bf16hi(u) : bf16lo(u), f);
        }
        *reinterpret_cast<uint2*>(turned + (cl * 8 + j) * kFp8Block + ((rg ^ cl) & 15) * 8) =
            make_uint2(e4m3_pack4(q[0], q[1], q[2], q[3]), e4m3_pack4(q[4], q[5], q[6], q[7]));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 16 + (tid >> 4);  // a column of x
        const int64_t k = kb * kFp8Block + row, m = mb * kFp8Block + cl * 8;
        const uint2 v = *reinterpret_cast<const uint2*>(turned + row * kFp8Block + ((cl ^ (row >> 3)) & 15) * 8);
        if (k < p.K && m < p.M) fp8_store8(p.codes_t + k * p.ldct + m, v.x, v.y, p.M - m);
    }
}

}  // namespace fp4q
