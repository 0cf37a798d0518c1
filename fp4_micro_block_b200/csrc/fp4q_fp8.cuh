// fp4q_fp8.cuh -- E4M3 codes under one FP32 scale per block of 128: the format's
// device helpers and the quantizer.
//
//   s = amax_block / 448,  code = E4M3(x / s)  (nearest even, saturating)
//
// One read of x gives the codes of x, of its transpose, or both: the blocks of
// the transpose run down the columns, so a CTA holds a whole 128 x 128 tile.
#pragma once

#include "fp4q_unit.cuh"

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

// Test build only: whether CTA 0 withholds the copies that it has armed its barrier
// for the i-th time for (p.skip_copy, -1: none), so that the waits for them run out.
template <typename P>
__device__ __forceinline__ bool withheld(const P& p, int64_t i) {
#ifdef FP4Q_TEST_HOOKS
    return blockIdx.x == 0 && i == p.skip_copy;
#else
    return false;
#endif
}

// All CTAs of the cluster have arrived, and see each other's shared memory.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at shared-memory address `saddr` of the cluster's CTA `rank`.
__device__ __forceinline__ float ld_cluster(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// A pair of fp32 values and operations on both (each rounded as alone).
__device__ __forceinline__ uint64_t f2_pack(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// Block scale s = amax / 448 and, where div_split's preconditions hold for every
// |x| <= amax, the negated parts of its split reciprocal (else nrz = 0: IEEE
// divisions).
struct __align__(16) Fp8Scale {
    float s, nrn, nrz, nlo;
};
__device__ __forceinline__ Fp8Scale fp8_scale(float amax) {
    Fp8Scale r;
    r.s = __fdiv_rn(amax, kE4m3Max);
    r.nrn = r.nrz = r.nlo = 0.0f;
    if (div_fast_ok(r.s, amax)) {
        const Rcp c = make_rcp(r.s);
        r.nrn = -c.rn;
        r.nrz = -c.rz;
        r.nlo = -c.lo;
    }
    return r;
}
// The scale that lane `src` of the warp holds.
__device__ __forceinline__ Fp8Scale fp8_scale_of(const Fp8Scale& f, int src) {
    Fp8Scale r;
    r.s = __shfl_sync(0xffffffffu, f.s, src);
    r.nrn = __shfl_sync(0xffffffffu, f.nrn, src);
    r.nrz = __shfl_sync(0xffffffffu, f.nrz, src);
    r.nlo = __shfl_sync(0xffffffffu, f.nlo, src);
    return r;
}
// s == 0: the block has zeros and NaN alone, which give the codes 0 and 0x7f.
__device__ __noinline__ uint32_t fp8_codes_ieee(uint32_t u0, uint32_t u1, float s) {
    if (s == 0.0f) {
        auto code = [](float v) { return fabsf(v) * 0.0f; };
        return e4m3_pack4(code(bf16lo(u0)), code(bf16hi(u0)), code(bf16lo(u1)), code(bf16hi(u1)));
    }
    return e4m3_pack4(__fdiv_rn(bf16lo(u0), s), __fdiv_rn(bf16hi(u0), s), __fdiv_rn(bf16lo(u1), s), __fdiv_rn(bf16hi(u1), s));
}
// The four codes of two words of bf16 pairs: x / s as div_split computes it,
// two elements an instruction (fp8_codes_fast: f.nrz != 0).
__device__ __forceinline__ uint32_t fp8_codes_fast(uint32_t u0, uint32_t u1, const Fp8Scale& f) {
    uint32_t q[4];
    const uint32_t u[2] = {u0 ^ 0x80008000u, u1 ^ 0x80008000u};  // -x
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint64_t nx = f2_pack(u[i] << 16, u[i] & 0xffff0000u);
        const uint64_t q0 = f2_fma(nx, f2_both(f.nrz), f2_mul(nx, f2_both(f.nlo)));
        const uint64_t e = f2_fma(q0, f2_both(f.s), nx);
        const uint64_t r = f2_fma(e, f2_both(f.nrn), q0);
        q[2 * i] = (uint32_t)r;
        q[2 * i + 1] = (uint32_t)(r >> 32);
    }
    return e4m3_pack4(__uint_as_float(q[0]), __uint_as_float(q[1]), __uint_as_float(q[2]), __uint_as_float(q[3]));
}
__device__ __forceinline__ uint32_t fp8_codes(uint32_t u0, uint32_t u1, const Fp8Scale& f) {
    return f.nrz != 0.0f ? fp8_codes_fast(u0, u1, f) : fp8_codes_ieee(u0, u1, f.s);
}

// Maxima of bf16 magnitudes, two at a time; a NaN loses to a number.
__device__ __forceinline__ uint32_t bf16x2_abs(uint32_t u) { return u & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// One number's larger half (NaN only if both are: counts as 0).
__device__ __forceinline__ float bf16x2_top(uint32_t u) { return fmaxf(fmaxf(bf16lo(u), bf16hi(u)), 0.0f); }
__device__ __forceinline__ uint32_t amax8x2(const uint4& w) {
    return bf16x2_max(bf16x2_max(bf16x2_abs(w.x), bf16x2_abs(w.y)), bf16x2_max(bf16x2_abs(w.z), bf16x2_abs(w.w)));
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
#ifdef FP4Q_TEST_HOOKS
    int64_t skip_copy;       // withheld()
#endif
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

__device__ __forceinline__ float amax8(const uint4& w) { return bf16x2_top(amax8x2(w)); }

// Row blocks alone: 16 lanes hold one 1 x 128 block, eight elements each, and
// four blocks of a K block's neighbouring rows at once; lane i of the 16 works
// out the scale of block i % 4 for all of them (a division and a reciprocal
// cost more than a block's codes: 34 us without the sharing).  Memory bounds it:
// 8192x4096 19.1 us, 0.82 of the 6458 GB/s copy rate (23.3 with tests per piece).
constexpr int kFp8RowThreads = 256, kFp8RowBlocks = 4;
__global__ void __launch_bounds__(kFp8RowThreads) fp8_row_kernel(const Fp8QuantParams p) {
    pdl_wait();
    pdl_trigger();
    constexpr int N = kFp8RowBlocks;
    const uint32_t l16 = threadIdx.x & 15, lane = threadIdx.x & 31, n_kb = (uint32_t)p.n_kb;
    const uint32_t half = (threadIdx.x >> 4) & 1, step = gridDim.x * (kFp8RowThreads / 16);
    // (rows N r .., block kb) of this half-warp, which moves on by `step` items;
    // both halves of a warp make the same number of trips (the shuffles' lanes)
    const uint32_t first = blockIdx.x * (kFp8RowThreads / 16) + (threadIdx.x >> 4);
    uint32_t r4 = first / n_kb, kb = first - r4 * n_kb;
    const uint32_t dr = step / n_kb, dkb = step - dr * n_kb;
    for (int64_t base = first - half; base < p.n_items; base += step) {
        const int64_t c = (int64_t)kb * kFp8Block + l16 * 8, r0 = (int64_t)r4 * N;
        uint4 w[N];
        const bool whole = r0 + N <= p.M && c + 8 <= p.K;
        if (whole) {
            const uint16_t* src = p.x + r0 * p.ldx + c;
#pragma unroll
            for (int k = 0; k < N; ++k) w[k] = __ldg(reinterpret_cast<const uint4*>(src + k * p.ldx));
        } else {
#pragma unroll 1
            for (int k = 0; k < N; ++k) {  // zeros past the last row and column
                const uint4 x = fp8_load8(p, r0 + k, c);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (i == k) w[i] = x;
            }
        }
        uint32_t m[N / 2];
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {  // two rows' maxima in a word
            const uint32_t a = amax8x2(w[2 * k]), b = amax8x2(w[2 * k + 1]);
            m[k] = bf16x2_max(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) m[k] = bf16x2_max(m[k], __shfl_xor_sync(0xffffffffu, m[k], o));
        }
        const uint32_t mine = (l16 & 2) ? m[1] : m[0];
        const Fp8Scale f = fp8_scale(fmaxf((l16 & 1) ? bf16hi(mine) : bf16lo(mine), 0.0f));
        if (l16 < N && r0 + l16 < p.M) p.scales[kb * p.lds + r0 + l16] = f.s;
        uint8_t* dst = p.codes + r0 * p.ldc + c;
        if (__all_sync(0xffffffffu, whole && f.nrz != 0.0f)) {  // no tests per block
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const Fp8Scale fk = fp8_scale_of(f, (lane & 16) + k);
                *reinterpret_cast<uint2*>(dst + k * p.ldc) = make_uint2(fp8_codes_fast(w[k].x, w[k].y, fk), fp8_codes_fast(w[k].z, w[k].w, fk));
            }
        } else {
#pragma unroll 1
            for (int k = 0; k < N; ++k) {
                const Fp8Scale fk = fp8_scale_of(f, (lane & 16) + k);
                uint4 x = w[0];
#pragma unroll
                for (int i = 1; i < N; ++i)
                    if (i == k) x = w[i];
                if (r0 + k < p.M && c < p.K) fp8_store8(dst + k * p.ldc, fp8_codes(x.x, x.y, fk), fp8_codes(x.z, x.w, fk), p.K - c);
            }
        }
        r4 += dr;
        kb += dkb;
        if (kb >= n_kb) {
            kb -= n_kb;
            ++r4;
        }
    }
}

// A 128 x 128 tile at a time, for the transpose and for tile scales: TMA brings
// the next tile (two boxes of 64 columns, 128-byte swizzle) while this one is
// worked on.  Thread (rg, cl) has rows 8 rg .. 8 rg + 7, columns 8 cl .. 8 cl + 7,
// so that a row's 128 columns are the 16 lanes of a half-warp (whole 128-byte
// runs of codes, row maxima by shuffles, two rows packed in a word) and a
// column's eight rows are one 8-byte piece of the transpose.  Those pieces cross
// the CTA through 16 KiB of shared memory whose 8-byte units are swizzled by the
// column group, so that neither side has bank conflicts.  8192x4096: tiles alone
// 17.3 us, 0.90 of the 6458 GB/s copy rate, which bounds them; both directions 33.8,
// with two quotients and two conversions an element (issue slots 54 %, ALU 51 %, FMA
// 30 % busy: no one unit is full).
constexpr int kFp8TileThreads = 256;
constexpr int kFp8TileBytes = 2 * kFp8Block * kFp8Block;
constexpr int kFp8TileStages = 2;
constexpr int kFp8TurnedOff = kFp8TileStages * kFp8TileBytes;
constexpr int kFp8PartOff = kFp8TurnedOff + kFp8Block * kFp8Block;
constexpr int kFp8ColOff = kFp8PartOff + 8 * (kFp8Block / 2) * 4;
constexpr int kFp8TileBarOff = kFp8ColOff + kFp8Block * 16;
static_assert(kFp8TileStages == 2, "this tile and the next one");
constexpr int kFp8TileSmem = 1024 + kFp8TileBarOff + 8 * kFp8TileStages;
constexpr int kFp8TileCtas = 2;  // per SM

template <bool TILE>
__global__ void __launch_bounds__(kFp8TileThreads, kFp8TileCtas)
    fp8_tile_kernel(const __grid_constant__ CUtensorMap map_x, const Fp8QuantParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = align_shared<1024>(smem_raw);
    uint8_t* turned = smem + kFp8TurnedOff;
    uint32_t(*part)[kFp8Block / 2] = reinterpret_cast<uint32_t(*)[kFp8Block / 2]>(smem + kFp8PartOff);
    Fp8Scale* col_scale = reinterpret_cast<Fp8Scale*>(smem + kFp8ColOff);
    const uint32_t full0 = smem_u32(smem + kFp8TileBarOff);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cl = tid & 15, rg = tid >> 4;
    if (tid == 0) {
        prefetch_tmap(&map_x);
        for (int i = 0; i < kFp8TileStages; ++i) mbar_init(full0 + 8 * i, 1);
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const uint32_t n_kb = (uint32_t)p.n_kb, n_items = (uint32_t)p.n_items;
    auto fetch = [&](uint32_t item, int stage) {  // one thread
        const uint32_t mb = item / n_kb, kb = item - mb * n_kb;
        const uint32_t dst = smem_u32(smem + stage * kFp8TileBytes), bar = full0 + 8 * stage;
        mbar_arrive_expect_tx(bar, kFp8TileBytes);
        if (withheld(p, item / gridDim.x)) return;
        tma_load_2d(dst, &map_x, (int32_t)(kb * kFp8Block), (int32_t)(mb * kFp8Block), bar);
        tma_load_2d(dst + kFp8TileBytes / 2, &map_x, (int32_t)(kb * kFp8Block + 64), (int32_t)(mb * kFp8Block), bar);
    };
    if (tid == 0)
        for (int i = 0; i < kFp8TileStages; ++i)
            if (blockIdx.x + i * gridDim.x < n_items) fetch(blockIdx.x + i * gridDim.x, i);
    int stage = 0;
    uint32_t phase = 0;
    for (uint32_t item = blockIdx.x; item < n_items; item += gridDim.x) {
        if (!__syncthreads_and(mbar_wait(full0 + 8 * stage, phase))) {
            if (tid == 0) {
                atomicOr(&g_device_error, kErrWaitTimeout);
                // the copies on their way land before the CTA exits: this tile's, and the next one's
                (void)mbar_wait(full0 + 8 * stage, phase);
                if (item + gridDim.x < n_items) (void)mbar_wait(full0 + 8 * (stage ^ 1), phase ^ (uint32_t)stage);
            }
            __syncthreads();
            return;
        }
        const uint32_t mb = item / n_kb, kb = item - mb * n_kb;
        const int64_t r0 = (int64_t)mb * kFp8Block + rg * 8, c = (int64_t)kb * kFp8Block + cl * 8;
        uint4 w[8];
        const uint8_t* tile = smem + stage * kFp8TileBytes + (cl >> 3) * (kFp8TileBytes / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = *reinterpret_cast<const uint4*>(tile + (8 * rg + i) * 128 + (((cl & 7) ^ i) << 4));

        Fp8Scale whole;
        if constexpr (TILE) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = bf16x2_max(m, amax8x2(w[i]));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) m = bf16x2_max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane == 0) part[warp][0] = m;
        } else if (p.codes_t) {
            uint32_t m[4] = {0, 0, 0, 0};  // columns 2j, 2j + 1 of the eight
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[0] = bf16x2_max(m[0], bf16x2_abs(w[i].x));
                m[1] = bf16x2_max(m[1], bf16x2_abs(w[i].y));
                m[2] = bf16x2_max(m[2], bf16x2_abs(w[i].z));
                m[3] = bf16x2_max(m[3], bf16x2_abs(w[i].w));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] = bf16x2_max(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
            if (lane < 16) *reinterpret_cast<uint4*>(&part[warp][cl * 4]) = make_uint4(m[0], m[1], m[2], m[3]);
        }
        __syncthreads();  // the maxima are there, and every thread has its part of the tile
        if (tid == 0 && item + kFp8TileStages * gridDim.x < n_items) fetch(item + kFp8TileStages * gridDim.x, stage);
        if (++stage == kFp8TileStages) {
            stage = 0;
            phase ^= 1;
        }
        // a whole tile, and scales that the quick quotients take: no tests per piece
        const bool whole_tile = (int64_t)(mb + 1) * kFp8Block <= p.M && (int64_t)(kb + 1) * kFp8Block <= p.K;
        bool quick = true, cols_quick = false;
        if constexpr (TILE) {
            uint32_t m = part[0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) m = bf16x2_max(m, part[i][0]);
            whole = fp8_scale(bf16x2_top(m));
            if (tid == 0) {
                if (p.codes) p.scales[kb * p.lds + mb] = whole.s;
                if (p.codes_t) p.scales_t[mb * p.ldst + kb] = whole.s;
            }
            cols_quick = whole.nrz != 0.0f;
        } else if (p.codes_t) {
            if (tid < kFp8Block) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = bf16x2_max(m, part[i][tid >> 1]);
                const Fp8Scale f = fp8_scale(fmaxf((tid & 1) ? bf16hi(m) : bf16lo(m), 0.0f));
                col_scale[(tid & 7) * 16 + (tid >> 3)] = f;  // (read by neighbouring column groups at once)
                const int64_t k = (int64_t)kb * kFp8Block + tid;
                if (k < p.K) p.scales_t[mb * p.ldst + k] = f.s;
                quick = f.nrz != 0.0f;
            }
            cols_quick = __syncthreads_and(quick);
        }

        if (p.codes) {
            Fp8Scale rows{};  // !TILE: of row cl % 8 of this half-warp's eight
            if constexpr (!TILE) {
                uint32_t m[4];  // maxima of rows 2i, 2i + 1 in one word
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = amax8x2(w[2 * i]), b = amax8x2(w[2 * i + 1]);
                    m[i] = bf16x2_max(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) m[i] = bf16x2_max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
                }
                const uint32_t mine = (cl & 4) ? ((cl & 2) ? m[3] : m[2]) : ((cl & 2) ? m[1] : m[0]);
                rows = fp8_scale(fmaxf((cl & 1) ? bf16hi(mine) : bf16lo(mine), 0.0f));
                if (cl < 8 && r0 + cl < p.M) p.scales[kb * p.lds + r0 + cl] = rows.s;
            }
            uint8_t* dst = p.codes + r0 * p.ldc + c;
            if (whole_tile && (TILE ? cols_quick : __all_sync(0xffffffffu, rows.nrz != 0.0f))) {
#pragma unroll
                for (int i = 0; i < 8; ++i, dst += p.ldc) {
                    const Fp8Scale f = TILE ? whole : fp8_scale_of(rows, (lane & 16) + i);
                    *reinterpret_cast<uint2*>(dst) = make_uint2(fp8_codes_fast(w[i].x, w[i].y, f), fp8_codes_fast(w[i].z, w[i].w, f));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i, dst += p.ldc) {
                    const Fp8Scale f = TILE ? whole : fp8_scale_of(rows, (lane & 16) + i);
                    if (r0 + i < p.M && c < p.K)
                        fp8_store8(dst, fp8_codes(w[i].x, w[i].y, f), fp8_codes(w[i].z, w[i].w, f), p.K - c);
                }
            }
        }
        if (!p.codes_t) continue;
        auto turn = [&](auto&& codes) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // columns 2j, 2j + 1: their rows two by two
                uint32_t u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = j == 0 ? w[i].x : j == 1 ? w[i].y : j == 2 ? w[i].z : w[i].w;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const Fp8Scale f = TILE ? whole : col_scale[(2 * j + h) * 16 + cl];
                    const uint32_t sel = h ? 0x7632 : 0x5410;
                    *reinterpret_cast<uint2*>(turned + (cl * 8 + 2 * j + h) * kFp8Block + ((rg ^ cl) & 15) * 8) =
                        make_uint2(codes(__byte_perm(u[0], u[1], sel), __byte_perm(u[2], u[3], sel), f),
                                   codes(__byte_perm(u[4], u[5], sel), __byte_perm(u[6], u[7], sel), f));
                }
            }
        };
        if (cols_quick)
            turn([](uint32_t a, uint32_t b, const Fp8Scale& f) { return fp8_codes_fast(a, b, f); });
        else
            turn([](uint32_t a, uint32_t b, const Fp8Scale& f) { return fp8_codes(a, b, f); });
        __syncthreads();
        const int64_t m0 = (int64_t)mb * kFp8Block + cl * 8;
        uint8_t* dst = p.codes_t + ((int64_t)kb * kFp8Block + rg) * p.ldct + m0;
#pragma unroll
        for (int i = 0; i < 8; ++i, dst += 16 * p.ldct) {
            const int row = i * 16 + rg;  // a column of x
            const uint2 v = *reinterpret_cast<const uint2*>(turned + row * kFp8Block + ((cl ^ (row >> 3)) & 15) * 8);
            if (whole_tile)
                *reinterpret_cast<uint2*>(dst) = v;
            else if ((int64_t)kb * kFp8Block + row < p.K && m0 < p.M)
                fp8_store8(dst, v.x, v.y, p.M - m0);
        }
        // (the next tile's first barrier keeps its maxima and pieces behind these reads)
    }
}

}  // namespace fp4q
