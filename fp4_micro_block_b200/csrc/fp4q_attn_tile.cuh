// fp4q_attn_tile.cuh -- the cache attention for many queries: 128 rows (query i,
// head g of the group: row i * G + g) of one K/V head per CTA on the 5th-generation
// tensor cores, 128 keys at a time.
//
//   S = Q K^T   (128 x 128)  A = Q in tensor memory, B = K as fp16 in shared memory
//   P = exp2(S - m)          fp16, in tensor memory in S's place
//   O += P V    (128 x D)    A = P, B = V^T as fp16 in shared memory
//
// The codes come as E4M3 by TMA and are converted to fp16 by a warpgroup of
// their own (exact; V is transposed on the way, so that both products have
// K-major operands).  Numerics as in fp4q_attn.cuh: the page scales of K and V
// are applied to S and P, which are fp32 until P is rounded.
//
// Warpgroups: 0     warp 0 TMA, warp 1 MMA issue;
//             1, 2  softmax of the even and of the odd tiles: thread = row, each
//                   with a maximum and a denominator of its own (one warp per SM
//                   quarter leaves most issue slots empty);
//             3     output: thread = row, O in registers; P V of a tile is added
//                   under the larger of the two maxima;
//             4     conversion.
// Two chunks of 1000 queries over 4096 keys, 8 K/V heads of 128 in groups of 4:
// 173 to 175 us, 574 TFLOP/s.  No pipe is full (tensor a third, ALU and exponentials
// nearly two fifths): the chain S, softmax, P V over two buffers bounds it.  Half
// tiles of 64 keys with O in tensor memory took 195 us, K's conversion shared with
// the output's warpgroup 177.
// Every wait is bounded; one that runs out sets g_device_error, and the role stops.
#pragma once

#include "fp4q_attn.cuh"
#include "fp4q_fp8_gemm.cuh"

namespace fp4q {

constexpr int kTileRows = 128, kTileKeys = 128;

template <int D>
struct AttnTileGeo {
    static constexpr int threads = 640;
    static constexpr int k8 = kTileKeys * D;          // bytes of a tile's K (or V) codes
    static constexpr int k16 = 2 * kTileKeys * D;     // as fp16
    static constexpr int raw_off = 0;                 // two stages of K and V codes
    static constexpr int kf_off = raw_off + 4 * k8;   // two buffers of K, two of V^T
    static constexpr int vf_off = kf_off + 2 * k16;
    static constexpr int mref_off = vf_off + 2 * k16;               // [4][128]: the maximum each tile's P is under
    static constexpr int ml_off = mref_off + 4 * kTileRows * 4;     // [2][2][128]: maxima, denominators
    static constexpr int qs_off = ml_off + 4 * kTileRows * 4;       // [128]: the queries' scales
    static constexpr int nan_off = qs_off + kTileRows * 4;      // [D]: first key with a NaN in V's column
    static constexpr int sc_off = nan_off + D * 4;              // [8][8]: scales of the tiles' runs of 16 keys
    static constexpr int bar_off = sc_off + 8 * 8 * 16;
    static constexpr int num_bars = 21;
    static constexpr int slot_off = bar_off + 8 * num_bars;
    static constexpr int smem = 1024 + slot_off + 16;
    static_assert(smem <= 227 * 1024, "shared memory");
    // tensor memory columns
    static constexpr uint32_t s_col = 0, pv_col = 256, q_col = 384;
};
// Registers of the five warpgroups: 5 * 96 at launch.
constexpr int kTileRegsRoles = 32, kTileRegsSoftmax = 96, kTileRegsOut = 168, kTileRegsConvert = 88;
static_assert(kTileRegsRoles + 2 * kTileRegsSoftmax + kTileRegsOut + kTileRegsConvert == 5 * 96, "register split");

// kind::f16, D fp32, A and B fp16, both K-major, M = 128.
__host__ __device__ constexpr uint32_t f16_idesc(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[smem]^T, K = 16.
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 16 words into this thread's TMEM lane; complete after tmem_wait_st.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A NaN code of V reaches the rows that see its key and no other: it counts as 0
// in the product, and nan_key keeps the first such key of each of four dims.
__device__ __noinline__ void attn_note_nans(int* nan_key, uint32_t bytes, int key) {
    for (int e = 0; e < 4; ++e)
        if (bytes >> (8 * e) & 1u) atomicMin(nan_key + e, key);
}

// SPLIT: a CTA has one run of the keys, and attn_join_kernel finishes the rows.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(640, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const AttnParams p, const AttnSplit sp) {
    using G = AttnTileGeo<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = align_shared<1024>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wg = warp >> 2;
    const uint32_t bars = smem_u32(smem + G::bar_off);
    const uint32_t full8 = bars, empty8 = bars + 16, kfull = bars + 32, kfree = bars + 48, vfull = bars + 64,
                   vfree = bars + 80, sfull = bars + 96, pfull = bars + 112, pvfull = bars + 128, pvfree = bars + 136,
                   qfull = bars + 144, lfull = bars + 152, done_bar = bars + 160;
    float* mref = reinterpret_cast<float*>(smem + G::mref_off);
    float* q_scale = reinterpret_cast<float*>(smem + G::qs_off);
    float* ml = reinterpret_cast<float*>(smem + G::ml_off);
    int* nan_key = reinterpret_cast<int*>(smem + G::nan_off);
    float4(*run_scale)[8] = reinterpret_cast<float4(*)[8]>(smem + G::sc_off);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::slot_off);
    if (tid == 0) {
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
        for (int i = 0; i < 2; ++i) {
            mbar_init(full8 + 8 * i, 2);
            mbar_init(empty8 + 8 * i, 4);
            mbar_init(kfull + 8 * i, 4);
            mbar_init(kfree + 8 * i, 1);
            mbar_init(vfull + 8 * i, 4);
            mbar_init(vfree + 8 * i, 1);
            mbar_init(sfull + 8 * i, 1);
            mbar_init(pfull + 8 * i, 4);
        }
        mbar_init(pvfull, 1);
        mbar_init(pvfree, 4);
        mbar_init(qfull, 4);
        mbar_init(lfull, 8);
        mbar_init(done_bar, 1);
        fence_barrier_init();
    }
    for (int i = tid; i < D; i += 640) nan_key[i] = 0x7fffffff;
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    uint32_t u = blockIdx.x;  // the last row tiles, which see most, first
    const uint32_t split = SPLIT ? u % sp.splits : 0;
    if (SPLIT) u /= sp.splits;
    const uint32_t rt = sp.row_tiles - 1 - u % sp.row_tiles;
    u /= sp.row_tiles;
    const int hk = (int)(u % (uint32_t)p.c.heads);
    const int64_t b = u / (uint32_t)p.c.heads;
    const AttnSeq s = attn_seq(p, b, tid == 0);
    const int r0 = (int)rt * kTileRows, n_rows = s.n * p.group;
    const int rows = min(n_rows - r0, kTileRows);
    // this split's keys k0 .. most - 1 of those that the tile sees (the last row sees most)
    const int all = rows > 0 ? attn_limit(p, s, r0 + rows - 1) : 0;
    const int k0 = SPLIT ? (int)min64((int64_t)split * sp.chunk, all) : 0, most = SPLIT ? min(all - k0, sp.chunk) + k0 : all;
    const int every = rows > 0 ? attn_limit(p, s, r0) : 0;            // keys below are seen by every row
    const int tiles = (most - k0 + kTileKeys - 1) / kTileKeys;
    const int run0 = k0 / kAttnStep;  // its first run of 16 keys
    const int per_page = p.c.page / kAttnStep, shift = per_page == 1 ? 0 : per_page == 2 ? 1 : per_page == 4 ? 2 : 3;

    if (wg == 0) {
        reg_dec<kTileRegsRoles>();
        if (warp == 0) {
            // -------------------------------------------- TMA: lane i < 8 brings keys 16 i .. of each tile
            // It also leaves the scales of these runs in shared memory, eight tiles deep
            // (the copies are at most six tiles ahead of the softmax): the softmax warps
            // would stall on a page's id and then on its scale (two chunks of 1000 over
            // 4096 keys: 181 us so, 174 with this).
            int j = 0;
            int32_t next = lane < 8 && k0 + lane * kAttnStep < most ? attn_page(p, b, (run0 + lane) >> shift, true) : 0;
            for (; j < tiles; ++j) {
                const int st = j & 1;
                const int boxes = min(8, (most - k0 - j * kTileKeys + kAttnStep - 1) / kAttnStep);
                const int32_t id = next;
                float ks = 0.0f, vs = 0.0f;
                if (lane < boxes) {
                    ks = __ldg(p.c.k_scale + (int64_t)id * p.c.heads + hk);
                    vs = __ldg(p.c.v_scale + (int64_t)id * p.c.heads + hk);
                }
                if (lane < 8 && k0 + (j + 1) * kTileKeys + lane * kAttnStep < most)
                    next = attn_page(p, b, (run0 + 8 * (j + 1) + lane) >> shift, true);
                if (j >= 2 && !__all_sync(0xffffffffu, mbar_wait(empty8 + 8 * st, (uint32_t)(((j >> 1) - 1) & 1)))) {
                    if (lane == 0) atomicOr(&g_device_error, kErrWaitTimeout);
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(full8 + 8 * st, boxes * 2 * kAttnStep * D);
                __syncwarp();
                if (lane < boxes && !withheld(p, j)) {
                    const int32_t row = (id * p.c.heads + hk) * p.c.page + ((8 * j + lane) & (per_page - 1)) * kAttnStep;
                    const uint32_t dst = smem_u32(smem + G::raw_off) + st * 2 * G::k8 + lane * kAttnStep * D;
                    tma_load_2d(dst, &map_k, 0, row, full8 + 8 * st);
                    tma_load_2d(dst + G::k8, &map_v, 0, row, full8 + 8 * st);
                }
                const float2 f = attn_page_scales(ks, vs);
                if (lane < 8) run_scale[j & 7][lane] = make_float4(f.x, f.y * kAttnWeight, attn_log2_scale(f.y), 0.0f);
                __syncwarp();
                if (lane == 0) mbar_arrive(full8 + 8 * st);
            }
            // every copy lands before the CTA may exit
            for (int i = j > 2 ? j - 2 : 0; i < j; ++i) (void)mbar_wait(full8 + 8 * (i & 1), (uint32_t)((i >> 1) & 1));
        } else if (warp == 1 && tiles > 0) {
            // -------------------------------------------- MMA: S runs two tiles ahead of P V
            // The whole warp goes through the loop, and one lane issues.
            const bool one = elect_one();
            const uint32_t t0 = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t kd = sw128_desc_lo(smem_u32(smem + G::kf_off)), vd = sw128_desc_lo(smem_u32(smem + G::vf_off));
            bool ok = __all_sync(0xffffffffu, mbar_wait(qfull, 0));
            auto issue_s = [&](int j) {
                const int st = j & 1;
                ok = ok && __all_sync(0xffffffffu, mbar_wait(kfull + 8 * st, (uint32_t)((j >> 1) & 1)));
                if (!ok) return;
                tc_fence_after();
                const uint32_t k = kd + st * (G::k16 >> 4);
                if (one) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        umma_f16_ts(t0 + G::s_col + 128 * st, t0 + G::q_col + 8 * i,
                                    sw128_desc_of(k + (((i >> 2) * (kTileKeys * 128) + (i & 3) * 32) >> 4)), f16_idesc(kTileKeys), i > 0);
                    tc_commit(kfree + 8 * st);
                    tc_commit(sfull + 8 * st);
                }
                __syncwarp();
            };
            issue_s(0);
            if (tiles > 1) issue_s(1);
            for (int j = 0; j < tiles && ok; ++j) {
                const int st = j & 1;
                ok = mbar_wait(vfull + 8 * st, (uint32_t)((j >> 1) & 1)) && mbar_wait(pfull + 8 * st, (uint32_t)((j >> 1) & 1)) &&
                     (j == 0 || mbar_wait(pvfree, (uint32_t)((j - 1) & 1)));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t v = vd + st * (G::k16 >> 4);
                if (one) {
#pragma unroll
                    for (int i = 0; i < kTileKeys / 16; ++i)
                        umma_f16_ts(t0 + G::pv_col, t0 + G::s_col + 128 * st + 8 * i,
                                    sw128_desc_of(v + (((i >> 2) * (D * 128) + (i & 3) * 32) >> 4)), f16_idesc(D), i > 0);
                    tc_commit(vfree + 8 * st);
                    tc_commit(pvfull);
                }
                __syncwarp();
                if (j + 2 < tiles) issue_s(j + 2);  // over P of tile j, in order behind its product
            }
            if (!ok && one) atomicOr(&g_device_error, kErrWaitTimeout);
            // all MMAs complete before TMEM is freed
            if (one) tc_commit(done_bar);
            if (!mbar_wait(done_bar, 0) && one) atomicOr(&g_device_error, kErrWaitTimeout);
        }
    } else if (wg <= 2) {
        // ------------------------------------------------ softmax: thread = row
        const int odd = wg - 1;
        const int t = tid & 127, r = r0 + t;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's TMEM lanes
        const int lim = rows > 0 ? attn_limit(p, s, r) : 0;
        if (!odd) {
            // the row's query as fp16, scaled by a power of two to a maximum of 2^14, its sign that of the softmax scale
            const bool live = t < rows;
            const uint32_t rr = live ? r : 0, tok = rr / (uint32_t)p.group, h = hk * p.group + (rr - tok * p.group);
            const uint16_t* src = p.q + (s.first + tok) * p.ldq + (int64_t)h * D;
            uint4 x[D / 8];
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                x[c] = live ? __ldg(reinterpret_cast<const uint4*>(src + 8 * c)) : make_uint4(0, 0, 0, 0);
                m = bf16x2_max(m, amax8x2(x[c]));
            }
            const float amax = bf16x2_top(m);
            int e = amax == 0.0f ? 0 : 14 + 127 - (int)(__float_as_uint(fmaxf(amax, 0x1p-126f)) >> 23);
            const int e1 = e / 2, e2 = e - e1;
            const float u1 = __int_as_float((127 + e1) << 23) * (p.scale_log2 < 0.0f ? -1.0f : 1.0f), u2 = __int_as_float((127 + e2) << 23);
            q_scale[t] = __int_as_float((127 - e1) << 23) * __int_as_float((127 - e2) << 23) * fabsf(p.scale_log2);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t q4[4] = {x[4 * c + k].x, x[4 * c + k].y, x[4 * c + k].z, x[4 * c + k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[4 * k + i] = f16x2_pack(bf16lo(q4[i]) * u1 * u2, bf16hi(q4[i]) * u1 * u2);
                }
                tmem_st16(tmem + lanes + G::q_col + 16 * c, w);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
        }
        float m = -INFINITY, l = 0.0f;
        bool ok = __all_sync(0xffffffffu, mbar_wait(qfull, 0));
        const float qs = q_scale[t];
        for (int j = odd; j < tiles && ok; j += 2) {
            const int st = j & 1;
            const float4* sc = run_scale[j & 7];
            const int left = lim - k0 - j * kTileKeys;  // keys of the tile that this row sees
            const bool edge = k0 + (j + 1) * kTileKeys > every;
            ok = __all_sync(0xffffffffu, mbar_wait(sfull + 8 * st, (uint32_t)((j >> 1) & 1)));
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = tmem + lanes + G::s_col + 128 * st;
            // (The loops stay rolled: with all roles unrolled the code did not fit the
            // instruction caches, and a tile took twice as long.)
            float top = -INFINITY;
#pragma unroll 1
            for (int col = 0; col < kTileKeys; col += 32) {
                uint32_t x[32];
                tmem_start(sa + col, x);
                tmem_wait(x);
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = i < left - col ? x[i] : 0xff800000u;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx[i] = fmaxf(fmaxf(__uint_as_float(x[16 * h + i]), __uint_as_float(x[16 * h + 4 + i])),
                                      fmaxf(__uint_as_float(x[16 * h + 8 + i]), __uint_as_float(x[16 * h + 12 + i])));
                    const int run = col / 16 + h;
                    top = fmaxf(top, fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), sc[run].x * qs, sc[run].z));  // (-inf * 0 is no number: skipped)
                }
            }
            const float mn = fmaxf(m, top), h = mn == -INFINITY ? 1.0f : exp2_approx(0.5f * (m - mn)), base = mn == -INFINITY ? 0.0f : mn;
            m = mn;
            l = l * h * h;
            mref[(j & 3) * kTileRows + t] = mn;
            // P goes where S was: columns c .. of P overwrite columns of S that have been read
            uint64_t sum = 0;
            const uint64_t nb = f2_both(-base);
            auto weights = [&](auto&& seen) {
#pragma unroll 1
                for (int col = 0; col < kTileKeys; col += 32) {
                    uint32_t x[32], w[16];
                    tmem_start(sa + col, x);
                    tmem_wait(x);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int run = col / 16 + h;
                        const uint64_t f = f2_both(sc[run].x * qs), wv = f2_both(sc[run].y);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const uint64_t z = f2_fma(f2_pack(x[16 * h + i], x[16 * h + i + 1]), f, nb);
                            const uint64_t e = f2_pack(__float_as_uint(seen(16 * h + i, left - col, exp2_approx(f2_lo(z)))),
                                                       __float_as_uint(seen(16 * h + i + 1, left - col, exp2_approx(f2_hi(z)))));
                            sum = f2_fma(e, f2_both(kAttnUnlift), sum);
                            const uint64_t y = f2_mul(e, wv);
                            w[8 * h + i / 2] = f16x2_pack(f2_lo(y), f2_hi(y));
                        }
                    }
                    tmem_st16(sa + col / 2, w);
                }
            };
            if (edge)
                weights([](int i, int n, float e) { return i < n ? e : 0.0f; });
            else
                weights([](int, int, float e) { return e; });
            l += f2_lo(sum) + f2_hi(sum);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pfull + 8 * st);
        }
        if (!ok && lane == 0) atomicOr(&g_device_error, kErrWaitTimeout);
        ml[2 * odd * kTileRows + t] = m;
        ml[(2 * odd + 1) * kTileRows + t] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(lfull);
    } else if (wg == 3) {
        // ------------------------------------------------ output: thread = row
        reg_inc<kTileRegsOut>();
        const int t = tid & 127, r = r0 + t;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        uint64_t o[D / 2];
#pragma unroll
        for (int d = 0; d < D / 2; ++d) o[d] = 0;
        float mo = -INFINITY;
        bool ok = true;
        for (int j = 0; j < tiles; ++j) {
            ok = __all_sync(0xffffffffu, mbar_wait(pvfull, (uint32_t)(j & 1)));
            if (!ok) break;
            tc_fence_after();
            const float mj = mref[(j & 3) * kTileRows + t], mn = fmaxf(mo, mj);
            // (-inf: nothing seen so far, or in this tile)
            const uint64_t a = f2_both(mo == -INFINITY ? 1.0f : exp2_approx(mo - mn)), w = f2_both(mj == -INFINITY ? 1.0f : exp2_approx(mj - mn));
            mo = mn;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                uint32_t x[16];
                tmem_start(tmem + lanes + G::pv_col + 16 * c, x);
                tmem_wait(x);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[8 * c + i] = f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), w, f2_mul(o[8 * c + i], a));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pvfree);
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(lfull, 0));
        if (!ok && lane == 0) atomicOr(&g_device_error, kErrWaitTimeout);
        float l = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float mk = ml[2 * k * kTileRows + t];
            const float h = mk == -INFINITY ? 1.0f : exp2_approx(0.5f * (mk - mo));
            l = fmaf(ml[(2 * k + 1) * kTileRows + t] * h, h, l);
        }
        const int lim = attn_limit(p, s, r);
        if constexpr (SPLIT) {
            // A warp's 32 rows through the K buffers, which no product reads any more, so
            // that they leave in whole lines (64 queries over 4096 keys 20.8 us, 23.8 with
            // each thread writing its own row).
            if (ok && (split == 0 || tiles > 0)) {
                constexpr int P = D / 4;  // 16-byte pieces of a row, swizzled by the row
                float4* st = reinterpret_cast<float4*>(smem + G::kf_off) + (warp & 3) * 32 * P;
#pragma unroll
                for (int c = 0; c < P; ++c) {
                    float v[4] = {f2_lo(o[2 * c]), f2_hi(o[2 * c]), f2_lo(o[2 * c + 1]), f2_hi(o[2 * c + 1])};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (nan_key[4 * c + i] < lim) v[i] = __int_as_float(0x7fffffff);
                    st[lane * P + (c ^ (lane & 7))] = make_float4(v[0], v[1], v[2], v[3]);
                }
                __syncwarp();
                const int w0 = t & ~31;  // the warp's first row
                float* slots = sp.ws + (((int64_t)(b * p.c.heads + hk) * sp.row_tiles + rt) * sp.slot_rows * sp.splits + split) * kAttnSlot<D>;
#pragma unroll 4
                for (int i = lane; i < 32 * P; i += 32) {
                    const int row = i / P, c = i % P;
                    if (w0 + row < rows)
                        *reinterpret_cast<float4*>(slots + (int64_t)(w0 + row) * sp.splits * kAttnSlot<D> + 4 * c) = st[row * P + (c ^ (row & 7))];
                }
                if (t < rows) *reinterpret_cast<float2*>(slots + (int64_t)t * sp.splits * kAttnSlot<D> + D) = make_float2(mo, l);
            }
        } else if (t < rows) {
            const float inv = l == 0.0f ? 0.0f : kAttnUnweight / l;
            const uint32_t tok = (uint32_t)r / (uint32_t)p.group, h = hk * p.group + (r - tok * p.group);
            uint4* dst = reinterpret_cast<uint4*>(p.o + (s.first + tok) * p.ldo + (int64_t)h * D);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = f2_lo(o[4 * c + i]) * inv;
                    v[2 * i + 1] = f2_hi(o[4 * c + i]) * inv;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (nan_key[8 * c + i] < lim) v[i] = __int_as_float(0x7fffffff);
                dst[c] = make_uint4(bf16x2_pack(v[0], v[1]), bf16x2_pack(v[2], v[3]), bf16x2_pack(v[4], v[5]), bf16x2_pack(v[6], v[7]));
            }
            if (p.lse) p.lse[(s.first + tok) * p.q_heads + h] = l == 0.0f ? -INFINITY : (mo + kAttnLift + log2f(l)) * kLn2;
        }
    } else {
        // ------------------------------------------------ conversion of the codes to fp16
        reg_dec<kTileRegsConvert>();
        const int t = tid & 127;
        // K, eight codes of a key (one 16-byte piece of fp16) at a time: piece kc of keys
        // kk, kk + kstep, ..; a row of a box or of the result is its key times the row's
        // size further, at the same swizzle (kstep is a multiple of 8)
        constexpr int kstep = 128 / (D / 8);
        const int kc = t % (D / 8), kk = t / (D / 8);
        const uint32_t ksrc = kk * D + (AttnTile<D>::at(kk & 15, 8 * kc) - (kk & 15) * D);
        const uint32_t kdst = (kc >> 3) * (kTileKeys * 128) + kk * 128 + (((kc ^ kk) & 7) << 4);
        // V, eight keys (run q) of four dims (word w0 + 8 i of a row): lanes are 4 runs x 8
        // words, so that eight neighbouring stores fall into different banks
        const int q = (t & 3) | (t >> 5) << 2, w0 = (t >> 2) & 7;
        bool ok = true;
        for (int j = 0; j < tiles; ++j) {
            const int st = j & 1, key0 = k0 + j * kTileKeys;
            const uint32_t ph = (uint32_t)((j >> 1) & 1);
            ok = mbar_wait(full8 + 8 * st, ph) && (j < 2 || mbar_wait(kfree + 8 * st, ph ^ 1u));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint8_t* raw = smem + G::raw_off + st * 2 * G::k8;
            const uint32_t kf = smem_u32(smem + G::kf_off) + st * G::k16 + kdst;
            constexpr int kn = kTileKeys / kstep;
#pragma unroll
            for (int i0 = 0; i0 < kn; i0 += 8) {
                uint2 x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const uint2*>(raw + ksrc + (i0 + i) * kstep * D);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const Half4 a = e4m3x4_f16(x[i].x), d = e4m3x4_f16(x[i].y);
                    sts_v4(kf + (i0 + i) * kstep * 128, a.lo, a.hi, d.lo, d.hi);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(kfull + 8 * st);
            ok = __all_sync(0xffffffffu, j < 2 || mbar_wait(vfree + 8 * st, ph ^ 1u));
            if (!ok) break;
            const uint32_t vf = smem_u32(smem + G::vf_off) + st * G::k16 + (q >> 3) * (D * 128) + 4 * w0 * 128;
            const uint8_t* vsrc = raw + G::k8 + 8 * q * D + ((4 * w0) & 15);
            const bool edge = key0 + kTileKeys > every;
#pragma unroll 2
            for (int i = 0; i < D / 32; ++i) {
                uint32_t x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)  // key 8 q + k: the row's 16-byte pieces are swizzled by its place in the box
                    x[k] = *reinterpret_cast<const uint32_t*>(vsrc + AttnTile<D>::at(8 * (q & 1) + k, ((4 * w0) & 16) + 32 * i) - 8 * (q & 1) * D);
                if (edge) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int key = key0 + 8 * q + k;
                        if (key >= most) x[k] = 0;  // beyond the last row's keys: whatever lies there
                        const uint32_t n = nan_bytes(x[k]);
                        if (n) attn_note_nans(nan_key + 4 * w0 + 32 * i, n, key);
                        x[k] &= ~n;
                    }
                }
                uint32_t y[4][4];  // [dim][pair of keys]
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const Half4 a = e4m3x4_f16(__byte_perm(x[2 * k], x[2 * k + 1], 0x5140)), d = e4m3x4_f16(__byte_perm(x[2 * k], x[2 * k + 1], 0x7362));
                    y[0][k] = a.lo;
                    y[1][k] = a.hi;
                    y[2][k] = d.lo;
                    y[3][k] = d.hi;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sts_v4(vf + (32 * i + k) * 128 + (((q ^ (4 * w0 + k)) & 7) << 4), y[k][0], y[k][1], y[k][2], y[k][3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(vfull + 8 * st);
                mbar_arrive(empty8 + 8 * st);
            }
        }
        if (!ok && lane == 0) atomicOr(&g_device_error, kErrWaitTimeout);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace fp4q
