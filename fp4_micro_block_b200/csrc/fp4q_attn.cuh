// fp4q_attn.cuh -- attention of bf16 queries over the paged 8-bit cache,
//   o = softmax(scale q K^T) V,  lse = ln sum exp(scale q K^T),
// K and V = E4M3 code * the page's scale.
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
#ifdef FP4Q_TEST_HOOKS
    int64_t skip_copy;       // withheld()
#endif
};

constexpr float kLn2 = 0.693147180559945309f;

// Rows and keys of sequence b, clamped to what exists; reports what it clamps.
struct AttnSeq {
    int64_t first;
    int32_t n, len;  // (rows and keys of a call are counted in 31 bits)
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
    s.n = (int32_t)(hi - lo);
    s.len = (int32_t)len;
    return s;
}

// Page id of the sequence's page pg, clamped into the pool.
__device__ __forceinline__ int32_t attn_page(const AttnParams& p, int64_t b, int32_t pg, bool tell) {
    int32_t id = p.c.table[b * p.c.table_stride + pg];
    if (id < 0 || id >= p.c.num_pages) {
        if (tell) atomicOr(&g_device_error, kErrBadIndex);
        id = 0;
    }
    return id;
}

// A page's scales of K and V as the kernels use them.  A V scale that is no number
// (or infinite) would turn the weights of masked keys, which are 0, to NaN: the
// page's scores are NaN in its place (vs - vs is 0 for numbers), which masking
// replaces.  (As a select between the two it took a microsecond of 76.)
__device__ __forceinline__ float2 attn_page_scales(float ks, float vs) {
    return make_float2(ks + (vs - vs), fminf(vs, 3.4028234e38f));
}

// ------------------------------------------------------------------ few queries
//
// One CTA: one sequence, one K/V head, 16 rows (query i, head g of the group:
// row i * G + g) and one run of keys; four warps take turns of 32 keys, two tiles
// of 16 that lie within a page each.  Decoding is bound by reading the cache: each warp keeps a
// ring of such tiles on its way (TMA boxes of 16 rows, swizzled so that the reads
// below have no bank conflicts), and lanes read whole 16-byte pieces of codes:
// which of a product's k (or n) indices a lane's bytes stand for is free as long
// as both operands agree.
//   S = Q K^T: lane (g, t) = (lane / 4, lane % 4) holds dims D/4 t .. of key g
//     (and 8 + g); its next four bytes are the k indices 2t, 2t+1, 2t+8, 2t+9
//     of the next m16n8k16 step.
//   O = P V: the lane's keys are 2t, 2t+1, 2t+8, 2t+9 (as S leaves them) and its
//     dims D/8 g ..; byte j of each makes column g of output tile j, dim D/8 g + j.
// E4M3 values are exact in fp16, and so is a bf16 query scaled by a power of
// two to a row maximum of 2^14 (dims 2^-28 below it lose bits).
//
// Softmax, one pass: with the page's V scale vs, the weights enter P V as
// w = exp2(s + log2 vs - m) 2^14 <= 2^14, m the running maximum of s + log2 vs,
// in fp16: full precision whatever the V scales are, and down to 2^-28 of the
// largest before fp16's subnormals.  The denominator sums w 2^-14 / vs in fp32.
// Neither passes fp32's range for scales up to 2^127: the exponential is
// e = exp2(s - (m - 24)), so that it keeps 2^-23 of a row's largest under them (its
// subnormals are flushed), w = e (vs 2^-10), and e 2^-24 goes into the denominator.
// Sums move to a new maximum by h = exp2((m - m') / 2) twice: a denominator is far
// above 1 under a small V scale, and counts where h h itself is below fp32's range.
//
// 32 tokens over 6000 keys on average, 8 K/V heads of 128 in groups of 4: 76 us,
// 0.80 of the 6458 GB/s copy rate (the codes' conversion keeps the ALU at 42 %); one
// token over 500 7.6 us, the latency of its steps.

constexpr float kAttnLift = 24.0f, kAttnUnlift = 0x1p-24f;  // exponentials are 2^24 of what they stand for
constexpr float kAttnWeight = 0x1p-10f;                     // and weights 2^14: 2^24 of them in the exponential
constexpr float kAttnUnweight = 0x1p-14f;

// log2 of a page's V scale as it enters the maxima, which are 24 below what they stand
// for.  Scales below 2^-100 (and 0) weigh as 2^-100 in the maximum only.
__device__ __forceinline__ float attn_log2_scale(float vs) { return log2f(fmaxf(vs, 0x1p-100f)) - kAttnLift; }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t f16x2_pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What one split leaves for the others: rows of D sums, then the row's maximum
// and denominator.  Up to eight splits of a row tile are a cluster, whose CTAs
// read each other's slots in shared memory; the slots of more are in the
// workspace, for a second kernel.
template <int D>
constexpr int kAttnSlot = D + 4;  // (whole 16-byte pieces)

constexpr int kAttnRows = 16, kAttnStep = 16;
constexpr int kAttnMaxChunk = 4096;   // keys of one split: its pages' ids and scales are in shared memory

struct AttnSplit {
    uint32_t row_tiles, splits;
    int32_t chunk;      // keys per split, a multiple of 128
    uint32_t tile_rows; // kAttnRows or kTileRows
    uint32_t slot_rows; // rows of a tile that may exist: min(tile_rows, max_q * G)
    float* ws;          // NULL: one split, or a cluster of them
};

// Smallest v such that keys >= v of the row are masked.
__device__ __forceinline__ int attn_limit(const AttnParams& p, const AttnSeq& s, int32_t r) {
    const int32_t i = (int32_t)((uint32_t)r / (uint32_t)p.group);
    const int32_t lim = p.causal ? s.len - s.n + i + 1 : s.len;
    return i < s.n && lim > 0 ? lim : 0;
}

// A tile's codes of K or V in shared memory: boxes of 16 rows x min(D, 128)
// bytes, whose 16-byte pieces the TMA's swizzle permutes within a row.
template <int D>
struct AttnTile {
    static constexpr int box_cols = D < 128 ? D : 128;
    static constexpr int bytes = kAttnStep * D;
    // Offset of byte c (a multiple of 8) of row r.
    __device__ static __forceinline__ uint32_t at(int r, int c) {
        if constexpr (D == 64)
            return r * 64 + ((((c >> 4) ^ (r >> 1)) & 3) << 4) + (c & 15);
        else
            return (c >> 7) * (kAttnStep * 128) + r * 128 + ((((c >> 4) ^ r) & 7) << 4) + (c & 15);
    }
};

// N words of row r from byte c.
template <int D, int N>
__device__ __forceinline__ void ld_words(uint32_t (&w)[N], const uint8_t* tile, int r, int c) {
    if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(tile + AttnTile<D>::at(r, c));
        w[0] = x.x;
        w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(tile + AttnTile<D>::at(r, c + 4 * i));
            w[i] = x.x;
            w[i + 1] = x.y;
            w[i + 2] = x.z;
            w[i + 3] = x.w;
        }
    }
}

// Shared memory of attn_rows_kernel.
template <int D>
struct AttnGeo {
    static constexpr int warps = 4;
    static constexpr int stages = D == 64 ? 3 : 2;                // turns (two tiles) on their way per warp
    static constexpr int ctas = D == 256 ? 1 : D == 128 ? 3 : 4;  // per SM, for the register budget
    static constexpr int tile_bytes = 2 * AttnTile<D>::bytes;     // K and V
    static constexpr int stage_bytes = 2 * tile_bytes;
    static constexpr int ring = warps * stages * stage_bytes;
    static constexpr int pages = kAttnMaxChunk / 16;
    // in the ring's place at the end: the warps' sums, and this split's slots for a cluster
    static constexpr int red = warps * kAttnRows * (D + 4) * 4;
    static constexpr int slots = red + kAttnRows * kAttnSlot<D> * 4;
    static constexpr int qf_off = ring > slots ? ring : slots;
    static constexpr int ids_off = qf_off + D / 16 * 32 * 16;
    static constexpr int ml_off = ids_off + 4 * 4 * pages;
    static constexpr int bar_off = ml_off + 2 * 4 * warps * kAttnRows;
    static constexpr int smem = 1024 + bar_off + 8 * warps * stages;
};

// A NaN code of V reaches the rows that see its key and no other: it is taken out
// of the product (vf), and the rows that see one are counted with products of 0s
// and 1s.  key: the lane's first key; limits of rows g and g + 8.
template <int D>
__device__ __forceinline__ void attn_take_nans(uint32_t (&vf)[4][D / 32], float (&o)[D / 8][4], int key, int lim0, int lim1) {
    uint32_t see[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // row g, row g + 8 of keys 2t, 2t + 1; then of keys 8 + 2t, 9 + 2t
        const int kk = key + 8 * (i >> 1);
        const int lim = (i & 1) ? lim1 : lim0;
        see[i] = (kk < lim ? 0x3c00u : 0u) | (kk + 1 < lim ? 0x3c000000u : 0u);
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t one[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t lo = (nan_bytes(vf[2 * h][w]) >> (8 * e)) & 1u, hi = (nan_bytes(vf[2 * h + 1][w]) >> (8 * e)) & 1u;
                one[h] = (lo ? 0x3c00u : 0u) | (hi ? 0x3c000000u : 0u);
            }
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_f16(c, see[0], see[1], see[2], see[3], one[0], one[1]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c[i] > 0.0f) o[4 * w + e][i] = __int_as_float(0x7fffffff);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) vf[i][w] &= ~nan_bytes(vf[i][w]);
    }
}

template <int D>
__global__ void __launch_bounds__(32 * AttnGeo<D>::warps, AttnGeo<D>::ctas)
    attn_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const AttnParams p, const AttnSplit sp) {
    using G = AttnGeo<D>;
    constexpr int KW = D / 16, NJ = D / 8, kWarps = G::warps, S = G::stages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = align_shared<1024>(smem_raw);
    float* red = reinterpret_cast<float*>(smem);
    uint4(*qf)[32] = reinterpret_cast<uint4(*)[32]>(smem + G::qf_off);  // the queries as fragments, for every warp
    int32_t* ids = reinterpret_cast<int32_t*>(smem + G::ids_off);       // the split's pages: row / page, scales
    float *ks = reinterpret_cast<float*>(ids + G::pages), *vs = ks + G::pages, *lvs = vs + G::pages;
    float(*red_m)[kAttnRows] = reinterpret_cast<float(*)[kAttnRows]>(smem + G::ml_off);
    float(*red_l)[kAttnRows] = red_m + kWarps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * (S * G::stage_bytes);
    const uint32_t full0 = smem_u32(smem + G::bar_off) + 8 * S * warp;
    if (lane == 0) {
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
        for (int i = 0; i < S; ++i) mbar_init(full0 + 8 * i, 1);
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    uint32_t u = blockIdx.x;  // (32-bit divisions: each 64-bit one here costs a tenth of a microsecond)
    const bool joined = sp.splits > 1 && !sp.ws;  // a cluster: every CTA of it stays to the end
    uint32_t split;
    if (joined) {
        split = u % sp.splits;
        u /= sp.splits;
    } else {
        // The first splits, most of them full, go first, and the later ones, of which
        // less is left, fill in behind them (32 tokens over 2048 to 8192 keys: 76 us;
        // a row tile's splits one after the other 86; 8 over 500 to 2000: 16.0 / 15.6).
        const uint32_t items = gridDim.x / sp.splits;
        split = u / items;
        u -= split * items;
    }
    const uint32_t rt = u % sp.row_tiles;
    u /= sp.row_tiles;
    const int hk = (int)(u % (uint32_t)p.c.heads);
    const int64_t b = u / (uint32_t)p.c.heads;
    const AttnSeq s = attn_seq(p, b, threadIdx.x == 0);
    const int r0 = (int)rt * kAttnRows;
    const int rows = min(s.n * p.group - r0, kAttnRows);
    if (rows <= 0) return;
    // keys this tile sees (the last row sees most), and this split's part of them
    const int most = attn_limit(p, s, r0 + rows - 1);
    const int k0 = (int)min64((int64_t)split * sp.chunk, most), k1 = min(most - k0, sp.chunk) + k0;
    if (split > 0 && k0 >= k1 && !joined) return;
    const int every = attn_limit(p, s, r0);  // keys below are seen by every row of the tile
    const int lim0 = attn_limit(p, s, r0 + g), lim1 = attn_limit(p, s, r0 + g + 8);

    // a tile is 16 keys, a turn of a warp two tiles
    const int tiles = k0 < k1 ? (int)((k1 - k0 + kAttnStep - 1) / kAttnStep) : 0;
    const int turns = (tiles + 1) / 2;
    const int per_page = p.c.page / kAttnStep, shift = per_page == 1 ? 0 : per_page == 2 ? 1 : per_page == 4 ? 2 : 3;
    auto fetch = [&](int turn, int stage, auto&& id) {  // one lane
        const uint32_t bar = full0 + 8 * stage;
        const int n = min(2, tiles - 2 * turn);
        mbar_arrive_expect_tx(bar, n * G::tile_bytes);
        if (withheld(p, turn)) return;
        for (int j = 0; j < n; ++j) {
            const int tile = 2 * turn + j;
            const int32_t row = id(tile >> shift) * p.c.page + (tile & (per_page - 1)) * kAttnStep;
            const uint32_t dst = smem_u32(ring + stage * G::stage_bytes + j * G::tile_bytes);
#pragma unroll
            for (int c = 0; c < D; c += AttnTile<D>::box_cols) {
                tma_load_2d(dst + c * kAttnStep, &map_k, c, row, bar);
                tma_load_2d(dst + AttnTile<D>::bytes + c * kAttnStep, &map_v, c, row, bar);
            }
        }
    };
    // the first turns' codes are on their way before anything else is known of the pages
    const int page0 = (k0 / kAttnStep) >> shift;
    if (lane == 0)
        for (int i = 0; i < S && warp + i * kWarps < turns; ++i)
            fetch(warp + i * kWarps, i, [&](int pg) { return (int32_t)(attn_page(p, b, page0 + pg, false) * p.c.heads + hk); });
    const int n_pages = (tiles + per_page - 1) >> shift;
    for (int i = threadIdx.x; i < n_pages; i += 32 * kWarps) {
        const int64_t at = attn_page(p, b, page0 + i, true) * p.c.heads + hk;
        ids[i] = (int32_t)at;
        const float2 f = attn_page_scales(p.c.k_scale[at], p.c.v_scale[at]);
        ks[i] = f.x * p.scale_log2;
        vs[i] = f.y;
        lvs[i] = attn_log2_scale(vs[i]);
    }

    // this lane's part of the queries: rows g and g + 8, dims D/4 t .. D/4 t + D/4 - 1, scaled by a power of two
    float qs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool live = r0 + g + 8 * i < s.n * p.group;
        const uint32_t r = live ? r0 + g + 8 * i : 0, tok = r / (uint32_t)p.group, h = hk * p.group + (r - tok * p.group);
        const uint16_t* src = p.q + (s.first + tok) * p.ldq + (int64_t)h * D + t * (D / 4);
        uint4 x[D / 32];
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            x[c] = live ? __ldg(reinterpret_cast<const uint4*>(src + 8 * c)) : make_uint4(0, 0, 0, 0);
            amax = fmaxf(amax, amax8(x[c]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // up = 2^(14 - floor(log2 amax)), as two factors (it may pass fp32's range); undone through qs
        int e = 14 + 127 - (int)(__float_as_uint(fmaxf(amax, 0x1p-126f)) >> 23);
        if (amax == 0.0f) e = 0;
        const int e1 = e / 2, e2 = e - e1;
        const float u1 = __int_as_float((127 + e1) << 23), u2 = __int_as_float((127 + e2) << 23);
        qs[i] = __int_as_float((127 - e1) << 23) * __int_as_float((127 - e2) << 23);
        if (warp == 0) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                for (int h = 0; h < 4; ++h)  // word h of the piece: k step 2c + h/2, its lower or upper two indices
                    reinterpret_cast<uint32_t*>(&qf[2 * c + h / 2][lane])[i + 2 * (h & 1)] =
                        f16x2_pack(bf16lo(w[h]) * u1 * u2, bf16hi(w[h]) * u1 * u2);
            }
        }
    }
    __syncthreads();

    float o[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;

    int stage = 0;
    uint32_t phase = 0;
#pragma unroll 1
    for (int turn = warp; turn < turns; turn += kWarps) {
        if (!__all_sync(0xffffffffu, mbar_wait(full0 + 8 * stage, phase))) {
            if (lane == 0) {
                atomicOr(&g_device_error, kErrWaitTimeout);
                // the turns on their way land before the ring is used again
                for (int i = turn; i < turns && i < turn + S * kWarps; i += kWarps) {
                    (void)mbar_wait(full0 + 8 * stage, phase);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            __syncwarp();
            break;
        }
        // The last turn may have one tile: what lies in the other's place is of
        // keys that no row sees.
        const uint8_t* at = ring + stage * G::stage_bytes;
        const int key = k0 + turn * (2 * kAttnStep);
        const int page[2] = {(2 * turn) >> shift, min(2 * turn + 1, tiles - 1) >> shift};

        float sc[2][2][4] = {};  // [tile][keys 2t, 2t+1 / 8+2t, 9+2t][row g: 0, 1; row g + 8: 2, 3]
        {
            uint32_t kf[2][2][KW];  // codes of this lane: keys g, 8 + g
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) ld_words<D>(kf[j][i], at + j * G::tile_bytes, g + 8 * i, t * (D / 4));
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const uint4 a = qf[w][lane];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const Half4 k = e4m3x4_f16(kf[j][i][w]);
                        mma_f16(sc[j][i], a.x, a.y, a.z, a.w, k.lo, k.hi);
                    }
            }
        }
        float x[2][8];  // [tile][row g: keys 2t, 2t+1, 8+2t, 9+2t; row g + 8: the same]
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float f = ks[page[j]], f0 = f * qs[0], f1 = f * qs[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[j][i] = sc[j][i >> 1][i & 1] * f0;
                x[j][4 + i] = sc[j][i >> 1][2 + (i & 1)] * f1;
            }
        }
        const bool edge = key + 2 * kAttnStep > every;  // some row does not see some key of this turn
        if (edge) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kk = key + kAttnStep * j + 2 * t + (i & 1) + 8 * (i >> 1);
                    if (kk >= lim0) x[j][i] = -INFINITY;
                    if (kk >= lim1) x[j][4 + i] = -INFINITY;
                }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float lv = lvs[page[j]];
            t0 = fmaxf(t0, fmaxf(fmaxf(x[j][0], x[j][1]), fmaxf(x[j][2], x[j][3])) + lv);
            t1 = fmaxf(t1, fmaxf(fmaxf(x[j][4], x[j][5]), fmaxf(x[j][6], x[j][7])) + lv);
        }
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
        if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {
            const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
            const float h0 = n0 == -INFINITY ? 1.0f : exp2_approx(0.5f * (m0 - n0)), h1 = n1 == -INFINITY ? 1.0f : exp2_approx(0.5f * (m1 - n1));
            const float a0 = h0 * h0, a1 = h1 * h1;
            m0 = n0;
            m1 = n1;
            l0 = l0 * h0 * h0;
            l1 = l1 * h1 * h1;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                o[j][0] *= a0;
                o[j][1] *= a0;
                o[j][2] *= a1;
                o[j][3] *= a1;
            }
        }
        const float b0 = m0 == -INFINITY ? 0.0f : m0, b1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[j][i] = exp2_approx(x[j][i] - b0);
                x[j][4 + i] = exp2_approx(x[j][4 + i] - b1);
                l0 = fmaf(x[j][i], kAttnUnlift, l0);
                l1 = fmaf(x[j][4 + i], kAttnUnlift, l1);
            }
            const float wv = vs[page[j]] * kAttnWeight;
            const uint32_t p0 = f16x2_pack(x[j][0] * wv, x[j][1] * wv), p1 = f16x2_pack(x[j][4] * wv, x[j][5] * wv),
                           p2 = f16x2_pack(x[j][2] * wv, x[j][3] * wv), p3 = f16x2_pack(x[j][6] * wv, x[j][7] * wv);
            uint32_t vf[4][D / 32];  // codes of this lane: keys 2t, 2t+1, 8+2t, 9+2t
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ld_words<D>(vf[i], at + j * G::tile_bytes + AttnTile<D>::bytes, 2 * t + (i & 1) + 8 * (i >> 1), g * (D / 8));
            if (edge) {
                const int tk = key + kAttnStep * j;
                bool nans = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool dead = tk + 2 * t + (i & 1) + 8 * (i >> 1) >= most;
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        if (dead) vf[i][w] = 0;  // beyond the last row's keys: whatever lies there
                        nans = nans || nan_bytes(vf[i][w]) != 0;
                    }
                }
                if (__any_sync(0xffffffffu, nans)) attn_take_nans<D>(vf, o, tk + 2 * t, lim0, lim1);
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const Half4 a = e4m3x4_f16(__byte_perm(vf[0][w], vf[1][w], 0x5140)), b = e4m3x4_f16(__byte_perm(vf[2][w], vf[3][w], 0x5140));
                const Half4 c = e4m3x4_f16(__byte_perm(vf[0][w], vf[1][w], 0x7362)), d = e4m3x4_f16(__byte_perm(vf[2][w], vf[3][w], 0x7362));
                mma_f16(o[4 * w], p0, p1, p2, p3, a.lo, b.lo);
                mma_f16(o[4 * w + 1], p0, p1, p2, p3, a.hi, b.hi);
                mma_f16(o[4 * w + 2], p0, p1, p2, p3, c.lo, d.lo);
                mma_f16(o[4 * w + 3], p0, p1, p2, p3, c.hi, d.hi);
            }
        }
        // every lane has its codes: the stage takes the turn S turns on
        __syncwarp();
        if (lane == 0 && turn + S * kWarps < turns) fetch(turn + S * kWarps, stage, [&](int pg) { return ids[pg]; });
        if (++stage == S) {
            stage = 0;
            phase ^= 1;
        }
    }

    // join the four warps: sums under the common maximum
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (t == 0) {
        red_m[warp][g] = m0;
        red_m[warp][g + 8] = m1;
        red_l[warp][g] = l0;
        red_l[warp][g + 8] = l1;
    }
    __syncthreads();  // also: every warp is done with its ring
    float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        top0 = fmaxf(top0, red_m[w][g]);
        top1 = fmaxf(top1, red_m[w][g + 8]);
    }
    const float a0 = m0 == -INFINITY ? 0.0f : exp2_approx(m0 - top0), a1 = m1 == -INFINITY ? 0.0f : exp2_approx(m1 - top1);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {  // columns 2t, 2t + 1 of tile j: dims D/8 (2t) + j, D/8 (2t + 1) + j
        float* row0 = red + (warp * kAttnRows + g) * (D + 4);
        float* row1 = row0 + 8 * (D + 4);
        row0[2 * t * NJ + j] = o[j][0] * a0;
        row0[(2 * t + 1) * NJ + j] = o[j][1] * a0;
        row1[2 * t * NJ + j] = o[j][2] * a1;
        row1[(2 * t + 1) * NJ + j] = o[j][3] * a1;
    }
    __syncthreads();
    // a warp finishes four rows, a lane D / 32 dims of each
    for (int r = warp; r < rows; r += kWarps) {
        float top = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float h = red_m[w][r] == -INFINITY ? 1.0f : exp2_approx(0.5f * (red_m[w][r] - top));
            l = fmaf(red_l[w][r] * h, h, l);
        }
        float v[D / 32];
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
            v[d] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v[d] += red[(w * kAttnRows + r) * (D + 4) + lane * (D / 32) + d];
        }
        if (sp.splits > 1) {
            float* slot = joined ? red + G::red / 4 + r * kAttnSlot<D> : sp.ws + ((((int64_t)(b * p.c.heads + hk) * sp.row_tiles + rt) * sp.slot_rows + r) * sp.splits + split) * kAttnSlot<D>;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) slot[lane * (D / 32) + d] = v[d];
            if (lane == 0) {
                slot[D] = top;
                slot[D + 1] = l;
            }
        } else {
            const uint32_t row = r0 + r, i = row / (uint32_t)p.group;
            const int64_t tok = s.first + i, h = hk * p.group + (row - i * p.group);
            const float inv = l == 0.0f ? 0.0f : kAttnUnweight / l;
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + tok * p.ldo + h * D + lane * (D / 32));
#pragma unroll
            for (int d = 0; d < D / 32; d += 2) dst[d / 2] = bf16x2_pack(v[d] * inv, v[d + 1] * inv);
            if (p.lse && lane == 0) p.lse[tok * p.q_heads + h] = l == 0.0f ? -INFINITY : (top + kAttnLift + log2f(l)) * kLn2;
        }
    }
    if (joined) {
        cluster_sync();
        // CTA i of the cluster finishes rows i, i + splits, ..; a warp a row, a lane D / 32 dims
        for (int r = (int)split + warp * (int)sp.splits; r < rows; r += kWarps * (int)sp.splits) {
            const uint32_t slot = smem_u32(red) + G::red + r * kAttnSlot<D> * 4;
            float m[8], z[8], top = -INFINITY, l = 0.0f, v[D / 32] = {};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m[i] = i < (int)sp.splits ? ld_cluster(slot + 4 * D, i) : -INFINITY;
                z[i] = i < (int)sp.splits ? ld_cluster(slot + 4 * D + 4, i) : 0.0f;
                top = fmaxf(top, m[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= (int)sp.splits) break;
                const float h = m[i] == -INFINITY ? 1.0f : exp2_approx(0.5f * (m[i] - top)), a = h * h;
                l = fmaf(z[i] * h, h, l);
#pragma unroll
                for (int d = 0; d < D / 32; ++d) v[d] = fmaf(ld_cluster(slot + 4 * (lane * (D / 32) + d), i), a, v[d]);
            }
            const uint32_t row = r0 + r, i = row / (uint32_t)p.group;
            const int64_t tok = s.first + i, h = hk * p.group + (row - i * p.group);
            const float inv = l == 0.0f ? 0.0f : kAttnUnweight / l;
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + tok * p.ldo + h * D + lane * (D / 32));
#pragma unroll
            for (int d = 0; d < D / 32; d += 2) dst[d / 2] = bf16x2_pack(v[d] * inv, v[d + 1] * inv);
            if (p.lse && lane == 0) p.lse[tok * p.q_heads + h] = l == 0.0f ? -INFINITY : (top + kAttnLift + log2f(l)) * kLn2;
        }
        cluster_sync();  // no CTA leaves while another reads its slots
    }
}

// Joins the splits of a row: one CTA per row, its four warps take turns of the
// splits, four at a time.
template <int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnParams p, const AttnSplit sp) {
    __shared__ float part[4][D + 2];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t u = blockIdx.x;
    const float* slots = sp.ws + (int64_t)u * sp.splits * kAttnSlot<D>;
    const uint32_t in_tile = u % sp.slot_rows;
    u /= sp.slot_rows;
    const int row = (int)(u % sp.row_tiles * sp.tile_rows + in_tile);
    u /= sp.row_tiles;
    const int hk = (int)(u % (uint32_t)p.c.heads);
    const int64_t b = u / (uint32_t)p.c.heads;
    const AttnSeq s = attn_seq(p, b, false);
    if (row >= s.n * p.group) return;
    // the splits that its row tile filled (the first always)
    const int last = min(s.n * p.group, (row / (int)sp.tile_rows + 1) * (int)sp.tile_rows) - 1;
    const int most = attn_limit(p, s, last);
    const int n = most > sp.chunk ? (most - 1) / sp.chunk + 1 : 1;
    float top = -INFINITY, l = 0.0f, v[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d) v[d] = 0.0f;
    for (int i0 = warp; i0 < n; i0 += 16) {
        float m[4], z[4], x[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + 4 * k;
            const float* slot = slots + min(i, n - 1) * kAttnSlot<D>;
            m[k] = i < n ? slot[D] : -INFINITY;
            z[k] = i < n ? slot[D + 1] : 0.0f;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) x[k][d] = i < n ? slot[lane * (D / 32) + d] : 0.0f;
        }
        const float t4 = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), top);
        const float hk = top == -INFINITY ? 1.0f : exp2_approx(0.5f * (top - t4)), keep = hk * hk;  // (nothing, or NaN, so far)
        l = l * hk * hk;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) v[d] *= keep;
        top = t4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float h = m[k] == -INFINITY ? 1.0f : exp2_approx(0.5f * (m[k] - top)), a = h * h;
            l = fmaf(z[k] * h, h, l);
#pragma unroll
            for (int d = 0; d < D / 32; ++d) v[d] = fmaf(x[k][d], a, v[d]);
        }
    }
#pragma unroll
    for (int d = 0; d < D / 32; ++d) part[warp][lane * (D / 32) + d] = v[d];
    if (lane == 0) {
        part[warp][D] = top;
        part[warp][D + 1] = l;
    }
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    top = fmaxf(fmaxf(part[0][D], part[1][D]), fmaxf(part[2][D], part[3][D]));
    const int d = 2 * threadIdx.x;
    float x0 = 0.0f, x1 = 0.0f;
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float h = part[w][D] == -INFINITY ? 1.0f : exp2_approx(0.5f * (part[w][D] - top)), a = h * h;
        l = fmaf(part[w][D + 1] * h, h, l);
        x0 = fmaf(part[w][d], a, x0);
        x1 = fmaf(part[w][d + 1], a, x1);
    }
    const uint32_t i = (uint32_t)row / (uint32_t)p.group;
    const int64_t tok = s.first + i, h = hk * p.group + (row - i * p.group);
    const float inv = l == 0.0f ? 0.0f : kAttnUnweight / l;
    *reinterpret_cast<uint32_t*>(p.o + tok * p.ldo + h * D + d) = bf16x2_pack(x0 * inv, x1 * inv);
    if (p.lse && threadIdx.x == 0) p.lse[tok * p.q_heads + h] = l == 0.0f ? -INFINITY : (top + kAttnLift + log2f(l)) * kLn2;
}

}  // namespace fp4q
