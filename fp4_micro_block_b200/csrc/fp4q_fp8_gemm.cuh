// fp4q_fp8_gemm.cuh -- D = A B^T of E4M3 codes under block-128 scales, on the
// 5th-generation tensor cores (tcgen05, kind::f8f6f4):
//
//   D[m, n] = sum_kb SA[kb, m] SB[kb, n] sum_{k in kb} A[m, k] B[n, k]
//
// The inner sum of one block is four MMAs (K = 32 each) into fp32 in tensor
// memory; the scales differ per row and block and are no power of two, so each
// block's sum is read back, scaled and added in fp32 registers.  Two TMEM
// buffers let the MMAs of block kb + 1 run under that.
//
// One operand's rows are the 128 TMEM lanes (a thread = a row), the other's are
// the accumulator's columns:
//   wide kernel    lanes = rows of A, 256 columns = rows of B; persistent;
//   narrow kernel  lanes = rows of B (the weights), 16..128 columns = rows of
//                  A: few rows of A do not waste lanes, and the K blocks of a
//                  tile are split over a cluster of CTAs whose partial sums
//                  are added through distributed shared memory in rank order.
//
// CTA roles: warp 0 lane 0 streams the K blocks of both operands by TMA into a
// ring; warp 1 allocates TMEM and issues the MMAs (as a whole, one lane elected:
// 141 us for 8192x4096x4096, with a branch on lane 0 158); the other warps (groups of four, each with
// its columns) scale and accumulate, then store.
// Every wait is bounded; a wait that runs out sets g_device_error and the role
// stops; the CTA drains its copies and MMAs and frees TMEM before it exits.
#pragma once

#include "fp4q_fp8.cuh"
#include "fp4q_mma.cuh"

namespace fp4q {

constexpr int kF8Lanes = 128;
constexpr int kF8MaxSplit = 8;                      // CTAs of a portable cluster
constexpr int kF8LaneBytes = kF8Lanes * kFp8Block;  // 16 KiB of the lane operand per K block

struct Fp8GemmParams {
    int64_t RL, RC;          // rows of the lane and the column operand
    int32_t n_kb;            // K blocks
    int64_t n_lt, n_tiles;   // lane tiles; tiles (lane tile fastest)
    const float *sl, *sc;    // scales [n_kb, ld]
    int64_t ldsl, ldsc;
    int32_t l_tile;          // narrow kernel: B's scales are per 128 x 128 tile
    void* d;
    int64_t ldd;
    int32_t out_bf16;
    int32_t tma_store;       // wide kernel: D's rows begin and end on 16 bytes
    int32_t split;           // narrow kernel: CTAs of the cluster that share a tile's K blocks
#ifdef FP4Q_TEST_HOOKS
    int64_t skip_copy;       // withheld()
#endif
};

// kind::f8f6f4 instruction descriptor: D fp32 (1 at [4,6)), A and B E4M3 (0 at
// [7,10), [10,13)), both K-major, N >> 3 at [17,23), M >> 4 at [24,29).
__host__ __device__ constexpr uint32_t f8_idesc(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kF8Lanes >> 4) << 24);
}

// sw128_desc in two parts: the low word, to which offsets / 16 are added, and the rest.
__device__ __forceinline__ uint32_t sw128_desc_lo(uint32_t saddr) { return (uint32_t)sw128_desc(saddr); }
__device__ __forceinline__ uint64_t sw128_desc_of(uint32_t lo) {
    return (uint64_t)lo | ((uint64_t)((1024u >> 4) | 1u << 14 | 2u << 29) << 32);
}
// One lane of the (converged) warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}
// D[tmem] (+)= A * B^T, E4M3 operands, M = 128, K = 32.
__device__ __forceinline__ void umma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Starts the load of 32 or 16 consecutive fp32 columns of this thread's TMEM lane; the
// registers hold them after tmem_wait of the same array.
__device__ __forceinline__ void tmem_start(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
          "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
          "+r"(r[30]), "+r"(r[31])
        :
        : "memory");
}
__device__ __forceinline__ void tmem_start(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// One element of D.
__device__ __forceinline__ void f8_store(const Fp8GemmParams& p, int64_t m, int64_t n, float v) {
    if (p.out_bf16)
        static_cast<uint16_t*>(p.d)[m * p.ldd + n] = (uint16_t)bf16x2_pack(v, 0.0f);
    else
        static_cast<float*>(p.d)[m * p.ldd + n] = v;
}

// acc += scale * (one K block's sums), columns [0, C) of TMEM at taddr, 16 at a
// time, the next on their way under the arithmetic of these (8192x4096x4096: 140
// us, 32 at a time without the overlap 144).  VEC: column scales from shared
// memory (broadcast reads), else f covers both scales.  read(): called once the
// last columns have arrived.
template <int C, bool VEC, typename Read>
__device__ __forceinline__ void f8_accumulate(uint32_t taddr, float f, const float* sc, float (&acc)[C], Read&& read) {
    constexpr int W = 16;
    uint32_t v[2][W];
    tmem_start(taddr, v[0]);
#pragma unroll
    for (int h = 0; h < C / W; ++h) {
        tmem_wait(v[h & 1]);
        if (h + 1 < C / W)
            tmem_start(taddr + (h + 1) * W, v[(h + 1) & 1]);
        else
            read();
#pragma unroll
        for (int c = 0; c < W; c += 4) {
            float4 s = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
            if constexpr (VEC) s = *reinterpret_cast<const float4*>(sc + h * W + c);
            const float k[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = __uint_as_float(v[h & 1][c + i]);
                float& o = acc[h * W + c + i];
                o = VEC ? fmaf(x * f, k[i], o) : fmaf(x, f, o);
            }
        }
    }
}

// ------------------------------------------------------------------ narrow kernel
//
// Few rows of A: the time is a launch, a ring's latency and the reading of B.
// 1x4096x4096 5.8 us (K over 4 CTAs), 37x4096x4352 8.5 us.

template <int NT>
struct F8Narrow {
    static constexpr int groups = NT >= 64 ? 2 : 1;      // epilogue groups of four warps
    static constexpr int cols = NT / groups;             // accumulator columns of a thread
    static constexpr int threads = 64 + 128 * groups;
    static constexpr int stage_bytes = kF8LaneBytes + NT * kFp8Block;
    static constexpr int stages = (192 * 1024) / stage_bytes;
    static constexpr int ring = stages * stage_bytes;
    static constexpr int sc_off = ring;                  // column scales, two buffers
    static constexpr int bar_off = sc_off + 2 * NT * 4;
    static constexpr int num_bars = 2 * stages + 5;
    static constexpr int slot_off = bar_off + num_bars * 8;
    static constexpr int smem = 1024 + slot_off + 16;
    static constexpr uint32_t tmem_cols = 2 * NT;        // two buffers
    static_assert(stage_bytes % 1024 == 0, "stages keep the 1024-byte alignment of the swizzle");
    static_assert(smem <= 227 * 1024, "shared memory");
    static_assert(ring >= NT * kF8Lanes * 4, "the ring holds the partial sums of the split");
};

template <int NT>
__global__ void __launch_bounds__(F8Narrow<NT>::threads, 1)
    fp8_gemm_narrow_kernel(const __grid_constant__ CUtensorMap map_l, const __grid_constant__ CUtensorMap map_c,
                           const Fp8GemmParams p) {
    using G = F8Narrow<NT>;
    constexpr int S = G::stages, C = G::cols;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = align_shared<1024>(smem_raw);
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t full0 = smem_u32(smem + G::bar_off), empty0 = full0 + 8 * S;
    const uint32_t accf = empty0 + 8 * S, acce = accf + 16, done_bar = acce + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::slot_off);

    if (tid == 0) {
        prefetch_tmap(&map_l);
        prefetch_tmap(&map_c);
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf + 8 * i, 1);
            mbar_init(acce + 8 * i, 4 * G::groups);  // one arrival per epilogue warp
        }
        mbar_init(done_bar, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), G::tmem_cols);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // this CTA's tile and its share of the K blocks
    const int64_t tile = blockIdx.x / p.split;
    const int rank = (int)(blockIdx.x - tile * p.split);
    const int64_t lt = tile % p.n_lt, ct = tile / p.n_lt;
    const int kb0 = (int)((int64_t)p.n_kb * rank / p.split);
    const int kbs = (int)((int64_t)p.n_kb * (rank + 1) / p.split) - kb0;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int g = 0, s = 0;
            uint32_t ph = 1;
            for (; g < kbs; ++g) {
                if (g >= S && !mbar_wait(empty0 + 8 * s, ph)) {
                    atomicOr(&g_device_error, kErrWaitTimeout);
                    break;
                }
                uint8_t* st = smem + s * G::stage_bytes;
                const uint32_t bar = full0 + 8 * s;
                mbar_arrive_expect_tx(bar, G::stage_bytes);
                if (!withheld(p, g)) {
                    tma_load_2d(smem_u32(st), &map_l, (kb0 + g) * kFp8Block, (int32_t)(lt * kF8Lanes), bar);
                    tma_load_2d(smem_u32(st + kF8LaneBytes), &map_c, (kb0 + g) * kFp8Block, (int32_t)(ct * NT), bar);
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
            }
            // every issued copy lands before the CTA may exit
            for (int k = (g > S ? g - S : 0); k < g; ++k)
                (void)mbar_wait(full0 + 8 * (k % S), (uint32_t)((k / S) & 1));
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        // The whole warp goes through the loop, and one lane issues.
        const bool one = elect_one();
        const uint32_t t0 = __shfl_sync(0xffffffffu, tmem_base, 0);
        const uint32_t ring = sw128_desc_lo(smem_u32(smem));
        bool ok = true;
        int s = 0;
        uint32_t ph = 0;
        for (int g = 0; g < kbs; ++g) {
            const int buf = (int)(g & 1);
            ok = mbar_wait(full0 + 8 * s, ph) && (g < 2 || mbar_wait(acce + 8 * buf, (uint32_t)(((g >> 1) - 1) & 1)));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t st = ring + s * (G::stage_bytes >> 4);
            if (one) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    umma_f8(t0 + NT * buf, sw128_desc_of(st + 2 * j), sw128_desc_of(st + (kF8LaneBytes >> 4) + 2 * j),
                            f8_idesc(NT), j > 0 ? 1u : 0u);
                tc_commit(empty0 + 8 * s);
                tc_commit(accf + 8 * buf);
            }
            __syncwarp();
            if (++s == S) {
                s = 0;
                ph ^= 1;
            }
        }
        if (!ok && one) atomicOr(&g_device_error, kErrWaitTimeout);
        // all MMAs of this CTA complete before TMEM is freed
        if (one) tc_commit(done_bar);
        if (!mbar_wait(done_bar, 0) && one) atomicOr(&g_device_error, kErrWaitTimeout);
    } else {
        // ------------------------------------------------ scale, accumulate, store
        const uint32_t quarter = warp & 3;         // the TMEM lanes this warp may read
        const int grp = (int)(warp - 2) >> 2;
        const int t = (int)(quarter * 32 + lane);  // TMEM lane, also this thread's place in the group
        const uint32_t taddr = tmem_base + ((quarter * 32u) << 16) + (uint32_t)(grp * C);
        float* sc_buf = reinterpret_cast<float*>(smem + G::sc_off) + grp * 2 * C;
        const int64_t row = lt * kF8Lanes + t, c0 = ct * NT + grp * C;
        // scale addresses, clamped to rows that exist (the others' results are dropped)
        const float* sl = p.sl + (int64_t)kb0 * p.ldsl + (p.l_tile ? lt : min64(row, p.RL - 1));
        const float* sc = p.sc + (int64_t)kb0 * p.ldsc + min64(c0 + (t < C ? t : 0), p.RC - 1);
        float acc[C];
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = 0.0f;
        bool ok = true;
        int g = 0;
        auto block = [&](float l, float s) {
            const int buf = g & 1;
            if (t < C) sc_buf[buf * C + t] = s;
            bar_sync(1 + grp, 128);
            if (ok) {  // once a wait has run out, the rest is skipped
                ok = __all_sync(0xffffffffu, mbar_wait(accf + 8 * buf, (uint32_t)((g >> 1) & 1)));
                if (!ok && lane == 0) atomicOr(&g_device_error, kErrWaitTimeout);
            }
            tc_fence_after();
            auto read = [&] {  // this warp's reads of the buffer are done
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce + 8 * buf);
            };
            if (ok)
                f8_accumulate<C, true>(taddr + NT * buf, l, sc_buf + buf * C, acc, read);
            else
                read();
            ++g;
        };
        // two blocks a turn: the next two's scales are on their way meanwhile
        auto lane_scale = [&](int kb) { return __ldg(sl + min(kb, kbs - 1) * p.ldsl); };
        auto col_scale = [&](int kb) { return __ldg(sc + min(kb, kbs - 1) * p.ldsc); };
        float l0 = lane_scale(0), l1 = lane_scale(1), s0 = col_scale(0), s1 = col_scale(1);
#pragma unroll 1
        for (int kb = 0; kb < kbs; kb += 2) {
            const float m0 = lane_scale(kb + 2), m1 = lane_scale(kb + 3), n0 = col_scale(kb + 2), n1 = col_scale(kb + 3);
            block(l0, s0);
            if (kb + 1 < kbs) block(l1, s1);
            l0 = m0;
            l1 = m1;
            s0 = n0;
            s1 = n1;
        }
        if (p.split == 1) {
            // lanes are consecutive columns of D: a warp writes runs of 32
            if (row < p.RL) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (c0 + c < p.RC) f8_store(p, c0 + c, row, acc[c]);
            }
        } else {
            // every block of this CTA has been read: the ring holds its partial sums now
            float* part = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int c = 0; c < C; ++c) part[(grp * C + c) * kF8Lanes + t] = acc[c];
        }
    }

    if (p.split > 1) {
        __syncthreads();
        cluster_sync();
        // rank r adds columns r, r + split, ... of the tile, rank 0's part first
        if (warp >= 2) {
            const int t = (int)((warp & 3) * 32 + lane);
            const int64_t row = lt * kF8Lanes + t, c0 = ct * NT;
            const uint32_t part = smem_u32(smem) + 4 * t;
            // (the groups take turns of them)
            const int grp = (int)(warp - 2) >> 2;
            for (int c = rank + grp * p.split; c < NT && c0 + c < p.RC; c += G::groups * p.split) {
                float v[kF8MaxSplit];
#pragma unroll
                for (int r = 0; r < kF8MaxSplit; ++r)
                    v[r] = r < p.split ? ld_cluster(part + c * kF8Lanes * 4, r) : 0.0f;
#pragma unroll
                for (int r = 1; r < kF8MaxSplit; ++r) v[0] += v[r];
                if (row < p.RL) f8_store(p, c0 + c, row, v[0]);
            }
        }
        cluster_sync();  // no CTA leaves while another reads its sums
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, G::tmem_cols);
    }
}

// ------------------------------------------------------------------ wide kernel
//
// 8192x4096x4096 139 to 142 us (1.97 to 1.94 PFLOP/s) with tile scales, 166 in a long
// run under the power limit; 4096x4096x8190 with row scales and fp32 output (two
// multiplies a sum, column scales from shared memory) 209 to 223, 234 so.  The
// two TMEM buffers are all of tensor memory, and their hand-over between the MMAs
// and the warps that scale bounds it: the tensor pipe is busy 45 % of the time.
// Sixteen such warps took 159 us, CTA pairs 181.

// The wide kernel's register split: 384 threads start with 168 each; the first
// warpgroup gives up 96 so that the two epilogue ones, which hold 128 sums per
// thread, have 216 (72 + 2 * 216 = 3 * 168).
constexpr int kF8RegsRoles = 72, kF8RegsEpilogue = 216;
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

struct F8Wide {
    static constexpr int n = 256;                        // columns of a tile = rows of B
    static constexpr int groups = 2;                     // epilogue groups of four warps
    static constexpr int cols = n / groups;              // accumulator columns of a thread
    static constexpr int first_epi = 4;                  // first epilogue warp (whole warpgroups, see kF8Regs)
    static constexpr int threads = 32 * first_epi + 128 * groups;
    static constexpr int stage_bytes = kF8LaneBytes + n * kFp8Block;
    static constexpr int stages = 4;
    static constexpr int stg_off = stages * stage_bytes; // 4 KiB of output staging per epilogue warp
    static constexpr int sc_off = stg_off + 8 * 4096;    // column scales, two buffers per group
    static constexpr int bar_off = sc_off + groups * 2 * cols * 4;
    static constexpr int num_bars = 2 * stages + 5;
    static constexpr int slot_off = bar_off + num_bars * 8;
    static constexpr int smem = 896 + slot_off + 16;     // the base is 128-byte aligned, the ring 1024
    static constexpr uint32_t tmem_cols = 2 * n;         // two buffers
    static_assert(stage_bytes % 1024 == 0, "stages keep the 1024-byte alignment of the swizzle");
    static_assert(smem <= 227 * 1024, "shared memory");
};

// VEC: B's scales are per row; else per 128 x 128 tile.
template <bool VEC>
__global__ void __launch_bounds__(F8Wide::threads, 1)
    fp8_gemm_wide_kernel(const __grid_constant__ CUtensorMap map_l, const __grid_constant__ CUtensorMap map_c,
                         const __grid_constant__ CUtensorMap map_d, const Fp8GemmParams p) {
    using G = F8Wide;
    constexpr int NT = G::n;
    constexpr int S = G::stages, C = G::cols;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = align_shared<1024>(smem_raw);
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t full0 = smem_u32(smem + G::bar_off), empty0 = full0 + 8 * S;
    const uint32_t accf = empty0 + 8 * S, acce = accf + 16, done_bar = acce + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::slot_off);

    if (tid == 0) {
        prefetch_tmap(&map_l);
        prefetch_tmap(&map_c);
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(accf + 8 * i, 1);
            mbar_init(acce + 8 * i, 4 * G::groups);  // one arrival per epilogue warp
        }
        mbar_init(done_bar, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), G::tmem_cols);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int64_t unit = blockIdx.x, step = gridDim.x;
    const int kbs = p.n_kb;
    const int64_t n_my = p.n_tiles > unit ? (p.n_tiles - 1 - unit) / step + 1 : 0;

    const int epi = (int)warp - G::first_epi;
    const uint32_t quarter = warp & 3;  // the TMEM lanes a warp may read
    const int grp = epi >> 2;

    if (epi < 0) {
        reg_dec<kF8RegsRoles>();
    }
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            const int64_t total = n_my * kbs;
            int64_t g = 0;
            int s = 0, kb = 0;
            uint32_t ph = 1;
            int64_t t = unit;
            for (; g < total; ++g) {
                if (g >= S && !mbar_wait(empty0 + 8 * s, ph)) {
                    atomicOr(&g_device_error, kErrWaitTimeout);
                    break;
                }
                const int64_t lt = t % p.n_lt, ct = t / p.n_lt;
                uint8_t* st = smem + s * G::stage_bytes;
                const uint32_t bar = full0 + 8 * s;
                mbar_arrive_expect_tx(bar, G::stage_bytes);
                if (!withheld(p, g)) {
                    tma_load_2d(smem_u32(st), &map_l, kb * kFp8Block, (int32_t)(lt * kF8Lanes), bar);
                    tma_load_2d(smem_u32(st + kF8LaneBytes), &map_c, kb * kFp8Block, (int32_t)(ct * NT), bar);
                }
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
                if (++kb == kbs) {
                    kb = 0;
                    t += step;
                }
            }
            // every issued copy lands before the CTA may exit
            for (int64_t k = (g > S ? g - S : 0); k < g; ++k)
                (void)mbar_wait(full0 + 8 * (int)(k % S), (uint32_t)((k / S) & 1));
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        // The whole warp goes through the loop, and one lane issues.
        const bool one = elect_one();
        const uint32_t t0 = __shfl_sync(0xffffffffu, tmem_base, 0);
        const uint32_t ring = sw128_desc_lo(smem_u32(smem));
        bool ok = true;
        const int64_t total = n_my * kbs;
        int s = 0;
        uint32_t ph = 0;
        for (int64_t g = 0; g < total; ++g) {
            const int buf = (int)(g & 1);
            ok = mbar_wait(full0 + 8 * s, ph) && (g < 2 || mbar_wait(acce + 8 * buf, (uint32_t)(((g >> 1) - 1) & 1)));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t st = ring + s * (G::stage_bytes >> 4);
            if (one) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    umma_f8(t0 + NT * buf, sw128_desc_of(st + 2 * j), sw128_desc_of(st + (kF8LaneBytes >> 4) + 2 * j),
                            f8_idesc(NT), j > 0 ? 1u : 0u);
                tc_commit(empty0 + 8 * s);
                tc_commit(accf + 8 * buf);
            }
            __syncwarp();
            if (++s == S) {
                s = 0;
                ph ^= 1;
            }
        }
        if (!ok && one) atomicOr(&g_device_error, kErrWaitTimeout);
        // all MMAs of this CTA complete before TMEM is freed
        if (one) tc_commit(done_bar);
        if (!mbar_wait(done_bar, 0) && one) atomicOr(&g_device_error, kErrWaitTimeout);
    } else if (epi >= 0) {
        // ------------------------------------------------ scale, accumulate, store
        reg_inc<kF8RegsEpilogue>();
        float acc[C];
        const int t = (int)quarter * 32 + (int)lane;  // TMEM lane, also this thread's place in the group
        const uint32_t taddr = tmem_base + ((quarter * 32u) << 16) + (uint32_t)(grp * C);
        float* sc_buf = reinterpret_cast<float*>(smem + G::sc_off) + grp * 2 * C;
        const int stg = epi * 4096;
        int64_t g = 0;
        bool ok = true;
#pragma unroll 1
        for (int64_t i = 0; i < n_my; ++i) {
            const int64_t tile = unit + i * step;
            const int64_t lt = tile % p.n_lt, ct = tile / p.n_lt;
            const int64_t row = lt * kF8Lanes + t, c0 = ct * NT + grp * C;
            // scale addresses, clamped to rows that exist (the others' results are dropped)
            const float* sl = p.sl + min64(row, p.RL - 1);
            const float* sc = p.sc + (VEC ? min64(c0 + (t < C ? t : 0), p.RC - 1) : min64(c0, p.RC - 1) / kFp8Block);
#pragma unroll
            for (int c = 0; c < C; ++c) acc[c] = 0.0f;
            auto lane_scale = [&](int kb) { return __ldg(sl + min(kb, kbs - 1) * p.ldsl); };
            auto col_scale = [&](int kb) { return __ldg(sc + min(kb, kbs - 1) * p.ldsc); };
            auto block = [&](float l, float s) {
                const int buf = (int)(g & 1);
                if constexpr (VEC) {
                    if (t < C) sc_buf[buf * C + t] = s;
                    bar_sync(1 + grp, 128);
                }
                if (ok) {  // once a wait has run out, the rest is skipped
                    ok = __all_sync(0xffffffffu, mbar_wait(accf + 8 * buf, (uint32_t)((g >> 1) & 1)));
                    if (!ok && lane == 0) atomicOr(&g_device_error, kErrWaitTimeout);
                }
                tc_fence_after();
                auto read = [&] {  // this warp's reads of the buffer are done
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acce + 8 * buf);
                };
                if (ok)
                    f8_accumulate<C, VEC>(taddr + NT * buf, VEC ? l : l * s, sc_buf + buf * C, acc, read);
                else
                    read();
                ++g;
            };
            // two blocks a turn: the next two's scales are on their way meanwhile,
            // and nothing waits for them (moving them along each block would)
            float l0 = lane_scale(0), l1 = lane_scale(1), s0 = col_scale(0), s1 = col_scale(1);
#pragma unroll 1
            for (int kb = 0; kb < kbs; kb += 2) {
                const float m0 = lane_scale(kb + 2), m1 = lane_scale(kb + 3), t0 = col_scale(kb + 2), t1 = col_scale(kb + 3);
                block(l0, s0);
                if (kb + 1 < kbs) block(l1, s1);
                l0 = m0;
                l1 = m1;
                s0 = t0;
                s1 = t1;
            }
            if (p.tma_store) {
                // 32 rows x 128 bytes at a time through this warp's 4 KiB (128-byte swizzle)
                const uint32_t buf32 = smem_u32(smem + G::stg_off + stg);
#pragma unroll
                for (int h = 0; h < C / 32; ++h) {  // boxes of 32 fp32 columns, or halves of 64 bf16 ones
                    const bool first = !p.out_bf16 || (h & 1) == 0, last = !p.out_bf16 || (h & 1) == 1;
                    if (first) {
                        if (lane == 0) bulk_wait_read0();
                        __syncwarp();
                    }
                    if (p.out_bf16) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            sts_v4(buf32 + swz128(lane, 64 * (h & 1) + 16 * q),
                                   bf16x2_pack(acc[32 * h + 8 * q], acc[32 * h + 8 * q + 1]),
                                   bf16x2_pack(acc[32 * h + 8 * q + 2], acc[32 * h + 8 * q + 3]),
                                   bf16x2_pack(acc[32 * h + 8 * q + 4], acc[32 * h + 8 * q + 5]),
                                   bf16x2_pack(acc[32 * h + 8 * q + 6], acc[32 * h + 8 * q + 7]));
                    } else {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            sts_v4(buf32 + swz128(lane, 16 * q), __float_as_uint(acc[32 * h + 4 * q]),
                                   __float_as_uint(acc[32 * h + 4 * q + 1]), __float_as_uint(acc[32 * h + 4 * q + 2]),
                                   __float_as_uint(acc[32 * h + 4 * q + 3]));
                    }
                    if (last) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        const int64_t col = c0 + 32 * h - (p.out_bf16 ? 32 : 0), r0 = lt * kF8Lanes + quarter * 32;
                        if (lane == 0 && col < p.RC && r0 < p.RL) {
                            tma_store_2d(&map_d, (int32_t)col, (int32_t)r0, buf32);
                            bulk_commit();
                        }
                    }
                }
            } else if (row < p.RL) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (c0 + c < p.RC) f8_store(p, row, c0 + c, acc[c]);
            }
        }
        if (lane == 0) bulk_wait0();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, G::tmem_cols);
    }
}

}  // namespace fp4q
