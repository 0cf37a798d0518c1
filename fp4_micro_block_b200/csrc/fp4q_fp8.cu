// fp4q_fp8.cu -- the extern "C" boundary of the 8-bit operators: argument
// checks and launches.  All arithmetic runs in the kernels included below.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/fp4q.h"
#include "fp4q_attn.cuh"
#include "fp4q_attn_tile.cuh"
#include "fp4q_fp8.cuh"
#include "fp4q_fp8_gemm.cuh"
#include "fp4q_host.cuh"
#include "fp4q_kv.cuh"

namespace fp4q {

// This translation unit's device error word (read together with fp4q.cu's).
bool fp8_device_error(unsigned int* out) {
    unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(out, g_device_error, sizeof(*out)) != cudaSuccess) return false;
    return !*out || cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero)) == cudaSuccess;
}

}  // namespace fp4q

namespace {

using namespace fp4q;

int64_t spans(int64_t n, int64_t d) { return (n + d - 1) / d; }

#ifdef FP4Q_TEST_HOOKS
// Test build only: the copies that CTA 0 of the next launch of a kernel with TMA
// loads withholds (-1: none); consumed by that launch.
std::atomic<int64_t> g_test_skip_copy{-1};
#endif
template <typename P>
void take_skip(P& p) {
#ifdef FP4Q_TEST_HOOKS
    p.skip_copy = g_test_skip_copy.exchange(-1);
#endif
}

bool valid_block(fp4q_fp8_block b) { return b == FP4Q_FP8_ROW || b == FP4Q_FP8_TILE; }

// One side of a quantized matrix: codes [rows, ld] and scales [ceil(cols/128), lds].
fp4q_status check_fp8(const void* codes, int64_t rows, int64_t cols, int64_t ld, const void* scales, int64_t lds,
                      fp4q_fp8_block block) {
    const int64_t n = block == FP4Q_FP8_TILE ? spans(rows, kFp8Block) : rows;
    if (!codes || !scales || ld < cols || lds < n) return FP4Q_ERR_INVALID_ARG;
    if (ld >= kMaxDim || lds >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
    if (ld % 16 != 0 || lds % 4 != 0 || !aligned(codes, 16) || !aligned(scales, 16)) return FP4Q_ERR_ALIGNMENT;
    return FP4Q_OK;
}

template <bool TILE>
fp4q_status launch_fp8_tile(const Fp8QuantParams& p, cudaStream_t s) {
    auto kern = fp8_tile_kernel<TILE>;
    static std::atomic<uint64_t> done{0};
    int sms = 0;
    fp4q_status st;
    if ((st = sm_count(&sms)) != FP4Q_OK || (st = ensure_smem(kern, kFp8TileSmem, done)) != FP4Q_OK) return st;
    CUtensorMap map;
    if ((st = make_x_map(&map, p.x, p.M, p.K, p.ldx, kFp8Block)) != FP4Q_OK) return st;
    const int grid = (int)std::min<int64_t>(p.n_items, (int64_t)kFp8TileCtas * sms);
    return launch(kern, grid, kFp8TileThreads, kFp8TileSmem, s, map, p);
}

// Codes [rows, K] with row stride ld, boxes of 128 columns x box_rows with the
// 128-byte swizzle; columns past K and rows past `rows` read as zero codes.
fp4q_status make_f8_map(CUtensorMap* map, const void* codes, int64_t rows, int64_t K, int64_t ld, uint32_t box_rows) {
    EncodeTiledFn enc;
    fp4q_status st = encode_fn(&enc);
    if (st != FP4Q_OK) return st;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {(cuuint32_t)kFp8Block, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4Q_OK : FP4Q_ERR_CUDA;
}

// The wide kernel's output [M, N], stored in boxes of 128 bytes x 32 rows.
fp4q_status make_f8_out_map(CUtensorMap* map, void* d, int64_t M, int64_t N, int64_t ldd, int bf16) {
    EncodeTiledFn enc;
    fp4q_status st = encode_fn(&enc);
    if (st != FP4Q_OK) return st;
    const int64_t es = bf16 ? 2 : 4;
    cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
    cuuint64_t strides[1] = {(cuuint64_t)(ldd * es)};
    cuuint32_t box[2] = {(cuuint32_t)(128 / es), 32u};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, d, dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4Q_OK : FP4Q_ERR_CUDA;
}

struct Fp8Operand {
    const uint8_t* codes;
    int64_t rows, ld;
    const float* scales;
    int64_t lds;
    int tile;
};

template <typename... KArgs, typename... Args>
fp4q_status launch_cluster(void (*kern)(KArgs...), int64_t grid, int cluster, int threads, int smem, cudaStream_t s,
                           Args&&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) == cudaSuccess ? FP4Q_OK : FP4Q_ERR_CUDA;
}

void f8_operands(Fp8GemmParams& p, const Fp8Operand& l, const Fp8Operand& c, int64_t lane_rows, int64_t col_rows) {
    p.RL = l.rows;
    p.RC = c.rows;
    p.n_lt = spans(l.rows, lane_rows);
    p.n_tiles = p.n_lt * spans(c.rows, col_rows);
    p.sl = l.scales;
    p.ldsl = l.lds;
    p.l_tile = l.tile;
    p.sc = c.scales;
    p.ldsc = c.lds;
}

// CTAs that share a narrow tile's K blocks.
int64_t f8_split(int64_t tiles, int64_t n_kb, int sms) {
    return std::max<int64_t>(1, std::min<int64_t>({(int64_t)kF8MaxSplit, n_kb, sms / tiles}));
}

// Whether the wide kernel is the faster one, by what both took on one B200: per
// wave and K block 0.55 us with tile scales of B, 0.80 with row scales (narrow,
// 128 columns: 0.62), 4 us besides (narrow: 4, and 4 more for a split's join).
// Measured for N = K = 4096, tile scales, in us (wide / narrow): M = 100 20.6 /
// 11.3, 256 20.9 / 19.0, 512 21.3 / 23.2, 800 21.9 / 44.9; 300 x 1000 x 513
// 7.3 / 8.1; 1000 x 1024 x 2000 13.6 / 14.9; 200 x 16384 x 4096 23.2 / 45.4.
bool f8_take_wide(int64_t M, int64_t N, int64_t n_kb, bool tile, int sms) {
    if (M <= 64) return false;  // a wide tile would waste more than half of its lanes
    const int64_t wide = spans(spans(M, kF8Lanes) * spans(N, F8Wide::n), sms) * n_kb * (tile ? 55 : 80) + 400;
    const int64_t tiles = spans(M, 128) * spans(N, kF8Lanes), split = f8_split(tiles, n_kb, sms);
    const int64_t narrow = spans(tiles * split, sms) * spans(n_kb, split) * 62 + (split > 1 ? 800 : 400);
    return wide < narrow;
}

// A's rows as columns, B's as lanes; the K blocks of a tile are split over up to
// kF8MaxSplit CTAs while SMs are free.
template <int NT>
fp4q_status launch_f8_narrow(const Fp8Operand& a, const Fp8Operand& b, int64_t K, Fp8GemmParams p, int sms,
                             cudaStream_t s) {
    using G = F8Narrow<NT>;
    auto kern = fp8_gemm_narrow_kernel<NT>;
    static std::atomic<uint64_t> done{0};
    fp4q_status st = ensure_smem(kern, G::smem, done);
    if (st != FP4Q_OK) return st;
    f8_operands(p, b, a, kF8Lanes, NT);
    if (p.n_tiles >= kMaxDim / kF8MaxSplit) return FP4Q_ERR_UNSUPPORTED;
    CUtensorMap map_l, map_c;
    if ((st = make_f8_map(&map_l, b.codes, b.rows, K, b.ld, kF8Lanes)) != FP4Q_OK) return st;
    if ((st = make_f8_map(&map_c, a.codes, a.rows, K, a.ld, NT)) != FP4Q_OK) return st;
    p.split = (int32_t)f8_split(p.n_tiles, p.n_kb, sms);
    return launch_cluster(kern, p.n_tiles * p.split, p.split, G::threads, G::smem, s, map_l, map_c, p);
}

// 128 x 256 tiles, persistent.
template <bool VEC>
fp4q_status launch_f8_wide(const Fp8Operand& a, const Fp8Operand& b, int64_t K, Fp8GemmParams p, int sms,
                           cudaStream_t s) {
    auto kern = fp8_gemm_wide_kernel<VEC>;
    static std::atomic<uint64_t> done{0};
    fp4q_status st = ensure_smem(kern, F8Wide::smem, done);
    if (st != FP4Q_OK) return st;
    f8_operands(p, a, b, kF8Lanes, F8Wide::n);
    CUtensorMap map_a, map_b, map_d;
    if ((st = make_f8_map(&map_a, a.codes, a.rows, K, a.ld, kF8Lanes)) != FP4Q_OK) return st;
    if ((st = make_f8_map(&map_b, b.codes, b.rows, K, b.ld, F8Wide::n)) != FP4Q_OK) return st;
    map_d = map_a;  // a placeholder where no TMA store is made
    // the TMA writes whole 16-byte pieces: a row of D has to end with one
    const int64_t es = p.out_bf16 ? 2 : 4;
    p.tma_store = p.ldd * es % 16 == 0 && b.rows * es % 16 == 0;
    if (p.tma_store && (st = make_f8_out_map(&map_d, p.d, a.rows, b.rows, p.ldd, p.out_bf16)) != FP4Q_OK) return st;
    const int grid = (int)std::min<int64_t>(p.n_tiles, sms);
    return launch(kern, grid, F8Wide::threads, F8Wide::smem, s, map_a, map_b, map_d, p);
}

fp4q_status check_cache(const fp4q_kv_cache* c, KvCacheView* v) {
    if (!c) return FP4Q_ERR_INVALID_ARG;
    if (c->num_pages < 0 || c->num_kv_heads <= 0 || c->table_stride < 0 || c->page_size <= 0 || c->head_dim <= 0)
        return FP4Q_ERR_INVALID_ARG;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return FP4Q_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return FP4Q_ERR_UNSUPPORTED;
    // rows of the code matrix [pages * heads * page_size, head_dim] are counted in 31 bits
    if (c->num_kv_heads > 65536 || c->num_pages >= kMaxDim ||
        c->num_pages * c->num_kv_heads >= kMaxDim / c->page_size || c->table_stride >= kMaxDim)
        return FP4Q_ERR_UNSUPPORTED;
    v->k = c->k;
    v->v = c->v;
    v->k_scale = c->k_scale;
    v->v_scale = c->v_scale;
    v->num_pages = c->num_pages;
    v->heads = c->num_kv_heads;
    v->page = c->page_size;
    v->dim = c->head_dim;
    v->table = c->block_table;
    v->table_stride = c->table_stride;
    return FP4Q_OK;
}

// The cache's pointers, once there is work for them.
fp4q_status check_cache_pointers(const KvCacheView& v) {
    if (!v.k || !v.v || !v.k_scale || !v.v_scale || !v.table || v.num_pages == 0 || v.table_stride == 0)
        return FP4Q_ERR_INVALID_ARG;
    if (!aligned(v.k, 16) || !aligned(v.v, 16) || !aligned(v.k_scale, 4) || !aligned(v.v_scale, 4) ||
        !aligned(v.table, 4))
        return FP4Q_ERR_ALIGNMENT;
    return FP4Q_OK;
}

}  // namespace

FP4Q_API fp4q_status fp4q_quantize_fp8(const void* x, int64_t M, int64_t K, int64_t ldx, fp4q_fp8_block block,
                                       uint8_t* codes, int64_t ldc, float* scales, int64_t lds, uint8_t* codes_t,
                                       int64_t ldct, float* scales_t, int64_t ldst, fp4q_stream_t stream) {
    if (M < 0 || K <= 0 || ldx < K || !valid_block(block)) return FP4Q_ERR_INVALID_ARG;
    if (M >= kMaxDim || K >= kMaxDim || ldx >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
    if (M == 0) return FP4Q_OK;
    if (!x || (!codes && !codes_t)) return FP4Q_ERR_INVALID_ARG;
    if (ldx % 8 != 0 || !aligned(x, 16)) return FP4Q_ERR_ALIGNMENT;
    fp4q_status st;
    if (codes && (st = check_fp8(codes, M, K, ldc, scales, lds, block)) != FP4Q_OK) return st;
    if (codes_t && (st = check_fp8(codes_t, K, M, ldct, scales_t, ldst, block)) != FP4Q_OK) return st;
    Fp8QuantParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.M = M;
    p.K = K;
    p.ldx = ldx;
    p.codes = codes;
    p.ldc = ldc;
    p.scales = scales;
    p.lds = lds;
    p.codes_t = codes_t;
    p.ldct = ldct;
    p.scales_t = scales_t;
    p.ldst = ldst;
    p.n_kb = spans(K, kFp8Block);
    if (block == FP4Q_FP8_ROW && !codes_t) {
        int sms = 0;
        if ((st = sm_count(&sms)) != FP4Q_OK) return st;
        p.n_items = spans(M, kFp8RowBlocks) * p.n_kb;
        if (p.n_items >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
        const int64_t per = kFp8RowThreads / 16;
        const int grid = (int)std::min<int64_t>(spans(p.n_items, per), (int64_t)sms * 4);
        return launch(fp8_row_kernel, grid, kFp8RowThreads, 0, (cudaStream_t)stream, p);
    }
    take_skip(p);
    p.n_items = spans(M, kFp8Block) * p.n_kb;
    if (p.n_items >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
    return block == FP4Q_FP8_TILE ? launch_fp8_tile<true>(p, (cudaStream_t)stream) : launch_fp8_tile<false>(p, (cudaStream_t)stream);
}

FP4Q_API fp4q_status fp4q_gemm_fp8(const uint8_t* a_codes, int64_t lda, const float* a_scales, int64_t ldas,
                                   const uint8_t* b_codes, int64_t ldb, const float* b_scales, int64_t ldbs,
                                   fp4q_fp8_block b_block, int64_t M, int64_t N, int64_t K, void* d, int64_t ldd,
                                   int d_bf16, fp4q_stream_t stream) {
    if (M < 0 || N <= 0 || K <= 0 || ldd < N || !valid_block(b_block)) return FP4Q_ERR_INVALID_ARG;
    if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim || ldd >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
    if (d_bf16 != 0 && d_bf16 != 1) return FP4Q_ERR_INVALID_ARG;
    if (M == 0) return FP4Q_OK;
    fp4q_status st;
    if ((st = check_fp8(a_codes, M, K, lda, a_scales, ldas, FP4Q_FP8_ROW)) != FP4Q_OK) return st;
    if ((st = check_fp8(b_codes, N, K, ldb, b_scales, ldbs, b_block)) != FP4Q_OK) return st;
    if (!d) return FP4Q_ERR_INVALID_ARG;
    if (!aligned(d, 16)) return FP4Q_ERR_ALIGNMENT;
    int sms = 0;
    if ((st = sm_count(&sms)) != FP4Q_OK) return st;
    Fp8Operand a{a_codes, M, lda, a_scales, ldas, 0}, b{b_codes, N, ldb, b_scales, ldbs, b_block == FP4Q_FP8_TILE};
    Fp8GemmParams p{};
    p.n_kb = (int32_t)spans(K, kFp8Block);
    p.d = d;
    p.ldd = ldd;
    p.out_bf16 = d_bf16;
    p.split = 1;
    take_skip(p);
    if (f8_take_wide(M, N, p.n_kb, b.tile != 0, sms)) {
        if (b.tile) return launch_f8_wide<false>(a, b, K, p, sms, (cudaStream_t)stream);
        return launch_f8_wide<true>(a, b, K, p, sms, (cudaStream_t)stream);
    }
    if (M <= 16) return launch_f8_narrow<16>(a, b, K, p, sms, (cudaStream_t)stream);
    if (M <= 32) return launch_f8_narrow<32>(a, b, K, p, sms, (cudaStream_t)stream);
    if (M <= 64) return launch_f8_narrow<64>(a, b, K, p, sms, (cudaStream_t)stream);
    return launch_f8_narrow<128>(a, b, K, p, sms, (cudaStream_t)stream);
}

FP4Q_API fp4q_status fp4q_kv_append_fp8(const void* k, int64_t ldk, const void* v, int64_t ldv, int64_t tokens,
                                        const fp4q_kv_cache* cache, const int32_t* cu_new, const int32_t* lens,
                                        int64_t batch, int64_t max_new, fp4q_stream_t stream) {
    KvAppendParams p{};
    fp4q_status st = check_cache(cache, &p.c);
    if (st != FP4Q_OK) return st;
    const int64_t row = (int64_t)p.c.heads * p.c.dim;
    if (tokens < 0 || batch < 0 || max_new < 0 || ldk < row || ldv < row) return FP4Q_ERR_INVALID_ARG;
    if (tokens >= kMaxDim || batch >= kMaxDim || max_new >= kMaxDim || ldk >= kMaxDim || ldv >= kMaxDim)
        return FP4Q_ERR_UNSUPPORTED;
    if (tokens == 0 || batch == 0 || max_new == 0) return FP4Q_OK;
    if (!k || !v || !cu_new || !lens) return FP4Q_ERR_INVALID_ARG;
    if ((st = check_cache_pointers(p.c)) != FP4Q_OK) return st;
    if (ldk % 8 != 0 || ldv % 8 != 0 || !aligned(k, 16) || !aligned(v, 16) || !aligned(cu_new, 4) || !aligned(lens, 4))
        return FP4Q_ERR_ALIGNMENT;
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.ldk = ldk;
    p.ldv = ldv;
    p.tokens = tokens;
    p.cu = cu_new;
    p.lens = lens;
    p.max_new = max_new;
    const int64_t pages = (max_new + p.c.page - 2) / p.c.page + 1;
    if (pages * batch >= kMaxDim / (2 * p.c.heads)) return FP4Q_ERR_UNSUPPORTED;
    p.pages_per_seq = (uint32_t)pages;
    p.per_row_log2 = p.c.dim == 64 ? 3 : p.c.dim == 128 ? 4 : 5;
    // threads for a page's rows, or for the few that a sequence can bring
    const int64_t pieces = std::min<int64_t>(p.c.page, max_new) << p.per_row_log2;
    const int threads = (int)std::min<int64_t>(kKvMaxThreads, std::max<int64_t>(spans(pieces, kKvPieces * 32) * 32, std::min<int64_t>(64, spans(pieces, 32) * 32)));
    return launch(kv_append_kernel, (int)(2 * p.c.heads * pages * batch), threads, 0, (cudaStream_t)stream, p);
}

namespace {

// How the rows and keys of a call are cut.  The keys of a row tile are split
// where there are too few tiles to fill the GPU (by the lengths' bound, since
// the lengths are on the device).
struct AttnPlan {
    bool tile;     // attn_tile_kernel
    bool cluster;  // the splits of a row tile join within a cluster
    int64_t tile_rows, row_tiles, splits, chunk, slot_rows;
    size_t ws_bytes;
};

constexpr int64_t kAttnMost = (int64_t)1 << 30;
constexpr int64_t kAttnCluster = 8;

// Keys of one split of attn_tile_kernel: as many splits as fill the GPU, of 512
// keys at least (a tile of 128 keys takes 1.45 us, the join 4 us and more).
int64_t attn_tile_chunk(int64_t items, int64_t max_len, int sms) {
    const int64_t want = std::max<int64_t>(1, sms / items);
    return std::max<int64_t>(512, spans(spans(max_len, want), kTileKeys) * kTileKeys);
}

// Whether attn_tile_kernel (128 rows a CTA) is the faster one, by what it and
// attn_rows_kernel (16 rows) took on one B200 at D = 128, in ns: 7000 and 1450 a
// wave and 128 keys, with 4000 and 0.35 a row of a slot where the keys are split,
// against 6000, 18 a key for each of the 3 CTAs an SM holds, and 64 a row tile for
// the join.  Measured, in us (tile / rows), 8 K/V heads of 4: 32 queries over 512
// keys 13.6 / 13.1, 64 over 512 13.7 / 19.9, 16 over 4096 17.5 / 17.2, 32 over 4096
// 19.5 / 25.9, 64 over 4096 20.8 / 40.2 (keys not split 51.7), 128 over 4096 30.0 /
// 62.8 (51.8), two of 100 over 4096 44.0 / 77.1 (51.9), two of 400 92 / 207; one K/V
// head, 64 over 4096 16.9 / 14.5; 16 sequences of 8 queries in groups of 8 over 2000
// 29.8 / 46.4.
bool attn_take_tile(int64_t row_items, int64_t tile_items, int64_t max_len, int64_t rows, int sms) {
    if (rows <= kAttnRows) return false;
    const double by_rows = 6000.0 + 18.0 * row_items * max_len / (3.0 * sms) + (row_items < 3 * (int64_t)sms ? 64.0 * row_items : 0.0);
    const int64_t chunk = attn_tile_chunk(tile_items, max_len, sms), splits = std::max<int64_t>(1, spans(max_len, chunk));
    const double by_tile = 7000.0 + 1450.0 * spans(tile_items * splits, sms) * spans(std::min(max_len, chunk), kTileKeys) +
                           (splits > 1 ? 4000.0 + 0.35 * tile_items * splits * std::min<int64_t>(rows, kTileRows) : 0.0);
    return by_tile < by_rows;
}

// Rows and keys are counted in 31 bits, with room for the last tile, and so are
// the row tiles of a call (of 128 rows here; the kernel of 16 needs more room,
// attn_plan).  Everything else that attn_plan multiplies stays within 64 bits then.
fp4q_status attn_bounds(int64_t batch, int64_t max_q, int64_t max_len, int64_t q_heads, int64_t kv_heads) {
    if (max_len > kAttnMost || max_q > kAttnMost / (q_heads / kv_heads)) return FP4Q_ERR_UNSUPPORTED;
    const int64_t heads = batch * kv_heads;  // (each below 2^31)
    if (heads >= kMaxDim || heads * spans(max_q * (q_heads / kv_heads), kTileRows) >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
    return FP4Q_OK;
}

// For sizes that attn_bounds takes.
fp4q_status attn_plan(int64_t batch, int64_t max_q, int64_t max_len, int64_t q_heads, int64_t kv_heads, int64_t dim,
                      int sms, AttnPlan* out) {
    AttnPlan a{};
    const int64_t rows = max_q * (q_heads / kv_heads), heads = batch * kv_heads;
    a.tile = dim <= 128 && attn_take_tile(heads * spans(rows, kAttnRows), heads * spans(rows, kTileRows), max_len, rows, sms);
    a.tile_rows = a.tile ? kTileRows : kAttnRows;
    a.row_tiles = spans(rows, a.tile_rows);
    a.slot_rows = std::min<int64_t>(a.tile_rows, rows);
    if (a.row_tiles >= kMaxDim / kv_heads || a.row_tiles * kv_heads >= kMaxDim / batch) return FP4Q_ERR_UNSUPPORTED;
    const int64_t items = batch * kv_heads * a.row_tiles;
    if (a.tile) {
        a.chunk = attn_tile_chunk(items, max_len, sms);
    } else {  // three CTAs fit on an SM
        const int64_t want = std::max<int64_t>(1, spans(3 * (int64_t)sms, items));
        a.chunk = std::min<int64_t>(kAttnMaxChunk, std::max<int64_t>(128, spans(spans(max_len, want), 128) * 128));
    }
    a.splits = std::max<int64_t>(1, spans(max_len, a.chunk));
    // A cluster saves the second launch (4 us of the host's time, none of the GPU's)
    // but holds its CTAs until the last is done: 32 x 8192 keys in clusters of two
    // took 111 us, with the second kernel 85.  So only where all have an SM to
    // themselves.
    a.cluster = !a.tile && a.splits > 1 && a.splits <= kAttnCluster && items * a.splits <= sms;
    if (a.splits >= kMaxDim / items || (a.splits > 1 && items >= kMaxDim / a.tile_rows)) return FP4Q_ERR_UNSUPPORTED;
    a.ws_bytes = a.splits > 1 && !a.cluster ? (size_t)(items * a.splits * a.slot_rows * (dim + 4)) * sizeof(float) : 0;
    *out = a;
    return FP4Q_OK;
}

// One side of a cache as [pages * heads * page_size, head_dim] codes, in boxes of
// 16 rows x min(head_dim, 128) bytes (swizzled by the box's width).
fp4q_status make_kv_map(CUtensorMap* map, const KvCacheView& c, const uint8_t* codes) {
    EncodeTiledFn enc;
    fp4q_status st = encode_fn(&enc);
    if (st != FP4Q_OK) return st;
    cuuint64_t dims[2] = {(cuuint64_t)c.dim, (cuuint64_t)(c.num_pages * c.heads * c.page)};
    cuuint64_t strides[1] = {(cuuint64_t)c.dim};
    cuuint32_t box[2] = {(cuuint32_t)std::min(c.dim, 128), (cuuint32_t)kAttnStep};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, c.dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FP4Q_OK : FP4Q_ERR_CUDA;
}

AttnSplit attn_split(const AttnPlan& a, void* ws) {
    return {(uint32_t)a.row_tiles, (uint32_t)a.splits, (int32_t)a.chunk, (uint32_t)a.tile_rows, (uint32_t)a.slot_rows,
            a.ws_bytes > 0 ? static_cast<float*>(ws) : nullptr};
}

template <int D, bool SPLIT>
fp4q_status launch_attn_tile(const AttnParams& p, const AttnPlan& a, void* ws, cudaStream_t s) {
    using G = AttnTileGeo<D>;
    const AttnSplit sp = attn_split(a, ws);
    auto kern = attn_tile_kernel<D, SPLIT>;
    static std::atomic<uint64_t> done{0};
    fp4q_status st = ensure_smem(kern, G::smem, done);
    if (st != FP4Q_OK) return st;
    CUtensorMap map_k, map_v;
    if ((st = make_kv_map(&map_k, p.c, p.c.k)) != FP4Q_OK || (st = make_kv_map(&map_v, p.c, p.c.v)) != FP4Q_OK) return st;
    const int64_t items = p.batch * p.c.heads * a.row_tiles;
    st = launch(kern, (int)(items * a.splits), G::threads, G::smem, s, map_k, map_v, p, sp);
    if (st != FP4Q_OK || a.ws_bytes == 0) return st;
    return launch(attn_join_kernel<D>, (int)(items * a.slot_rows), 128, 0, s, p, sp);
}

template <int D>
fp4q_status launch_attn(const AttnParams& p, const AttnPlan& a, void* ws, cudaStream_t s) {
    using G = AttnGeo<D>;
    const AttnSplit sp = attn_split(a, ws);
    auto kern = attn_rows_kernel<D>;
    static std::atomic<uint64_t> done{0};
    fp4q_status st = ensure_smem(kern, G::smem, done);
    if (st != FP4Q_OK) return st;
    CUtensorMap map_k, map_v;
    if ((st = make_kv_map(&map_k, p.c, p.c.k)) != FP4Q_OK || (st = make_kv_map(&map_v, p.c, p.c.v)) != FP4Q_OK) return st;
    const int64_t items = p.batch * p.c.heads * a.row_tiles;
    st = launch_cluster(kern, items * a.splits, a.cluster ? (int)a.splits : 1, 32 * G::warps, G::smem, s, map_k, map_v, p, sp);
    if (st != FP4Q_OK || a.ws_bytes == 0) return st;
    return launch(attn_join_kernel<D>, (int)(items * a.slot_rows), 128, 0, s, p, sp);
}

}  // namespace

FP4Q_API size_t fp4q_attention_fp8_workspace_bytes(int64_t batch, int64_t max_q, int64_t max_len, int32_t num_q_heads,
                                                   int32_t num_kv_heads, int32_t head_dim) {
    const size_t bad = (size_t)-1;
    if (batch < 0 || max_q < 0 || max_len < 0 || num_kv_heads <= 0 || num_q_heads <= 0 ||
        num_q_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256) || batch >= kMaxDim || max_q >= kMaxDim || max_len >= kMaxDim)
        return bad;
    if (batch == 0 || max_q == 0) return 0;
    int sms = 0;
    AttnPlan a;
    if (attn_bounds(batch, max_q, max_len, num_q_heads, num_kv_heads) != FP4Q_OK || sm_count(&sms) != FP4Q_OK ||
        attn_plan(batch, max_q, max_len, num_q_heads, num_kv_heads, head_dim, sms, &a) != FP4Q_OK)
        return bad;
    return a.ws_bytes;
}

FP4Q_API fp4q_status fp4q_attention_fp8(const void* q, int64_t ldq, int64_t tokens, int32_t num_q_heads,
                                        const fp4q_kv_cache* cache, const int32_t* cu_q, const int32_t* lens,
                                        int64_t batch, int64_t max_q, int64_t max_len, int causal,
                                        float softmax_scale, void* o, int64_t ldo, float* lse, void* workspace,
                                        size_t workspace_bytes, fp4q_stream_t stream) {
    AttnParams p{};
    fp4q_status st = check_cache(cache, &p.c);
    if (st != FP4Q_OK) return st;
    if (num_q_heads <= 0 || num_q_heads % p.c.heads != 0 || tokens < 0 || batch < 0 || max_q < 0 || max_len < 0 ||
        (causal != 0 && causal != 1) || !std::isfinite(softmax_scale))
        return FP4Q_ERR_INVALID_ARG;
    const int64_t row = (int64_t)num_q_heads * p.c.dim;
    if (ldq < row || ldo < row) return FP4Q_ERR_INVALID_ARG;
    if (tokens >= kMaxDim || batch >= kMaxDim || max_q >= kMaxDim || max_len >= kMaxDim || ldq >= kMaxDim ||
        ldo >= kMaxDim)
        return FP4Q_ERR_UNSUPPORTED;
    if (tokens == 0 || batch == 0 || max_q == 0) return FP4Q_OK;
    if (!q || !o || !cu_q || !lens) return FP4Q_ERR_INVALID_ARG;
    if ((st = check_cache_pointers(p.c)) != FP4Q_OK) return st;
    if (ldq % 8 != 0 || ldo % 8 != 0 || !aligned(q, 16) || !aligned(o, 16) || !aligned(cu_q, 4) ||
        !aligned(lens, 4) || !aligned(lse, 4))
        return FP4Q_ERR_ALIGNMENT;
    p.q = static_cast<const uint16_t*>(q);
    p.ldq = ldq;
    p.tokens = tokens;
    p.q_heads = num_q_heads;
    p.group = num_q_heads / p.c.heads;
    p.cu = cu_q;
    p.lens = lens;
    p.batch = batch;
    p.max_q = max_q;
    p.max_len = max_len;
    p.causal = causal;
    p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
    p.o = static_cast<uint16_t*>(o);
    p.ldo = ldo;
    p.lse = lse;
    int sms = 0;
    AttnPlan a;
    if ((st = attn_bounds(batch, max_q, max_len, num_q_heads, p.c.heads)) != FP4Q_OK) return st;
    if ((st = sm_count(&sms)) != FP4Q_OK) return st;
    if ((st = attn_plan(batch, max_q, max_len, num_q_heads, p.c.heads, p.c.dim, sms, &a)) != FP4Q_OK) return st;
    if (a.ws_bytes > 0) {
        if (!workspace || workspace_bytes < a.ws_bytes) return FP4Q_ERR_INVALID_ARG;
        if (!aligned(workspace, 16)) return FP4Q_ERR_ALIGNMENT;
    }
    take_skip(p);
    if (a.tile)
        return a.splits > 1 ? (p.c.dim == 64 ? launch_attn_tile<64, true> : launch_attn_tile<128, true>)(p, a, workspace, (cudaStream_t)stream)
                            : (p.c.dim == 64 ? launch_attn_tile<64, false> : launch_attn_tile<128, false>)(p, a, workspace, (cudaStream_t)stream);
    if (p.c.dim == 64) return launch_attn<64>(p, a, workspace, (cudaStream_t)stream);
    if (p.c.dim == 128) return launch_attn<128>(p, a, workspace, (cudaStream_t)stream);
    return launch_attn<256>(p, a, workspace, (cudaStream_t)stream);
}

#ifdef FP4Q_TEST_HOOKS
// Test build only (not declared in include/fp4q.h): makes CTA 0 of the next launch
// of the two-way quantizer, the FP8 GEMM or the cache attention arm its barrier for
// copies number i (a tile, a K block, a turn of 32 keys or a tile of 128) and never
// issue them, so that the bounded waits for them run out.
FP4Q_API void fp4q_test_skip_copy(int64_t i) { g_test_skip_copy.store(i); }
#endif
