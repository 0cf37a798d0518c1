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
        p.n_items = M * p.n_kb;
        const int64_t per = kFp8RowThreads / 16;
        const int grid = (int)std::min<int64_t>(spans(p.n_items, per), (int64_t)sms * 8);
        return launch(fp8_row_kernel, grid, kFp8RowThreads, 0, (cudaStream_t)stream, p);
    }
    p.n_items = spans(M, kFp8Block) * p.n_kb;
    if (p.n_items >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
    if (block == FP4Q_FP8_TILE)
        return launch(fp8_tile_kernel<true>, (int)p.n_items, kFp8TileThreads, 0, (cudaStream_t)stream, p);
    return launch(fp8_tile_kernel<false>, (int)p.n_items, kFp8TileThreads, 0, (cudaStream_t)stream, p);
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
    Fp8GemmParams p{};
    p.a = a_codes;
    p.b = b_codes;
    p.sa = a_scales;
    p.sb = b_scales;
    p.lda = lda;
    p.ldb = ldb;
    p.ldas = ldas;
    p.ldbs = ldbs;
    p.M = M;
    p.N = N;
    p.K = K;
    p.d = d;
    p.ldd = ldd;
    p.out_bf16 = d_bf16;
    p.b_tile = b_block == FP4Q_FP8_TILE;
    p.n_nt = spans(N, kFp8SimpleTile);
    const int64_t tiles = spans(M, kFp8SimpleTile) * p.n_nt;
    if (tiles >= kMaxDim) return FP4Q_ERR_UNSUPPORTED;
    return launch(fp8_gemm_simple_kernel, (int)tiles, 256, 0, (cudaStream_t)stream, p);
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
    p.pages_per_seq = (max_new + p.c.page - 2) / p.c.page + 1;
    if (p.pages_per_seq * batch >= kMaxDim / (2 * p.c.heads)) return FP4Q_ERR_UNSUPPORTED;
    return launch(kv_append_kernel, (int)(2 * p.c.heads * p.pages_per_seq * batch), kKvThreads, 0,
                  (cudaStream_t)stream, p);
}

FP4Q_API size_t fp4q_attention_fp8_workspace_bytes(int64_t batch, int64_t max_q, int64_t max_len, int32_t num_q_heads,
                                                   int32_t num_kv_heads, int32_t head_dim) {
    if (batch < 0 || max_q < 0 || max_len < 0 || num_kv_heads <= 0 || num_q_heads <= 0 ||
        num_q_heads % num_kv_heads != 0 || head_dim <= 0)
        return (size_t)-1;
    return 0;
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
    const int64_t warps = max_q * batch;
    if (warps >= kMaxDim / num_q_heads) return FP4Q_ERR_UNSUPPORTED;
    const int grid = (int)spans(warps * num_q_heads, 4);
    if (p.c.dim == 64) return launch(attn_simple_kernel<64>, grid, 128, 0, (cudaStream_t)stream, p);
    if (p.c.dim == 128) return launch(attn_simple_kernel<128>, grid, 128, 0, (cudaStream_t)stream, p);
    return launch(attn_simple_kernel<256>, grid, 128, 0, (cudaStream_t)stream, p);
}
