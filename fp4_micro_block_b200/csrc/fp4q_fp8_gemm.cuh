// fp4q_fp8_gemm.cuh -- D = A B^T of E4M3 codes under block-128 scales:
//   D[m, n] = sum_kb SA[kb, m] SB[kb, n] sum_{k in kb} A[m, k] B[n, k]
#pragma once

#include "fp4q_fp8.cuh"

namespace fp4q {

struct Fp8GemmParams {
    const uint8_t *a, *b;
    const float *sa, *sb;
    int64_t lda, ldb, ldas, ldbs;
    int64_t M, N, K;
    void* d;
    int64_t ldd;
    int out_bf16, b_tile;
    int64_t n_nt;
};

constexpr int kFp8SimpleTile = 64;
__global__ void __launch_bounds__(256) fp8_gemm_simple_kernel(const Fp8GemmParams p) {
    __shared__ float as[32][kFp8SimpleTile + 1], bs[32][kFp8SimpleTile + 1];
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / p.n_nt) * kFp8SimpleTile, n0 = (int64_t)(blockIdx.x % p.n_nt) * kFp8SimpleTile;
    float acc[4][4] = {};
    for (int64_t kb = 0; kb * kFp8Block < p.K; ++kb) {
        float sum[4][4] = {};
        for (int k0 = 0; k0 < kFp8Block; k0 += 32) {
            for (int e = threadIdx.x; e < kFp8SimpleTile * 32; e += 256) {
                const int r = e >> 5, k = e & 31;
                const int64_t kk = kb * kFp8Block + k0 + k;
                as[k][r] = m0 + r < p.M && kk < p.K ? e4m3_decode(p.a[(m0 + r) * p.lda + kk]) : 0.0f;
                bs[k][r] = n0 + r < p.N && kk < p.K ? e4m3_decode(p.b[(n0 + r) * p.ldb + kk]) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < 32; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) sum[i][j] = fmaf(as[k][ty + 16 * i], bs[k][tx + 16 * j], sum[i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m < p.M && n < p.N)
                    acc[i][j] = fmaf(sum[i][j], p.sa[kb * p.ldas + m] * p.sb[kb * p.ldbs + (p.b_tile ? n / kFp8Block : n)],
                                     acc[i][j]);
            }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= p.M || n >= p.N) continue;
            if (p.out_bf16)
                static_cast<uint16_t*>(p.d)[m * p.ldd + n] = (uint16_t)bf16x2_pack(acc[i][j], 0.0f);
            else
                static_cast<float*>(p.d)[m * p.ldd + n] = acc[i][j];
        }
}

}  // namespace fp4q
