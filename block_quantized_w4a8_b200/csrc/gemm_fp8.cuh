// FP8 (e4m3) matmul with 128-wide blocks: activations with one scale per row and block of
// the contracted axis, weights with one scale per 128 x 128 tile.
#pragma once

#include "fp8_quant.cuh"

namespace w4a8 {
namespace fp8 {

__device__ __forceinline__ float decode(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// One thread per output: out[m][c] = sum_b sa[b][m] * sw * sum_{r in b} a[m][r] * w(r, c), the
// contracted axis r of length R, output columns c < C. TRANS = false: w(r, c) = q[c * R + r]
// (forward: C = N, R = K); true: q[r * C + c] (input gradient: C = K, R = N).
template <bool TRANS>
__global__ void __launch_bounds__(256) gemm_simple_kernel(int M, int C, int R, const uint8_t* __restrict__ a, int pitch,
                                                          const float* __restrict__ sa, int64_t sarow, int64_t sablk,
                                                          const uint8_t* __restrict__ q, const float* __restrict__ sw,
                                                          int swcols, void* __restrict__ out, Epilogue epi) {
    const int c = blockIdx.y * 32 + (threadIdx.x & 31);
    const int m = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (c >= C || m >= M) return;
    float acc = 0.0f;
    for (int b = 0; b * kBlk < R; ++b) {
        float p = 0.0f;
        const int r1 = min(R, (b + 1) * kBlk);
        for (int r = b * kBlk; r < r1; ++r)
            p = fmaf(decode(a[int64_t(m) * pitch + r]), decode(TRANS ? q[int64_t(r) * C + c] : q[int64_t(c) * R + r]), p);
        const float w = TRANS ? sw[int64_t(b) * swcols + c / kBlk] : sw[int64_t(c / kBlk) * swcols + b];
        acc = fmaf(p, __fmul_rn(sa[m * sarow + b * sablk], w), acc);
    }
    epi_store(out, int64_t(m) * C + c, c, acc, epi);
}

}  // namespace fp8
}  // namespace w4a8
