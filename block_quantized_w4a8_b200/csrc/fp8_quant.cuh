// FP8 (e4m3) quantisation with blocks of 128: activations with one f32 scale per row and
// 128 columns, weights with one f32 scale per 128 x 128 tile.
//
//   s = max(amax / 448, 2^-126),  q = e4m3(x * (1/s)), each f32 step rounded to nearest,
// where 448 is the largest e4m3 value. The floor on s keeps 1/s finite; a block of zeros
// then has codes 0. amax ignores NaN; a NaN keeps its NaN code (0x7F), an infinity makes the
// block's scale infinite, so either one reaches every output that uses the block.
#pragma once

#include <cuda_fp8.h>

#include "device_common.cuh"

namespace w4a8 {
namespace fp8 {

constexpr int kBlk = 128;  // elements per scale along a row (and rows per weight tile)

__device__ __forceinline__ float block_scale(float amax) {
    return fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f);  // 2^-126
}

// Eight codes of eight values times inv (conversion: nearest even, saturating, NaN kept).
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[2 * i], inv), __fmul_rn(v[2 * i + 1], inv)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Eight consecutive elements idx .. idx+7 of row-major x, zeros from element `left` on.
// VEC: idx is a multiple of 8 and the eight elements are either all inside or all outside.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* x, int64_t idx, int left, float (&v)[8]) {
    if (VEC) {
        float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
        if (left > 0) {
            if (BF16) {
                const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(x) + idx);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // a bf16 is the top half of an f32
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
                return;
            }
            load4<false>(x, idx, a);
            load4<false>(x, idx + 4, b);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0.0f;
            if (i < left)
                v[i] = BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x)[idx + i])
                            : reinterpret_cast<const float*>(x)[idx + i];
        }
    }
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
    return a;
}

// Rows of length L: 8 lanes per 128-block, 16 elements each (half the scale arithmetic per
// element of 16 lanes: the kernel is bound by its instructions, not by the bytes, for bf16).
// Codes at q[m * pitch + k] (pitch a multiple of 16; with a pitch beyond L the rest of the row's
// last 16 are written with zeros), the scale of (row m, block b) at s[m * srow + b * sblk].
// early: the next kernel may start while this one runs (the contraction of the same call, which
// waits before it reads q and s). Not for a caller's q and s: those of one row are also a weight
// of one row, and weights are read before that wait.
// VEC: L a multiple of 16. One block per group of lanes (two or four were no faster). 2048 x 4096
// bf16: 4.8 us, 25 MB at 5.3 TB/s.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) quant_rows_kernel(const void* __restrict__ x, int M, int L, int pitch,
                                                         uint8_t* __restrict__ q, float* __restrict__ s, int64_t srow,
                                                         int64_t sblk, int early) {
    if (early) pdl_launch_dependents();
    const uint32_t nb = uint32_t(L + kBlk - 1) / kBlk, n = uint32_t(M) * nb;  // n < 2^28 per launch
    const uint32_t i = blockIdx.x * 32u + (threadIdx.x >> 3);
    const int lane = threadIdx.x & 7;
    const uint32_t m = i / nb, b = i - m * nb;
    const int k = int(b) * kBlk + lane * 16, left = i < n ? L - k : 0;
    float v[2][8];
    load8<BF16, VEC>(x, int64_t(m) * L + k, left, v[0]);
    load8<BF16, VEC>(x, int64_t(m) * L + k + 8, left - 8, v[1]);
    const float sc = block_scale(warp_max8(fmaxf(amax8(v[0]), amax8(v[1]))));
    if (i >= n) return;
    const float inv = __frcp_rn(sc);
    if (k < L) {
        const uint2 lo = codes8(v[0], inv), hi = codes8(v[1], inv);
        *reinterpret_cast<uint4*>(q + int64_t(m) * pitch + k) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    if (lane == 0) s[m * srow + b * sblk] = sc;
}

// One CTA per 128 x 128 tile of an N x K weight (K a multiple of 16), the tile held in
// registers between the maximum and the codes: each element is read once. 14300 x 4000 f32:
// 42.4 us, 286 MB at the copy rate.
template <bool BF16>
__global__ void __launch_bounds__(256) pack_tile_kernel(const void* __restrict__ w, int N, int K,
                                                        uint8_t* __restrict__ q, float* __restrict__ s) {
    __shared__ float wmax[8];
    const int kb = blockIdx.x, nb = blockIdx.y;
    const int k = kb * kBlk + (threadIdx.x & 15) * 8, r0 = nb * kBlk + (threadIdx.x >> 4);
    float v[8][8];
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        load8<BF16, true>(w, int64_t(r) * K + k, r < N ? K - k : 0, v[i]);
        a = fmaxf(a, amax8(v[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, wmax[i]);
    const float sc = block_scale(a), inv = __frcp_rn(sc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r < N && k < K) *reinterpret_cast<uint2*>(q + int64_t(r) * K + k) = codes8(v[i], inv);
    }
    if (threadIdx.x == 0) s[int64_t(nb) * gridDim.x + kb] = sc;
}

}  // namespace fp8
}  // namespace w4a8
