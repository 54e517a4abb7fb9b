// Mixture-of-experts layer for a few tokens with Q4_0 experts and Q8_0 activations:
//   router   l = x . Wr^T, the top_k largest logits, p = softmax over them or over all
//   experts  g, u = xq . Wg^T, xq . Wu^T;  h = g / (1 + exp(-g)) * u;  hq = Q8_0(h)
//   output   y[t] = sum over slots s of p[t][s] * (hq[t][s] . Wd[e(t, s)]^T)
// with the block dots of w4a8_gemm (exact integers, rescaled per 32-block in f32).
#pragma once

#include "device_common.cuh"

namespace w4a8 {
namespace moe {

constexpr int kMaxExperts = 256;
constexpr int kMaxTopK = 16;

// ------------------------------------------------------------------ router
// Order-preserving map of a float to an unsigned key (larger float, larger key; a NaN of
// either sign maps to 0, below every number).
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0u;
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <bool BF16>
__device__ __forceinline__ void load8f(const void* p, int64_t idx, float (&v)[8]) {
    float a[4], b[4];
    load4<BF16>(p, idx, a);
    load4<BF16>(p, idx + 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

// One CTA per token: a warp per expert for the logits, then one warp for the top_k.
template <bool XB, bool WB>
__global__ void __launch_bounds__(256) route_kernel(int E, int H, int top_k, int renorm, const void* __restrict__ x,
                                                    const void* __restrict__ wr, int* __restrict__ ids,
                                                    float* __restrict__ weights) {
    __shared__ float logit[kMaxExperts];
    const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = warp; e < E; e += 8) {
        float s = 0.0f;
        for (int k = lane * 8; k < H; k += 256) {
            float a[8], b[8];
            load8f<XB>(x, int64_t(t) * H + k, a);
            load8f<WB>(wr, int64_t(e) * H + k, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) logit[e] = s;
    }
    __syncthreads();
    if (warp != 0) return;
    uint32_t key[kMaxExperts / 32];
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) key[i] = lane + 32 * i < E ? order_key(logit[lane + 32 * i]) : 0u;
    uint32_t taken = 0u;  // bit i: this lane's expert lane + 32 i is chosen
    float top = 0.0f, sum = 0.0f, mine = 0.0f;
    for (int s = 0; s < top_k; ++s) {
        uint32_t best = 0u;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = kMaxExperts / 32 - 1; i >= 0; --i)  // the lowest index among equals
            if (lane + 32 * i < E && !((taken >> i) & 1u) && key[i] >= best) {
                best = key[i];
                at = lane + 32 * i;
            }
        const uint32_t m = __reduce_max_sync(0xffffffffu, at != 0x7fffffff ? best : 0u);
        const int e = int(__reduce_min_sync(0xffffffffu, unsigned(at != 0x7fffffff && best == m ? at : 0x7fffffff)));
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        const float l = logit[e];
        if (s == 0) top = l;
        const float p = expf(l - top);
        sum += p;
        if (lane == s) mine = p;
        if (lane == 0) ids[int64_t(t) * top_k + s] = e;
    }
    if (!renorm) {
        sum = 0.0f;
        for (int e = lane; e < E; e += 32) sum += expf(logit[e] - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < top_k) weights[int64_t(t) * top_k + lane] = __fdiv_rn(mine, sum);
}

// ------------------------------------------------------------------ experts
// Dot of one Q4_0 row with one Q8_0 row of B blocks, by one warp (the result in every lane).
__device__ __forceinline__ float warp_dot(const uint8_t* q, const uint16_t* d, const int8_t* xq, const float* xd, int B,
                                          int lane) {
    float acc = 0.0f;
    for (int b = lane; b < B; b += 32) {
        const uint4 w = reinterpret_cast<const uint4*>(q)[b];
        const uint4 lo = reinterpret_cast<const uint4*>(xq)[2 * b], hi = reinterpret_cast<const uint4*>(xq)[2 * b + 1];
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w}, xl[4] = {lo.x, lo.y, lo.z, lo.w}, xh[4] = {hi.x, hi.y, hi.z, hi.w};
        int s = 0;  // 16 * sum (q - 8) * xq
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s = __dp4a(int((ww[i] << 4 & 0xF0F0F0F0u) ^ 0x80808080u), int(xl[i]), s);
            s = __dp4a(int((ww[i] & 0xF0F0F0F0u) ^ 0x80808080u), int(xh[i]), s);
        }
        acc = fmaf(float(s), __fmul_rn(__half2float(__ushort_as_half(d[b])) * 0.0625f, xd[b]), acc);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    return acc;
}

// h[t][s][i], one warp per value; slots without an expert give 0.
__global__ void __launch_bounds__(256) gate_up_simple_kernel(int64_t n, int E, int H, int I, int top_k,
                                                             const int8_t* xq, const float* xd, const int* ids,
                                                             const uint8_t* wq, const uint16_t* wd, float* h) {
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> 5;
    if (i >= n) return;
    const int64_t slot = i / I, t = slot / top_k;
    const int e = ids[slot], B = H / 32, lane = threadIdx.x & 31;
    float v = 0.0f;
    if (e >= 0 && e < E) {
        const int64_t r = int64_t(e) * 2 * I + i % I;
        const float g = warp_dot(wq + r * (H / 2), wd + r * B, xq + t * H, xd + t * B, B, lane);
        const float u = warp_dot(wq + (r + I) * (H / 2), wd + (r + I) * B, xq + t * H, xd + t * B, B, lane);
        v = __fmul_rn(__fdiv_rn(g, 1.0f + expf(-g)), u);
    }
    if (lane == 0) h[i] = v;
}

// y[t][n], one warp per value.
__global__ void __launch_bounds__(256) down_simple_kernel(int64_t n, int E, int H, int I, int top_k, const int8_t* hq,
                                                          const float* hd, const int* ids, const float* weights,
                                                          const uint8_t* wq, const uint16_t* wd, void* y,
                                                          int out_bf16) {
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) >> 5;
    if (i >= n) return;
    const int64_t t = i / H;
    const int B = I / 32, lane = threadIdx.x & 31;
    float v = 0.0f;
    for (int s = 0; s < top_k; ++s) {
        const int64_t slot = t * top_k + s;
        const int e = ids[slot];
        if (e < 0 || e >= E) continue;
        const int64_t r = int64_t(e) * H + i % H;
        v = fmaf(weights[slot], warp_dot(wq + r * (I / 2), wd + r * B, hq + slot * I, hd + slot * B, B, lane), v);
    }
    if (lane == 0) {
        if (out_bf16)
            reinterpret_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
        else
            reinterpret_cast<float*>(y)[i] = v;
    }
}

}  // namespace moe
}  // namespace w4a8
