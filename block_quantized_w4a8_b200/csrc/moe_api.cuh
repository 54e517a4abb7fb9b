// Entry points of the mixture-of-experts layer (argument checks, workspace, launches).
// Included by w4a8.cu, whose helpers it uses.
#pragma once

#include "moe.cuh"

namespace {

inline bool moe_dims_ok(int T, int E, int H, int I, int top_k) {
    return T > 0 && E > 0 && top_k > 0 && dims_ok(H, I) && H % 32 == 0 && I % 32 == 0;
}
inline bool moe_supported(int T, int E, int I, int top_k) {
    return T <= W4A8_MOE_MAX_TOKENS && E <= W4A8_MOE_MAX_EXPERTS && top_k <= W4A8_MOE_MAX_TOPK && top_k <= E &&
           I <= W4A8_MAX_DIM / 2;
}

struct MoeWs {
    int8_t* xq;  // Q8_0 of x
    float* xd;
    float* h;    // experts' activations, one row per slot
    int8_t* hq;  // Q8_0 of h
    float* hd;
    size_t bytes;
};
MoeWs moe_ws(void* ws, int T, int H, int I, int top_k) {
    MoeWs w{};
    char* base = static_cast<char*>(ws);
    const size_t rows = size_t(T) * top_k;
    size_t off = 0;
    w.xq = reinterpret_cast<int8_t*>(base + off); off = align256(off + size_t(T) * H);
    w.xd = reinterpret_cast<float*>(base + off); off = align256(off + size_t(T) * (H / 32) * 4);
    w.h = reinterpret_cast<float*>(base + off); off = align256(off + rows * I * 4);
    w.hq = reinterpret_cast<int8_t*>(base + off); off = align256(off + rows * I);
    w.hd = reinterpret_cast<float*>(base + off); off = align256(off + rows * (I / 32) * 4);
    w.bytes = off;
    return w;
}

w4a8_status check_route(int T, int E, int H, int top_k, const void* x, w4a8_dtype xdt, const void* wr, w4a8_dtype wdt,
                        const void* ids, const void* weights) {
    if (T <= 0 || E <= 0 || top_k <= 0 || !dims_ok(T, H) || H % 32 != 0 || !x || !wr || !ids || !weights)
        return W4A8_ERR_INVALID_ARG;
    if ((xdt != W4A8_F32 && xdt != W4A8_BF16) || (wdt != W4A8_F32 && wdt != W4A8_BF16)) return W4A8_ERR_UNSUPPORTED;
    if (E > W4A8_MOE_MAX_EXPERTS || top_k > W4A8_MOE_MAX_TOPK || top_k > E) return W4A8_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(wr) || !aligned16(ids) || !aligned16(weights)) return W4A8_ERR_MISALIGNED;
    return W4A8_OK;
}

w4a8_status run_route(int T, int E, int H, int top_k, int renorm, const void* x, w4a8_dtype xdt, const void* wr,
                      w4a8_dtype wdt, int* ids, float* weights, cudaStream_t stream) {
    if (xdt == W4A8_BF16) {
        if (wdt == W4A8_BF16)
            moe::route_kernel<true, true><<<T, 256, 0, stream>>>(E, H, top_k, renorm, x, wr, ids, weights);
        else
            moe::route_kernel<true, false><<<T, 256, 0, stream>>>(E, H, top_k, renorm, x, wr, ids, weights);
    } else {
        if (wdt == W4A8_BF16)
            moe::route_kernel<false, true><<<T, 256, 0, stream>>>(E, H, top_k, renorm, x, wr, ids, weights);
        else
            moe::route_kernel<false, false><<<T, 256, 0, stream>>>(E, H, top_k, renorm, x, wr, ids, weights);
    }
    return launch_status();
}

w4a8_status check_moe(int T, int E, int H, int I, int top_k, const void* x, w4a8_dtype dt, const void* ids,
                      const void* weights, const void* gq, const void* gd, const void* dq, const void* dd,
                      w4a8_dtype odt, const void* y, const void* ws, size_t ws_bytes) {
    if (!moe_dims_ok(T, E, H, I, top_k) || !x || !ids || !weights || !gq || !gd || !dq || !dd || !y)
        return W4A8_ERR_INVALID_ARG;
    if (!moe_supported(T, E, I, top_k)) return W4A8_ERR_UNSUPPORTED;
    if ((dt != W4A8_F32 && dt != W4A8_BF16) || (odt != W4A8_F32 && odt != W4A8_BF16)) return W4A8_ERR_UNSUPPORTED;
    for (const void* p : {x, ids, weights, gq, gd, dq, dd, y})
        if (!aligned16(p)) return W4A8_ERR_MISALIGNED;
    if (!ws || ws_bytes < moe_ws(nullptr, T, H, I, top_k).bytes) return W4A8_ERR_WORKSPACE;
    if (!aligned16(ws)) return W4A8_ERR_MISALIGNED;
    return W4A8_OK;
}

w4a8_status run_experts(int T, int E, int H, int I, int top_k, const void* x, w4a8_dtype dt, const int* ids,
                        const float* weights, const uint8_t* gq, const uint16_t* gd, const uint8_t* dq,
                        const uint16_t* dd, w4a8_dtype odt, void* y, void* ws, cudaStream_t stream) {
    const MoeWs w = moe_ws(ws, T, H, I, top_k);
    w4a8_status st = run_quant_rowmajor(x, dt, T, H, w.xq, w.xd, nullptr, stream);
    if (st != W4A8_OK) return st;
    const int64_t nh = int64_t(T) * top_k * I, ny = int64_t(T) * H;
    moe::gate_up_simple_kernel<<<unsigned(cdiv(nh, 8)), 256, 0, stream>>>(nh, E, H, I, top_k, w.xq, w.xd, ids, gq, gd,
                                                                          w.h);
    if ((st = launch_status()) != W4A8_OK) return st;
    st = run_quant_rowmajor(w.h, W4A8_F32, T * top_k, I, w.hq, w.hd, nullptr, stream);
    if (st != W4A8_OK) return st;
    moe::down_simple_kernel<<<unsigned(cdiv(ny, 8)), 256, 0, stream>>>(ny, E, H, I, top_k, w.hq, w.hd, ids, weights, dq,
                                                                       dd, y, odt == W4A8_BF16 ? 1 : 0);
    return launch_status();
}

}  // namespace

extern "C" {

w4a8_status w4a8_moe_route(int T, int E, int H, int top_k, int renorm, const void* x, w4a8_dtype dtype, const void* wr,
                           w4a8_dtype wr_dtype, int32_t* ids, float* weights, cudaStream_t stream) {
    const w4a8_status st = check_route(T, E, H, top_k, x, dtype, wr, wr_dtype, ids, weights);
    if (st != W4A8_OK) return st;
    return run_route(T, E, H, top_k, renorm, x, dtype, wr, wr_dtype, ids, weights, stream);
}

size_t w4a8_moe_workspace_bytes(int T, int E, int H, int I, int top_k) {
    if (!moe_dims_ok(T, E, H, I, top_k) || !moe_supported(T, E, I, top_k)) return 0;
    return moe_ws(nullptr, T, H, I, top_k).bytes;
}

w4a8_status w4a8_moe_q4_0(int T, int E, int H, int I, int top_k, const void* x, w4a8_dtype dtype, const int32_t* ids,
                          const float* weights, const uint8_t* gu_qs, const uint16_t* gu_d, const uint8_t* dn_qs,
                          const uint16_t* dn_d, w4a8_dtype out_dtype, void* y, void* ws, size_t ws_bytes,
                          cudaStream_t stream) {
    const w4a8_status st = check_moe(T, E, H, I, top_k, x, dtype, ids, weights, gu_qs, gu_d, dn_qs, dn_d, out_dtype, y,
                                     ws, ws_bytes);
    if (st != W4A8_OK) return st;
    return run_experts(T, E, H, I, top_k, x, dtype, ids, weights, gu_qs, gu_d, dn_qs, dn_d, out_dtype, y, ws, stream);
}

w4a8_status w4a8_moe_layer_q4_0(int T, int E, int H, int I, int top_k, int renorm, const void* x, w4a8_dtype dtype,
                                const void* wr, w4a8_dtype wr_dtype, const uint8_t* gu_qs, const uint16_t* gu_d,
                                const uint8_t* dn_qs, const uint16_t* dn_d, int32_t* ids, float* weights,
                                w4a8_dtype out_dtype, void* y, void* ws, size_t ws_bytes, cudaStream_t stream) {
    w4a8_status st = check_moe(T, E, H, I, top_k, x, dtype, ids, weights, gu_qs, gu_d, dn_qs, dn_d, out_dtype, y, ws,
                               ws_bytes);
    if (st != W4A8_OK) return st;
    st = check_route(T, E, H, top_k, x, dtype, wr, wr_dtype, ids, weights);
    if (st != W4A8_OK) return st;
    st = run_route(T, E, H, top_k, renorm, x, dtype, wr, wr_dtype, ids, weights, stream);
    if (st != W4A8_OK) return st;
    return run_experts(T, E, H, I, top_k, x, dtype, ids, weights, gu_qs, gu_d, dn_qs, dn_d, out_dtype, y, ws, stream);
}

}  // extern "C"
