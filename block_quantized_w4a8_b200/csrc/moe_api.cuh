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
    uint8_t* xq;  // Q8_0 of x and of every slot's h, in the layout of moe.cuh
    float* xd;
    uint8_t* hq;
    float* hd;
    size_t bytes;
};
MoeWs moe_ws(void* ws, int T, int H, int I, int top_k) {
    MoeWs w{};
    char* base = static_cast<char*>(ws);
    const size_t rows = size_t(T) * top_k, hb = moe::padded_blocks(H), ib = moe::padded_blocks(I);
    size_t off = 0;
    w.xq = reinterpret_cast<uint8_t*>(base + off); off = align256(off + T * hb * 32);
    w.xd = reinterpret_cast<float*>(base + off); off = align256(off + T * hb * 4);
    w.hq = reinterpret_cast<uint8_t*>(base + off); off = align256(off + rows * ib * 32);
    w.hd = reinterpret_cast<float*>(base + off); off = align256(off + rows * ib * 4);
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

template <int DEEP>
auto* route_of(bool xb, bool wb) {
    return xb ? (wb ? moe::route_kernel<true, true, true, DEEP> : moe::route_kernel<true, true, false, DEEP>)
              : (wb ? moe::route_kernel<true, false, true, DEEP> : moe::route_kernel<true, false, false, DEEP>);
}

// One launch: the router (wr != nullptr) and the Q8_0 form of x (xq != nullptr).
w4a8_status run_route(int T, int E, int H, int top_k, int renorm, const void* x, w4a8_dtype xdt, const void* wr,
                      w4a8_dtype wdt, int* ids, float* weights, uint8_t* xq, float* xd, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(T) * moe::kRouteCtas);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = moe::kRouteCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = wr ? 1 : 0;
    const bool xb = xdt == W4A8_BF16, wb = wdt == W4A8_BF16;
    auto* kernel = !wr ? (xb ? moe::route_kernel<false, true, false, 1> : moe::route_kernel<false, false, false, 1>)
                       : T >= moe::kShallowTokens ? route_of<4>(xb, wb) : route_of<8>(xb, wb);
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, E, H, top_k, renorm, x, wr, ids, weights, xq, xd));
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

// Tensor maps of Q4_0 rows: codes in boxes of 128 bytes (8 blocks) x 16 rows with the
// 128-byte swizzle; scales in boxes of 8 x 16, when their rows' pitch allows TMA.
bool moe_maps(CUtensorMap* tq, CUtensorMap* ts, int* sc_tma, const uint8_t* q, const uint16_t* d, int64_t rows, int K) {
    *sc_tma = K % 256 == 0 ? 1 : 0;
    memset(ts, 0, sizeof(*ts));
    return encode_2d(tq, q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(K / 2), uint64_t(rows), uint64_t(K / 2), 128, 16,
                     CU_TENSOR_MAP_SWIZZLE_128B) &&
           (!*sc_tma || encode_2d(ts, d, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, uint64_t(K / 32), uint64_t(rows),
                                  uint64_t(K / 32) * 2, 8, 16));
}

w4a8_status run_experts(int T, int E, int H, int I, int top_k, const int* ids, const float* weights, const uint8_t* gq,
                        const uint16_t* gd, const uint8_t* dq, const uint16_t* dd, w4a8_dtype odt, void* y,
                        const MoeWs& w, cudaStream_t stream) {
    CUtensorMap gtq, gts, dtq, dts;
    int gsc, dsc;
    if (!moe_maps(&gtq, &gts, &gsc, gq, gd, int64_t(E) * 2 * I, H) ||
        !moe_maps(&dtq, &dts, &dsc, dq, dd, int64_t(E) * H, I))
        return W4A8_ERR_CUDA;
    // limits for the largest lists, so that one setting serves every call
    const int n = T * top_k, td = T < moe::kDownTokens ? T : moe::kDownTokens;
    const int64_t items = int64_t(moe::max_groups(E, n, moe::kGroup)) * (I / 32);
    const int64_t slots = int64_t(sm_count()) * 2;
    // 64 rows per item where that still leaves every CTA two of them, which halves what an item costs
    // beside its boxes (64 tokens, top 8 of 64, 2048 x 1024: 108 us against 111 with 32 rows; 16 tokens
    // 59.3 / 61.2; one token, with 8 experts' items: 17.0 / 16.0)
    auto* gate_up = I % 64 == 0 && items >= 4 * slots ? moe::gate_up_kernel<4> : moe::gate_up_kernel<2>;
    cudaError_t e = smem_limit_once(gate_up,
                                    int(moe::gate_up_smem(moe::kMaxExperts, moe::kMaxTokens * moe::kMaxTopK)));
    if (e == cudaSuccess)
        e = smem_limit_once(moe::down_kernel, int(moe::down_smem(moe::kDownTokens, moe::kMaxExperts,
                                                                 moe::kDownTokens * moe::kMaxTopK)));
    if (e != cudaSuccess) return cuda_status(e);
    e = launch_pdl(gate_up, dim3(unsigned(items < slots ? items : slots)), dim3(256),
                   moe::gate_up_smem(E, n), stream, T, E, H, I, top_k, ids, weights, (const uint8_t*)w.xq,
                   (const float*)w.xd, gtq, gts, gsc, gd, w.hq, w.hd);
    if (e != cudaSuccess) return cuda_status(e);
    const int tz = int(cdiv(T, moe::kDownTokens));
    int cs = 8;  // the largest cluster whose grid is resident at once
    while (cs > 1 && int64_t(H / 32) * tz * cs > slots) cs >>= 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(cs), unsigned(H / 32), unsigned(tz));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = moe::down_smem(td, E, td * top_k);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cs);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, moe::down_kernel, T, E, H, I, top_k, ids, weights,
                                          (const uint8_t*)w.hq, (const float*)w.hd, dtq, dts, dsc, dd, y,
                                          odt == W4A8_BF16 ? 1 : 0));
}

}  // namespace

extern "C" {

w4a8_status w4a8_moe_route(int T, int E, int H, int top_k, int renorm, const void* x, w4a8_dtype dtype, const void* wr,
                           w4a8_dtype wr_dtype, int32_t* ids, float* weights, cudaStream_t stream) {
    const w4a8_status st = check_route(T, E, H, top_k, x, dtype, wr, wr_dtype, ids, weights);
    if (st != W4A8_OK) return st;
    return run_route(T, E, H, top_k, renorm, x, dtype, wr, wr_dtype, ids, weights, nullptr, nullptr, stream);
}

size_t w4a8_moe_workspace_bytes(int T, int E, int H, int I, int top_k) {
    if (!moe_dims_ok(T, E, H, I, top_k) || !moe_supported(T, E, I, top_k)) return 0;
    return moe_ws(nullptr, T, H, I, top_k).bytes;
}

w4a8_status w4a8_moe_q4_0(int T, int E, int H, int I, int top_k, const void* x, w4a8_dtype dtype, const int32_t* ids,
                          const float* weights, const uint8_t* gu_qs, const uint16_t* gu_d, const uint8_t* dn_qs,
                          const uint16_t* dn_d, w4a8_dtype out_dtype, void* y, void* ws, size_t ws_bytes,
                          cudaStream_t stream) {
    w4a8_status st = check_moe(T, E, H, I, top_k, x, dtype, ids, weights, gu_qs, gu_d, dn_qs, dn_d, out_dtype, y, ws,
                               ws_bytes);
    if (st != W4A8_OK) return st;
    const MoeWs w = moe_ws(ws, T, H, I, top_k);
    st = run_route(T, E, H, top_k, 0, x, dtype, nullptr, W4A8_F32, nullptr, nullptr, w.xq, w.xd, stream);
    if (st != W4A8_OK) return st;
    return run_experts(T, E, H, I, top_k, ids, weights, gu_qs, gu_d, dn_qs, dn_d, out_dtype, y, w, stream);
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
    const MoeWs w = moe_ws(ws, T, H, I, top_k);
    st = run_route(T, E, H, top_k, renorm, x, dtype, wr, wr_dtype, ids, weights, w.xq, w.xd, stream);
    if (st != W4A8_OK) return st;
    return run_experts(T, E, H, I, top_k, ids, weights, gu_qs, gu_d, dn_qs, dn_d, out_dtype, y, w, stream);
}

}  // extern "C"
