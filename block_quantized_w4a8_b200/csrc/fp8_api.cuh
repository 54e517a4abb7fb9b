// Entry points of the FP8 block-scaled matmul (argument checks, workspace, launches).
// Included by w4a8.cu, whose helpers it uses.
#pragma once

#include "gemm_fp8.cuh"

namespace {

inline int fp8_blocks(int n) { return int(cdiv(n, fp8::kBlk)); }

w4a8_status check_fp8_dtype(w4a8_dtype dt) {
    return (dt == W4A8_F32 || dt == W4A8_BF16) ? W4A8_OK : W4A8_ERR_UNSUPPORTED;
}

// Quantises M rows of length L into codes of the given pitch and scales of the given
// strides, in launches of less than 2^28 blocks.
w4a8_status run_fp8_quant(const void* x, w4a8_dtype dt, int M, int L, int pitch, uint8_t* q, float* s, int64_t srow,
                          int64_t sblk, cudaStream_t stream) {
    const int nb = fp8_blocks(L);
    const int chunk = int((int64_t(1) << 27) / nb);
    const bool vec = L % 8 == 0;
    for (int m0 = 0; m0 < M; m0 += chunk) {
        const int mc = M - m0 < chunk ? M - m0 : chunk;
        const dim3 grid(unsigned(cdiv(int64_t(mc) * nb, 16)));
        const void* xc = static_cast<const char*>(x) + int64_t(m0) * L * (dt == W4A8_BF16 ? 2 : 4);
        uint8_t* qc = q + int64_t(m0) * pitch;
        float* sc = s + m0 * srow;
        if (dt == W4A8_BF16) {
            if (vec)
                fp8::quant_rows_kernel<true, true><<<grid, 256, 0, stream>>>(xc, mc, L, pitch, qc, sc, srow, sblk);
            else
                fp8::quant_rows_kernel<true, false><<<grid, 256, 0, stream>>>(xc, mc, L, pitch, qc, sc, srow, sblk);
        } else {
            if (vec)
                fp8::quant_rows_kernel<false, true><<<grid, 256, 0, stream>>>(xc, mc, L, pitch, qc, sc, srow, sblk);
            else
                fp8::quant_rows_kernel<false, false><<<grid, 256, 0, stream>>>(xc, mc, L, pitch, qc, sc, srow, sblk);
        }
        const w4a8_status st = launch_status();
        if (st != W4A8_OK) return st;
    }
    return W4A8_OK;
}

// Workspace of a contraction over R columns: the quantised rows (codes of pitch
// round_up(R, 16), block-major scales of pitch round_up(M, 4)).
struct Fp8Ws {
    uint8_t* q;
    float* s;
    int pitch, spitch;
    size_t bytes;
};
Fp8Ws fp8_ws(void* ws, int M, int R) {
    Fp8Ws w{};
    char* base = static_cast<char*>(ws);
    size_t off = 0;
    w.pitch = int(cdiv(R, 16) * 16);
    w.spitch = int(cdiv(M, 4) * 4);
    w.q = reinterpret_cast<uint8_t*>(base + off); off = align256(off + size_t(M) * w.pitch);
    w.s = reinterpret_cast<float*>(base + off); off = align256(off + size_t(w.spitch) * fp8_blocks(R) * 4);
    w.bytes = off;
    return w;
}

inline bool fp8_dims_ok(int M, int N, int K) { return dims_ok(M, N) && dims_ok(K, 1) && K % 16 == 0; }

// out (M x C) = in (M x R) . w, w = W^T (TRANS = false) or W (the input gradient).
template <bool TRANS>
w4a8_status fp8_gemm_impl(int M, int N, int K, const void* in, w4a8_dtype dt, const uint8_t* q, const float* s,
                          void* out, const Epilogue& epi, void* ws, size_t ws_bytes, cudaStream_t stream) {
    if (!fp8_dims_ok(M, N, K) || !in || !q || !s || !out) return W4A8_ERR_INVALID_ARG;
    if (check_fp8_dtype(dt) != W4A8_OK) return W4A8_ERR_UNSUPPORTED;
    if (!aligned16(in) || !aligned16(q) || !aligned16(s) || !aligned16(out)) return W4A8_ERR_MISALIGNED;
    const int R = TRANS ? N : K, C = TRANS ? K : N;
    const Fp8Ws w = fp8_ws(ws, M, R);
    if (!ws || ws_bytes < w.bytes) return W4A8_ERR_WORKSPACE;
    if (!aligned16(ws)) return W4A8_ERR_MISALIGNED;
    w4a8_status st = run_fp8_quant(in, dt, M, R, w.pitch, w.q, w.s, 1, w.spitch, stream);
    if (st != W4A8_OK) return st;
    const dim3 grid(unsigned(cdiv(M, 8)), unsigned(cdiv(C, 32)));
    fp8::gemm_simple_kernel<TRANS><<<grid, 256, 0, stream>>>(M, C, R, w.q, w.pitch, w.s, 1, w.spitch, q, s,
                                                            fp8_blocks(K), out, epi);
    return launch_status();
}

}  // namespace

extern "C" {

w4a8_status w4a8_quant_act_fp8(const void* x, w4a8_dtype dtype, int M, int K, uint8_t* q, float* s,
                               cudaStream_t stream) {
    if (!fp8_dims_ok(M, 1, K) || !x || !q || !s) return W4A8_ERR_INVALID_ARG;
    if (check_fp8_dtype(dtype) != W4A8_OK) return W4A8_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return W4A8_ERR_MISALIGNED;
    return run_fp8_quant(x, dtype, M, K, K, q, s, fp8_blocks(K), 1, stream);
}

w4a8_status w4a8_pack_fp8(const void* w, w4a8_dtype dtype, int N, int K, uint8_t* q, float* s, cudaStream_t stream) {
    if (!fp8_dims_ok(1, N, K) || !w || !q || !s) return W4A8_ERR_INVALID_ARG;
    if (check_fp8_dtype(dtype) != W4A8_OK) return W4A8_ERR_UNSUPPORTED;
    if (!aligned16(w) || !aligned16(q) || !aligned16(s)) return W4A8_ERR_MISALIGNED;
    const dim3 grid(unsigned(fp8_blocks(K)), unsigned(fp8_blocks(N)));
    if (dtype == W4A8_BF16)
        fp8::pack_tile_kernel<true><<<grid, 256, 0, stream>>>(w, N, K, q, s);
    else
        fp8::pack_tile_kernel<false><<<grid, 256, 0, stream>>>(w, N, K, q, s);
    return launch_status();
}

size_t w4a8_fp8_workspace_bytes(int M, int N, int K) {
    if (!fp8_dims_ok(M, N, K)) return 0;
    const size_t a = fp8_ws(nullptr, M, K).bytes, b = fp8_ws(nullptr, M, N).bytes;
    return a > b ? a : b;
}

w4a8_status w4a8_gemm_fp8(int M, int N, int K, const void* x, w4a8_dtype dtype, const uint8_t* q, const float* s,
                          const w4a8_epilogue* epi, void* y, void* ws, size_t ws_bytes, cudaStream_t stream) {
    Epilogue e;
    const w4a8_status st = make_epilogue(epi, &e);
    if (st != W4A8_OK) return st;
    return fp8_gemm_impl<false>(M, N, K, x, dtype, q, s, y, e, ws, ws_bytes, stream);
}

w4a8_status w4a8_gemm_fp8_backward(int M, int N, int K, const void* dy, w4a8_dtype dtype, const uint8_t* q,
                                   const float* s, w4a8_dtype dx_dtype, void* dx, void* ws, size_t ws_bytes,
                                   cudaStream_t stream) {
    if (check_fp8_dtype(dx_dtype) != W4A8_OK) return W4A8_ERR_UNSUPPORTED;
    const Epilogue e{nullptr, 0, dx_dtype == W4A8_BF16 ? 1 : 0};
    return fp8_gemm_impl<true>(M, N, K, dy, dtype, q, s, dx, e, ws, ws_bytes, stream);
}

}  // extern "C"
