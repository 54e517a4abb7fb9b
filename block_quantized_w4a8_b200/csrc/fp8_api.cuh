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
                          int64_t sblk, bool early, cudaStream_t stream) {
    const int chunk = int((int64_t(1) << 27) / fp8_blocks(L));
    const bool vec = L % 16 == 0;
    for (int m0 = 0; m0 < M; m0 += chunk) {
        const int mc = M - m0 < chunk ? M - m0 : chunk;
        const void* xc = static_cast<const char*>(x) + int64_t(m0) * L * (dt == W4A8_BF16 ? 2 : 4);
        uint8_t* qc = q + int64_t(m0) * pitch;
        float* sc = s + m0 * srow;
        const dim3 grid(unsigned(cdiv(int64_t(mc) * fp8_blocks(L), 32)));
        auto* kernel = dt == W4A8_BF16 ? (vec ? fp8::quant_rows_kernel<true, true> : fp8::quant_rows_kernel<true, false>)
                                       : (vec ? fp8::quant_rows_kernel<false, true> : fp8::quant_rows_kernel<false, false>);
        kernel<<<grid, 256, 0, stream>>>(xc, mc, L, pitch, qc, sc, srow, sblk, early ? 1 : 0);
        const w4a8_status st = launch_status();
        if (st != W4A8_OK) return st;
    }
    return W4A8_OK;
}

// Token tile of the few-token kernel, and the pitch of the block-major scales: whole tiles
// are copied, so the rows are padded to the largest tile a path may take (256 for CTA pairs).
inline int fp8_token_tile(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }
inline int fp8_scale_pitch(int M) { return M <= 64 ? fp8_token_tile(M) : int(cdiv(M, 256) * 256); }

// Workspace of a contraction over R columns: the quantised rows (codes of pitch
// round_up(R, 16), block-major scales).
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
    w.spitch = fp8_scale_pitch(M);
    w.q = reinterpret_cast<uint8_t*>(base + off); off = align256(off + size_t(M) * w.pitch);
    w.s = reinterpret_cast<float*>(base + off); off = align256(off + size_t(w.spitch) * fp8_blocks(R) * 4);
    w.bytes = off;
    return w;
}

inline bool fp8_dims_ok(int M, int N, int K) { return dims_ok(M, N) && dims_ok(K, 1) && K % 16 == 0; }

// CTA pairs on 256 x 256 tiles once the few-token kernel's tiles (64 tokens x 128 columns) are more
// than the SMs. Measured with K = 4096, pairs against the few-token kernel: 128 x 14336 (224 tiles)
// 26.1 against 28.6 us, 192 x 14336 (336) 26.5 / 51.1, 256 x 6144 (192) 23.5 / 27.9, 320 x 4096
// (160) 23.6 / 27.0; 256 x 4096 (128) 22.8 / 17.5, 1024 x 1024 (128) 23.1 / 18.1, 64 x 14336 (112)
// 24.8 / 19.2; K = 1024: 300 x 4096 (160) 10.9 / 12.6; K = 8192: 512 x 2048 (128) 38.4 / 27.9.
inline bool fp8_use_pair(int M, int C) { return M > 64 && cdiv(M, 64) * cdiv(C, 128) > sm_count(); }

// Split of the contracted axis for the few-token kernel: the largest power of two whose CTAs are
// all resident, two per SM, sets the blocks per CTA, and CTAs that would have none are not launched, so
// that the cluster may be of any size up to 8 (one token of 4096 columns, 9, 13, 17 and 33 blocks: 5, 7, 6 and
// 7 CTAs take 5.2, 5.4, 5.4 and 6.5 us; the next smaller splits of 3 and 4 CTAs 5.4, 5.5, 5.9 and 7.1).
// Tiles of 64 tokens stop at 4, since every CTA's partial sums are read by the others (64 tokens at
// 4096 x 4096: 4 CTAs per tile 9.6 us, 8 CTAs 11.0; one token: 8 CTAs 6.3, 4 CTAs 6.8).
struct Fp8Split {
    int ks, kbs;  // CTAs per output tile, blocks per CTA
};
Fp8Split fp8_split(int M, int C, int R) {
    const int tt = fp8_token_tile(M), nblk = fp8_blocks(R);
    const int64_t tiles = cdiv(C, 128) * cdiv(M, tt), slots = int64_t(sm_count()) * 2;
    int ks = tt == 64 ? 4 : fp8::kMaxSplit;
    while (ks > 1 && (tiles * ks > slots || ks > nblk)) ks >>= 1;
    const int kbs = int(cdiv(nblk, ks));
    return Fp8Split{int(cdiv(nblk, kbs)), kbs};  // every CTA has at least one block
}
// Whether the few-token kernel quantises the activation itself: rows that can be read eight
// elements at a time, and at most 64 token blocks per CTA (two rounds of its 8 groups of
// lanes), each done again by every column tile. One token at 4096 x 4096: 6.3 us against 7.0 with
// the kernel of its own, and one launch less; 16 tokens: 8.0 against 7.5 on the device, less
// than the launch costs the host.
bool fp8_fused(int M, int C, int R) {
    if (M > 16 || R % 8 != 0) return false;
    const Fp8Split sp = fp8_split(M, C, R);
    return sp.kbs <= fp8::RowsGeo<16, true>::XBLK && M * sp.kbs <= 64;
}

template <int MN, bool TRANS, bool FUSE, bool BF16>
w4a8_status launch_fp8_rows(int M, int C, int R, const CUtensorMap& tw, const Fp8Ws& w, const void* x, const float* s,
                            int swcols, void* out, const Epilogue& epi, cudaStream_t stream) {
    using G = fp8::RowsGeo<MN, FUSE>;
    const cudaError_t ea = smem_limit_once(fp8::gemm_rows_kernel<MN, TRANS, FUSE, BF16>, G::SMEM);
    if (ea != cudaSuccess) return cuda_status(ea);
    CUtensorMap tx = tw;  // not read by the fused form
    if (!FUSE && !encode_2d(&tx, w.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(R), uint64_t(M), uint64_t(w.pitch), 128,
                            MN, CU_TENSOR_MAP_SWIZZLE_128B))
        return W4A8_ERR_CUDA;
    const Fp8Split sp = fp8_split(M, C, R);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(sp.ks), unsigned(cdiv(C, 128)), unsigned(cdiv(M, MN)));
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = G::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(sp.ks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, fp8::gemm_rows_kernel<MN, TRANS, FUSE, BF16>, M, C, R, tw, tx,
                                          (const float*)w.s, w.spitch, x, s, swcols, sp.kbs, out, epi));
}

template <bool TRANS>
w4a8_status launch_fp8_pair(int M, int C, int R, const CUtensorMap& tw, const Fp8Ws& w, const float* s, int swcols,
                            void* out, const Epilogue& epi, cudaStream_t stream) {
    using G = fp8::PairGeo;
    const cudaError_t ea = smem_limit_once(fp8::gemm_pair_fp8_kernel<TRANS>, G::SMEM);
    if (ea != cudaSuccess) return cuda_status(ea);
    CUtensorMap tx;
    if (!encode_2d(&tx, w.q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(R), uint64_t(M), uint64_t(w.pitch), 128, 128,
                   CU_TENSOR_MAP_SWIZZLE_128B))
        return W4A8_ERR_CUDA;
    // the output, in pieces of 32 rows x 128 bytes, when its rows are whole 16-byte units
    const int esize = epi.out_bf16 ? 2 : 4;
    const int tma_out = C % (16 / esize) == 0;
    CUtensorMap to = tx;
    if (tma_out && !encode_2d(&to, out, epi.out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                              esize, uint64_t(C), uint64_t(M), uint64_t(C) * esize, uint32_t(128 / esize), 32,
                              CU_TENSOR_MAP_SWIZZLE_128B))
        return W4A8_ERR_CUDA;
    const int tm = int(cdiv(M, 256)), tc = int(cdiv(C, 256));
    const int64_t tiles = int64_t(tm) * tc;
    const int pairs = int(tiles < sm_count() / 2 ? tiles : sm_count() / 2);
    return cuda_status(launch_pdl(fp8::gemm_pair_fp8_kernel<TRANS>, dim3(unsigned(2 * pairs)), dim3(G::THREADS),
                                  size_t(G::SMEM), stream, M, C, R, tw, tx, to, tma_out, (const float*)w.s, w.spitch, s,
                                  swcols, tm, tc, out, epi));
}

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
    // one box = 128 x 128 codes, either way round
    CUtensorMap tw;
    if (!encode_2d(&tw, q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, uint64_t(K), uint64_t(N), uint64_t(K), 128, 128,
                   CU_TENSOR_MAP_SWIZZLE_128B))
        return W4A8_ERR_CUDA;
    const int swcols = fp8_blocks(K);
    const bool pair = fp8_use_pair(M, C);
    if (!pair && fp8_fused(M, C, R))
        return dt == W4A8_BF16 ? launch_fp8_rows<16, TRANS, true, true>(M, C, R, tw, w, in, s, swcols, out, epi, stream)
                               : launch_fp8_rows<16, TRANS, true, false>(M, C, R, tw, w, in, s, swcols, out, epi, stream);
    const w4a8_status st = run_fp8_quant(in, dt, M, R, w.pitch, w.q, w.s, 1, w.spitch, true, stream);
    if (st != W4A8_OK) return st;
    if (pair) return launch_fp8_pair<TRANS>(M, C, R, tw, w, s, swcols, out, epi, stream);
    switch (fp8_token_tile(M)) {
        case 16: return launch_fp8_rows<16, TRANS, false, false>(M, C, R, tw, w, in, s, swcols, out, epi, stream);
        case 32: return launch_fp8_rows<32, TRANS, false, false>(M, C, R, tw, w, in, s, swcols, out, epi, stream);
        default: return launch_fp8_rows<64, TRANS, false, false>(M, C, R, tw, w, in, s, swcols, out, epi, stream);
    }
}

}  // namespace

extern "C" {

w4a8_status w4a8_quant_act_fp8(const void* x, w4a8_dtype dtype, int M, int K, uint8_t* q, float* s,
                               cudaStream_t stream) {
    if (!fp8_dims_ok(M, 1, K) || !x || !q || !s) return W4A8_ERR_INVALID_ARG;
    if (check_fp8_dtype(dtype) != W4A8_OK) return W4A8_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return W4A8_ERR_MISALIGNED;
    return run_fp8_quant(x, dtype, M, K, K, q, s, fp8_blocks(K), 1, false, stream);
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
