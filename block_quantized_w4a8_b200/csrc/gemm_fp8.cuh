// FP8 (e4m3) matmul with 128-wide blocks: activations with one scale per row and block of
// the contracted axis, weights with one scale per 128 x 128 tile.
//
//   out[m][c] = sum_b sa[b][m] * sw(b, c/128) * P_b[m][c],   P_b = sum_{r in b} a[m][r] * w(r, c)
//
// over blocks b of 128 of the contracted axis r. Forward: c = n, r = k, w(r, c) = q[c][r];
// input gradient (TRANS): c = k, r = n, w(r, c) = q[r][c]. Each P_b is four
// tcgen05.mma.kind::f8f6f4 of K = 32 into a fresh tensor-memory tile; the epilogue reads the
// tile and adds it, times the two scales, to f32 accumulators in registers. Both weight
// orders are read by the same TMA boxes of 128 x 128 bytes with the 128-byte swizzle: the
// forward's box is a K-major operand, the gradient's the same bytes as an MN-major one.
#pragma once

#include <cuda.h>

#include "fp8_quant.cuh"

namespace w4a8 {
namespace fp8 {

constexpr int kTile = 128 * 128;  // bytes of one operand tile

// Shared-memory matrix descriptors with the 128-byte swizzle (atoms of 8 rows x 128 bytes,
// 1024 bytes apart): for a K-major operand the 8-row groups follow one another along M/N,
// for an MN-major one along K; one 128-byte row spans the whole K block, or the whole M/N
// extent, so the other stride is never used.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}
// Byte offset of the kk-th K = 32 slice inside a tile.
template <bool MN_MAJOR>
__device__ __forceinline__ uint32_t k_offset(int kk) {
    return MN_MAJOR ? uint32_t(kk) * 32u * 128u : uint32_t(kk) * 32u;
}
// Instruction descriptor, kind::f8f6f4: A and B e4m3, D f32; ta / tb: operand is MN-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool ta, bool tb) {
    return (1u << 4) | (ta ? 1u << 15 : 0u) | (tb ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ void tmem_load(uint32_t t, uint32_t (&r)[16]) { tmem_ld_32x32_x16(t, r); }
__device__ __forceinline__ void tmem_load(uint32_t t, uint32_t (&r)[32]) { tmem_ld_32x32(t, r); }
__device__ __forceinline__ void tmem_load(uint32_t t, uint32_t (&r)[64]) { tmem_ld_32x32_x64(t, r); }
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[64]) { tmem_wait_ld64(r); }
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) { tmem_wait_ld16(r); }
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) { tmem_wait_ld(r); }

// bounded_wait_warp without a call: the register split of the CTA-pair kernel (setmaxnreg) rules
// out calls.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait_nohint<CLUSTER>(bar, parity)), 1)) return true;
    const unsigned long long t0 = global_timer_ns();
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xffffffffu, mbar_try_wait<CLUSTER>(bar, parity))) return true;
        if ((it & 15u) == 0u) {
            const bool late = global_timer_ns() - t0 > kWaitLimitNs;
            if (late && (threadIdx.x & 31u) == 0u) {
                atomicOr(&g_device_status, kDevErrTimeout);
                *abort = 1u;
            }
            if (__any_sync(0xffffffffu, late || *abort != 0u)) return false;
        }
    }
}

// drain_wait_warp without a call.
__device__ __forceinline__ void drain_inline(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
    const unsigned long long t0 = global_timer_ns();
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        if (__any_sync(0xffffffffu, global_timer_ns() - t0 > limit_ns)) return;
}

constexpr int kMaxStages = 8;
constexpr int kMaxBufs = 8;
constexpr int kMaxSplit = 8;  // CTAs that share the contracted axis (a portable cluster)

// ------------------------------------------------------------------ few tokens
// Weights on the MMA's 128 rows, MN tokens (16, 32 or 64) as its columns: each weight tile is
// read once per token tile. The blocks of the contracted axis are split over a cluster of up
// to 8 CTAs, whose partial sums are added through distributed shared memory in a fixed order.
// FUSE (a handful of token blocks per CTA): the CTA quantises its share of the activation
// itself, while the first weight tiles arrive, and no other kernel runs. The weights' bytes are the
// bound: 16 x 14336 x 4096 takes 16.2 us with the quantisation (58.7 MB at 3.6 TB/s; 224 CTAs leave
// half of the SMs with one), one token at 4096 x 4096 6.3 us, mostly the latency of a launch, the first
// tiles and the join. mma.sync would need the codes widened in registers; tcgen05 reads them as they lie.
template <int MN_, bool FUSE>
struct RowsGeo {
    static constexpr int MN = MN_;
    static constexpr int STAGE = kTile + (FUSE ? 0 : MN * 128);
    static constexpr int NS = FUSE ? 5 : MN == 16 ? 6 : MN == 32 ? 5 : 4;
    static constexpr int NBUF = 4;                            // tensor-memory tiles
    static constexpr int COLS = MN * NBUF;
    static constexpr int CW = MN;                             // columns per epilogue warp
    static constexpr int EPI_WARPS = 4;
    static constexpr int LD = CW < 32 ? 16 : 32;
    static constexpr int COPY_WARP = EPI_WARPS, MMA_WARP = EPI_WARPS + 1;
    static constexpr int THREADS = (EPI_WARPS + 2) * 32;
    static constexpr int XBLK = 12;                           // FUSE: blocks of the quantised activation
    static constexpr int OFF_X = NS * STAGE;
    static constexpr int OFF_SX = OFF_X + (FUSE ? XBLK * MN * 128 : 0);  // token scales, one row per stage (block)
    static constexpr int OFF_CTRL = OFF_SX + (FUSE ? XBLK : NS) * MN * 4;
    static constexpr int SMEM = OFF_CTRL + 512 + 1024;
    static_assert(128 * MN * 4 <= NS * STAGE, "partial sums fit the stages");
    static_assert(NS <= kMaxStages && NBUF <= kMaxBufs && SMEM <= 115712, "two CTAs per SM");
    static_assert(!FUSE || MN == 16, "the fused form is for a few tokens");
};
struct RowsCtrl {
    unsigned long long full[kMaxStages];   // TMA: 1 arrival + bytes
    unsigned long long empty[kMaxStages];  // one arrival per epilogue warp
    unsigned long long tfull[kMaxBufs];    // MMA commit
    unsigned long long tempty[kMaxBufs];   // one arrival per epilogue warp
    unsigned long long drain;
    unsigned long long xready;             // FUSE: one arrival per epilogue warp
    uint32_t tmem_base;
    uint32_t abort;
};
static_assert(sizeof(RowsCtrl) <= 512, "control block");

// Grid: x = split of the contracted axis (the cluster), y = 128-column tile, z = token tile.
// The activation: codes through tm_x and scales sx, or (FUSE) x itself, BF16 or f32, R a
// multiple of 8.
template <int MN, bool TRANS, bool FUSE, bool BF16>
__global__ void __launch_bounds__(RowsGeo<MN, FUSE>::THREADS, 2)
    gemm_rows_kernel(int M, int C, int R, const __grid_constant__ CUtensorMap tm_w,
                     const __grid_constant__ CUtensorMap tm_x, const float* __restrict__ sx, int spitch,
                     const void* x, const float* __restrict__ sw, int swcols, int kbs, void* __restrict__ out,
                     Epilogue epi) {
    using G = RowsGeo<MN, FUSE>;
    constexpr int NS = G::NS, NBUF = G::NBUF, CW = G::CW, LD = G::LD;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    RowsCtrl* ctrl = reinterpret_cast<RowsCtrl*>(smem + G::OFF_CTRL);
    float* ssx = reinterpret_cast<float*>(smem + G::OFF_SX);
    volatile uint32_t* abort = &ctrl->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nblk = (R + kBlk - 1) / kBlk;
    const int b0 = blockIdx.x * kbs;
    const int Bl = min(nblk, b0 + kbs) - b0;  // at least 1 (host)
    const int c0 = blockIdx.y * 128, m0 = blockIdx.z * MN;
    auto bar = [](unsigned long long* p) { return smem_addr(p); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar(&ctrl->full[s]), 1);
            mbar_init(bar(&ctrl->empty[s]), G::EPI_WARPS);
        }
        for (int j = 0; j < NBUF; ++j) {
            mbar_init(bar(&ctrl->tfull[j]), 1);
            mbar_init(bar(&ctrl->tempty[j]), G::EPI_WARPS);
        }
        mbar_init(bar(&ctrl->drain), 1);
        mbar_init(bar(&ctrl->xready), G::EPI_WARPS);
        ctrl->abort = 0;
        mbar_init_fence();
    }
    if (warp == G::MMA_WARP) {
        tmem_alloc(smem_addr(&ctrl->tmem_base), G::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctrl->tmem_base;
    pdl_launch_dependents();
    const uint32_t smem0 = smem_addr(smem);

    float acc[CW];  // epilogue warps: this thread's output column (lane) for CW tokens
    if (warp == G::COPY_WARP) {
        const bool leader = elect_one();
        auto load_w = [&](int it) {
            const uint32_t fb = bar(&ctrl->full[it % NS]);
            mbar_arrive_expect_tx(fb, uint32_t(FUSE ? kTile : G::STAGE + MN * 4));
            const int r = (b0 + it) * kBlk;
            tma_load_2d<1>(smem0 + (it % NS) * G::STAGE, &tm_w, TRANS ? c0 : r, TRANS ? r : c0, fb);
        };
        auto load_x = [&](int it) {
            if (FUSE) return;
            const uint32_t fb = bar(&ctrl->full[it % NS]);
            tma_load_2d<1>(smem0 + (it % NS) * G::STAGE + kTile, &tm_x, (b0 + it) * kBlk, m0, fb);
            bulk_g2s(smem_addr(ssx + (it % NS) * MN), sx + int64_t(b0 + it) * spitch + m0, MN * 4, fb);
        };
        // the weights do not depend on the preceding kernel (the activation's quantisation)
        const int pre = min(NS, Bl);
        if (leader)
            for (int it = 0; it < pre; ++it) load_w(it);
        if (!FUSE) pdl_wait_primary();
        if (leader)
            for (int it = 0; it < pre; ++it) load_x(it);
        __syncwarp();
        int issued = pre;
        for (int it = pre; it < Bl; ++it) {
            if (!bounded_wait_warp(bar(&ctrl->empty[it % NS]), ((it / NS) & 1) ^ 1, abort)) break;
            if (leader) {
                load_w(it);
                load_x(it);
            }
            __syncwarp();
            issued = it + 1;
        }
        for (int it = max(0, issued - NS); it < issued; ++it)
            drain_wait_warp(bar(&ctrl->full[it % NS]), (it / NS) & 1, 200000ull);
    } else if (warp == G::MMA_WARP) {
        const bool leader = elect_one();
        uint32_t local_abort = 0;
        constexpr uint32_t idesc = idesc_e4m3(128, MN, TRANS, false);
        const bool go = !FUSE || bounded_wait_warp(bar(&ctrl->xready), 0, abort);
        for (int it = 0; it < Bl && go; ++it) {
            const int slot = it % NS, buf = it % NBUF;
            if (!bounded_wait_warp(bar(&ctrl->full[slot]), (it / NS) & 1, abort)) break;
            if (!bounded_wait_warp(bar(&ctrl->tempty[buf]), ((it / NBUF) & 1) ^ 1, abort)) break;
            tc_fence_after();
            if (leader) {
                const uint32_t w = smem0 + slot * G::STAGE;
                const uint32_t xa = FUSE ? smem0 + G::OFF_X + it * MN * 128 : w + kTile;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f8(tmem_base + buf * MN, desc_sw128(w + k_offset<TRANS>(kk)), desc_sw128(xa + k_offset<false>(kk)),
                           idesc, kk != 0);
                tc_commit(bar(&ctrl->tfull[buf]));
            }
            __syncwarp();
        }
        if (leader) tc_commit(bar(&ctrl->drain));
        __syncwarp();
        bounded_wait_warp(bar(&ctrl->drain), 0, &local_abort);
    } else {
        const uint32_t lane_base = tmem_base + (uint32_t(warp * 32) << 16);
        if constexpr (FUSE) {
            // 16 lanes of 8 elements per token and block, the arithmetic of quant_rows_kernel; codes into
            // the operand's layout (rows of 128 bytes, 128-byte swizzle). Rows past M keep what the memory held: they
            // only reach columns that are not stored.
            pdl_wait_primary();
            const int sub = lane & 15, tokens = min(MN, M - m0), n = tokens * Bl;
            for (int w0 = warp * 2; w0 < n; w0 += 32) {  // the same trips for both half-warps
                float v[4][8];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = w0 + (lane >> 4) + 8 * u, b = i / tokens, j = i - b * tokens, k = (b0 + b) * kBlk + sub * 8;
                    load8<BF16, true>(x, int64_t(m0 + j) * R + k, i < n ? R - k : 0, v[u]);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = w0 + (lane >> 4) + 8 * u, b = i / tokens, j = i - b * tokens;
                    float a = amax8(v[u]);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o, 16));
                    const float sc = block_scale(a);
                    if (i < n) {
                        *reinterpret_cast<uint2*>(smem + G::OFF_X + b * MN * 128 + j * 128 + (((sub >> 1) ^ (j & 7)) << 4) +
                                                  (sub & 1) * 8) = codes8(v[u], __frcp_rn(sc));
                        if (sub == 0) ssx[b * MN + j] = sc;
                    }
                }
            }
            fence_proxy_async_smem();  // read by the tensor core
            named_barrier(1, 128);     // the scales are read by all four warps
            if (lane == 0) mbar_arrive(bar(&ctrl->xready));
        }
#pragma unroll
        for (int j = 0; j < CW; ++j) acc[j] = 0.0f;
        const float* swp = TRANS ? sw + int64_t(b0) * swcols + blockIdx.y : sw + int64_t(blockIdx.y) * swcols + b0;
        const int64_t swstep = TRANS ? swcols : 1;
        float wnext = __ldg(swp);
        for (int it = 0; it < Bl; ++it) {
            const int slot = it % NS, buf = it % NBUF;
            const float w = wnext;
            if (it + 1 < Bl) wnext = __ldg(swp + (it + 1) * swstep);
            if (!bounded_wait_warp(bar(&ctrl->tfull[buf]), (it / NBUF) & 1, abort)) break;
            if (!FUSE && !bounded_wait_warp(bar(&ctrl->full[slot]), (it / NS) & 1, abort)) break;  // the scales' copy
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < CW; h += LD) {
                uint32_t p[LD];
                tmem_load(lane_base + buf * MN + h, p);
                float s[LD];
#pragma unroll
                for (int j = 0; j < LD; j += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(ssx + (FUSE ? it : slot) * MN + h + j);
                    s[j] = v.x; s[j + 1] = v.y; s[j + 2] = v.z; s[j + 3] = v.w;
                }
                tmem_wait(p);
                if (h + LD == CW) {  // tile and scales are in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_after(bar(&ctrl->empty[slot]), s[LD - 1]);
                        mbar_arrive(bar(&ctrl->tempty[buf]));
                    }
                }
#pragma unroll
                for (int j = 0; j < LD; ++j)
                    acc[h + j] = fmaf(__uint_as_float(p[j]), __fmul_rn(w, s[j]), acc[h + j]);
            }
        }
    }

    // The tensor memory goes back before the CTA waits for its cluster: one that held columns while it
    // waited for a CTA that still waits for columns of another kernel (whose own CTAs may need these)
    // could close a circle.
    tc_fence_before();
    __syncthreads();
    if (warp == G::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem_base, G::COLS);
    }

    const int ks = gridDim.x;
    const int tokens = min(MN, M - m0);
    if (ks > 1) {
        // partial sums [token][128] over the stages, which every MMA has finished reading
        float* red = reinterpret_cast<float*>(smem);
        if (warp < G::EPI_WARPS) {
#pragma unroll
            for (int j = 0; j < CW; ++j) red[j * 128 + warp * 32 + lane] = acc[j];
        }
        cluster_sync();
        if (!*abort) {
            // this CTA's share of the tokens, four columns per thread; the partial sums of all
            // CTAs are requested before the first is added
            const int per = (tokens + ks - 1) / ks, t1 = min(tokens, (int(blockIdx.x) + 1) * per);
            const int col = (threadIdx.x & 31) * 4, c = c0 + col;
            if (c < C) {
#pragma unroll 2
                for (int t = blockIdx.x * per + (threadIdx.x >> 5); t < t1; t += G::THREADS / 32) {
                    const uint32_t at = smem0 + uint32_t(t * 128 + col) * 4;
                    float4 v[kMaxSplit];
#pragma unroll
                    for (int z = 0; z < kMaxSplit; ++z)
                        if (z < ks) v[z] = ld_cluster4(mapa_shared(at, z));
                    float4 a = v[0];
#pragma unroll
                    for (int z = 1; z < kMaxSplit; ++z)
                        if (z < ks) {
                            a.x = __fadd_rn(a.x, v[z].x);
                            a.y = __fadd_rn(a.y, v[z].y);
                            a.z = __fadd_rn(a.z, v[z].z);
                            a.w = __fadd_rn(a.w, v[z].w);
                        }
                    const int64_t o = int64_t(m0 + t) * C + c;
                    if ((C & 3) == 0) {
                        epi_store4(out, o, c, a.x, a.y, a.z, a.w, epi);
                    } else {
                        epi_store(out, o, c, a.x, epi);
                        if (c + 1 < C) epi_store(out, o + 1, c + 1, a.y, epi);
                        if (c + 2 < C) epi_store(out, o + 2, c + 2, a.z, epi);
                        if (c + 3 < C) epi_store(out, o + 3, c + 3, a.w, epi);
                    }
                }
            }
        }
        cluster_sync();  // no CTA leaves while another reads its partial sums
    } else if (warp < G::EPI_WARPS && !*abort) {
        const int c = c0 + warp * 32 + lane;
        if (c < C) {
#pragma unroll
            for (int j = 0; j < CW; ++j)
                if (j < tokens) epi_store(out, int64_t(m0 + j) * C + c, c, acc[j], epi);
        }
    }
}

// ------------------------------------------------------------------ many tokens
// CTA pairs (cta_group::2), persistent: tiles of 256 tokens x 256 output columns, each CTA
// holding 128 tokens (its TMEM lanes) and staging half of the weight tile. Two tensor-memory
// tiles of 256 columns alternate, so the MMAs of the next block run while the epilogue adds
// the last one; the output of a tile is stored while the next tile's first blocks run. A stage
// is handed back by its MMAs' commit, not by the epilogue, which takes the token scales from
// global memory a block ahead. 4096 x 14336 x 4096: 289 us with the quantisation (1.66 PFLOP/s); bound by
// the chain MMA commit, tensor-memory read, release over two tiles (about 0.65 us per block of
// 0.28 us of MMA), of which no part alone is most: without three quarters of the MMAs 20 % less time, without the
// multiply-adds 6 %. 256-column MMAs, since each reads the token operand from shared memory: two of
// 128 columns with hand-offs of their own were 7 % slower, and polling instead of suspending
// waits 3 %.
struct PairGeo {
    static constexpr int STAGE = 2 * kTile;  // token tile, weight half
    static constexpr int NS = 6;
    static constexpr int NBUF = 2;
    static constexpr int CW = 128;           // columns per epilogue warp
    static constexpr int LD = 64;            // columns per tensor-memory load
    static constexpr int EPI_WARPS = 8;      // two warpgroups
    static constexpr int COPY_WARP = 8, MMA_WARP = 9;
    static constexpr int THREADS = 384;
    // Registers: launched with 168 per thread (three warpgroups on 64 K registers); the third
    // warpgroup keeps 40, the epilogue takes 232 each for 128 accumulators and a piece of 64
    // columns: 2 * 232 + 40 = 3 * 168. Measured on the gradient of 1024 x 4096 x 4096 (whole
    // call): 30.2 us; pieces of 32 columns, which spill in the loop, 40.9; sixteen warps of 64
    // columns 35.3.
    static constexpr int OFF_STG = NS * STAGE;
    static constexpr int OFF_CTRL = OFF_STG + EPI_WARPS * 32 * 32 * 4;
    static constexpr int SMEM = OFF_CTRL + 512 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};
struct PairCtrl {
    unsigned long long full[kMaxStages];    // this CTA's copies (1 arrival + bytes)
    unsigned long long empty[kMaxStages];   // pair commit of the stage's MMAs, on both CTAs
    unsigned long long pfull[kMaxStages];   // even CTA: the odd CTA's stage is ready
    unsigned long long tfull[2];            // pair commit, on both CTAs
    unsigned long long tempty[2];           // even CTA: one arrival per epilogue warp of both
    unsigned long long drain;
    uint32_t tmem_base;
    uint32_t abort;
};
static_assert(sizeof(PairCtrl) <= 512, "control block");

// Tile order: column tiles fastest within bands of 16 of them, then token tiles, so that the CTAs
// running at one time share weights and tokens in L2.
__device__ __forceinline__ void pair_tile(int t, int tm, int tc, int& mt, int& ct) {
    constexpr int BAND = 16;
    const int band = t / (tm * BAND), in = t - band * tm * BAND;
    const int w = min(BAND, tc - band * BAND);
    mt = in / w;
    ct = band * BAND + in - mt * w;
}

__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A warp's 32 x 32 f32 staging area: word c of row r at r * 32 + (c ^ 2 (r & 15)), so that both the
// writes (a row per lane, two words at a time) and the reads (a row per half-warp) touch
// every bank once.
__device__ __forceinline__ uint32_t stage_word(int r, int c) { return uint32_t(r * 32 + (c ^ ((r & 15) * 2))); }

// The staged piece to rows m0.. and columns c0.. of the output (M x C), with the epilogue: two
// columns per lane, two rows per store.
__device__ __forceinline__ void store_piece(void* out, const float* stg, int m0, int M, int c0, int C, const Epilogue& epi) {
    const int lane = threadIdx.x & 31, cc = (lane & 15) * 2, c = c0 + cc;
    if (c >= C) return;
    const int rows = min(32, M - m0);
    const bool two = c + 1 < C, wide = (C & 1) == 0;
    const bool bias = epi.bias != nullptr;
    const float b0 = epi_value(epi, c, 0.0f), b1 = two ? epi_value(epi, c + 1, 0.0f) : 0.0f;
#pragma unroll 8
    for (int i = lane >> 4; i < rows; i += 2) {
        float2 v = *reinterpret_cast<const float2*>(stg + stage_word(i, cc));
        if (bias) {
            v.x = __fadd_rn(v.x, b0);
            v.y = __fadd_rn(v.y, b1);
        }
        const int64_t o = int64_t(m0 + i) * C + c;
        if (epi.out_bf16) {
            __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(out) + o;
            const __nv_bfloat162 w = __floats2bfloat162_rn(v.x, v.y);
            if (wide) {
                *reinterpret_cast<__nv_bfloat162*>(p) = w;
            } else {
                p[0] = w.x;
                if (two) p[1] = w.y;
            }
        } else {
            float* p = reinterpret_cast<float*>(out) + o;
            if (wide) {
                *reinterpret_cast<float2*>(p) = v;
            } else {
                p[0] = v.x;
                if (two) p[1] = v.y;
            }
        }
    }
}

// A lane's row of a staged piece of 128 bytes, which a TMA store takes to the output: 16-byte
// chunk c of row r at (c ^ (r & 7)) (the 128-byte swizzle). `acc` holds the row's sums in pairs
// from column c0 on: 64 bf16 (BF16) or 32 f32 columns.
template <bool BF16>
__device__ __forceinline__ void stage_row(uint32_t row, int lane, const unsigned long long* acc, int c0, int C,
                                          const Epilogue& epi) {
    constexpr int PER = BF16 ? 8 : 4;  // columns per chunk
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
        float v[PER];
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) unpack2(acc[ch * PER / 2 + j], v[2 * j], v[2 * j + 1]);
        if (epi.bias) {
#pragma unroll
            for (int j = 0; j < PER; ++j) v[j] = epi_value(epi, min(c0 + ch * PER + j, C - 1), v[j]);
        }
        uint32_t w[4];
        if constexpr (BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(v[j]);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(row + uint32_t((ch ^ (lane & 7)) << 4)), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
    }
}

// Loads that stay where they are written (a plain __ldg may be moved down to its use).
__device__ __forceinline__ float load_ahead(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

template <bool TRANS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairGeo::THREADS, 1)
    gemm_pair_fp8_kernel(int M, int C, int R, const __grid_constant__ CUtensorMap tm_w,
                         const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_out, int tma_out,
                         const float* sx, int spitch, const float* __restrict__ sw, int swcols, int tiles_m, int tiles_c,
                         void* __restrict__ out, Epilogue epi) {
    using G = PairGeo;
    constexpr int NS = G::NS, NBUF = G::NBUF, CW = G::CW, LD = G::LD;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PairCtrl* ctrl = reinterpret_cast<PairCtrl*>(smem + G::OFF_CTRL);
    volatile uint32_t* abort = &ctrl->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int nblk = (R + kBlk - 1) / kBlk;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int ntiles = tiles_m * tiles_c;
    auto bar = [](unsigned long long* p) { return smem_addr(p); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(bar(&ctrl->full[s]), 1);
            mbar_init(bar(&ctrl->empty[s]), 1);
            mbar_init(bar(&ctrl->pfull[s]), 1);
        }
        for (int j = 0; j < NBUF; ++j) {
            mbar_init(bar(&ctrl->tfull[j]), 1);
            mbar_init(bar(&ctrl->tempty[j]), 2 * G::EPI_WARPS);
        }
        mbar_init(bar(&ctrl->drain), 1);
        ctrl->abort = 0;
        mbar_init_fence();
    }
    if (warp == G::MMA_WARP) {
        tmem_alloc_pair(smem_addr(&ctrl->tmem_base), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();  // barriers of both CTAs initialised, tensor memory allocated
    tc_fence_after();
    const uint32_t tmem_base = ctrl->tmem_base;
    pdl_launch_dependents();
    const uint32_t smem0 = smem_addr(smem);
    pdl_wait_primary();  // the token operand and its scales are written by the preceding kernel

    if (warp >= G::COPY_WARP) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == G::COPY_WARP) {
        const bool leader = elect_one();
        int it = 0;
        bool go = true;
        for (int t = pair; t < ntiles && go; t += npairs) {
            int mt, ct;
            pair_tile(t, tiles_m, tiles_c, mt, ct);
            const int m0 = mt * 256 + int(rank) * 128, c0 = ct * 256 + int(rank) * 128;
            for (int b = 0; b < nblk; ++b, ++it) {
                const int slot = it % NS;
                if (!wait_inline<true>(bar(&ctrl->empty[slot]), ((it / NS) & 1) ^ 1, abort)) {
                    go = false;
                    break;
                }
                if (leader) {
                    const uint32_t fb = bar(&ctrl->full[slot]);
                    mbar_arrive_expect_tx(fb, uint32_t(G::STAGE));
                    const uint32_t st = smem0 + slot * G::STAGE;
                    tma_load_2d<1>(st, &tm_x, b * kBlk, m0, fb);
                    tma_load_2d<1>(st + kTile, &tm_w, TRANS ? c0 : b * kBlk, TRANS ? b * kBlk : c0, fb);
                }
                __syncwarp();
            }
        }
        for (int i = max(0, it - NS); i < it; ++i) drain_inline(bar(&ctrl->full[i % NS]), (i / NS) & 1, 200000ull);
    } else if (warp == G::MMA_WARP) {
        const bool leader = elect_one();
        uint32_t local_abort = 0;
        int total = 0;  // blocks of all this pair's tiles
        for (int t = pair; t < ntiles; t += npairs) total += nblk;
        if (rank == 0) {
            constexpr uint32_t idesc = idesc_e4m3(256, 256, false, TRANS);
            for (int it = 0; it < total; ++it) {
                const int slot = it % NS, buf = it % NBUF;
                if (!wait_inline<false>(bar(&ctrl->full[slot]), (it / NS) & 1, abort)) break;
                if (!wait_inline<true>(bar(&ctrl->pfull[slot]), (it / NS) & 1, abort)) break;
                if (!wait_inline<true>(bar(&ctrl->tempty[buf]), ((it / NBUF) & 1) ^ 1, abort)) break;
                tc_fence_after();
                if (leader) {
                    const uint32_t x = smem0 + slot * G::STAGE, w = x + kTile;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8_pair(tmem_base + buf * 256, desc_sw128(x + k_offset<false>(kk)),
                                    desc_sw128(w + k_offset<TRANS>(kk)), idesc, kk != 0);
                    tc_commit_pair(bar(&ctrl->tfull[buf]), 3);
                    tc_commit_pair(bar(&ctrl->empty[slot]), 3);
                }
                __syncwarp();
            }
            if (leader) tc_commit_pair(bar(&ctrl->drain), 3);
        } else {
            const uint32_t pfull0 = mapa_shared(bar(&ctrl->pfull[0]), 0);
            for (int it = 0; it < total; ++it) {
                if (!wait_inline<false>(bar(&ctrl->full[it % NS]), (it / NS) & 1, abort)) break;
                if (leader) mbar_arrive_remote(pfull0 + uint32_t(it % NS) * 8u);
                __syncwarp();
            }
        }
        __syncwarp();
        wait_inline<false>(bar(&ctrl->drain), 0, &local_abort);
    } else if (warp < G::EPI_WARPS) {
        const int q = warp & 3, cg = warp >> 2;  // TMEM lane quarter, half of the columns
        const int r = q * 32 + lane;             // this thread's token within the CTA's 128
        const uint32_t lane_base = tmem_base + (uint32_t(q * 32) << 16) + cg * CW;
        const uint32_t tempty0 = rank == 0 ? bar(&ctrl->tempty[0]) : mapa_shared(bar(&ctrl->tempty[0]), 0);
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        unsigned long long acc[CW / 2];
        int it = 0;
        bool go = true;
        for (int t = pair; t < ntiles && go; t += npairs) {
            int mt, ct;
            pair_tile(t, tiles_m, tiles_c, mt, ct);
            const int m = mt * 256 + int(rank) * 128 + r;
            const int cb = ct * 2 + cg;  // weight scale column of this warp
            const bool inside = cb * 128 < C;
            const float* swp = TRANS ? sw + cb : sw + int64_t(cb) * swcols;
            const int64_t swstep = TRANS ? swcols : 1;
            const float* sxp = sx + m;  // the scales' rows are padded to whole tiles
#pragma unroll
            for (int j = 0; j < CW / 2; ++j) acc[j] = 0ull;
            float wnext = inside ? load_ahead(swp) : 0.0f, snext = load_ahead(sxp);
#pragma unroll 1
            for (int b = 0; b < nblk; ++b, ++it) {
                const int buf = it % NBUF;
                const float f = __fmul_rn(snext, wnext);
                if (b + 1 < nblk) {
                    sxp += spitch;
                    snext = load_ahead(sxp);
                    swp += swstep;
                    if (inside) wnext = load_ahead(swp);
                }
                const unsigned long long f2 = pack2(f, f);
                if (!wait_inline<true>(bar(&ctrl->tfull[buf]), (it / NBUF) & 1, abort)) {
                    go = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < CW / LD; ++h) {
                    uint32_t p[LD];
                    tmem_load(lane_base + buf * 256 + h * LD, p);
                    tmem_wait(p);
                    if (h + 1 == CW / LD) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (rank == 0)
                                mbar_arrive(tempty0 + uint32_t(buf) * 8u);
                            else
                                mbar_arrive_remote(tempty0 + uint32_t(buf) * 8u);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < LD / 2; ++j)
                        acc[h * LD / 2 + j] = fma2(pack2(__uint_as_float(p[2 * j]), __uint_as_float(p[2 * j + 1])),
                                                   f2, acc[h * LD / 2 + j]);
                }
            }
            // The tile leaves through shared memory, in pieces of 32 rows x 128 bytes that TMA stores
            // take to the output while the next tile runs (rows of a multiple of 16 bytes), or 32 rows
            // x 32 columns at a time, so that the stores of a warp lie in whole rows. Either way the
            // accumulators are read with fixed indexes.
            const int c0 = ct * 256 + cg * CW, mrow = mt * 256 + int(rank) * 128 + q * 32;
            float* stg = reinterpret_cast<float*>(smem + G::OFF_STG) + warp * 32 * 32;
            if (tma_out) {
                const uint32_t stg0 = smem_addr(stg), row = stg0 + uint32_t(lane) * 128u;
                auto send = [&](int c) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && go && c < C && mrow < M) {
                        if (epi.out_bf16)
                            tma_store_2d<2>(&tm_out, c, mrow, stg0);
                        else
                            tma_store_2d<4>(&tm_out, c, mrow, stg0);
                        bulk_commit();
                    }
                    __syncwarp();
                };
                auto staged = [&]() {  // the previous piece has left
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                };
                if (epi.out_bf16) {
#pragma unroll
                    for (int h = 0; h < CW / 64; ++h) {
                        staged();
                        stage_row<true>(row, lane, acc + h * 32, c0 + h * 64, C, epi);
                        send(c0 + h * 64);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < CW / 32; ++h) {
                        staged();
                        stage_row<false>(row, lane, acc + h * 16, c0 + h * 32, C, epi);
                        send(c0 + h * 32);
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < CW / 32; ++h) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        *reinterpret_cast<unsigned long long*>(stg + stage_word(lane, 2 * j)) = acc[h * 16 + j];
                    __syncwarp();
                    if (go) store_piece(out, stg, mrow, M, c0 + h * 32, C, epi);
                    __syncwarp();
                }
            }
        }
        if (lane == 0) bulk_wait();
        __syncwarp();
    }

    tc_fence_before();
    cluster_sync();
    if (warp == G::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace fp8
}  // namespace w4a8
