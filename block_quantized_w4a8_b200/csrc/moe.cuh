// Mixture-of-experts layer for a few tokens with Q4_0 experts and Q8_0 activations:
//   router   l = x . Wr^T, the top_k largest logits, p = softmax over them or over all
//   experts  g, u = xq . Wg^T, xq . Wu^T;  h = g / (1 + exp(-g)) * u;  hq = Q8_0(h)
//   output   y[t] = sum over slots s of p[t][s] * (hq[t][s] . Wd[e(t, s)]^T)
// with the block dots of w4a8_gemm (exact integers, rescaled per 32-block in f32).
//
// Three launches, chained by programmatic dependent launch: route (the router, a cluster per
// token, and the Q8_0 form of x), gate_up (g, u, h and its Q8_0 form) and down (the weighted
// sum).
//
// The weights of the chosen experts are read once and are nearly all the traffic, so both
// expert kernels are built around their stream: every warp runs a ring of its own, two TMA boxes
// (16 rows x 8 blocks each) per stage, with no barrier between warps until their rows are
// summed. The integer dots are exact. Groups of one token use dp4a, a row per lane;
// larger ones mma.sync.m16n8k32 on int8, one per 16 rows and quant block: the instruction's K
// is the block, its A fragment is the packed codes as they lie in memory (one ldmatrix word
// holds the low and high nibbles of both K halves), and 8 tokens cost what one costs. tcgen05
// would need the codes expanded to shared or tensor memory first, and reads its accumulators
// back per block; at these sizes the memory is the bound, not the matrix rate.
#pragma once

#include <cuda.h>

#include "device_common.cuh"
#include "ring_count.cuh"

namespace w4a8 {
namespace moe {

constexpr int kMaxExperts = 256;
constexpr int kMaxTopK = 16;
constexpr int kMaxTokens = 64;
constexpr int kMaxSlotsPerThread = kMaxTokens * kMaxTopK / 256;

// ------------------------------------------------------------------ router
// Order-preserving map of a float to an unsigned key (larger float, larger key; a NaN of
// either sign maps to 0, below every number).
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 0u;
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Eight consecutive elements (idx a multiple of 8), widened to f32.
template <bool BF16>
__device__ __forceinline__ void load8f(const void* p, int64_t idx, float (&v)[8]) {
    if (BF16) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p) + idx);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // a bf16 is the top half of an f32
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + idx);
        const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + idx + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// Activations as the expert kernels read them: rows of K/32 blocks padded to a multiple of 8.
// Codes: per group of 4 blocks 128 bytes [lane quarter 0..3][block 0..3][K half 0..1][4
// codes], so that a lane's B fragments of 4 blocks are two 16-byte loads; scales: d / 16 per
// block (the weight codes enter the dots as 16 (q - 8)), 0 in the padding.
__host__ __device__ __forceinline__ int padded_blocks(int K) { return (K / 32 + 7) / 8 * 8; }
// Byte offset, within a row, of the word of codes 4w .. 4w+3 of block b.
__device__ __forceinline__ int word_offset(int b, int w) {
    return (b >> 2) * 128 + (w & 3) * 32 + (b & 3) * 8 + (w >> 2) * 4;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

constexpr int kRouteCtas = 8;  // CTAs per token (the cluster)
// Tokens from which the router keeps 4 steps of loads in flight per warp instead of 8, whose
// registers leave two CTAs per SM (whole layers, 4 against 8: one token, 256 experts, H = 4096
// 26.2 / 23.7 us; 4 tokens, 8 experts 121.8 / 121.2; 13 tokens, 11 experts 20.3 / 20.9; 64 tokens,
// 64 experts 107.0 / 108.2; 64 tokens, 256 experts of 1024 x 256 61.0 / 68.9).
constexpr int kShallowTokens = 8;

// Grid: kRouteCtas CTAs (a cluster) per token. Every CTA quantises its share of the token's
// blocks (xq != nullptr) and, with ROUTE, computes the logits of its experts, a warp each;
// they meet in the first CTA's shared memory, where one warp takes the top_k. Bound by latency,
// not bytes: about a tenth of the 106 us of a layer of 64 tokens and 64 experts of 2048 x 1024.
// DEEP: steps of 256 columns whose loads are in flight together per warp.
template <bool ROUTE, bool XB, bool WB, int DEEP>
__global__ void __launch_bounds__(256, 1) route_kernel(int E, int H, int top_k, int renorm, const void* __restrict__ x,
                                                    const void* __restrict__ wr, int* __restrict__ ids,
                                                    float* __restrict__ weights, uint8_t* __restrict__ xq,
                                                    float* __restrict__ xd) {
    __shared__ float logit[kMaxExperts];
    __shared__ __align__(16) uint32_t keys[kMaxExperts];
    __shared__ int chosen[kMaxTopK];
    const int t = blockIdx.x / kRouteCtas, rank = blockIdx.x % kRouteCtas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    if (ROUTE) {
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        bool waited = false;
        for (int e = rank + kRouteCtas * warp; e < E; e += kRouteCtas * 8) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll DEEP
            for (int k = lane * 8; k < H; k += 256) {
                float a[8], b[8];
                load8f<XB>(x, int64_t(t) * H + k, a);
                load8f<WB>(wr, int64_t(e) * H + k, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i & 3] = fmaf(a[i], b[i], s[i & 3]);
            }
            float v = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (!waited) {  // the first CTA runs: its shared memory can be written
                asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
                waited = true;
            }
            if (lane == 0) st_cluster(mapa_shared(smem_addr(&logit[e]), 0), v);
        }
        if (!waited) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        // the logits are on their way; this CTA's codes are written while they arrive (the
        // release orders stores before it: the codes' global stores come after)
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    if (xq) {
        const int B = H / 32, Bp = padded_blocks(H), sub = threadIdx.x & 7;
        for (int b0 = rank * 32; b0 < Bp; b0 += 32 * kRouteCtas) {
            const int b = b0 + int(threadIdx.x >> 3);
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (b < B) load4<XB>(x, int64_t(t) * H + b * 32 + sub * 4, v);
            const float amax = warp_max8(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
            // the maximum passes over a NaN, whose code is 0: the block's scale carries it on
            const uint32_t nans = __ballot_sync(0xffffffffu, v[0] != v[0] || v[1] != v[1] || v[2] != v[2] || v[3] != v[3]);
            const bool nan = (nans >> (threadIdx.x & 24u)) & 0xFFu;
            const float d = nan ? __int_as_float(0x7FC00000) : __fdiv_rn(amax, 127.0f);
            const float id = d != 0.0f ? __frcp_rn(d) : 0.0f;
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w |= (uint32_t(max(-127, min(127, int(roundf(__fmul_rn(v[i], id)))))) & 0xFFu) << (8 * i);
            if (b < Bp) {
                *reinterpret_cast<uint32_t*>(xq + int64_t(t) * Bp * 32 + word_offset(b, sub)) = w;
                if (sub == 0) xd[int64_t(t) * Bp + b] = __fmul_rn(d, 0.0625f);
            }
        }
    }
    if (!ROUTE) return;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
    // An expert's rank is the number of experts before it (larger, or equal with a lower
    // index): no chain of dependent maxima.
    for (int e = threadIdx.x; e < (E + 3) / 4 * 4; e += 256) keys[e] = e < E ? order_key(logit[e]) : 0u;
    __syncthreads();
    if (threadIdx.x < E) {
        const int me = threadIdx.x;
        const uint32_t key = keys[me];
        int before = 0;
#pragma unroll 4
        for (int e = 0; e < E; e += 4) {  // keys are below 2^32 - 1; the padding stands behind every expert
            const uint4 k = *reinterpret_cast<const uint4*>(keys + e);
            before += int(k.x >= key + (e >= me ? 1u : 0u)) + int(k.y >= key + (e + 1 >= me ? 1u : 0u)) +
                      int(k.z >= key + (e + 2 >= me ? 1u : 0u)) + int(k.w >= key + (e + 3 >= me ? 1u : 0u));
        }
        if (before < top_k) chosen[before] = me;
    }
    __syncthreads();
    if (warp != 0) return;
    const int mine = lane < top_k ? chosen[lane] : 0;
    const float top = logit[chosen[0]];
    const float p = lane < top_k ? expf(logit[mine] - top) : 0.0f;
    float sum = p;
    if (!renorm) {
        sum = 0.0f;
        for (int e = lane; e < E; e += 32) sum += expf(logit[e] - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < top_k) {
        ids[int64_t(t) * top_k + lane] = mine;
        weights[int64_t(t) * top_k + lane] = __fdiv_rn(p, sum);
    }
}

// ------------------------------------------------------------------ who uses which expert
// Built by every CTA in shared memory from the T x top_k slots. A slot that names its
// token's expert again is folded into the first one (their weights added), so a token is at
// most once in an expert's list. Lists longer than `group` tokens are cut into groups, each a
// pass of its own over the expert's weights.
struct Lists {
    float* w;        // [n] weight of a slot (folded)
    uint16_t* ord;   // [n] entries by expert: slot | token << 10
    uint16_t* act;   // [groups] expert of a group, in rising order
    uint16_t* from;  // [groups] first entry
    uint8_t* cnt;    // [groups] tokens
    int* nact;       // groups
    int* id;         // scratch: [n] expert of a slot, -1: empty or folded
    int* cur;        // scratch: [E]
    uint8_t* hist;   // scratch: [n / 32][E] tokens of an expert in each 32 slots
};
__host__ __device__ __forceinline__ int max_groups(int E, int n, int group) { return (E < n ? E : n) + n / group; }
__host__ __device__ __forceinline__ size_t lists_bytes(int E, int n, int group) {
    return 16 + size_t(n) * 4 + (size_t(max_groups(E, n, group)) * 5 + size_t(n) * 2 + 15) / 16 * 16;
}
constexpr int kSlotMask = 1023;  // slots are below kMaxTokens * kMaxTopK
static_assert(kMaxTokens * kMaxTopK <= kSlotMask + 1 && kMaxTokens <= 64, "slot and token fit 16 bits");
// `scratch`: at most 4 n + 4 E + E n / 32 bytes (13 KB), free once the lists are built.
__device__ __forceinline__ Lists lists_at(uint8_t* p, uint8_t* scratch, int E, int n, int group) {
    const int m = max_groups(E, n, group);
    Lists l;
    l.nact = reinterpret_cast<int*>(p);
    l.w = reinterpret_cast<float*>(p + 16);
    l.ord = reinterpret_cast<uint16_t*>(l.w + n);
    l.act = l.ord + n;
    l.from = l.act + m;
    l.cnt = reinterpret_cast<uint8_t*>(l.from + m);
    l.id = reinterpret_cast<int*>(scratch);
    l.cur = l.id + n;
    l.hist = reinterpret_cast<uint8_t*>(l.cur + E);
    return l;
}
// Entries stand in the order of the slots, so that every CTA cuts the same groups. All
// threads of the CTA call it and pass a barrier after it; ids and weights are read from
// L2.
__device__ __forceinline__ void build_lists(const Lists& l, const int* ids, const float* weights, int n, int top_k, int E,
                                            int group) {
    if (n <= 32 && n <= group * top_k) {  // one warp, one slot per lane, one group per expert
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x, id = lane < n ? __ldcg(ids + lane) : -1;
            float w = lane < n ? __ldcg(weights + lane) : 0.0f;
            const int t = lane / top_k;
            bool valid = id >= 0 && id < E;
            int pos = 0, grp = 0, cnt = 0, groups = 0;  // entries before this one, groups before it, its group's size
            uint32_t lead = 0u;                          // slots that open a group
            bool folded = false;
#pragma unroll 1
            for (int j = 0; j < n; ++j) {  // fold repeats within a token into the first
                const int idj = __shfl_sync(0xffffffffu, id, j);
                const float wj = __shfl_sync(0xffffffffu, w, j);
                const int tj = __shfl_sync(0xffffffffu, t, j);
                if (j != lane && tj == t && idj == id) {
                    if (j < lane)
                        folded = true;
                    else
                        w = __fadd_rn(w, wj);
                }
            }
            valid = valid && !folded;
            const int key = valid ? id : 0x7fffffff;
            const uint32_t same = __match_any_sync(0xffffffffu, key);
            lead = __ballot_sync(0xffffffffu, valid && (same & ((1u << lane) - 1u)) == 0u);
            cnt = __popc(same);
            groups = __popc(lead);
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const int kj = __shfl_sync(0xffffffffu, key, j);
                pos += kj < key || (kj == key && j < lane);
                grp += kj < key && ((lead >> j) & 1u);
            }
            if (valid) {
                l.ord[pos] = uint16_t(lane | t << 10);
                l.w[lane] = w;
                if ((lead >> lane) & 1u) {
                    l.act[grp] = uint16_t(id);
                    l.from[grp] = uint16_t(pos);
                    l.cnt[grp] = uint8_t(cnt);
                }
            }
            if (lane == 0) *l.nact = groups;
        }
        return;
    }
    for (int i = threadIdx.x; i < n; i += 256) {
        const int id = __ldcg(ids + i);
        l.id[i] = id >= 0 && id < E ? id : -1;
        l.w[i] = __ldcg(weights + i);
    }
    const int chunks = (n + 31) / 32;
    for (int e = threadIdx.x; e < chunks * E; e += 256) l.hist[e] = 0;
    __syncthreads();
    int mine[kMaxSlotsPerThread], tok[kMaxSlotsPerThread];
    int rank[kMaxSlotsPerThread];  // among the 32 slots of this warp's chunk
    float wsum[kMaxSlotsPerThread];
#pragma unroll
    for (int k = 0; k < kMaxSlotsPerThread; ++k) {
        const int i = threadIdx.x + 256 * k;
        mine[k] = i < n ? l.id[i] : -1;
        if (i - int(threadIdx.x & 31) >= n) continue;  // the whole warp
        tok[k] = i / top_k;
        if (mine[k] >= 0) {
            const int s0 = tok[k] * top_k, id = mine[k];
            wsum[k] = l.w[i];
            for (int s = s0; s < s0 + top_k; ++s)
                if (s != i && l.id[s] == id) {
                    if (s < i) mine[k] = -1;
                    wsum[k] = __fadd_rn(wsum[k], l.w[s]);
                }
        }
        const uint32_t same = __match_any_sync(0xffffffffu, mine[k]);
        rank[k] = __popc(same & ((1u << (threadIdx.x & 31)) - 1u));
        if (mine[k] >= 0 && rank[k] == 0) l.hist[(i >> 5) * E + mine[k]] = uint8_t(__popc(same));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256) {
        int run = 0;
        for (int c = 0; c < chunks; ++c) {
            const int h = l.hist[c * E + e];
            l.hist[c * E + e] = uint8_t(run);
            run += h;
        }
        l.cur[e] = run;
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // first entries and groups, 32 experts at a time (packed: entries | groups << 16)
        const int lane = threadIdx.x;
        uint32_t base = 0u;
#pragma unroll 1
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, c = e < E ? l.cur[e] : 0;
            const uint32_t one = uint32_t(c) | uint32_t((c + group - 1) / group) << 16;
            uint32_t sum = one;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t p = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += p;
            }
            const uint32_t at = base + sum - one;
            const int a = int(at & 0xFFFFu);
            int u = int(at >> 16);
            if (e < E) l.cur[e] = a;
            for (int g = 0; g < c; g += group, ++u) {
                l.act[u] = uint16_t(e);
                l.from[u] = uint16_t(a + g);
                l.cnt[u] = uint8_t(min(group, c - g));
            }
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) *l.nact = int(base >> 16);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMaxSlotsPerThread; ++k)
        if (mine[k] >= 0) {
            const int i = threadIdx.x + 256 * k;
            l.ord[l.cur[mine[k]] + l.hist[(i >> 5) * E + mine[k]] + rank[k]] = uint16_t(i | tok[k] << 10);
            l.w[i] = wsum[k];
        }
}

// ------------------------------------------------------------------ the stream
constexpr int kWarps = 8;
constexpr int kGroup = 8;          // tokens of a group: the MMA's columns
constexpr int kBoxBlocks = 8;      // quant blocks per box
constexpr int kChainBoxes = 16;    // boxes added to one f32 sum (128 blocks, as w4a8_gemm); sums of longer runs are added up
constexpr int kTileBytes = 2048;   // 16 rows x 8 blocks of codes, 128-byte swizzle
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kScaleBytes = 512;   // 2 x 16 rows x 8 fp16
constexpr int kRingBytes = kWarps * kStages * (kStageBytes + kScaleBytes);

// One warp's ring: two 16-row tiles of 8 blocks per stage.
struct Ring : RingCount {
    uint32_t codes, bars;  // shared addresses of this warp's stages and barriers
    uint8_t* scales;

    // Lane 0 of the warp: fetch box j of the rows r0 .. r0+15 and r1 .. r1+15.
    __device__ __forceinline__ void issue(const CUtensorMap* tq, const CUtensorMap* ts, int sc_tma, int j, int r0, int r1) {
        const int st = stage(issued);
        const uint32_t bar = bars + st * 8, q = codes + st * kStageBytes;
        mbar_arrive_expect_tx(bar, kStageBytes + (sc_tma ? kScaleBytes : 0));
        tma_load_2d<1>(q, tq, j * 128, r0, bar);
        tma_load_2d<1>(q + kTileBytes, tq, j * 128, r1, bar);
        if (sc_tma) {
            const uint32_t s = smem_addr(scales + st * kScaleBytes);
            tma_load_2d<2>(s, ts, j * kBoxBlocks, r0, bar);
            tma_load_2d<2>(s + 256, ts, j * kBoxBlocks, r1, bar);
        }
    }
    // Wait for the next box. Without sc_tma (scale rows whose pitch is not a multiple of 16
    // bytes) the warp fetches the box's scales itself, zeros past the row.
    __device__ __forceinline__ void wait(const uint16_t* wd, int sc_tma, int j, int r0, int r1, int B, volatile uint32_t* abort) {
        const int st = stage(used), lane = threadIdx.x & 31;
        if (!sc_tma) {
            uint32_t h[4] = {0u, 0u, 0u, 0u};
            const uint16_t* src = wd + int64_t((lane < 16 ? r0 : r1) + (lane & 15)) * B + j * kBoxBlocks;
#pragma unroll
            for (int i = 0; i < kBoxBlocks; ++i)
                if (j * kBoxBlocks + i < B) h[i >> 1] |= uint32_t(__ldg(src + i)) << (16 * (i & 1));
            *reinterpret_cast<uint4*>(scales + st * kScaleBytes + lane * 16) = make_uint4(h[0], h[1], h[2], h[3]);
            __syncwarp();
        }
        if (!dead && !bounded_wait_warp(bars + st * 8, parity(used), abort)) dead = true;
    }
    __device__ __forceinline__ void drain() {
        for (int i = first_pending(); i < issued; ++i) drain_wait_warp(bars + stage(i) * 8, parity(i), 200000ull);
    }
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding an integer below 2^22 to its bits adds it to its value
// D + kMagic as floats, D = A . B of 16 rows x 8 tokens over one block (|D| <= 16*8*127*32 < 2^22).
__device__ __forceinline__ void mma_s8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    const int m = 0x4B400000;
    int d[4];
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(m));
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __int_as_float(d[i]);
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Signed bytes 16 (q - 8) of the low (elements 0..15 of the block) and high nibbles.
__device__ __forceinline__ uint32_t low_codes(uint32_t r) { return ((r << 4) & 0xF0F0F0F0u) ^ 0x80808080u; }
__device__ __forceinline__ uint32_t high_codes(uint32_t r) { return (r & 0xF0F0F0F0u) ^ 0x80808080u; }
__device__ __forceinline__ float2 halves(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// Activations of a group: codes and scales of the token in column i at xq + row[i] * pitch and
// xd + row[i] * pitch / 32. L2: read past L1 (not used twice by an SM).
template <bool L2>
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
    return L2 ? __ldcg(reinterpret_cast<const uint4*>(p)) : *reinterpret_cast<const uint4*>(p);
}
template <bool L2>
__device__ __forceinline__ float4 load_scales(const float* p) {
    return L2 ? __ldcg(reinterpret_cast<const float4*>(p)) : *reinterpret_cast<const float4*>(p);
}

// This lane's part of a box of 8 tokens: B fragments (column lane/4) and scales (columns 2c,
// 2c+1) of its 8 blocks.
struct Frag {
    uint4 x[4];
    float4 d[4];  // [half box][column]
};
template <bool L2>
__device__ __forceinline__ Frag load_frag(const uint8_t* xb, const float* d0, const float* d1) {
    Frag f;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        f.x[2 * q] = load_codes<L2>(xb + q * 128);
        f.x[2 * q + 1] = load_codes<L2>(xb + q * 128 + 16);
        f.d[2 * q] = load_scales<L2>(d0 + q * 4);
        f.d[2 * q + 1] = load_scales<L2>(d1 + q * 4);
    }
    return f;
}

// One stage: 2 x 16 rows x 8 blocks times 8 tokens. acc[m][h] pairs tokens 2c, 2c+1 (c = lane &
// 3) of row lane/4 + 8 h of tile m. Per block D is exact, and acc += D * (d_w * d_x).
__device__ __forceinline__ void stage_mma(unsigned long long (&acc)[2][2], uint32_t codes, const uint8_t* scales,
                                          const Frag& f) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const uint32_t base = codes + uint32_t(lane >> 4) * kTileBytes + uint32_t((lane & 15) * 128);
    const unsigned long long magic = pack2(-kMagic, -kMagic);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint2 sw[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
            sw[m] = *reinterpret_cast<const uint2*>(scales + (m >> 1) * 256 + (g + (m & 1) * 8) * 16 + q * 8);
        const uint32_t bw[8] = {f.x[2 * q].x,     f.x[2 * q].y,     f.x[2 * q].z,     f.x[2 * q].w,
                                f.x[2 * q + 1].x, f.x[2 * q + 1].y, f.x[2 * q + 1].z, f.x[2 * q + 1].w};
        const float e0[4] = {f.d[2 * q].x, f.d[2 * q].y, f.d[2 * q].z, f.d[2 * q].w};
        const float e1[4] = {f.d[2 * q + 1].x, f.d[2 * q + 1].y, f.d[2 * q + 1].z, f.d[2 * q + 1].w};
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t r[4];
            ldmatrix4(base + uint32_t(((q * 4 + b) ^ (lane & 7)) << 4), r);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float v[4];
                mma_s8(v, low_codes(r[2 * m]), low_codes(r[2 * m + 1]), high_codes(r[2 * m]), high_codes(r[2 * m + 1]),
                       bw[2 * b], bw[2 * b + 1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 p = halves(b < 2 ? sw[2 * m + h].x : sw[2 * m + h].y);
                    const float w = (b & 1) ? p.y : p.x;
                    acc[m][h] = fma2(add2(pack2(v[2 * h], v[2 * h + 1]), magic),
                                     pack2(__fmul_rn(w, e0[b]), __fmul_rn(w, e1[b])), acc[m][h]);
                }
            }
        }
    }
}

// The same stage for a group of one token, a row per lane (row lane & 15 of tile lane >> 4), the
// token's codes broadcast: about 200 instructions against 300 for the MMA form. One token on 64
// experts of 2048 x 1024, top 8: 16.2 us against 17.6 with the MMA form alone; groups of two on
// dp4a as well were slower (4 tokens, top 2 of 8, 4096 x 14336: 125.2 against 122.3 us).
template <bool L2>
__device__ __forceinline__ void stage_dp4a(float& acc, uint32_t codes, const uint8_t* scales, const uint8_t* xb,
                                           const float* db) {
    const int lane = threadIdx.x & 31, row = lane & 15;
    const uint32_t base = codes + uint32_t(lane >> 4) * kTileBytes + uint32_t(row * 128);
    const uint4 sc = *reinterpret_cast<const uint4*>(scales + lane * 16);
    const uint32_t sw[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
    for (int b0 = 0; b0 < 8; b0 += 4) {  // the activations of four blocks are fetched together
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)  // word i % 4 of two blocks
            x[i] = load_codes<L2>(xb + (b0 >> 2) * 128 + (i & 3) * 32 + (i >> 2) * 16);
        const float4 dx = load_scales<L2>(db + b0);
#pragma unroll
        for (int k0 = 0; k0 < 4; k0 += 2) {
            const int b = b0 + k0;
            uint32_t w[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[k][0]), "=r"(w[k][1]), "=r"(w[k][2]), "=r"(w[k][3])
                             : "r"(base + uint32_t(((b + k) ^ (row & 7)) << 4)));
            const float2 dw = halves(sw[b >> 1]);
            int s0 = 0, s1 = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // words i of blocks b and b + 1: both K halves
                const uint4 v = x[2 * k0 + i];
                s0 = __dp4a(int(low_codes(w[0][i])), int(v.x), s0);
                s1 = __dp4a(int(low_codes(w[1][i])), int(v.z), s1);
                s0 = __dp4a(int(high_codes(w[0][i])), int(v.y), s0);
                s1 = __dp4a(int(high_codes(w[1][i])), int(v.w), s1);
            }
            acc = fmaf(float(s0), __fmul_rn(dw.x, k0 ? dx.z : dx.x), acc);
            acc = fmaf(float(s1), __fmul_rn(dw.y, k0 ? dx.w : dx.y), acc);
        }
    }
}

struct Ctrl {
    unsigned long long full[kWarps][kStages];
    uint32_t abort;
};
constexpr int kCtrlBytes = 256;
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");

__device__ __forceinline__ Ring make_ring(uint8_t* smem, Ctrl* ctrl) {
    const int warp = threadIdx.x >> 5;
    Ring r;
    r.codes = smem_addr(smem) + uint32_t(warp * kStages * kStageBytes);
    r.scales = smem + kWarps * kStages * kStageBytes + warp * kStages * kScaleBytes;
    r.bars = smem_addr(&ctrl->full[warp][0]);
    r.reset();
    return r;
}
// The scales' map is encoded, and so prefetched, only with sc_tma.
__device__ __forceinline__ void init_ctrl(Ctrl* ctrl, const CUtensorMap* tq, const CUtensorMap* ts, int sc_tma) {
    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int s = 0; s < kStages; ++s) mbar_init(smem_addr(&ctrl->full[w][s]), 1);
        ctrl->abort = 0;
        mbar_init_fence();
        asm volatile("prefetch.tensormap [%0];" ::"l"(tq) : "memory");
        if (sc_tma) asm volatile("prefetch.tensormap [%0];" ::"l"(ts) : "memory");
    }
}

// The activation rows a lane reads for a group: columns past the group repeat its last token
// (a column never reaches another).
struct Group {
    int first, cnt;
    int b, s0, s1;  // rows of columns lane/4, 2c, 2c+1
    // Rows by token (gate / up) or by slot (down).
    template <bool TOKEN>
    __device__ __forceinline__ void set(const Lists& l, int g) {
        const int lane = threadIdx.x & 31;
        auto row = [](int entry) { return TOKEN ? entry >> 10 : entry & kSlotMask; };
        first = l.from[g];
        cnt = l.cnt[g];
        b = row(int(l.ord[first + min(lane >> 2, cnt - 1)]));
        s0 = row(int(l.ord[first + min(2 * (lane & 3), cnt - 1)]));
        s1 = row(int(l.ord[first + min(2 * (lane & 3) + 1, cnt - 1)]));
    }
};
// Both forms' sums; the other one's stay zero.
struct Sums {
    unsigned long long m[2][2];
    float d;
    __device__ __forceinline__ void clear() {
        m[0][0] = m[0][1] = m[1][0] = m[1][1] = 0ull;
        d = 0.0f;
    }
};

// ------------------------------------------------------------------ gate, up and h
constexpr int kRedPitch = 9;
constexpr int kRedBytes = 4 * 64 * kRedPitch * 4;
__host__ __device__ __forceinline__ size_t gate_up_smem(int E, int n) {
    return 1024 + kRingBytes + kCtrlBytes + kRedBytes + lists_bytes(E, n, kGroup);
}

// Items: (group of at most 8 tokens of one expert, 16 RG rows of I), dealt round-robin to the
// CTAs. RG warps share a K slice's boxes (one per 16 gate and 16 up rows), 8 / RG slices; their
// sums meet in shared memory, where a warp per token and 32 rows forms h, its block's scale
// and codes. RG = 2 spreads few items over the GPU; RG = 4 (I a multiple of 64) halves what an
// item costs beside its boxes. Two CTAs per SM. 64 tokens, top 8 of 64 experts of 2048 x 1024:
// 65 us for 151 MB, bound by instruction issue (32 M warp instructions, 0.53 per cycle and
// scheduler); 4 tokens, top 2 of 8 experts of 4096 x 14336: 118 to 121 us for the whole layer, about
// two thirds of the copy rate, the rest uneven rounds of items.
template <int RG>
__global__ void __launch_bounds__(256, 2)
    gate_up_kernel(int T, int E, int H, int I, int top_k, const int* ids, const float* weights, const uint8_t* xq,
                   const float* xd, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_s,
                   int sc_tma, const uint16_t* __restrict__ wd, uint8_t* __restrict__ hq, float* __restrict__ hd) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + kRingBytes);
    float* red = reinterpret_cast<float*>(smem + kRingBytes + kCtrlBytes);
    const int n = T * top_k;
    const Lists l = lists_at(smem + kRingBytes + kCtrlBytes + kRedBytes, smem, E, n, kGroup);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int SLICES = kWarps / RG, ROWS = 16 * RG;
    const int rg = warp % RG, ksl = warp / RG;
    init_ctrl(ctrl, &tm_q, &tm_s, sc_tma);
    pdl_wait_primary();  // ids, xq and xd are written by the preceding kernel
    pdl_launch_dependents();
    build_lists(l, ids, weights, n, top_k, E, kGroup);
    fence_proxy_async_smem();  // the lists' scratch lies in the ring, which TMA writes next
    __syncthreads();
    const int B = H / 32, Bp = padded_blocks(H), nbox = Bp / kBoxBlocks;
    const int IB = I / 32, IBp = padded_blocks(I), IR = I / ROWS;
    const int nitems = *l.nact * IR;
    Ring ring = make_ring(smem, ctrl);
    // the next box to fetch: item, box, first gate row
    int pi = blockIdx.x, pj = ksl, pr = 0;
    auto row_of = [&](int item) {
        const int gi = item / IR;
        return int(l.act[gi]) * 2 * I + (item - gi * IR) * ROWS + rg * 16;
    };
    const bool any = ksl < nbox;
    if (any && pi < nitems) pr = row_of(pi);
    auto fetch = [&]() {
        if (!any || pi >= nitems || ring.dead) return;
        if (lane == 0) ring.issue(&tm_q, &tm_s, sc_tma, pj, pr, pr + I);
        ++ring.issued;
        pj += SLICES;
        if (pj >= nbox) {
            pj = ksl;
            pi += gridDim.x;
            if (pi < nitems) pr = row_of(pi);
        }
    };
    fetch();
    fetch();

    for (int item = blockIdx.x; item < nitems; item += gridDim.x) {
        const int gi = item / IR, ir = item - gi * IR;
        const int r = int(l.act[gi]) * 2 * I + ir * ROWS + rg * 16;
        Group gr;
        gr.template set<true>(l, gi);
        const bool one = gr.cnt == 1;
        const int pitch = Bp * 32;
        const uint8_t* xb = xq + gr.b * pitch;
        const float *d0 = xd + gr.s0 * Bp, *d1 = xd + gr.s1 * Bp;
        Sums acc;
        float* p = red + ksl * 2 * ROWS * kRedPitch;  // gate rows, up rows
        int j = ksl;
#pragma unroll 1
        for (bool first = true; first || j < nbox; first = false) {
            const int end = min(nbox, j + SLICES * kChainBoxes);
            acc.clear();
#pragma unroll 1
            for (; j < end; j += SLICES) {
                const int st = Ring::stage(ring.used);
                const uint32_t cq = ring.codes + st * kStageBytes;
                const uint8_t* cs = ring.scales + st * kScaleBytes;
                if (one) {
                    ring.wait(wd, sc_tma, j, r, r + I, B, &ctrl->abort);
                    stage_dp4a<false>(acc.d, cq, cs, xb + j * 256, d0 + j * 8);
                } else {
                    const Frag f = load_frag<false>(xb + (lane & 3) * 32 + j * 256, d0 + j * 8, d1 + j * 8);
                    ring.wait(wd, sc_tma, j, r, r + I, B, &ctrl->abort);
                    stage_mma(acc.m, cq, cs, f);
                }
                __syncwarp();
                ++ring.used;
                fetch();
            }
            // into this warp's words of the sums, each always the same lane's
            auto put = [&](float* q, float v) { *q = first ? v : __fadd_rn(*q, v); };
            if (one) {
                put(p + ((lane >> 4) * ROWS + rg * 16 + (lane & 15)) * kRedPitch, acc.d);
            } else {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    float a, b;
                    unpack2(acc.m[m >> 1][m & 1], a, b);
                    float* q = p + ((m >> 1) * ROWS + rg * 16 + (m & 1) * 8 + (lane >> 2)) * kRedPitch + 2 * (lane & 3);
                    put(q, a);
                    put(q + 1, b);
                }
            }
        }
        __syncthreads();
        for (int tb = warp; tb < gr.cnt * (RG / 2); tb += kWarps) {  // token, 32 rows of the item
            const int t = RG == 2 ? tb : tb >> 1, half = RG == 2 ? 0 : tb & 1;
            const int slot = l.ord[gr.first + t] & kSlotMask, ib = ir * (RG / 2) + half;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int s = 0; s < SLICES; ++s) {
                const float* q = red + (s * 2 * ROWS + half * 32 + lane) * kRedPitch + t;
                gate = __fadd_rn(gate, q[0]);
                up = __fadd_rn(up, q[ROWS * kRedPitch]);
            }
            const float hv = __fmul_rn(__fdiv_rn(gate, 1.0f + expf(-gate)), up);
            float amax = fabsf(hv);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // the maximum passes over a NaN, whose code is 0: the scale carries it on
            const bool nan = __any_sync(0xffffffffu, hv != hv);
            const float d = nan ? __int_as_float(0x7FC00000) : __fdiv_rn(amax, 127.0f);
            const float id = d != 0.0f ? __frcp_rn(d) : 0.0f;
            const int code = max(-127, min(127, int(roundf(__fmul_rn(hv, id)))));
            uint32_t w = (uint32_t(code) & 0xFFu) << (8 * (lane & 3));
            w |= __shfl_xor_sync(0xffffffffu, w, 1);
            w |= __shfl_xor_sync(0xffffffffu, w, 2);
            if ((lane & 3) == 0)
                *reinterpret_cast<uint32_t*>(hq + int64_t(slot) * IBp * 32 + word_offset(ib, lane >> 2)) = w;
            if (lane == 0) hd[int64_t(slot) * IBp + ib] = __fmul_rn(d, 0.0625f);
            if (ib == IB - 1 && lane < IBp - IB) hd[int64_t(slot) * IBp + IB + lane] = 0.0f;  // the padding
        }
        __syncthreads();
    }
    ring.drain();
}

// ------------------------------------------------------------------ down and the weighted sum
constexpr int kDownTokens = 32;  // tokens of one CTA: the warps' sums take 1 KB of shared memory each
constexpr int kYPitch = 33;
__host__ __device__ __forceinline__ size_t down_smem(int T, int E, int n) {
    return 1024 + kRingBytes + kCtrlBytes + size_t(kWarps) * T * kYPitch * 4 + lists_bytes(E, n, kGroup);
}

// Grid: x = split (the cluster), y = 32 rows of H, z = 32 tokens. The boxes of all used experts
// for those rows are dealt in runs to the warps of the cluster; each warp adds its sums,
// times the slots' weights, to a [token][row] array of its own, and the arrays are added in a
// fixed order (within the CTA, then across the cluster through distributed shared memory).
// 64 tokens, top 8 of 64 experts of 2048 x 1024: 50 us for 75 MB, bound by instruction issue.
__global__ void __launch_bounds__(256, 2)
    down_kernel(int Tall, int E, int H, int I, int top_k, const int* ids, const float* weights, const uint8_t* hq,
                const float* hd, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_s,
                int sc_tma, const uint16_t* __restrict__ wd, void* __restrict__ y, int out_bf16) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + kRingBytes);
    float* ybuf = reinterpret_cast<float*>(smem + kRingBytes + kCtrlBytes);
    // this CTA's tokens: ids, weights and h start at its first slot
    const int tok0 = blockIdx.z * kDownTokens, T = min(kDownTokens, Tall - tok0);
    const int n = T * top_k, YT = T * kYPitch;
    const int B = I / 32, Bp = padded_blocks(I), nbox = Bp / kBoxBlocks, pitch = Bp * 32;
    ids += tok0 * top_k;
    weights += tok0 * top_k;
    hq += int64_t(tok0) * top_k * pitch;
    hd += int64_t(tok0) * top_k * Bp;
    const Lists l = lists_at(reinterpret_cast<uint8_t*>(ybuf + kWarps * YT), smem, E, n, kGroup);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.y * 32, slices = gridDim.x * kWarps;
    init_ctrl(ctrl, &tm_q, &tm_s, sc_tma);
    for (int i = threadIdx.x; i < kWarps * YT; i += 256) ybuf[i] = 0.0f;
    // Read before the wait: ids and weights come from the kernel before the preceding one,
    // which has completed, since every CTA of the preceding kernel waits for it before it
    // lets this grid start (and the loads are from L2).
    build_lists(l, ids, weights, n, top_k, E, kGroup);
    fence_proxy_async_smem();
    __syncthreads();
    const int nact = *l.nact;
    Ring ring = make_ring(smem, ctrl);
    // this warp's boxes of all groups' boxes in order: one run, so that a group's sums are
    // flushed once per warp that meets it (and every kChainBoxes boxes)
    const int64_t total = int64_t(nact) * nbox, s = blockIdx.x * kWarps + warp;
    int left = int((s + 1) * total / slices - s * total / slices), pleft = left;
    int pg = int(s * total / slices / nbox), pj = int(s * total / slices - int64_t(pg) * nbox);  // the next box to fetch
    auto fetch = [&]() {
        if (pleft == 0 || ring.dead) return;
        if (lane == 0) {
            const int r = int(l.act[pg]) * H + n0;
            ring.issue(&tm_q, &tm_s, sc_tma, pj, r, r + 16);
        }
        ++ring.issued;
        --pleft;
        if (++pj == nbox) {
            pj = 0;
            ++pg;
        }
    };
    int ug = pg, uj = pj;  // the box in hand
    fetch();
    fetch();
    pdl_wait_primary();  // hq and hd

    float* yw = ybuf + warp * YT;
    auto flush = [&](const Group& gr, const Sums& acc) {
        if (gr.cnt == 1) {
            const int entry = l.ord[gr.first];
            float* p = yw + (entry >> 10) * kYPitch + lane;
            *p = fmaf(l.w[entry & kSlotMask], acc.d, *p);
        } else {
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                const int at = 2 * (lane & 3) + col;
                if (at >= gr.cnt) continue;
                const int entry = l.ord[gr.first + at];
                const float w = l.w[entry & kSlotMask];
                float* p = yw + (entry >> 10) * kYPitch + (lane >> 2);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    float v0, v1;
                    unpack2(acc.m[m >> 1][m & 1], v0, v1);
                    p[m * 8] = fmaf(w, col ? v1 : v0, p[m * 8]);
                }
            }
        }
        __syncwarp();
    };
#pragma unroll 1
    while (left > 0) {  // the run's part in one group, at most kChainBoxes boxes at a time
        const int end = min(uj + min(left, kChainBoxes), nbox);
        left -= end - uj;
        Group gr;
        gr.template set<false>(l, ug);
        const uint8_t* xb = hq + int64_t(gr.b) * pitch;
        const float *d0 = hd + int64_t(gr.s0) * Bp, *d1 = hd + int64_t(gr.s1) * Bp;
        const int r = int(l.act[ug]) * H + n0;
        Sums acc;
        acc.clear();
#pragma unroll 1
        for (; uj < end; ++uj) {
            const int st = Ring::stage(ring.used);
            const uint32_t cq = ring.codes + st * kStageBytes;
            const uint8_t* cs = ring.scales + st * kScaleBytes;
            if (gr.cnt == 1) {
                ring.wait(wd, sc_tma, uj, r, r + 16, B, &ctrl->abort);
                stage_dp4a<true>(acc.d, cq, cs, xb + uj * 256, d0 + uj * 8);
            } else {
                const Frag f = load_frag<true>(xb + (lane & 3) * 32 + uj * 256, d0 + uj * 8, d1 + uj * 8);
                ring.wait(wd, sc_tma, uj, r, r + 16, B, &ctrl->abort);
                stage_mma(acc.m, cq, cs, f);
            }
            __syncwarp();
            ++ring.used;
            fetch();
        }
        flush(gr, acc);
        if (uj == nbox) {
            uj = 0;
            ++ug;
        }
    }
    ring.drain();
    __syncthreads();
    for (int i = threadIdx.x; i < T * 32; i += 256) {
        float* p = ybuf + (i >> 5) * kYPitch + (i & 31);
        float v = p[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = __fadd_rn(v, p[w * YT]);
        p[0] = v;
    }
    const int cs = gridDim.x;
    if (cs > 1)
        cluster_sync();
    else
        __syncthreads();
    if (!*reinterpret_cast<volatile uint32_t*>(&ctrl->abort)) {
        for (int i = blockIdx.x * 256 + threadIdx.x; i < T * 32; i += cs * 256) {
            const uint32_t p = smem_addr(ybuf + (i >> 5) * kYPitch + (i & 31));
            float v = 0.0f;
            for (int z = 0; z < cs; ++z) {
                float u;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(mapa_shared(p, z)));
                v = __fadd_rn(v, u);
            }
            const int64_t o = int64_t(tok0 + (i >> 5)) * H + n0 + (i & 31);
            if (out_bf16)
                reinterpret_cast<__nv_bfloat16*>(y)[o] = __float2bfloat16_rn(v);
            else
                reinterpret_cast<float*>(y)[o] = v;
        }
    }
    if (cs > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

}  // namespace moe
}  // namespace w4a8
