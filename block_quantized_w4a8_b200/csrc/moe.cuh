// Mixture-of-experts layer for a few tokens with Q4_0 experts and Q8_0 activations:
//   router   l = x . Wr^T, the top_k largest logits, p = softmax over them or over all
//   experts  g, u = xq . Wg^T, xq . Wu^T;  h = g / (1 + exp(-g)) * u;  hq = Q8_0(h)
//   output   y[t] = sum over slots s of p[t][s] * (hq[t][s] . Wd[e(t, s)]^T)
// with the block dots of w4a8_gemm (exact integers, rescaled per 32-block in f32).
//
// Three launches: route (one cluster per token; also quantises x), gate_up (g, u, h and its
// Q8_0 form) and down (the weighted sum). The weights of the chosen experts are read once and
// are nearly all the traffic, so both expert kernels are built around the stream: every warp
// runs a ring of TMA boxes of its own (32 rows x 8 blocks), with no barrier between warps
// until its rows are summed. The dots are mma.sync.m16n8k32 on int8, one per 16 rows and
// quant block: the instruction's K is the block, its A fragment is the packed codes as they
// lie in memory (one ldmatrix word holds the low and high nibbles of both K halves), and 8
// tokens cost what one costs. tcgen05 would need the codes expanded to shared or tensor
// memory first, and reads its accumulators back per block; at these sizes the memory is the
// bound, not the matrix rate.
#pragma once

#include <cuda.h>

#include "device_common.cuh"

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

// Grid: kRouteCtas CTAs (a cluster) per token. Every CTA quantises its share of the token's
// blocks (xq != nullptr) and, with ROUTE, computes the logits of its experts, a warp each;
// they meet in the first CTA's shared memory, where one warp takes the top_k.
template <bool ROUTE, bool XB, bool WB>
__global__ void __launch_bounds__(256) route_kernel(int E, int H, int top_k, int renorm, const void* __restrict__ x,
                                                    const void* __restrict__ wr, int* __restrict__ ids,
                                                    float* __restrict__ weights, uint8_t* __restrict__ xq,
                                                    float* __restrict__ xd) {
    __shared__ float logit[kMaxExperts];
    const int t = blockIdx.x / kRouteCtas, rank = blockIdx.x % kRouteCtas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    if (ROUTE) {
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        bool waited = false;
        for (int e = rank + kRouteCtas * warp; e < E; e += kRouteCtas * 8) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
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
    }
    if (xq) {
        const int B = H / 32, Bp = padded_blocks(H), sub = threadIdx.x & 7;
        for (int b0 = rank * 32; b0 < Bp; b0 += 32 * kRouteCtas) {
            const int b = b0 + int(threadIdx.x >> 3);
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (b < B) load4<XB>(x, int64_t(t) * H + b * 32 + sub * 4, v);
            const float amax = warp_max8(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
            const float d = __fdiv_rn(amax, 127.0f);
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
    cluster_sync();  // the logits are in the first CTA
    if (rank != 0 || warp != 0) return;
    uint32_t key[kMaxExperts / 32];
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) key[i] = lane + 32 * i < E ? order_key(logit[lane + 32 * i]) : 0u;
    uint32_t taken = 0u;  // bit i: this lane's expert lane + 32 i is chosen
    float top = 0.0f, sum = 0.0f, mine = 0.0f;
    for (int s = 0; s < top_k; ++s) {
        uint32_t best = 0u;
        unsigned at = 0x7fffffffu;
#pragma unroll
        for (int i = kMaxExperts / 32 - 1; i >= 0; --i)  // the lowest index among equals
            if (lane + 32 * i < E && !((taken >> i) & 1u) && key[i] >= best) {
                best = key[i];
                at = unsigned(lane + 32 * i);
            }
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        const int e = int(__reduce_min_sync(0xffffffffu, best == m ? at : 0x7fffffffu));
        if ((e & 31) == lane) taken |= 1u << (e >> 5);
        const float l = logit[e];
        if (s == 0) top = l;
        const float p = expf(l - top);
        sum += p;
        if (lane == s) {
            mine = p;
            ids[int64_t(t) * top_k + s] = e;
        }
    }
    if (!renorm) {
        sum = 0.0f;
        for (int e = lane; e < E; e += 32) sum += expf(logit[e] - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < top_k) weights[int64_t(t) * top_k + lane] = __fdiv_rn(mine, sum);
}

// ------------------------------------------------------------------ who uses which expert
// Built by every CTA in shared memory from the T x top_k slots. A slot that names its
// token's expert again is folded into the first one (their weights added), so a token is at
// most once in an expert's list. Lists longer than `group` tokens are cut into groups, each a
// pass of its own over the expert's weights.
struct Lists {
    int* id;         // [n] expert of a slot, -1: empty or folded
    float* w;        // [n] weight of a slot (folded)
    int* cur;        // [E] scratch
    uint16_t* act;   // [max groups] expert of a group, in rising order
    uint16_t* from;  // first entry of a group
    uint16_t* ord;   // [n] slots by expert
    uint8_t* cnt;    // tokens of a group
    uint8_t* hist;   // [n / 32][E] scratch: tokens of an expert in each 32 slots
    int* nact;       // groups
};
__host__ __device__ __forceinline__ int max_groups(int E, int n, int group) { return (E < n ? E : n) + n / group; }
__host__ __device__ __forceinline__ size_t lists_bytes(int E, int n, int group) {
    return size_t(E + 1) * 4 + size_t(n) * 8 +
           (size_t(max_groups(E, n, group)) * 5 + size_t(n) * 2 + size_t(n + 31) / 32 * E + 15) / 16 * 16;
}
__device__ __forceinline__ Lists lists_at(uint8_t* p, int E, int n, int group) {
    const int m = max_groups(E, n, group);
    Lists l;
    l.id = reinterpret_cast<int*>(p);
    l.w = reinterpret_cast<float*>(l.id + n);
    l.cur = reinterpret_cast<int*>(l.w + n);
    l.nact = l.cur + E;
    l.act = reinterpret_cast<uint16_t*>(l.nact + 1);
    l.from = l.act + m;
    l.ord = l.from + m;
    l.cnt = reinterpret_cast<uint8_t*>(l.ord + n);
    l.hist = l.cnt + m;
    return l;
}
// Entries stand in the order of the slots, so that every CTA cuts the same groups. All
// threads of the CTA (256) call it; ids and weights are read from L2.
__device__ __forceinline__ void build_lists(const Lists& l, const int* ids, const float* weights, int n, int top_k, int E,
                                            int group) {
    for (int i = threadIdx.x; i < n; i += 256) {
        const int id = __ldcg(ids + i);
        l.id[i] = id >= 0 && id < E ? id : -1;
        l.w[i] = __ldcg(weights + i);
    }
    const int chunks = (n + 31) / 32;
    for (int e = threadIdx.x; e < chunks * E; e += 256) l.hist[e] = 0;
    __syncthreads();
    int mine[kMaxSlotsPerThread];
    int rank[kMaxSlotsPerThread];  // among the 32 slots of this warp's chunk
    float wsum[kMaxSlotsPerThread];
#pragma unroll
    for (int k = 0; k < kMaxSlotsPerThread; ++k) {
        const int i = threadIdx.x + 256 * k;
        mine[k] = i < n ? l.id[i] : -1;
        if (i - int(threadIdx.x & 31) >= n) continue;  // the whole warp
        if (mine[k] >= 0) {
            const int s0 = i / top_k * top_k, id = mine[k];
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
    if (threadIdx.x < 32) {  // first entries and groups: 8 experts per lane
        const int lane = threadIdx.x;
        int c[8], sum = 0, used = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = lane * 8 + i < E ? l.cur[lane * 8 + i] : 0;
            sum += c[i];
            used += (c[i] + group - 1) / group;
        }
        int a = sum, u = used;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int pa = __shfl_up_sync(0xffffffffu, a, o), pu = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) {
                a += pa;
                u += pu;
            }
        }
        if (lane == 31) *l.nact = u;
        a -= sum;
        u -= used;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane * 8 + i < E) {
                l.cur[lane * 8 + i] = a;
                for (int g = 0; g < c[i]; g += group, ++u) {
                    l.act[u] = uint16_t(lane * 8 + i);
                    l.from[u] = uint16_t(a + g);
                    l.cnt[u] = uint8_t(min(group, c[i] - g));
                }
                a += c[i];
            }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMaxSlotsPerThread; ++k)
        if (mine[k] >= 0) {
            const int i = threadIdx.x + 256 * k;
            l.ord[l.cur[mine[k]] + l.hist[(i >> 5) * E + mine[k]] + rank[k]] = uint16_t(i);
            l.w[i] = wsum[k];
        }
    __syncthreads();
}

// ------------------------------------------------------------------ the weight stream
constexpr int kWarps = 8;
constexpr int kStages = 2;         // boxes in flight per warp
constexpr int kBoxBlocks = 8;      // quant blocks per box
constexpr int kTileBytes = 2048;   // 16 rows x 8 blocks of codes, 128-byte swizzle
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kScaleBytes = 512;   // 2 x 16 rows x 8 fp16
constexpr int kRingBytes = kWarps * kStages * (kStageBytes + kScaleBytes);

// One warp's ring: two 16-row tiles of 8 blocks per stage.
struct Ring {
    uint32_t codes, bars;  // shared addresses of this warp's stages and barriers
    uint8_t* scales;
    int issued, used;
    bool dead;             // a wait ran out: nothing more is issued or waited for

    // Lane 0 of the warp: fetch box j of the rows r0 .. r0+15 and r1 .. r1+15.
    __device__ __forceinline__ void issue(const CUtensorMap* tq, const CUtensorMap* ts, int sc_tma, int j, int r0, int r1) {
        const int st = issued % kStages;
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
        const int st = used % kStages, lane = threadIdx.x & 31;
        uint32_t h[4] = {0u, 0u, 0u, 0u};
        if (!sc_tma) {
            const uint16_t* src = wd + int64_t((lane < 16 ? r0 : r1) + (lane & 15)) * B + j * kBoxBlocks;
#pragma unroll
            for (int i = 0; i < kBoxBlocks; ++i)
                if (j * kBoxBlocks + i < B) h[i >> 1] |= uint32_t(__ldg(src + i)) << (16 * (i & 1));
        }
        if (!dead && !bounded_wait_warp(bars + st * 8, (used / kStages) & 1, abort)) dead = true;
        if (!sc_tma) {
            *reinterpret_cast<uint4*>(scales + st * kScaleBytes + lane * 16) = make_uint4(h[0], h[1], h[2], h[3]);
            __syncwarp();
        }
    }
    __device__ __forceinline__ void drain() {
        for (int i = used; i < issued; ++i) drain_wait_warp(bars + (i % kStages) * 8, (i / kStages) & 1, 200000ull);
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
__device__ __forceinline__ float half_at(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __half2float(__ushort_as_half(uint16_t((i & 1) ? w >> 16 : w & 0xFFFFu)));
}

// Accumulators of a warp: per 8-token tile, for each of the two 16-row tiles, the pairs of
// tokens 2c, 2c+1 (c = lane & 3) of rows lane/4 and lane/4 + 8.
template <int NT>
struct Acc {
    unsigned long long v[NT][2][2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m) v[i][m >> 1][m & 1] = 0ull;
    }
};
// Rows of the activation matrix this lane reads for each 8-token tile: column lane/4 of the B
// fragment, columns 2c and 2c+1 for the scales. Columns past the list repeat its last entry.
template <int NT>
struct Rows {
    int b[NT], s0[NT], s1[NT];
};

// One box: 32 rows x 8 blocks times nt tiles of 8 tokens; xq, xd already at the box's columns.
// Per block the integer dot D is exact and enters as round(D * d_w) * d_x, added in f32.
template <int NT>
__device__ __forceinline__ void box_dots(Acc<NT>& acc, uint32_t codes, const uint8_t* scales, const uint8_t* xq,
                                         const float* xd, int pitch, int spitch, const Rows<NT>& rows, int nt) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t base = codes + uint32_t(lane >> 4) * kTileBytes + uint32_t((lane & 15) * 128);
    uint4 sw[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) sw[m] = *reinterpret_cast<const uint4*>(scales + (m >> 1) * 256 + (g + (m & 1) * 8) * 16);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t a[4][8];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            uint32_t r[4];
            ldmatrix4(base + uint32_t(((q * 4 + b) ^ (lane & 7)) << 4), r);
#pragma unroll
            for (int m = 0; m < 4; ++m) {  // 16 (q - 8) as signed bytes: low nibbles (K 0..15), high nibbles (K 16..31)
                a[b][(m >> 1) * 4 + (m & 1)] = ((r[m] << 4) & 0xF0F0F0F0u) ^ 0x80808080u;
                a[b][(m >> 1) * 4 + 2 + (m & 1)] = (r[m] & 0xF0F0F0F0u) ^ 0x80808080u;
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (i >= nt) break;
            const uint4* px = reinterpret_cast<const uint4*>(xq + rows.b[i] * pitch + q * 128 + c * 32);
            const uint4 x0 = px[0], x1 = px[1];
            const float4 d0 = *reinterpret_cast<const float4*>(xd + rows.s0[i] * spitch + q * 4);
            const float4 d1 = *reinterpret_cast<const float4*>(xd + rows.s1[i] * spitch + q * 4);
            const uint32_t bw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            const float e0[4] = {d0.x, d0.y, d0.z, d0.w}, e1[4] = {d1.x, d1.y, d1.z, d1.w};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const unsigned long long dx = pack2(e0[b], e1[b]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float f[4];
                    mma_s8(f, a[b][m * 4], a[b][m * 4 + 1], a[b][m * 4 + 2], a[b][m * 4 + 3], bw[2 * b], bw[2 * b + 1]);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float w = half_at(sw[m * 2 + r], q * 4 + b), n = __fmul_rn(-kMagic, w);  // exact
                        const unsigned long long v = fma2(pack2(f[2 * r], f[2 * r + 1]), pack2(w, w), pack2(n, n));
                        acc.v[i][m][r] = fma2(v, dx, acc.v[i][m][r]);
                    }
                }
            }
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
    r.issued = r.used = 0;
    r.dead = false;
    return r;
}
__device__ __forceinline__ void init_ctrl(Ctrl* ctrl) {
    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int s = 0; s < kStages; ++s) mbar_init(smem_addr(&ctrl->full[w][s]), 1);
        ctrl->abort = 0;
        mbar_init_fence();
    }
}

// ------------------------------------------------------------------ gate, up and h
constexpr int kRedPitch = 9;
constexpr int kRedBytes = 4 * 64 * kRedPitch * 4;
__host__ __device__ __forceinline__ size_t gate_up_smem(int E, int n, int group) {
    return 1024 + kRingBytes + kCtrlBytes + kRedBytes + lists_bytes(E, n, group);
}

// Items: (32 rows of I, group of tokens of one expert), dealt round-robin to the CTAs. Two warps share a
// K slice's boxes (one per 16 gate and 16 up rows), four slices; their sums meet in shared
// memory, where a warp per token forms h, its block's scale and codes. NT:
// 8-token tiles of a group.
template <int NT>
__global__ void __launch_bounds__(256, 2)
    gate_up_kernel(int T, int E, int H, int I, int top_k, const int* ids, const float* weights, const uint8_t* xq, const float* xd,
                   const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_s, int sc_tma,
                   const uint16_t* __restrict__ wd, uint8_t* __restrict__ hq, float* __restrict__ hd) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + kRingBytes);
    float* red = reinterpret_cast<float*>(smem + kRingBytes + kCtrlBytes);
    const int n = T * top_k;
    const Lists l = lists_at(smem + kRingBytes + kCtrlBytes + kRedBytes, E, n, 8 * NT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rg = warp & 1, ksl = warp >> 1;
    init_ctrl(ctrl);
    pdl_wait_primary();  // ids, xq and xd are written by the preceding kernel
    pdl_launch_dependents();
    build_lists(l, ids, weights, n, top_k, E, 8 * NT);  // its barriers also publish the control block
    const int B = H / 32, Bp = padded_blocks(H), nbox = Bp / kBoxBlocks;
    const int IB = I / 32, IBp = padded_blocks(I);
    const int nitems = *l.nact * IB;
    Ring ring = make_ring(smem, ctrl);
    int pi = blockIdx.x, pj = ksl;  // the next box to fetch: item, box
    auto row_of = [&](int item) { return int(l.act[item / IB]) * 2 * I + (item % IB) * 32 + rg * 16; };
    auto fetch = [&]() {
        if (ksl >= nbox || pi >= nitems || ring.dead) return;
        if (lane == 0) {
            const int r = row_of(pi);
            ring.issue(&tm_q, &tm_s, sc_tma, pj, r, r + I);
        }
        ++ring.issued;
        pj += 4;
        if (pj >= nbox) {
            pj = ksl;
            pi += gridDim.x;
        }
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) fetch();

    for (int item = blockIdx.x; item < nitems; item += gridDim.x) {
        const int gi = item / IB, ib = item - gi * IB;
        const int first = l.from[gi], cnt = l.cnt[gi], nt = (cnt + 7) / 8;
        const int r = row_of(item);
        Rows<NT> rows;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            auto at = [&](int col) { return int(l.ord[first + min(i * 8 + col, cnt - 1)]) / top_k; };
            rows.b[i] = at(lane >> 2);
            rows.s0[i] = at(2 * (lane & 3));
            rows.s1[i] = at(2 * (lane & 3) + 1);
        }
        Acc<NT> acc;
        acc.clear();
        for (int j = ksl; j < nbox; j += 4) {
            ring.wait(wd, sc_tma, j, r, r + I, B, &ctrl->abort);
            const int st = ring.used % kStages;
            box_dots<NT>(acc, ring.codes + st * kStageBytes, ring.scales + st * kScaleBytes, xq + j * 256,
                         xd + j * kBoxBlocks, Bp * 32, Bp, rows, nt);
            __syncwarp();
            ++ring.used;
            fetch();
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (i >= nt) break;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float a, b;
                    unpack2(acc.v[i][m][h], a, b);
                    float* p = red + (ksl * 64 + m * 32 + rg * 16 + h * 8 + (lane >> 2)) * kRedPitch + 2 * (lane & 3);
                    p[0] = a;
                    p[1] = b;
                }
            __syncthreads();
            if (i * 8 + warp < cnt) {
                const int slot = l.ord[first + i * 8 + warp];
                float gate = 0.0f, up = 0.0f;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    gate = __fadd_rn(gate, red[(s * 64 + lane) * kRedPitch + warp]);
                    up = __fadd_rn(up, red[(s * 64 + 32 + lane) * kRedPitch + warp]);
                }
                const float hv = __fmul_rn(__fdiv_rn(gate, 1.0f + expf(-gate)), up);
                float amax = fabsf(hv);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const float d = __fdiv_rn(amax, 127.0f);
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
    }
    ring.drain();
}

// ------------------------------------------------------------------ down and the weighted sum
constexpr int kYPitch = 33;
__host__ __device__ __forceinline__ size_t down_smem(int T, int E, int n, int group) {
    return 1024 + kRingBytes + kCtrlBytes + size_t(kWarps) * T * kYPitch * 4 + lists_bytes(E, n, group);
}

// Grid: x = split (the cluster), y = 32 rows of H. The boxes of all used experts for those
// rows are dealt round-robin to the warps of the cluster; each warp adds its sums, times the
// slots' weights, to a [token][row] array of its own, and the arrays are added in a fixed
// order (within the CTA, then across the cluster through distributed shared memory).
template <int NT>
__global__ void __launch_bounds__(256, 2)
    down_kernel(int T, int E, int H, int I, int top_k, const int* ids, const float* weights, const uint8_t* hq,
                const float* hd, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_s,
                int sc_tma, const uint16_t* __restrict__ wd, void* __restrict__ y, int out_bf16) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + kRingBytes);
    float* ybuf = reinterpret_cast<float*>(smem + kRingBytes + kCtrlBytes);
    const int n = T * top_k, YT = T * kYPitch;
    const Lists l = lists_at(reinterpret_cast<uint8_t*>(ybuf + kWarps * YT), E, n, 8 * NT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.y * 32, slices = gridDim.x * kWarps;
    init_ctrl(ctrl);
    for (int i = threadIdx.x; i < kWarps * YT; i += 256) ybuf[i] = 0.0f;
    // Read before the wait: ids and weights come from the kernel before the preceding one,
    // which has completed, since every CTA of the preceding kernel waits for it before it
    // lets this grid start (and the loads are from L2).
    build_lists(l, ids, weights, n, top_k, E, 8 * NT);
    const int B = I / 32, Bp = padded_blocks(I), nbox = Bp / kBoxBlocks;
    const int nchunks = *l.nact * nbox;
    Ring ring = make_ring(smem, ctrl);
    int pc = blockIdx.x * kWarps + warp;
    auto fetch = [&]() {
        if (pc >= nchunks || ring.dead) return;
        if (lane == 0) {
            const int r = int(l.act[pc / nbox]) * H + n0;
            ring.issue(&tm_q, &tm_s, sc_tma, pc % nbox, r, r + 16);
        }
        ++ring.issued;
        pc += slices;
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) fetch();
    pdl_wait_primary();  // hq and hd

    float* yw = ybuf + warp * YT;
    Acc<NT> acc;
    Rows<NT> rows;
    int a = -1, first = 0, cnt = 0, nt = 0;
    auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (i >= nt) break;
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                const int at = i * 8 + 2 * (lane & 3) + col;
                if (at >= cnt) continue;
                const int slot = l.ord[first + at];
                const float w = l.w[slot];
                float* p = yw + slot / top_k * kYPitch + (lane >> 2);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    float v0, v1;
                    unpack2(acc.v[i][m >> 1][m & 1], v0, v1);
                    p[m * 8] = fmaf(w, col ? v1 : v0, p[m * 8]);
                }
            }
        }
    };
    for (int c = blockIdx.x * kWarps + warp; c < nchunks; c += slices) {
        const int an = c / nbox, j = c - an * nbox;
        if (an != a) {
            if (a >= 0) flush();
            a = an;
            first = l.from[a];
            cnt = l.cnt[a];
            nt = (cnt + 7) / 8;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                auto at = [&](int col) { return int(l.ord[first + min(i * 8 + col, cnt - 1)]); };
                rows.b[i] = at(lane >> 2);
                rows.s0[i] = at(2 * (lane & 3));
                rows.s1[i] = at(2 * (lane & 3) + 1);
            }
            acc.clear();
        }
        const int r = int(l.act[a]) * H + n0;
        ring.wait(wd, sc_tma, j, r, r + 16, B, &ctrl->abort);
        const int st = ring.used % kStages;
        box_dots<NT>(acc, ring.codes + st * kStageBytes, ring.scales + st * kScaleBytes, hq + j * 256,
                     hd + j * kBoxBlocks, Bp * 32, Bp, rows, nt);
        __syncwarp();
        ++ring.used;
        fetch();
    }
    if (a >= 0) flush();
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
    if (!ctrl->abort) {
        for (int i = blockIdx.x * 256 + threadIdx.x; i < T * 32; i += cs * 256) {
            const uint32_t p = smem_addr(ybuf + (i >> 5) * kYPitch + (i & 31));
            float v = 0.0f;
            for (int z = 0; z < cs; ++z) {
                float u;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(mapa_shared(p, z)));
                v = __fadd_rn(v, u);
            }
            const int64_t o = int64_t(i >> 5) * H + n0 + (i & 31);
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
