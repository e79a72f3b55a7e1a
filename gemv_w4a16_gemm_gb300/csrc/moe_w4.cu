// moe_w4.cu -- a mixture-of-experts layer for 1 to 64 tokens whose experts'
// weights are in the packed W4 format:
//
//     l = x R^T;  score = softmax(l) or sigmoid(l);  the topk experts by l, or by score + bias;
//     weight = scale * score (divided by the chosen scores' sum);
//     out[m] = sum_chosen weight * W2_e (silu(gate_e x) * up_e x).
//
// What bounds it: the chosen experts' weights, 19/32 bytes each, are read once
// from HBM; with one token that is a few microseconds, so launches and the
// depth of dependent loads count more (8 of 128 experts of 2048 x 768: 20.8 us,
// 6.3 of them routing, for 3.4 of bytes).  With more tokens the products' 2.2
// instructions a weight and lane, at the latency of 3 warps a scheduler, take
// longer than the bytes (64 tokens, 2 of 16 experts of 6656 x 4096: 183 us for
// 115, half of the issue slots in use).
//
// Four launches, each started while its predecessor finishes:
//   route    one cluster of 8 CTAs: the logits as m16n8k16 MMAs (bf16 products,
//            fp32 sums) split over the cluster's 64 warps by experts and K;
//            CTA r joins those of tokens 8r .. 8r + 7 in its shared memory and
//            chooses, a warp a token; the first CTA sorts the choices by expert
//            for the products.  Other clusters meanwhile write x in the order
//            of the MMA fragments.
//   gate/up  h = silu(gate) * up for every (token, chosen expert)
//   down     y = W2 h, fp32
//   combine  out = sum of weight * y, in the order of choice
//
// The two products.  A unit is a pair of 16-row tiles of an expert (for gate/up
// the gate and the up tile of the same rows, for down two neighbours) times that
// expert's tokens.  The line of all units of the active experts, weighted by
// what their numbers of tokens cost, is cut into equal ranges, one per SM (one
// CTA of W warps).  A CTA takes the units of its range an expert at a time: their
// 256-column super-blocks, one after the other, are cut into W equal ranges, one
// per warp, and the units that warps share are joined in shared memory at the
// end, in the line's order.  A warp's tiles come through a ring of two pairs of
// its own in shared memory (cp.async; tiles loaded straight to registers left
// the tokens' rows waiting on the same few scoreboards).  The tokens' rows come
// from L2 through L1, which hardly keeps them: a register of them is loaded
// again, for the sub-block after the next, as soon as its group of 32 columns
// is done.  (Loaded one sub-block ahead, 64 tokens of 16 experts of 6656 x 4096
// took 198 us instead of 183, and 32 of 128 experts of 2048 x 768 61 instead of 60; if
// all of these loads hit L1 the former would take 158.  Whole units per warp,
// so that the warps read the same columns at the same time, changed neither.)
//
// Arithmetic.  A word of packed codes, masked, is a pair of bf16 subnormals
// q 2^-133 (low nibbles) or q 2^-129 (high nibbles); one bf16x2 fma with 2^127
// or 2^123 makes it (q - z) 2^-6, exactly.  The MMAs sum (q - z) x 2^-6 per
// group of 32 and acc += s * sum in fp32: the weights are never rounded.  h is
// rounded to bf16, as an activation between two of the library's linear layers
// is (in two parts where an output has few terms, see two_parts).
#include <cooperative_groups.h>

#include "common.cuh"
#include "decode.h"
#include "kernels.h"

#include <atomic>

namespace cg = cooperative_groups;

namespace w4q {

namespace {

constexpr int TILE_BYTES = 2432;
constexpr int MAX_EXPERTS = 512, MAX_TOKENS = 64;

// ------------------------------------------------------------------- route

constexpr int ROUTE_CTAS = 8, ROUTE_WARPS = 8, ROUTE_TOKENS = 8;
constexpr int MAX_ENTRIES = MAX_TOKENS * 16;

// What the products need of the choice: the active experts in order, each with
// its entries (token * topk + place, in order) and what the units before it cost.
struct Plan {
    int count, pad[3];
    int expert[MAX_EXPERTS];
    int before[MAX_EXPERTS + 4];  // [count + 1]
    int offset[MAX_EXPERTS + 4];  // [count + 1], into entries
    int entries[MAX_ENTRIES];
};

struct RouteParams {
    const __nv_bfloat16 *x, *router;
    const float *bias;
    uint16_t *xf;      // [tokens][hidden] in fragment order
    Plan *plan;
    float *weights;    // [tokens][topk]
    int32_t *ids_out;  // the caller's, or null
    float *weights_out;
    int tokens, hidden, experts, topk;
    bool sigmoid, renormalize;
    float scale;
    int groups;  // of 8 tokens that the products take at a time, at most
};

// What a super-block of a unit of an expert with n tokens costs, in eighths of
// a pass with up to 8: passes of 32 (with `most` = 4 groups of 8 at a time), 16
// (2) and 8 tokens.
__device__ __forceinline__ int step_cost(int n, int most)
{
    int cost = 0;
    if (most >= 4)
        for (; n > 16; n -= 32)
            cost += 20;
    if (most >= 2)
        for (; n > 8; n -= 16)
            cost += 14;
    return cost + (n > 0 ? (n + 7) / 8 * 8 : 0);
}

__device__ __forceinline__ uint32_t order_key(float v)  // larger for larger v, at least 1; NaN is the least
{
    const uint32_t b = __float_as_uint(v);
    const uint32_t k = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
    return v != v ? 1u : max(k, 1u);
}

// volatile: the compiler is not to move it down to its use
__device__ __forceinline__ uint4 ldg_row(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// TT groups of 8 tokens, up to 32 PER experts.
template <int TT, int PER>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) moe_route_kernel(const RouteParams p)
{
    // the cluster's warps' parts of this CTA's tokens' logits: [slice][16 experts' tile][token][expert]
    __shared__ float s_part[ROUTE_CTAS * ROUTE_WARPS][ROUTE_TOKENS * 16];
    __shared__ uint16_t s_ids[MAX_ENTRIES];            // the first CTA's: all choices
    __shared__ uint32_t s_mask[32 * PER][2];           // the tokens of an expert
    __shared__ uint16_t s_offset[32 * PER];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

    if (blockIdx.x >= ROUTE_CTAS) {
        pdl_wait();
        pdl_launch_dependents();
        const int me = (blockIdx.x - ROUTE_CTAS) * 32 * ROUTE_WARPS + tid, all = (gridDim.x - ROUTE_CTAS) * 32 * ROUTE_WARPS;
        // x in fragment order: of 64 columns, lane t's pairs 16j + 2t and 16j + 8 + 2t, j = 0..3
        const int per = p.hidden / 16;
        for (int i = me; i < p.tokens * per; i += all) {
            const int m = i / per, at = i - m * per;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(p.x + (int64_t)m * p.hidden) + (at / 4) * 32 + at % 4;
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = __ldg(src + 4 * j);
            uint4 *dst = reinterpret_cast<uint4 *>(p.xf + (int64_t)m * p.hidden) + 2 * at;
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return;
    }

    cg::cluster_group cluster = cg::this_cluster();
    const int rank = blockIdx.x;
    for (int i = tid; i < 64 * PER; i += 32 * ROUTE_WARPS)
        s_mask[i / 2][i % 2] = 0;
    cluster.sync();  // every CTA runs before anything is written to its shared memory
    pdl_wait();
    pdl_launch_dependents();

    float bias[PER];  // loaded long before it is used
#pragma unroll
    for (int i = 0; i < PER; ++i)
        bias[i] = p.sigmoid && p.bias && 32 * i + lane < p.experts ? __ldg(p.bias + 32 * i + lane) : 0.f;
    const int mt = (p.experts + 15) / 16;
    const int slices = ROUTE_CTAS * ROUTE_WARPS / mt;
    const int gw = rank * ROUTE_WARPS + warp;
    const int slice = gw / mt, tile = gw - slice * mt;
    if (slice < slices) {
        const int chunks = p.hidden / 32;
        const int c0 = chunks * slice / slices, c1 = chunks * (slice + 1) / slices;
        // rows past the last are its copies: their logits are not read
        const int e0 = min(tile * 16 + g, p.experts - 1), e1 = min(tile * 16 + 8 + g, p.experts - 1);
        const uint4 *ra = reinterpret_cast<const uint4 *>(p.router + (int64_t)e0 * p.hidden) + t;
        const uint4 *rb = reinterpret_cast<const uint4 *>(p.router + (int64_t)e1 * p.hidden) + t;
        const uint4 *rx[TT];
        float acc[TT][4];
#pragma unroll
        for (int n = 0; n < TT; ++n) {
            rx[n] = reinterpret_cast<const uint4 *>(p.x + (int64_t)min(n * 8 + g, p.tokens - 1) * p.hidden) + t;
            acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
        }
        constexpr int U = TT == 8 ? 2 : 4;  // chunks whose loads go out together
        for (int c = c0; c < c1; c += U) {
            uint4 a[U], b[U], x[U][TT];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int at = 4 * min(c + i, c1 - 1);
                a[i] = ldg_row(ra + at);
                b[i] = ldg_row(rb + at);
#pragma unroll
                for (int n = 0; n < TT; ++n)
                    x[i][n] = ldg_row(rx[n] + at);
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (c + i < c1) {
                    const uint32_t f0[4] = {a[i].x, b[i].x, a[i].y, b[i].y};
                    const uint32_t f1[4] = {a[i].z, b[i].z, a[i].w, b[i].w};
#pragma unroll
                    for (int n = 0; n < TT; ++n) {
                        mma_bf16(acc[n], f0, x[i][n].x, x[i][n].y, acc[n]);
                        mma_bf16(acc[n], f1, x[i][n].z, x[i][n].w, acc[n]);
                    }
                }
        }
#pragma unroll
        for (int n = 0; n < TT; ++n) {
            float *dst = cluster.map_shared_rank(&s_part[gw][0], n);
            dst[(2 * t) * 16 + g] = acc[n][0];
            dst[(2 * t + 1) * 16 + g] = acc[n][1];
            dst[(2 * t) * 16 + 8 + g] = acc[n][2];
            dst[(2 * t + 1) * 16 + 8 + g] = acc[n][3];
        }
    }
    cluster.sync();
    const int m = rank * ROUTE_TOKENS + warp;  // one warp per token
    if (m < p.tokens) {
        float score[PER];
        uint32_t key[PER];
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = 32 * i + lane;
            score[i] = -INFINITY;
            key[i] = 0u;
            if (e < p.experts) {
                float v = 0.f;
#pragma unroll 8
                for (int s = 0; s < slices; ++s)
                    v += s_part[s * mt + e / 16][warp * 16 + e % 16];
                score[i] = v;
                key[i] = order_key(v);
                top = fmaxf(top, v);
            }
        }
        if (p.sigmoid) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = 32 * i + lane;
                if (e < p.experts) {
                    score[i] = 1.f / (1.f + expf(-score[i]));
                    key[i] = order_key(score[i] + bias[i]);
                }
            }
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                score[i] = 32 * i + lane < p.experts ? expf(score[i] - top) : 0.f;
                sum += score[i];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(~0u, sum, o);
        }
        float mine = 0.f, chosen = 0.f;  // lane k: the k-th chosen score
        int id = 0;
        for (int k = 0; k < p.topk; ++k) {
            uint32_t best = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                best = max(best, key[i]);
            best = __reduce_max_sync(~0u, best);
            uint32_t at = ~0u;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i)
                if (key[i] == best)
                    at = 32 * i + lane;
            at = __reduce_min_sync(~0u, at);
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (32 * i + lane == (int)at) {
                    v = score[i];
                    key[i] = 0;
                }
            v = __shfl_sync(~0u, v, at & 31);
            chosen += v;
            if (lane == k) {
                mine = v;
                id = (int)at;
            }
        }
        if (lane < p.topk) {
            // a NaN logit makes every softmax score NaN (sum), whichever are chosen; a sigmoid's its own
            const float all = !p.sigmoid && (!p.renormalize || sum != sum) ? sum : p.renormalize ? chosen : 1.f;
            const float w = all == 0.f ? 0.f : mine / all * p.scale;
            p.weights[m * p.topk + lane] = w;
            cluster.map_shared_rank(s_ids, 0)[m * p.topk + lane] = (uint16_t)id;
            atomicOr(cluster.map_shared_rank(&s_mask[0][0], 0) + 2 * id + (m >> 5), 1u << (m & 31));
            if (p.ids_out)
                p.ids_out[m * p.topk + lane] = id;
            if (p.weights_out)
                p.weights_out[m * p.topk + lane] = w;
        }
    }
    if constexpr (TT > 1)
        cluster.sync();
    if (rank != 0)
        return;
    if constexpr (TT == 1)  // the first CTA has chosen for all tokens
        __syncthreads();
    // the choices by expert: an expert's tokens are bits of its mask
    if (warp == 0) {
        int count = 0, cost = 0, entries = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = 32 * i + lane, n = __popc(s_mask[e][0]) + __popc(s_mask[e][1]);
            const uint32_t active = __ballot_sync(~0u, n > 0);
            const int c = step_cost(n, p.groups);
            int xc = c, xn = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int yc = __shfl_up_sync(~0u, xc, o), yn = __shfl_up_sync(~0u, xn, o);
                if (lane >= o) {
                    xc += yc;
                    xn += yn;
                }
            }
            s_offset[e] = (uint16_t)(entries + xn - n);
            if (n > 0) {
                const int at = count + __popc(active & ((1u << lane) - 1));
                p.plan->expert[at] = e;
                p.plan->before[at] = cost + xc - c;
                p.plan->offset[at] = entries + xn - n;
            }
            count += __popc(active);
            cost += __shfl_sync(~0u, xc, 31);
            entries += __shfl_sync(~0u, xn, 31);
        }
        if (lane == 0) {
            p.plan->count = count;
            p.plan->before[count] = cost;
            p.plan->offset[count] = entries;
        }
    }
    __syncthreads();
    for (int i = tid; i < p.tokens * p.topk; i += 32 * ROUTE_WARPS) {
        const int e = s_ids[i], mm = i / p.topk;
        const uint32_t lo = s_mask[e][0], hi = s_mask[e][1], below = (1u << (mm & 31)) - 1;
        const int before = mm < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below);
        p.plan->entries[s_offset[e] + before] = i;
    }
}

// ------------------------------------------------------------ the products


// bf16 pairs
constexpr uint32_t BF_2P127 = 0x7F007F00u, BF_2P123 = 0x7D007D00u, NEG_2P127 = 0xFF00FF00u;

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

struct GemmParams {
    const uint8_t *packed;
    const uint16_t *xf;  // rows in fragment order
    const Plan *plan;
    uint16_t *h;         // gate/up: [entries][rows_out] in fragment order
    float *y;            // down: [entries][rows_out]
    int topk, experts;
    int K;         // columns
    int rows_out;  // rows per expert of the result
    int low;       // elements from h to what its rounding left, or 0
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}

// d = a b and d += a b; not volatile, so that independent chains interleave.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_more(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// a += s x, b += s y
__device__ __forceinline__ void fma_pair(float &a, float &b, float s, float x, float y)
{
    asm("{\n\t.reg .b64 s, x, c;\n\tmov.b64 s, {%2, %2};\n\tmov.b64 x, {%3, %4};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, s, x, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(s), "f"(x), "f"(y));
}

template <int V>
struct Count {
    static constexpr int value = V;
};

// A group of 32 columns of a tile times NT groups of 8 tokens: acc += s * sum (q - z) x 2^-6.  `zz`
// holds the zeros of rows g, g + 8 of this group in its lower (gr = 0) or upper half.
template <int NT, int LOW>
__device__ __forceinline__ void group_step(uint32_t q0, uint32_t q1, uint32_t sc, uint32_t zz, int gr,
                                           const uint4 (&x)[1 + LOW][NT], float (&acc)[NT][4])
{
    // -z 2^-6 of rows g, g + 8
    const uint32_t z0 = bf16x2_mul(prmt(zz, 0u, gr ? 0x4242u : 0x4040u), NEG_2P127);
    const uint32_t z1 = bf16x2_mul(prmt(zz, 0u, gr ? 0x4343u : 0x4141u), NEG_2P127);
    float d[NT][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t w = k ? q1 : q0, wh = w >> 8;
        const uint32_t a[4] = {bf16x2_fma(w & 0x000F000Fu, BF_2P127, z0), bf16x2_fma(wh & 0x000F000Fu, BF_2P127, z1),
                               bf16x2_fma(w & 0x00F000F0u, BF_2P123, z0), bf16x2_fma(wh & 0x00F000F0u, BF_2P123, z1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            if (k == 0)
                mma_first(d[nt], a, x[0][nt].x, x[0][nt].y);
            else
                mma_more(d[nt], a, x[0][nt].z, x[0][nt].w);
        if constexpr (LOW != 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_more(d[nt], a, k == 0 ? x[1][nt].x : x[1][nt].z, k == 0 ? x[1][nt].y : x[1][nt].w);
    }
    const float sa = bf16lo_to_f32(sc), sb = bf16hi_to_f32(sc);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        fma_pair(acc[nt][0], acc[nt][1], sa, d[nt][0], d[nt][1]);
        fma_pair(acc[nt][2], acc[nt][3], sb, d[nt][2], d[nt][3]);
    }
}

// NT groups of 8 tokens at a time, at most; W warps; LOW = 1: h is in two parts.
template <bool GATED, int NT, int W, int LOW_H>
__global__ void __launch_bounds__(32 * W, 1) moe_gemm_kernel(const GemmParams p)
{
    constexpr int LOW = GATED ? 0 : LOW_H;  // parts of a row of xf beyond the first
    extern __shared__ __align__(16) int s_before[];  // [experts + 1] each: costs before, offsets, numbers of the active experts
    int *s_offset = s_before + p.experts + 1, *s_expert = s_offset + p.experts + 1;
    uint8_t *s_ring = reinterpret_cast<uint8_t *>(s_before) + (12 * (p.experts + 1) + 15) / 16 * 16;  // [W][2][2 tiles]
    // a warp's parts of the unit that it continues and of the one that it begins: [W][2][2 * NT][128]
    float *s_part = reinterpret_cast<float *>(s_ring + W * 4 * TILE_BYTES);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int low = p.low / 8;  // from the first part of h to the second, in 16 bytes

    pdl_wait();
    pdl_launch_dependents();
    const int count = p.plan->count;
    for (int i = tid; i < p.experts + 1; i += 32 * W) {
        s_before[i] = p.plan->before[i];
        s_offset[i] = p.plan->offset[i];
        s_expert[i] = i < p.experts ? p.plan->expert[i] : 0;
    }
    __syncthreads();

    // A unit: an active expert's block of rows.  Share r of the whole cost ends at share * r +
    // min(r, extra).  (At most 512 experts, 64 x 16 choices, 2048 blocks: less than 2^24.)
    struct Unit {
        int a, blk;
    };
    const int KB = p.K / 256, blocks = p.rows_out / (GATED ? 16 : 32);
    const unsigned total = (unsigned)s_before[count] * blocks, share = total / gridDim.x, extra = total - share * gridDim.x;
    auto cut_at = [&](unsigned r) -> Unit {  // the first unit that begins at or past that end
        const unsigned at = share * r + min(r, extra);
        const int whole = (int)(at / (unsigned)blocks);
        int lo = 0, hi = count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_before[mid] <= whole)
                lo = mid;
            else
                hi = mid;
        }
        const unsigned each = s_before[lo + 1] - s_before[lo], blk = (at - (unsigned)s_before[lo] * blocks + each - 1) / each;
        return blk < (unsigned)blocks ? Unit{lo, (int)blk} : Unit{lo + 1, 0};
    };
    const Unit at = cut_at(blockIdx.x), end = cut_at(blockIdx.x + 1);

    // Segments: the units of one expert in the range, or, where no expert has more than 8 tokens and
    // each takes one pass, all of them.  Warp w's part of a segment of S steps (its units'
    // super-blocks) is S w / W .. S (w + 1) / W - 1.  All warps go through all segments.
    struct Segment {
        Unit first;
        int units;  // 0: no segment left
    };
    auto segment_at = [&](Unit at) -> Segment {
        if (at.a > end.a || (at.a == end.a && at.blk >= end.blk))
            return {at, 0};
        if constexpr (NT == 1)
            return {at, (end.a - at.a) * blocks + end.blk - at.blk};
        return {at, (at.a == end.a ? end.blk : blocks) - at.blk};
    };
    auto after = [&](const Segment &s) -> Segment { return segment_at(NT == 1 ? end : Unit{s.first.a + 1, 0}); };
    auto unit_of = [&](const Segment &s, int u) -> Unit {
        const int blk = s.first.blk + u, more = NT == 1 ? (unsigned)blk / (unsigned)blocks : 0;
        return {s.first.a + more, blk - more * blocks};
    };
    auto cut_of = [&](const Segment &s, int w) -> int { return s.units * KB * w / W; };  // < 2^22
    Segment seg = segment_at(at);
    if (seg.units == 0)
        return;  // the whole CTA
    // Where the pair of unit u, super-block b of a segment lies, in 16 bytes (32 bits reach 64 GB);
    // rows_out / 16 is a multiple of 16, so the pair's second tile lies `second`, and the next
    // super-block 8 tiles, from it.
    constexpr uint32_t TILE16 = TILE_BYTES / 16, NEXT_SB = 8 * TILE16, NONE = ~0u;
    const uint32_t second = GATED ? (uint32_t)(blocks >> 3) * KB * NEXT_SB : TILE16;
    auto place = [&](const Segment &s, int u, int b) -> uint32_t {
        const Unit at = unit_of(s, u);
        const int tl = s_expert[at.a] * 2 * blocks + (GATED ? at.blk : 2 * at.blk);
        return ((uint32_t)(tl >> 3) * KB + b) * NEXT_SB + (tl & 7) * TILE16;
    };
    auto first_place = [&](Segment s) -> uint32_t {  // of this warp's, from segment s on
        while (s.units > 0 && cut_of(s, warp) == cut_of(s, warp + 1))
            s = after(s);
        if (s.units == 0)
            return NONE;
        const int c = cut_of(s, warp), u = (unsigned)c / (unsigned)KB;
        return place(s, u, c - u * KB);
    };
    // The pair at `at` into one half of the warp's ring: 16 bytes a lane, 4864 in all.
    const uint64_t policy = policy_evict_first();
    const uint32_t ring = smem_addr(s_ring) + warp * (4 * TILE_BYTES);
    auto copy = [&](uint32_t at, int half) {
        if (at != NONE) {
            const uint8_t *src = p.packed + (uint64_t)at * 16 + 16 * lane;
            const uint32_t dst = ring + half * 2 * TILE_BYTES + 16 * lane;
#pragma unroll
            for (int r = 0; r < 2; ++r, src += (uint64_t)second * 16) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    copy16(dst + r * TILE_BYTES + 512 * i, src + 512 * i, policy);
                if (lane < 24)
                    copy16(dst + r * TILE_BYTES + 2048, src + 2048, policy);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t here = first_place(seg);
    int half = 0;
    copy(here, 0);

    for (; seg.units > 0; seg = after(seg)) {
        const int c0 = cut_of(seg, warp), c1 = cut_of(seg, warp + 1);
        const uint32_t there = c0 < c1 ? first_place(after(seg)) : here;
        auto tokens_of = [&](int a) -> int { return s_offset[a + 1] - s_offset[a]; };
        // the result of unit u for the 8 tokens from col0 on
        auto store = [&](const float (&v)[2][4], int col0, int u) {
            const Unit unit = unit_of(seg, u);
            const int blk = unit.blk, n = tokens_of(unit.a);
            const int *list = p.plan->entries + s_offset[unit.a];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = col0 + 2 * t + i;
                if (col >= n)
                    continue;
                const int entry = __ldg(list + col);
                if constexpr (GATED) {
                    // rows g and g + 8 of the 16, in fragment order
                    uint16_t *dst = p.h + (int64_t)entry * p.rows_out + (blk >> 2) * 64 + (g >> 1) * 16 + (blk & 3) * 4 + (g & 1);
#pragma unroll
                    for (int e8 = 0; e8 < 2; ++e8) {
                        const float gate = v[0][2 * e8 + i] * 64.f, up = v[1][2 * e8 + i] * 64.f;
                        const float h = gate / (1.f + __expf(-gate)) * up;
                        const __nv_bfloat16 hb = __float2bfloat16_rn(h);
                        dst[2 * e8] = *reinterpret_cast<const uint16_t *>(&hb);
                        if constexpr (LOW_H != 0) {
                            const __nv_bfloat16 lb = __float2bfloat16_rn(__hisinf(hb) ? 0.f : h - __bfloat162float(hb));
                            dst[p.low + 2 * e8] = *reinterpret_cast<const uint16_t *>(&lb);
                        }
                    }
                } else {
                    float *dst = p.y + (int64_t)entry * p.rows_out + blk * 32 + g;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        dst[16 * r] = v[r][i] * 64.f;
                        dst[16 * r + 8] = v[r][2 + i] * 64.f;
                    }
                }
            }
        };
        // an expert with more than 8 NT tokens takes several passes over its tiles
        auto pass = [&](auto groups_of_8, int n0) {
            constexpr int N = decltype(groups_of_8)::value;
            if (c0 < c1) {
                int u = (unsigned)c0 / (unsigned)KB, b = c0 - u * KB, a = unit_of(seg, u).a;
                const bool again = NT > 1 && n0 + 8 * N < tokens_of(a);
                const uint4 *row[N];  // tokens past the last are its copies, and are not stored
                auto find_rows = [&]() {
#pragma unroll
                    for (int nt = 0; nt < N; ++nt) {
                        const int entry = __ldg(p.plan->entries + s_offset[a] + min(n0 + nt * 8 + g, tokens_of(a) - 1));
                        row[nt] = reinterpret_cast<const uint4 *>(
                            p.xf + (int64_t)(GATED ? (unsigned)entry / (unsigned)p.topk : entry) * p.K + 16 * t);
                    }
                };
                find_rows();
                bool begun = b == 0;  // the unit's first super-block is this warp's
                uint32_t at = here;
                float acc[2][N][4];
                // the tokens' rows: a register is loaded again, for the sub-block after the next, as soon
                // as its group is done
                uint4 x[2][2][1 + LOW][N];
                auto begin_rows = [&]() {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int nt = 0; nt < N; ++nt)
#pragma unroll
                            for (int lo = 0; lo <= LOW; ++lo)
                                x[i >> 1][i & 1][lo][nt] = ldg_row(row[nt] + lo * low + b * 32 + 8 * (i >> 1) + (i & 1));
                };
                begin_rows();
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int nt = 0; nt < N; ++nt)
                        acc[r][nt][0] = acc[r][nt][1] = acc[r][nt][2] = acc[r][nt][3] = 0.f;
                for (int c = c0; c < c1; ++c) {
                    const bool more = c + 1 < c1, inside = b + 1 < KB;
                    const int b_next = inside ? b + 1 : 0;
                    const uint32_t next = more ? (inside ? at + NEXT_SB : place(seg, u + 1, 0)) : again ? here : there;
                    // this pair has come, and every lane has read the one before
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                    __syncwarp();
                    const uint32_t tiles = ring + half * 2 * TILE_BYTES;
                    half ^= 1;
                    copy(next, half);
                    uint4 sc[2][2], z[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        sc[r][0] = lds128(tiles + r * TILE_BYTES + 2048 + 16 * g);
                        sc[r][1] = lds128(tiles + r * TILE_BYTES + 2048 + 128 + 16 * g);
                        z[r] = lds128(tiles + r * TILE_BYTES + 2304 + 16 * g);
                    }
#pragma unroll
                    for (int sb = 0; sb < 4; ++sb) {
                        uint4 q[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            q[r] = lds128(tiles + r * TILE_BYTES + 512 * sb + 16 * lane);
#pragma unroll
                        for (int gr = 0; gr < 2; ++gr) {
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const uint4 &s = sc[r][sb >> 1];
                                group_step<N, LOW>(gr ? q[r].z : q[r].x, gr ? q[r].w : q[r].y,
                                              sb & 1 ? (gr ? s.w : s.z) : (gr ? s.y : s.x), (&z[r].x)[sb], gr, x[sb & 1][gr],
                                              acc[r]);
                            }
                            // (of a last step, columns that are not used)
#pragma unroll
                            for (int nt = 0; nt < N; ++nt)
#pragma unroll
                                for (int lo = 0; lo <= LOW; ++lo)
                                    x[sb & 1][gr][lo][nt] = ldg_row(
                                        row[nt] + lo * low + (sb < 2 ? b * 32 + 8 * (sb + 2) : b_next * 32 + 8 * (sb - 2)) + gr);
                        }
                    }
                    at = next;
                    ++b;
                    if (!inside || !more) {
#pragma unroll
                        for (int nt = 0; nt < N; ++nt) {
                            if (begun && !inside) {
                                const float v[2][4] = {{acc[0][nt][0], acc[0][nt][1], acc[0][nt][2], acc[0][nt][3]},
                                                       {acc[1][nt][0], acc[1][nt][1], acc[1][nt][2], acc[1][nt][3]}};
                                store(v, n0 + nt * 8, u);
                            } else {
#pragma unroll
                                for (int r = 0; r < 2; ++r)
                                    *reinterpret_cast<float4 *>(s_part + (((warp * 2 + begun) * NT + nt) * 2 + r) * 128 + lane * 4) =
                                        make_float4(acc[r][nt][0], acc[r][nt][1], acc[r][nt][2], acc[r][nt][3]);
                            }
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                acc[r][nt][0] = acc[r][nt][1] = acc[r][nt][2] = acc[r][nt][3] = 0.f;
                        }
                        ++u;
                        b = 0;
                        begun = true;
                        if (NT == 1 && more && unit_of(seg, u).a != a) {
                            a = unit_of(seg, u).a;
                            find_rows();
                            begin_rows();
                        }
                    }
                }
            }
            // --- the units that warps share: step x is warp ((x + 1) W - 1) / S's
            const int S = seg.units * KB;
            __syncthreads();
            for (int u = warp; u < seg.units; u += W) {
                const int w0 = (unsigned)((u * KB + 1) * W - 1) / (unsigned)S, w1 = (unsigned)((u + 1) * KB * W - 1) / (unsigned)S;
                if (w0 == w1)
                    continue;
#pragma unroll
                for (int nt = 0; nt < N; ++nt) {
                    float v[2][4] = {};
                    for (int w = w0; w <= w1; ++w) {
                        if (cut_of(seg, w) == cut_of(seg, w + 1))
                            continue;  // fewer steps than warps
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float4 y = *reinterpret_cast<const float4 *>(
                                s_part + (((w * 2 + (w == w0)) * NT + nt) * 2 + r) * 128 + lane * 4);
                            v[r][0] += y.x;
                            v[r][1] += y.y;
                            v[r][2] += y.z;
                            v[r][3] += y.w;
                        }
                    }
                    store(v, n0 + nt * 8, u);
                }
            }
            __syncthreads();  // the parts are read
        };
        const int n = NT == 1 ? 8 : tokens_of(seg.first.a);
        int n0 = 0;
        if constexpr (NT > 2)
            for (; n - n0 > 16; n0 += 32)
                pass(Count<4>(), n0);
        if constexpr (NT > 1)
            for (; n - n0 > 8; n0 += 16)
                pass(Count<2>(), n0);
        for (; n0 < n; n0 += 8)
            pass(Count<1>(), n0);
        here = there;
    }
}

// out[m] = sum over the choices of weight * y, four elements a thread
__global__ void __launch_bounds__(128) moe_combine_kernel(const float *y, const float *weights, __nv_bfloat16 *out,
                                                          int tokens, int topk, int hidden)
{
    pdl_wait();
    pdl_launch_dependents();
    const int i = blockIdx.x * 128 + threadIdx.x, per = hidden / 4;
    const int m = i / per, d = i % per;
    if (m >= tokens)
        return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < topk; ++k) {
        const float w = __ldg(weights + m * topk + k);
        const float4 v = __ldg(reinterpret_cast<const float4 *>(y + (int64_t)(m * topk + k) * hidden) + d);
        s.x = fmaf(w, v.x, s.x);
        s.y = fmaf(w, v.y, s.y);
        s.z = fmaf(w, v.z, s.z);
        s.w = fmaf(w, v.w, s.w);
    }
    __nv_bfloat162 o[2] = {__floats2bfloat162_rn(s.x, s.y), __floats2bfloat162_rn(s.z, s.w)};
    reinterpret_cast<uint2 *>(out + (int64_t)m * hidden)[d] = *reinterpret_cast<const uint2 *>(o);
}

template <bool GATED, int NT, int W, int LOW>
cudaError_t launch_variant(const GemmParams &p, int sm_count, cudaStream_t stream)
{
    constexpr int fixed = W * (4 * TILE_BYTES + NT * 2048);
    static std::atomic<unsigned long long> done{0};
    auto fn = moe_gemm_kernel<GATED, NT, W, LOW>;
    const cudaError_t e = smem_opt_in_once(done, fn, 12 * (MAX_EXPERTS + 1) + 16 + fixed);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(fn, dim3((unsigned)sm_count), dim3(32 * W), (12 * (p.experts + 1) + 15) / 16 * 16 + fixed, stream, p);
}

// Groups of 8 tokens at a time: with up to 8 tokens no expert has more; 32 at a time pay where the
// experts have more than 16 on average (64 tokens, 8 of 16 experts of 2048 x 768: 65 us, 73 by 16).
int groups_of(int tokens, int topk, int experts)
{
    return tokens <= 8 ? 1 : tokens * topk <= 16 * experts ? 2 : 4;
}

// h's rounding adds as much to the result's error as the result's own: the two
// together are 1.41 times the latter on average.  Over few terms, the topk *
// inter of an output's sum, that is uneven, because a few large h decide: one
// row in a hundred has 1.7 times with 256 terms, 1.66 with 2048, 1.6 with 4096,
// 1.56 with 8192 (gaussian weights).  Up to 4096 terms what the rounding left
// goes through the second product too, for any number of tokens, so that a
// row's precision does not depend on its batch.  (64 tokens, 2 of 8 experts of
// 2048 x 256: 30 us instead of 28; 8 tokens, 4 of 64 of 2048 x 1024: 36 instead of
// 33; 64 tokens, 8 of 16 of 2048 x 512: 66 instead of 58.  In every call it would
// cost 64 tokens, 2 of 16 of 6656 x 4096, 209 us instead of 183.)
constexpr int TWO_PARTS = 4096;
bool two_parts(int topk, int inter) { return topk * inter <= TWO_PARTS; }

template <bool GATED, int LOW>
cudaError_t launch_gemm(const GemmParams &p, int groups, int sm_count, cudaStream_t stream)
{
    return groups == 1   ? launch_variant<GATED, 1, 12, LOW>(p, sm_count, stream)
           : groups == 2 ? launch_variant<GATED, 2, 12, LOW>(p, sm_count, stream)
                         : launch_variant<GATED, 4, 8, LOW>(p, sm_count, stream);
}

struct Workspace {
    size_t xf, h, y, plan, weights, bytes;
};
Workspace layout(int tokens, int hidden, int inter, int topk)
{
    Workspace w;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += (n + 255) / 256 * 256;
        return was;
    };
    w.xf = take((size_t)tokens * hidden * 2);
    w.h = take((size_t)tokens * topk * inter * (two_parts(topk, inter) ? 4 : 2));
    w.y = take((size_t)tokens * topk * hidden * 4);
    w.plan = take(sizeof(Plan));
    w.weights = take((size_t)tokens * topk * 4);
    w.bytes = at;
    return w;
}

}  // namespace

size_t moe_workspace(int tokens, int hidden, int inter, int topk)
{
    return layout(tokens, hidden, inter, topk).bytes;
}

cudaError_t launch_moe(const Moe &a, int sm_count, void *workspace, cudaStream_t stream)
{
    const Workspace w = layout(a.tokens, a.hidden, a.inter, a.topk);
    char *base = static_cast<char *>(workspace);
    uint16_t *xf = reinterpret_cast<uint16_t *>(base + w.xf), *h = reinterpret_cast<uint16_t *>(base + w.h);
    float *y = reinterpret_cast<float *>(base + w.y), *weights = reinterpret_cast<float *>(base + w.weights);
    Plan *plan = reinterpret_cast<Plan *>(base + w.plan);

    const int groups = groups_of(a.tokens, a.topk, a.experts);
    RouteParams r = {static_cast<const __nv_bfloat16 *>(a.x), static_cast<const __nv_bfloat16 *>(a.router), a.bias, xf,
                     plan, weights, a.ids_out, a.weights_out, a.tokens, a.hidden, a.experts, a.topk, a.sigmoid,
                     a.renormalize, a.scale, groups};
    cudaLaunchConfig_t cfg = {};
    const long long items = (long long)a.tokens * a.hidden / 16, per_cluster = ROUTE_CTAS * 32 * ROUTE_WARPS;
    const int others = (int)(items <= per_cluster ? 1 : items >= 8 * per_cluster ? 8 : items / per_cluster);
    cfg.gridDim = dim3(ROUTE_CTAS * (1 + others));
    cfg.blockDim = dim3(32 * ROUTE_WARPS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ROUTE_CTAS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    using Route = void (*)(const RouteParams);
    static const Route routes[4][2] = {{moe_route_kernel<1, 4>, moe_route_kernel<1, 16>},
                                       {moe_route_kernel<2, 4>, moe_route_kernel<2, 16>},
                                       {moe_route_kernel<4, 4>, moe_route_kernel<4, 16>},
                                       {moe_route_kernel<8, 4>, moe_route_kernel<8, 16>}};
    const Route route = routes[a.tokens <= 8 ? 0 : a.tokens <= 16 ? 1 : a.tokens <= 32 ? 2 : 3][a.experts <= 128 ? 0 : 1];
    cudaError_t e = cudaLaunchKernelEx(&cfg, route, (const RouteParams)r);
    if (e != cudaSuccess)
        return e;

    const int low = two_parts(a.topk, a.inter) ? a.tokens * a.topk * a.inter : 0;
    GemmParams up = {static_cast<const uint8_t *>(a.w13), xf, plan, h, nullptr, a.topk, a.experts,
                     a.hidden, a.inter, low};
    GemmParams down = {static_cast<const uint8_t *>(a.w2), h, plan, nullptr, y, a.topk, a.experts,
                       a.inter, a.hidden, low};
    e = low ? launch_gemm<true, 1>(up, groups, sm_count, stream) : launch_gemm<true, 0>(up, groups, sm_count, stream);
    if (e == cudaSuccess)
        e = low ? launch_gemm<false, 1>(down, groups, sm_count, stream) : launch_gemm<false, 0>(down, groups, sm_count, stream);
    if (e != cudaSuccess)
        return e;
    const long long threads = (long long)a.tokens * (a.hidden / 4);
    return launch_pdl(moe_combine_kernel, dim3((unsigned)((threads + 127) / 128)), dim3(128), 0, stream,
                      static_cast<const float *>(y), static_cast<const float *>(weights),
                      static_cast<__nv_bfloat16 *>(a.out), a.tokens, a.topk, a.hidden);
}

}  // namespace w4q
