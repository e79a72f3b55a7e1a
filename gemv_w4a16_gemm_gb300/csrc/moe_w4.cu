// moe_w4.cu -- a mixture-of-experts layer for 1 to 64 tokens whose experts'
// weights are in the packed W4 format:
//
//     l = x R^T;  score = softmax(l) or sigmoid(l);  the topk experts by l, or by score + bias;
//     weight = scale * score (divided by the chosen scores' sum);
//     out[m] = sum_chosen weight * W2_e (silu(gate_e x) * up_e x).
//
// What bounds it: the chosen experts' weights, 19/32 bytes each, are read once
// from HBM; with one token that is a few microseconds, so launches and the
// depth of dependent loads count as much.
//
// Four launches, each started while its predecessor finishes:
//   route    one cluster of 8 CTAs per 8 tokens: the logits as m16n8k16 MMAs
//            (bf16 products, fp32 sums) split over the cluster's 64 warps by
//            experts and K, joined in the first CTA's shared memory, and the
//            choice there; x is written in the order of the MMA fragments.
//   gate/up  h = silu(gate) * up for every (token, chosen expert)
//   down     y = W2 h, fp32
//   combine  out = sum of weight * y, in the order of choice
//
// The two products.  A unit is RT 16-row tiles of one expert (a gate and an up
// half each for gate/up) times that expert's tokens; KW warps share its K, each
// streaming its 256-column super-blocks through a ring of its own in shared
// memory (cp.async, contiguous RT * 2432 bytes), so the warps meet only to add
// their sums.  The units of the active experts go round the resident CTAs.
// A super-block's x fragments come through L1 (the fragment order makes them
// two 16-byte loads per 64 columns), once for all RT tiles.
//
// Arithmetic.  A word of packed codes, masked, is a pair of bf16 subnormals
// q 2^-133 (low nibbles) or q 2^-129 (high nibbles); one bf16x2 fma with 2^127
// or 2^123 makes it (q - z) 2^-6, exactly.  The MMAs sum (q - z) x 2^-6 per
// group of 32 and acc += s * sum in fp32: the weights are never rounded.  h is
// rounded to bf16, as an activation between two of the library's linear layers
// is.
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "decode.h"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace w4q {

namespace {

constexpr int TILE_BYTES = 2432;
constexpr int MAX_EXPERTS = 512, MAX_TOPK = 16, MAX_TOKENS = 64;

// ------------------------------------------------------------------- route

constexpr int ROUTE_CTAS = 8, ROUTE_WARPS = 8, ROUTE_TOKENS = 8;

struct RouteParams {
    const __nv_bfloat16 *x, *router;
    const float *bias;
    uint16_t *xf;      // [tokens][hidden] in fragment order
    int32_t *ids;      // [tokens][topk]
    float *weights;    // [tokens][topk]
    int32_t *ids_out;  // the caller's, or null
    float *weights_out;
    int tokens, hidden, experts, topk;
    bool sigmoid, renormalize;
    float scale;
};

__device__ __forceinline__ uint32_t order_key(float v)  // larger for larger v, at least 1; NaN is the least
{
    const uint32_t b = __float_as_uint(v);
    const uint32_t k = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
    return v != v ? 1u : max(k, 1u);
}

__global__ void __launch_bounds__(32 * ROUTE_WARPS) moe_route_kernel(const RouteParams p)
{
    // partial logits of the cluster's warps, in the first CTA: [slice][expert][token]
    __shared__ float s_part[ROUTE_CTAS * ROUTE_WARPS * 16 * ROUTE_TOKENS];
    __shared__ float s_logit[ROUTE_TOKENS][MAX_EXPERTS];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int m0 = (blockIdx.x / ROUTE_CTAS) * ROUTE_TOKENS;
    cluster.sync();  // the first CTA runs before anything is written to its shared memory
    pdl_wait();
    pdl_launch_dependents();

    const int mt = (p.experts + 15) / 16;
    const int slices = ROUTE_CTAS * ROUTE_WARPS / mt;
    const int gw = rank * ROUTE_WARPS + warp;
    const int tile = gw % mt, slice = gw / mt;
    if (slice < slices) {
        const int chunks = p.hidden / 32;
        const int c0 = chunks * slice / slices, c1 = chunks * (slice + 1) / slices;
        const int e0 = tile * 16 + g, e1 = e0 + 8, m = m0 + g;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const uint4 *ra = reinterpret_cast<const uint4 *>(p.router + (int64_t)e0 * p.hidden) + t;
        const uint4 *rb = reinterpret_cast<const uint4 *>(p.router + (int64_t)e1 * p.hidden) + t;
        const uint4 *rx = reinterpret_cast<const uint4 *>(p.x + (int64_t)m * p.hidden) + t;
        const bool ha = e0 < p.experts, hb = e1 < p.experts, hx = m < p.tokens;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        constexpr int U = 4;
        for (int c = c0; c < c1; c += U) {
            uint4 a[U], b[U], x[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const bool in = c + i < c1;
                a[i] = in && ha ? __ldg(ra + 4 * (c + i)) : zero;
                b[i] = in && hb ? __ldg(rb + 4 * (c + i)) : zero;
                x[i] = in && hx ? __ldg(rx + 4 * (c + i)) : zero;
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const uint32_t f0[4] = {a[i].x, b[i].x, a[i].y, b[i].y};
                const uint32_t f1[4] = {a[i].z, b[i].z, a[i].w, b[i].w};
                mma_bf16(acc, f0, x[i].x, x[i].y, acc);
                mma_bf16(acc, f1, x[i].z, x[i].w, acc);
            }
        }
        float *dst = cluster.map_shared_rank(s_part, 0) + gw * 128;
        dst[g * 8 + 2 * t] = acc[0];
        dst[g * 8 + 2 * t + 1] = acc[1];
        dst[(g + 8) * 8 + 2 * t] = acc[2];
        dst[(g + 8) * 8 + 2 * t + 1] = acc[3];
    }
    // x in fragment order: of 64 columns, lane t's pairs 16j + 2t and 16j + 8 + 2t, j = 0..3
    for (int i = rank * 32 * ROUTE_WARPS + tid; i < ROUTE_TOKENS * p.hidden / 16; i += ROUTE_CTAS * 32 * ROUTE_WARPS) {
        const int m = m0 + i / (p.hidden / 16), at = i % (p.hidden / 16);
        if (m < p.tokens) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(p.x + (int64_t)m * p.hidden) + (at / 4) * 32 + at % 4;
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[2 * j] = __ldg(src + 8 * j);
                w[2 * j + 1] = __ldg(src + 8 * j + 4);
            }
            uint4 *dst = reinterpret_cast<uint4 *>(p.xf + (int64_t)m * p.hidden) + 2 * at;
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
    cluster.sync();
    if (rank != 0)
        return;
    for (int i = tid; i < ROUTE_TOKENS * p.experts; i += 32 * ROUTE_WARPS) {
        const int m = i % ROUTE_TOKENS, e = i / ROUTE_TOKENS;
        float v = 0.f;
        for (int s = 0; s < slices; ++s)
            v += s_part[(s * mt + e / 16) * 128 + (e % 16) * 8 + m];
        s_logit[m][e] = v;
    }
    __syncthreads();
    // one warp per token
    const int m = m0 + warp;
    if (m >= p.tokens)
        return;
    constexpr int PER = MAX_EXPERTS / 32;
    float score[PER];
    uint32_t key[PER];
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 32 * i + lane;
        score[i] = e < p.experts ? s_logit[warp][e] : -INFINITY;
        key[i] = e < p.experts ? order_key(score[i]) : 0u;
        top = fmaxf(top, score[i]);
    }
    if (p.sigmoid) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = 32 * i + lane;
            if (e < p.experts) {
                score[i] = 1.f / (1.f + expf(-score[i]));
                key[i] = order_key(score[i] + (p.bias ? __ldg(p.bias + e) : 0.f));
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
        const float all = p.renormalize ? chosen : (p.sigmoid ? 1.f : sum);
        const float w = all > 0.f ? mine / all * p.scale : 0.f;
        p.ids[m * p.topk + lane] = id;
        p.weights[m * p.topk + lane] = w;
        if (p.ids_out)
            p.ids_out[m * p.topk + lane] = id;
        if (p.weights_out)
            p.weights_out[m * p.topk + lane] = w;
    }
}

// ------------------------------------------------------------ the products

constexpr int GW = 4;  // warps of a CTA

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
    const int32_t *ids;  // [entries]
    uint16_t *h;         // gate/up: [entries][rows_out] in fragment order
    float *y;            // down: [entries][rows_out]
    int entries, topk, experts;
    int K;         // columns
    int rows_out;  // rows per expert of the result
    int KW;        // warps that share a unit's K
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}

template <bool GATED, int RT, int NT, int S>
struct GemmSmem {
    static constexpr int STEP = RT * TILE_BYTES;
    static constexpr int RING = GW * S * STEP;
    static constexpr int SUMS = GW * RT * NT * 128 * 4;
    static size_t bytes(int entries, int experts) { return RING + SUMS + entries * 4 + experts * 4 + 64 * 4; }
};

// RT tiles a step: gate/up RT / 2 gate tiles, then the up tiles of the same
// rows; down RT consecutive tiles.  NT groups of 8 tokens at a time.
template <bool GATED, int RT, int NT, int S, int CPS>
__global__ void __launch_bounds__(32 * GW, CPS) moe_gemm_kernel(const GemmParams p)
{
    using SM = GemmSmem<GATED, RT, NT, S>;
    extern __shared__ __align__(16) uint8_t smem[];
    float *s_sum = reinterpret_cast<float *>(smem + SM::RING);                     // [warp][RT][NT][128]
    int *s_ids = reinterpret_cast<int *>(smem + SM::RING + SM::SUMS);              // [entries]
    int *s_active = s_ids + p.entries;                                             // [active experts]
    __shared__ uint32_t s_mask[MAX_EXPERTS / 32];
    __shared__ int s_count;
    __shared__ int s_list[GW][MAX_TOKENS];  // a warp's tokens: entries of its expert
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const uint64_t policy = policy_evict_first();

    if (tid < MAX_EXPERTS / 32)
        s_mask[tid] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    for (int i = tid; i < p.entries; i += 32 * GW) {
        const int e = __ldg(p.ids + i);
        s_ids[i] = e;
        atomicOr(&s_mask[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (warp == 0) {  // the active experts in order
        const uint32_t m = lane < MAX_EXPERTS / 32 ? s_mask[lane] : 0u;
        int n = __popc(m), at = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, at, o);
            if (lane >= o)
                at += y;
        }
        if (lane == 31)
            s_count = at;
        at -= n;
        for (uint32_t r = m; r != 0; r &= r - 1)
            s_active[at++] = 32 * lane + __ffs(r) - 1;
    }
    __syncthreads();

    constexpr int ROWS = GATED ? RT / 2 : RT;  // tiles of the result a unit covers
    const int KB = p.K / 256, blocks = p.rows_out / (16 * ROWS);
    const int units = s_count * blocks;
    const int KW = p.KW, kw = warp % KW, group = warp / KW, groups = GW / KW;
    const int first = blockIdx.x * groups + group, stride = gridDim.x * groups;
    const int steps = kw < KB ? (KB - kw + KW - 1) / KW : 0;  // of this warp in a unit

    const uint32_t ring = smem_addr(smem) + warp * (S * SM::STEP);
    // the copies run S - 1 steps ahead, across units
    int fu = first, fs = 0, fstage = 0;
    auto fetch = [&]() {
        if (fu < units && steps > 0) {
            const int e = s_active[fu / blocks], blk = fu % blocks, b = kw + fs * KW;
            const int tile = GATED ? e * (2 * p.rows_out / 16) + blk * ROWS : e * (p.rows_out / 16) + blk * ROWS;
            const uint32_t dst = ring + fstage * SM::STEP;
            auto part = [&](int tl, uint32_t to, int bytes) {
                const uint8_t *src = p.packed + (((int64_t)(tl >> 3) * KB + b) * 8 + (tl & 7)) * TILE_BYTES;
                for (int i = lane * 16; i < bytes; i += 512)
                    cp16(to + i, src + i, policy);
            };
            if constexpr (GATED) {
                part(tile, dst, ROWS * TILE_BYTES);
                part(tile + p.rows_out / 16, dst + ROWS * TILE_BYTES, ROWS * TILE_BYTES);
            } else {
                part(tile, dst, RT * TILE_BYTES);
            }
            if (++fs == steps) {
                fs = 0;
                fu += stride;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        fstage = fstage + 1 == S ? 0 : fstage + 1;
    };

    int stage = 0, last_e = -1, n = 0;
    // An expert with more than 8 NT tokens takes several passes; the ring's order is that of one
    // pass, so the further passes read their tiles again, without running ahead.
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        fetch();
    for (int u = first; u < units; u += stride) {
        const int e = s_active[u / blocks], blk = u % blocks;
        if (e != last_e) {
            n = 0;
            for (int i0 = 0; i0 < p.entries; i0 += 32) {
                const bool is = i0 + lane < p.entries && s_ids[i0 + lane] == e;
                const uint32_t m = __ballot_sync(~0u, is);
                if (is)
                    s_list[warp][n + __popc(m & ((1u << lane) - 1))] = i0 + lane;
                n += __popc(m);
            }
            __syncwarp();
            last_e = e;
        }
        for (int n0 = 0; n0 < n; n0 += 8 * NT) {
            const uint16_t *row[NT];
            bool have[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                have[nt] = n0 + nt * 8 + g < n;
                const int entry = have[nt] ? s_list[warp][n0 + nt * 8 + g] : 0;
                row[nt] = p.xf + (int64_t)(GATED ? entry / p.topk : entry) * p.K + 16 * t;
            }
            const bool second = NT > 1 && n0 + 8 < n;
            float acc[RT][NT][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    acc[r][nt][0] = acc[r][nt][1] = acc[r][nt][2] = acc[r][nt][3] = 0.f;
            for (int s = 0; s < steps; ++s) {
                const int b = kw + s * KW;
                uint32_t src = ring + stage * SM::STEP;
                if (n0 == 0) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
                    __syncwarp();  // every lane's copies are here, and the previous step's stage is read
                    fetch();
                } else {
                    // a further pass: this step's tiles once more, into the ring's free stage
                    src = ring + fstage * SM::STEP;
                    const int tile = GATED ? e * (2 * p.rows_out / 16) + blk * ROWS : e * (p.rows_out / 16) + blk * ROWS;
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const int tl = GATED && r >= ROWS ? tile + p.rows_out / 16 + r - ROWS : tile + r;
                        const uint8_t *from = p.packed + (((int64_t)(tl >> 3) * KB + b) * 8 + (tl & 7)) * TILE_BYTES;
                        for (int i = lane * 16; i < TILE_BYTES; i += 512)
                            cp16(src + r * TILE_BYTES + i, from + i, policy);
                    }
                    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
                    __syncwarp();
                }
#pragma unroll
                for (int sb = 0; sb < 4; ++sb) {
                    uint4 x[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        x[nt][0] = x[nt][1] = make_uint4(0, 0, 0, 0);
                        if (have[nt]) {
                            const uint4 *q = reinterpret_cast<const uint4 *>(row[nt] + b * 256 + sb * 64);
                            x[nt][0] = __ldg(q);
                            x[nt][1] = __ldg(q + 1);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const uint32_t base = src + r * TILE_BYTES;
                        const uint4 q = lds128(base + 512 * sb + 16 * lane);
                        uint32_t sc[2], zz;
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                     : "=r"(sc[0]), "=r"(sc[1])
                                     : "r"(base + 2048 + 128 * (sb >> 1) + 16 * g + 8 * (sb & 1)));
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(zz) : "r"(base + 2304 + 16 * g + 4 * sb));
#pragma unroll
                        for (int gr = 0; gr < 2; ++gr) {
                            // -z 2^-6 of rows g, g + 8
                            const uint32_t z0 = bf16x2_mul(prmt(zz, 0u, gr ? 0x4242u : 0x4040u), NEG_2P127);
                            const uint32_t z1 = bf16x2_mul(prmt(zz, 0u, gr ? 0x4343u : 0x4141u), NEG_2P127);
                            float d[NT][4];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.f;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t w = (&q.x)[2 * gr + k], wh = w >> 8;
                                const uint32_t a[4] = {bf16x2_fma(w & 0x000F000Fu, BF_2P127, z0), bf16x2_fma(wh & 0x000F000Fu, BF_2P127, z1),
                                                       bf16x2_fma(w & 0x00F000F0u, BF_2P123, z0), bf16x2_fma(wh & 0x00F000F0u, BF_2P123, z1)};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    if (nt == 0 || second)
                                        mma_bf16(d[nt], a, k ? x[nt][gr].z : x[nt][gr].x, k ? x[nt][gr].w : x[nt][gr].y, d[nt]);
                            }
                            const float s0 = bf16lo_to_f32(sc[gr]), s1 = bf16hi_to_f32(sc[gr]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                acc[r][nt][0] = fmaf(s0, d[nt][0], acc[r][nt][0]);
                                acc[r][nt][1] = fmaf(s0, d[nt][1], acc[r][nt][1]);
                                acc[r][nt][2] = fmaf(s1, d[nt][2], acc[r][nt][2]);
                                acc[r][nt][3] = fmaf(s1, d[nt][3], acc[r][nt][3]);
                            }
                        }
                    }
                }
                if (n0 == 0)
                    stage = stage + 1 == S ? 0 : stage + 1;
            }
            // --- the sums of the warps that share the unit, and the result
            float *mine = s_sum + warp * (RT * NT * 128);
            if (KW > 1) {
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        *reinterpret_cast<float4 *>(mine + (r * NT + nt) * 128 + lane * 4) =
                            make_float4(acc[r][nt][0], acc[r][nt][1], acc[r][nt][2], acc[r][nt][3]);
                asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * KW) : "memory");
            }
            // fragment f of the result goes to warp f % KW
            for (int f = kw; f < ROWS * NT; f += KW) {
                float v[2][4];
#pragma unroll
                for (int half = 0; half < (GATED ? 2 : 1); ++half) {
                    const int fr = f + half * ROWS * NT;
                    if (KW > 1) {
                        v[half][0] = v[half][1] = v[half][2] = v[half][3] = 0.f;
                        for (int w = 0; w < KW; ++w) {
                            const float4 x = *reinterpret_cast<const float4 *>(
                                s_sum + (group * KW + w) * (RT * NT * 128) + fr * 128 + lane * 4);
                            v[half][0] += x.x;
                            v[half][1] += x.y;
                            v[half][2] += x.z;
                            v[half][3] += x.w;
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < RT; ++r)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                if (r * NT + nt == fr)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        v[half][i] = acc[r][nt][i];
                    }
                }
                const int tile = blk * ROWS + f / NT, col = n0 + (f % NT) * 8 + 2 * t;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (col + i >= n)
                        continue;
                    const int entry = s_list[warp][col + i];
                    if constexpr (GATED) {
                        // rows g (even half of the fragment order) and g + 8 of the 16
                        uint16_t *dst = p.h + (int64_t)entry * p.rows_out + (tile >> 2) * 64 + (g >> 1) * 16 + (tile & 3) * 4 + (g & 1);
#pragma unroll
                        for (int e8 = 0; e8 < 2; ++e8) {
                            const float gate = v[0][2 * e8 + i] * 64.f, up = v[1][2 * e8 + i] * 64.f;
                            const float hv = gate / (1.f + __expf(-gate)) * up;
                            const __nv_bfloat16 hb = __float2bfloat16_rn(hv);
                            dst[2 * e8] = *reinterpret_cast<const uint16_t *>(&hb);
                        }
                    } else {
                        float *dst = p.y + (int64_t)entry * p.rows_out + tile * 16 + g;
                        dst[0] = v[0][i] * 64.f;
                        dst[8] = v[0][2 + i] * 64.f;
                    }
                }
            }
            if (KW > 1)  // the sums are read
                asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * KW) : "memory");
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
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

template <bool GATED, int RT, int NT, int S, int CPS>
cudaError_t launch_gemm(GemmParams p, int sm_count, cudaStream_t stream)
{
    using SM = GemmSmem<GATED, RT, NT, S>;
    static std::atomic<unsigned long long> done{0};
    auto fn = moe_gemm_kernel<GATED, RT, NT, S, CPS>;
    cudaError_t e = smem_opt_in_once(done, fn, (int)SM::bytes(MAX_TOKENS * MAX_TOPK, MAX_EXPERTS));
    if (e != cudaSuccess)
        return e;
    const int KB = p.K / 256;
    p.KW = KB >= 4 ? 4 : (KB >= 2 ? 2 : 1);
    const int most = p.entries < p.experts ? p.entries : p.experts;
    const long long ctas = ((long long)most * (p.rows_out / (16 * (GATED ? RT / 2 : RT))) * p.KW + GW - 1) / GW;
    const long long grid = ctas < (long long)sm_count * CPS ? ctas : (long long)sm_count * CPS;
    return launch_pdl(fn, dim3((unsigned)grid), dim3(32 * GW), SM::bytes(p.entries, p.experts), stream, p);
}

struct Workspace {
    size_t xf, h, y, ids, weights, bytes;
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
    w.h = take((size_t)tokens * topk * inter * 2);
    w.y = take((size_t)tokens * topk * hidden * 4);
    w.ids = take((size_t)tokens * topk * 4);
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
    int32_t *ids = reinterpret_cast<int32_t *>(base + w.ids);

    RouteParams r = {static_cast<const __nv_bfloat16 *>(a.x), static_cast<const __nv_bfloat16 *>(a.router), a.bias, xf,
                     ids, weights, a.ids_out, a.weights_out, a.tokens, a.hidden, a.experts, a.topk, a.sigmoid,
                     a.renormalize, a.scale};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.tokens + ROUTE_TOKENS - 1) / ROUTE_TOKENS * ROUTE_CTAS));
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, moe_route_kernel, r);
    if (e != cudaSuccess)
        return e;

    GemmParams up = {static_cast<const uint8_t *>(a.w13), xf, ids, h, nullptr, a.tokens * a.topk, a.topk, a.experts,
                     a.hidden, a.inter, 1};
    GemmParams down = {static_cast<const uint8_t *>(a.w2), h, ids, nullptr, y, a.tokens * a.topk, a.topk, a.experts,
                       a.inter, a.hidden, 1};
    if (a.tokens <= 8) {
        e = launch_gemm<true, 2, 1, 2, 4>(up, sm_count, stream);
        if (e == cudaSuccess)
            e = launch_gemm<false, 2, 1, 2, 4>(down, sm_count, stream);
    } else {
        e = launch_gemm<true, 4, 2, 2, 2>(up, sm_count, stream);
        if (e == cudaSuccess)
            e = launch_gemm<false, 4, 2, 2, 2>(down, sm_count, stream);
    }
    if (e != cudaSuccess)
        return e;
    const long long threads = (long long)a.tokens * (a.hidden / 4);
    return launch_pdl(moe_combine_kernel, dim3((unsigned)((threads + 127) / 128)), dim3(128), 0, stream,
                      static_cast<const float *>(y), static_cast<const float *>(weights),
                      static_cast<__nv_bfloat16 *>(a.out), a.tokens, a.topk, a.hidden);
}

}  // namespace w4q
