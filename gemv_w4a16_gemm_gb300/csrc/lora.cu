// lora.cu -- low-rank adapters of many requests beside a shared projection:
//
//     out[m] = bf16(y[m] + c_a * B_a (A_a x[m])),  a = ids[m]
//
// with A_a [rank][K], B_a [N][rank] in bf16 and out[m] = y[m] for a token
// without an adapter.  Two launches: the first forms h = A_a x (fp32 sums of
// exact products), the second adds B_a h; small adapters take one launch of
// thread-block clusters, which do both.
//
// Every warp finds the (at most 64) tokens' adapters by itself, so an adapter's weights
// are read once for each 16 of its tokens (from L2 but the first time: whoever has many
// tokens an adapter has few adapters).  Both products are m16n8k16 MMAs with the weights
// of 16 ranks or outputs as their rows and tokens as their columns.  A dot product does
// not depend on the order of its terms, so k runs in the order in which 16-byte pieces of
// a row lie in the lanes' registers, and the weights need no rearrangement.  h enters the
// second product as the sum of three bf16, which is all of its 24 bits, so that a row is as
// precise alone as in any batch.  (As two, 16 bits, one result in 600 was another bf16 than the
// exact sum's, one in 4000 to 11000 so; the third costs nothing for up to 2 tokens of an
// adapter, 0.3 us in 11 for 8 of rank 32, and 5 in 25 for 64 of rank 256, where two warps a CTA
// multiply.)
//
// What bounds it: the used adapters' bytes, read once each, for large ones (64 adapters of
// rank 64, 6656 to 19968: 220 MB in 46.0 us, 4.8 TB/s with both launches' beginnings, of
// which the second product runs at 7); for few the chain of dependent loads (rank 16,
// 4096 to 4096: 4.8 us).  In the second product every warp streams its own pieces of the
// weights through a ring of bulk copies in shared memory, so that some 100 KB an SM are in
// flight whatever the MMAs and their registers need.
#include <atomic>
#include <cfloat>

#include "common.cuh"
#include "decode.h"
#include "kernels.h"

namespace w4q {

namespace {

constexpr int TILE = 16;      // tokens of one adapter that are taken together
constexpr int MAX_PARTS = 8;  // partial sums of h that the second launch adds up

constexpr int NEEDS = 3;

struct LoraArgs {
    const __nv_bfloat16 *x, *y, *A, *B;
    const int32_t *ids;
    const float *scales;
    __nv_bfloat16 *out;
    float *h;  // [parts][tokens][rank]
    unsigned *err;
    int64_t x_stride, y_stride, out_stride;
    int tokens, K, N, rank, adapters;
    int grid1;      // CTAs of the first launch
    int warps;      // of a CTA that multiply in the second, and stages of each one's ring
    int stages;
    int sms;
    int cluster;    // CTAs of a cluster
    int room;       // clusters that leave some of the device to the next launch's beginning
    int need[NEEDS];  // clusters of a tile with which a warp has one unit, at most two, three
    bool vec;       // the rows of y and out keep 8-byte alignment
    bool in_place;  // out is y: tokens without an adapter are there already
};

// The tokens by adapter, cut into tiles of up to 16 of one adapter's tokens.  Every
// warp finds them for itself, two tokens a lane (its own number and 32 more), so that
// no warp waits for another: a token leads a tile if a multiple of 16 tokens before it
// have its adapter; tiles are numbered by their leaders, those without an adapter last.
struct Tiles {
    int id[2];    // adapter, -1: none, -2: no token
    int same[2];  // earlier tokens of the adapter
    int rank[2];  // number of the tile that the token leads, or -1
    int used, all;  // tiles with an adapter; with those without one
};

__device__ __forceinline__ Tiles find_tiles(const LoraArgs &p)
{
    const int lane = threadIdx.x & 31;
    const uint32_t before = (1u << lane) - 1u, full = 0xffffffffu;
    Tiles g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = lane + 32 * h;
        g.id[h] = -2;
        if (t < p.tokens) {
            const int id = __ldcg(p.ids + t);
            g.id[h] = id < 0 || id >= p.adapters ? -1 : id;
        }
    }
    g.same[0] = __popc(__match_any_sync(full, g.id[0]) & before);
    g.same[1] = 0;
    if (p.tokens > 32) {
        g.same[1] = __popc(__match_any_sync(full, g.id[1]) & before);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            g.same[1] += __shfl_sync(full, g.id[0], i) == g.id[1];
    }
    uint32_t with[2], none[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool leads = g.same[h] % TILE == 0;
        with[h] = __ballot_sync(full, leads && g.id[h] >= 0);
        none[h] = __ballot_sync(full, leads && g.id[h] == -1);
    }
    g.used = __popc(with[0]) + __popc(with[1]);
    g.all = g.used + __popc(none[0]) + __popc(none[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        g.rank[h] = -1;
        if (with[h] >> lane & 1)
            g.rank[h] = (h ? __popc(with[0]) : 0) + __popc(with[h] & before);
        if (none[h] >> lane & 1)
            g.rank[h] = g.used + (h ? __popc(none[0]) : 0) + __popc(none[h] & before);
    }
    return g;
}

// Tile j's adapter and, into tok[0 .. count), its tokens in order; a whole warp.
__device__ __forceinline__ int tile_tokens(const Tiles &g, int j, int *tok, int &count)
{
    const int lane = threadIdx.x & 31;
    const uint32_t before = (1u << lane) - 1u, full = 0xffffffffu;
    const uint32_t lead0 = __ballot_sync(full, g.rank[0] == j), lead1 = __ballot_sync(full, g.rank[1] == j);
    const int from = __ffs(lead0 ? lead0 : lead1) - 1;
    const int id = __shfl_sync(full, lead0 ? g.id[0] : g.id[1], from);
    const int base = __shfl_sync(full, lead0 ? g.same[0] : g.same[1], from);
    const bool in0 = g.id[0] == id && g.same[0] >= base && g.same[0] < base + TILE;
    const bool in1 = g.id[1] == id && g.same[1] >= base && g.same[1] < base + TILE;
    const uint32_t m0 = __ballot_sync(full, in0), m1 = __ballot_sync(full, in1);
    __syncwarp();
    if (in0)
        tok[__popc(m0 & before)] = lane;
    if (in1)
        tok[__popc(m0) + __popc(m1 & before)] = lane + 32;
    count = __popc(m0) + __popc(m1);
    __syncwarp();
    return id;
}

// Bulk copy of weights into this CTA's shared memory, counted on the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// The whole warp waits for a stage; false if the wait ran out.
__device__ __forceinline__ bool stage_ready(uint32_t bar, uint32_t parity, unsigned *err)
{
    const bool got = mbar_wait_sleep(bar, parity);
    if (__all_sync(0xffffffffu, got))
        return true;
    if ((threadIdx.x & 31) == 0)
        report_error(err, ERR_FULL_WAIT);
    return false;
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16 *p, bool on)
{
    return on ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ h = A x

// A stage: 16 ranks by 1024 columns, one bulk copy of up to 2 KB a row (copies of 256
// bytes were bound by their number: 54 MB in 18 us against 12), rows 64 bytes further
// apart, so that two rows' 64-byte pieces lie in different banks.
constexpr int STAGE_K = 1024, ROW_PITCH = 2 * STAGE_K + 64, DOWN_STAGE = 16 * ROW_PITCH, DOWN_STAGES = 3;
constexpr int DOWN_WARPS = 8, DOWN_THREADS = 32 * (DOWN_WARPS + 1);  // the last warp copies
constexpr int WARP_K = STAGE_K / DOWN_WARPS, UNITS = WARP_K / 32;    // a warp's columns of a stage, in steps of 32
constexpr int DOWN_SMEM = DOWN_STAGES * DOWN_STAGE;

// The first launch's work is a line: tiles of tokens, for each its ranks by 16, for each
// up to MAX_PARTS pieces of K.  It is cut evenly among the CTAs; those that share an item
// (tile, 16 ranks) leave a partial sum each, in the order of the line.
struct Line {
    int ranks, pieces, piece_k;  // items of a tile, pieces of an item, columns of a piece
    int total, ctas;
};
__device__ __forceinline__ Line line_of(const LoraArgs &p, int tiles)
{
    Line l;
    const int stages = (p.K + STAGE_K - 1) / STAGE_K, each = (stages + MAX_PARTS - 1) / MAX_PARTS;
    l.ranks = (p.rank + 15) / 16;
    l.pieces = (stages + each - 1) / each;
    l.piece_k = each * STAGE_K;
    l.total = tiles * l.ranks * l.pieces;
    l.ctas = min(p.grid1, l.total);
    return l;
}
// The CTA that has piece u: the largest c with c * total / ctas <= u.
__device__ __forceinline__ int owner(const Line &l, int u) { return ((u + 1) * l.ctas - 1) / l.total; }

// What a CTA whose pieces end before `end` has, from piece u on, of one item: columns k0
// to k1, and which of the item's partial sums that gives.
struct Share {
    int tile, rank0, k0, k1, part;
};
__device__ __forceinline__ Share share_of(const LoraArgs &p, const Line &l, int u, int end, int &next)
{
    const int item = u / l.pieces, from = item * l.pieces;
    next = min(end, from + l.pieces);
    return {item / l.ranks, item % l.ranks * 16, (u - from) * l.piece_k, min((next - from) * l.piece_k, p.K),
            (int)blockIdx.x - owner(l, from)};
}

// A warp's columns of a stage, from k on, of tokens first to first + 7, a lane's one of them.
__device__ __forceinline__ void load_tokens(const LoraArgs &p, const int *toks, int first, int count, int k, int k1, uint4 (&v)[UNITS])
{
    const int lane = threadIdx.x & 31, t = first + (lane >> 2), c = lane & 3;
    const __nv_bfloat16 *x = p.x + (t < count ? toks[t] : 0) * p.x_stride + k + 8 * c;
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
        v[i] = load16(x + 32 * i, t < count && k + 32 * i + 8 * c < k1);
}

__global__ void __maxnreg__(128) lora_down_kernel(const LoraArgs p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int toks[2][DOWN_WARPS + 1][TILE];
    __shared__ float red[DOWN_WARPS][TILE * 16];
    __shared__ alignas(8) uint64_t bars[2 * DOWN_STAGES];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const uint32_t full = smem_addr(bars), empty = full + 8 * DOWN_STAGES;
    if (threadIdx.x == 0) {
        for (int s = 0; s < DOWN_STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, DOWN_WARPS);
        }
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();
    // only now: the second launch reads its other inputs before it waits for this one
    pdl_launch_dependents();
    const Tiles g = find_tiles(p);
    const Line l = line_of(p, g.used);
    if ((int)blockIdx.x >= l.ctas)
        return;
    const int begin = blockIdx.x * l.total / l.ctas, end = (blockIdx.x + 1) * l.total / l.ctas;
    int stage = 0;  // stages so far

    if (warp == DOWN_WARPS) {
        bool alive = true;
        for (int u = begin, next; u < end && alive; u = next) {
            const Share h = share_of(p, l, u, end, next);
            const int rows = min(16, p.rank - h.rank0);
            int count;
            const int adapter = tile_tokens(g, h.tile, toks[0][warp], count);
            const __nv_bfloat16 *A = p.A + ((size_t)adapter * p.rank + h.rank0 + min(lane, rows - 1)) * p.K;
            for (int k = h.k0; k < h.k1; k += STAGE_K, ++stage) {
                const int slot = stage % DOWN_STAGES;
                if (stage >= DOWN_STAGES) {
                    const bool got = mbar_wait_sleep(empty + 8 * slot, stage / DOWN_STAGES - 1 & 1);
                    if (!__all_sync(0xffffffffu, got)) {
                        report_error(p.err, ERR_EMPTY_WAIT);
                        alive = false;
                        break;
                    }
                }
                const uint32_t bytes = 2 * min(STAGE_K, h.k1 - k);
                if (lane == 0)
                    mbar_arrive_expect_tx(full + 8 * slot, bytes * rows);
                __syncwarp();
                if (lane < rows)
                    bulk_load(smem_addr(smem + slot * DOWN_STAGE + lane * ROW_PITCH), A + k, bytes, full + 8 * slot);
            }
        }
        // what is in flight lands in this CTA's memory
        for (int s = max(0, stage - DOWN_STAGES); s < stage; ++s)
            if (!mbar_wait_sleep(full + 8 * (s % DOWN_STAGES), s / DOWN_STAGES & 1)) {
                report_error(p.err, ERR_DRAIN_WAIT);
                break;
            }
        return;
    }

    // The first 8 tokens' columns are loaded a stage ahead: they come from L2, whose latency
    // was longer than a stage's time.  (Tiles of more tokens have few adapters to stream.)
    bool alive = true;
    float acc[2][4] = {};
    uint4 v[UNITS];
    int next, buf = 0, count;
    Share h = share_of(p, l, begin, end, next);
    tile_tokens(g, h.tile, toks[0][warp], count);
    load_tokens(p, toks[0][warp], 0, count, h.k0 + warp * WARP_K, h.k1, v);
    while (true) {
        Share after = h;
        int after_next = next, after_count = 0;
        if (next < end) {
            after = share_of(p, l, next, end, after_next);
            tile_tokens(g, after.tile, toks[buf ^ 1][warp], after_count);
        }
        const bool half = h.rank0 + 8 >= p.rank;  // only 8 ranks
        for (int k0 = h.k0; k0 < h.k1; k0 += STAGE_K, ++stage) {
            const int slot = stage % DOWN_STAGES, k = k0 + warp * WARP_K;
            const uint8_t *rows = smem + slot * DOWN_STAGE + r * ROW_PITCH + 2 * WARP_K * warp + 16 * c;
            uint4 ahead[UNITS], more[UNITS];
            if (count > 8)
                load_tokens(p, toks[buf][warp], 8, count, k, h.k1, more);
            if (k0 + STAGE_K < h.k1)
                load_tokens(p, toks[buf][warp], 0, count, k + STAGE_K, h.k1, ahead);
            else
                load_tokens(p, toks[buf ^ 1][warp], 0, after_count, after.k0 + warp * WARP_K, after.k1, ahead);
            if (alive)
                alive = stage_ready(full + 8 * slot, stage / DOWN_STAGES & 1, p.err);
            if (alive) {
#pragma unroll
                for (int i = 0; i < UNITS; ++i) {
                    uint4 w0 = *reinterpret_cast<const uint4 *>(rows + 64 * i), w1 = *reinterpret_cast<const uint4 *>(rows + 8 * ROW_PITCH + 64 * i);
                    if (k + 32 * i + 8 * c >= h.k1)  // what lies behind the columns is not theirs
                        w0 = w1 = make_uint4(0u, 0u, 0u, 0u);
                    if (half)
                        w1 = make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t f0[4] = {w0.x, w1.x, w0.y, w1.y}, f1[4] = {w0.z, w1.z, w0.w, w1.w};
                    mma_bf16(acc[0], f0, v[i].x, v[i].y, acc[0]);
                    mma_bf16(acc[0], f1, v[i].z, v[i].w, acc[0]);
                    if (count > 8) {
                        mma_bf16(acc[1], f0, more[i].x, more[i].y, acc[1]);
                        mma_bf16(acc[1], f1, more[i].z, more[i].w, acc[1]);
                    }
                }
                __syncwarp();  // every lane has read the stage
                if (lane == 0)
                    mbar_arrive(empty + 8 * slot);
            }
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
                v[i] = ahead[i];
        }
        // this CTA's share of the item: the warps' sums are added up in their order
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                red[warp][(8 * n + 2 * c + (e & 1)) * 16 + r + 8 * (e >> 1)] = acc[n][e];
                acc[n][e] = 0.f;
            }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * DOWN_WARPS) : "memory");
        for (int i = threadIdx.x; i < count * 16; i += 32 * DOWN_WARPS) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < DOWN_WARPS; ++w)
                s += red[w][i];
            if (h.rank0 + i % 16 < p.rank)
                p.h[((size_t)h.part * p.tokens + toks[buf][warp][i / 16]) * p.rank + h.rank0 + i % 16] = s;
        }
        if (next >= end)
            break;
        asm volatile("bar.sync 1, %0;" ::"n"(32 * DOWN_WARPS) : "memory");
        h = after;
        next = after_next;
        count = after_count;
        buf ^= 1;
    }
}

// -------------------------------------------------------------- out = y + B h

// A warp works on 32 outputs at a time: 32 rows of B, one contiguous piece, and so
// one bulk copy.
constexpr int COLS = 32;
constexpr int UP_MAX_STAGES = 8;
constexpr int UP_SMEM = 112 * 1024;  // for two CTAs an SM, beside 1 KB of static shared memory

// Warps of a CTA that multiply: fewer for the larger pieces of high ranks.  Beside two of them
// others help to add up h (rank 256, 33 tokens of one adapter, 4096 to 4096: by 6 us, now 16.9);
// with four it costs more than it saves, since a CTA of both launches then has no room on an SM
// (32 of rank 128: 19.4 without, 20.1 with).
constexpr int UP_WARPS = 8;
__host__ __device__ constexpr int up_warps(int rank) { return rank <= 64 ? UP_WARPS : (rank <= 128 ? 4 : 2); }
__host__ __device__ constexpr int up_block_warps(int rank) { return rank <= 128 ? up_warps(rank) : UP_WARPS; }

// h lies in shared memory as the MMAs' operand of 8 columns, NT tiles of them: up to 2
// tokens: 1 tile, the first bf16 of each in columns 0 and 1, the second in 2 and 3, the third
// in 4 and 5; up to 4: 2 tiles, the first bf16 in columns 0 to 3 of one, the second in 4 to 7,
// the third in 0 to 3 of the other; up to 8: 3 tiles, one for each bf16; up to 16: 6.
// (With the tokens as the 16 rows of the other operand, twice the MMAs, 64 adapters of rank 64
// took 49 us instead of 45.6.)
__host__ __device__ constexpr int h_tiles(int count) { return count <= 2 ? 1 : (count <= 4 ? 2 : (count <= 8 ? 3 : 6)); }
__host__ __device__ constexpr int h_sums(int nt) { return (nt + 2) / 3; }  // tiles of results

// Bytes from column to column of h: two columns' 16-byte pieces (ranks in 32s), or four
// columns' 8-byte pieces, lie in different banks.
__host__ __device__ constexpr int h_pitch(int rank)
{
    return rank % 32 == 0 ? 2 * rank + (rank % 64 == 0 ? 64 : 0) : 32 * ((rank + 15) / 16 | 1);
}

// Four ranks from k on of token t's h, as three bf16 each; slots: 2, 4, 8 or 16 tokens' places.
__device__ __forceinline__ void store_h(uint8_t *h, int pitch, int slots, int t, int k, float4 s)
{
    const float f[4] = {s.x, s.y, s.z, s.w};
    uint32_t b[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        // the first 8 bits, which stay finite; what is not finite is the first part alone
        const bool finite = fabsf(f[e]) <= FLT_MAX;
        b[0][e] = finite ? __float_as_uint(f[e]) >> 16 : __bfloat16_as_ushort(__float2bfloat16_rn(f[e]));
        float rest = finite ? f[e] - bf16hi_to_f32(__float_as_uint(f[e])) : 0.f;
#pragma unroll
        for (int i = 1; i < 3; ++i) {
            const __nv_bfloat16 v = __float2bfloat16_rn(rest);
            b[i][e] = __bfloat16_as_ushort(v);
            rest -= __bfloat162float(v);
        }
    }
    const int col = slots == 16 ? t % 8 + t / 8 * 24 : t, step = slots == 16 ? 8 : slots;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        *reinterpret_cast<uint2 *>(h + (col + i * step) * pitch + 2 * k) = make_uint2(b[i][0] | b[i][1] << 16, b[i][2] | b[i][3] << 16);
}
// Zeros, from rank k on, in the columns of a tile that no token has.
__device__ __forceinline__ void store_h_rest(uint8_t *h, int pitch, int slots, int t, int k)
{
    if (slots <= 4)
        for (int col = 3 * slots + t; col < (slots == 2 ? 8 : 16); col += slots)
            *reinterpret_cast<uint2 *>(h + col * pitch + 2 * k) = make_uint2(0u, 0u);
}
__device__ __forceinline__ int h_slots(int count) { return count <= 2 ? 2 : (count <= 4 ? 4 : (count <= 8 ? 8 : 16)); }

// h of a tile's tokens, the parts added up in their order; zeros in the columns of other
// tokens and behind the last rank.
__device__ __forceinline__ void load_h(const LoraArgs &p, const Line &l, int tile, const int *toks, int count, int pitch, uint8_t *h)
{
    const int quads = (p.rank + 15) / 16 * 4, slots = h_slots(count);
    for (int i = threadIdx.x; i < slots * quads; i += blockDim.x) {
        const int t = i / quads, k = i % quads * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < count && k < p.rank) {
            const float *src = p.h + (size_t)toks[t] * p.rank + k;
            const int piece = (tile * l.ranks + k / 16) * l.pieces, parts = owner(l, piece + l.pieces - 1) - owner(l, piece) + 1;
            float4 v[MAX_PARTS];
#pragma unroll
            for (int q = 0; q < MAX_PARTS; ++q)
                v[q] = q < parts ? __ldcg(reinterpret_cast<const float4 *>(src + (size_t)q * p.tokens * p.rank)) : s;
#pragma unroll
            for (int q = 0; q < MAX_PARTS; ++q)
                s.x += v[q].x, s.y += v[q].y, s.z += v[q].z, s.w += v[q].w;
        }
        store_h(h, pitch, slots, t, k, s);
        store_h_rest(h, pitch, slots, t, k);
    }
}

// delta of 32 outputs: row q of tile i is output 4 q + 2 i, row q + 8 output 4 q + 2 i + 1, so
// that a lane's results of a token are 4 outputs in a row.
// WIDE (ranks in 32s): 16-byte pieces, 8 ranks a lane; where a row is a multiple of 128
// bytes the odd rows' pairs of pieces are read in the other order, so that two rows' pieces
// never lie in the same banks.  Else 8-byte pieces, 4 ranks a lane.
template <bool WIDE, int NT>
__device__ __forceinline__ void multiply(const LoraArgs &p, const uint8_t *stage, const uint8_t *h, int pitch,
                                         float (&acc)[2][h_sums(NT)][4])
{
    const int lane = threadIdx.x & 31, q = lane >> 2, c = lane & 3, row = 2 * p.rank;
    const uint8_t *from = stage + 4 * q * row;
    if (WIDE) {
        const int odd = p.rank % 64 == 0 ? q & 1 : 0;
        for (int k = 0; k < p.rank; k += 64) {
            uint4 w[2][2][2];  // 32 ranks, tile, half
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint8_t *at = from + (2 * i + e) * row + 2 * k + 16 * c;
                    const uint4 a = *reinterpret_cast<const uint4 *>(at + 64 * odd);
                    uint4 b = a;
                    if (k + 32 < p.rank)
                        b = *reinterpret_cast<const uint4 *>(at + 64 - 64 * odd);
                    w[0][i][e] = odd ? b : a;
                    w[1][i][e] = odd ? a : b;
                }
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (k + 32 * b < p.rank)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(h + (8 * n + q) * pitch + 2 * k + 64 * b + 16 * c);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t f0[4] = {w[b][i][0].x, w[b][i][1].x, w[b][i][0].y, w[b][i][1].y};
                            mma_bf16(acc[i][n / 3], f0, v.x, v.y, acc[i][n / 3]);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t f1[4] = {w[b][i][0].z, w[b][i][1].z, w[b][i][0].w, w[b][i][1].w};
                            mma_bf16(acc[i][n / 3], f1, v.z, v.w, acc[i][n / 3]);
                        }
                    }
        }
    } else {
        for (int k = 0; k < p.rank; k += 16) {
            uint2 w[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    w[i][e] = k + 4 * c < p.rank ? *reinterpret_cast<const uint2 *>(from + (2 * i + e) * row + 2 * k + 8 * c)
                                                 : make_uint2(0u, 0u);  // what lies behind the row is not its
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 v = *reinterpret_cast<const uint2 *>(h + (8 * n + q) * pitch + 2 * k + 8 * c);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t f[4] = {w[i][0].x, w[i][1].x, w[i][0].y, w[i][1].y};
                    mma_bf16(acc[i][n / 3], f, v.x, v.y, acc[i][n / 3]);
                }
            }
        }
    }
}

// y of a lane's tokens and its 4 outputs from n on.
template <int TOKS>
struct Base {
    uint2 v[TOKS];
};
template <int TOKS>
__device__ __forceinline__ Base<TOKS> load_base(const LoraArgs &p, const int (&tok)[TOKS], int n)
{
    Base<TOKS> b;
#pragma unroll
    for (int e = 0; e < TOKS; ++e)
        b.v[e] = tok[e] >= 0 && p.vec && n + 4 <= p.N ? *reinterpret_cast<const uint2 *>(p.y + tok[e] * p.y_stride + n) : make_uint2(0u, 0u);
    return b;
}

// Four results of a token: out = bf16(y + scale * delta).
__device__ __forceinline__ void add_store(const LoraArgs &p, int tok, int n, const float (&d)[4], float scale, uint2 base)
{
    __nv_bfloat16 *o = p.out + tok * p.out_stride + n;
    if (p.vec && n + 4 <= p.N) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(fmaf(scale, d[0], bf16lo_to_f32(base.x)), fmaf(scale, d[1], bf16hi_to_f32(base.x)));
        const __nv_bfloat162 b = __floats2bfloat162_rn(fmaf(scale, d[2], bf16lo_to_f32(base.y)), fmaf(scale, d[3], bf16hi_to_f32(base.y)));
        *reinterpret_cast<uint2 *>(o) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        const __nv_bfloat16 *y = p.y + tok * p.y_stride + n;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < p.N)
                o[j] = __float2bfloat16_rn(fmaf(scale, d[j], __bfloat162float(y[j])));
    }
}

// Units whose y is loaded ahead: a unit of a low rank takes less time than that (with one, 64
// tokens of as many adapters of rank 8, 2048 to 50000, took 45 us, 34 so, and 33 with four).
__host__ __device__ constexpr int y_ahead(int nt) { return nt <= 3 ? 2 : 1; }

// A warp's ring in the second launch.
struct UpRing {
    uint8_t *mem;
    uint32_t bar, parity;
    int slot, stages, stage_bytes;
    bool alive;
};

// The weights of unit u into slot s of the ring, of B (an adapter's).
__device__ __forceinline__ void issue_unit(const LoraArgs &p, const UpRing &ring, const __nv_bfloat16 *B, int u, int s)
{
    if ((threadIdx.x & 31) == 0) {
        const uint32_t bytes = min(COLS, p.N - u * COLS) * p.rank * 2;
        mbar_arrive_expect_tx(ring.bar + 8 * s, bytes);
        bulk_load(smem_addr(ring.mem + s * ring.stage_bytes), B + (size_t)u * COLS * p.rank, bytes, ring.bar + 8 * s);
    }
}

// Waits for unit u of u, u + step, ... below u1; false if that or an earlier wait ran out.
__device__ __forceinline__ bool unit_ready(const LoraArgs &p, UpRing &ring, int u, int u1, int step)
{
    if (!ring.alive)
        return false;
    if (stage_ready(ring.bar + 8 * ring.slot, ring.parity, p.err))
        return true;
    // what else is in flight still lands in this CTA's memory
    for (int i = 0, v = u; i < ring.stages && v < u1; ++i, v += step) {
        const bool wraps = ring.slot + i >= ring.stages;
        if (!mbar_wait_sleep(ring.bar + 8 * (ring.slot + i - (wraps ? ring.stages : 0)), ring.parity ^ (wraps ? 1u : 0u)))
            report_error(p.err, ERR_DRAIN_WAIT);
    }
    return ring.alive = false;
}
// Every lane has read unit u: the next one's weights into its slot.
__device__ __forceinline__ void unit_done(const LoraArgs &p, UpRing &ring, const __nv_bfloat16 *B, int u, int u1, int step)
{
    __syncwarp();
    if (u + ring.stages * step < u1)
        issue_unit(p, ring, B, u + ring.stages * step, ring.slot);
    if (++ring.slot == ring.stages) {
        ring.slot = 0;
        ring.parity ^= 1;
    }
}

// A warp's units u0, u0 + step, ... below u1 of a tile with NT tiles of h, the first of
// whose weights are on their way.
template <bool WIDE, int NT>
__device__ __forceinline__ void add_units(const LoraArgs &p, UpRing &ring, const __nv_bfloat16 *B, const int *toks, int count, float scale,
                                          int u0, int u1, int step, const uint8_t *h, int pitch)
{
    // NT = 1 and 2: lane column c adds the parts of one token; else it has two tokens of each 8
    constexpr int TOKS = NT <= 2 ? 1 : (NT == 3 ? 2 : 4);
    const int lane = threadIdx.x & 31, q = lane >> 2, c = lane & 3;
    int tok[TOKS];
#pragma unroll
    for (int e = 0; e < TOKS; ++e) {
        const int t = NT == 1 ? (c < 2 ? c : count) : (NT == 2 ? 2 * (c & 1) + (c >> 1) : 8 * (e / 2) + 2 * c + e % 2);
        tok[e] = t < count ? toks[t] : -1;
    }
    constexpr int AHEAD = y_ahead(NT);
    Base<TOKS> bases[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        bases[i] = load_base<TOKS>(p, tok, u0 + i * step < u1 ? (u0 + i * step) * COLS + 4 * q : p.N);
    for (int u = u0; u < u1; u += step) {
        const Base<TOKS> base = bases[0];
#pragma unroll
        for (int i = 0; i < AHEAD - 1; ++i)
            bases[i] = bases[i + 1];
        const int v = u + AHEAD * step;
        bases[AHEAD - 1] = load_base<TOKS>(p, tok, v < u1 ? v * COLS + 4 * q : p.N);
        if (!unit_ready(p, ring, u, u1, step))
            continue;
        float acc[2][h_sums(NT)][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < h_sums(NT); ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][n][e] = 0.f;
        multiply<WIDE, NT>(p, ring.mem + ring.slot * ring.stage_bytes, h, pitch, acc);
        unit_done(p, ring, B, u, u1, step);
        const int n = u * COLS + 4 * q;
        if (NT <= 2) {
            float d[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float first = acc[j / 2][0][2 * (j & 1)], second = acc[j / 2][0][2 * (j & 1) + 1];  // columns 2 c and 2 c + 1
                if (NT == 1) {  // a token's parts are in lane columns 0 to 2: token 0 goes to column 0, token 1 to 1
                    const float got = __shfl_xor_sync(0xffffffffu, c & 1 ? first : second, 1);
                    const float sum = c < 2 ? (c ? second : first) + got : (c == 2 ? first : got);
                    d[j] = sum + __shfl_xor_sync(0xffffffffu, sum, 2);
                } else {  // the lane two columns on holds the second parts of the same tokens
                    d[j] = (c < 2 ? first : second) + __shfl_xor_sync(0xffffffffu, c < 2 ? second : first, 2);
                }
            }
            if (tok[0] >= 0 && n < p.N)
                add_store(p, tok[0], n, d, scale, base.v[0]);
        } else {
#pragma unroll
            for (int e = 0; e < TOKS; ++e)
                if (tok[e] >= 0 && n < p.N) {
                    const float d[4] = {acc[0][e / 2][e % 2], acc[0][e / 2][2 + e % 2], acc[1][e / 2][e % 2], acc[1][e / 2][2 + e % 2]};
                    add_store(p, tok[e], n, d, scale, base.v[e]);
                }
        }
    }
}

// The same for one token and a rank of R: a lane has an output and all of h, in fp32, in registers, which
// takes a third of the instructions (16 tokens of as many adapters of rank 16, 6656 to 19968: 10.7
// -> 8.8 us).
template <int R>
__device__ __forceinline__ void add_units_one(const LoraArgs &p, UpRing &ring, const __nv_bfloat16 *B, int tok, float scale, int u0, int u1,
                                              int step, const uint8_t *h)
{
    const int lane = threadIdx.x & 31;
    float2 hv[R / 2];
#pragma unroll
    for (int k = 0; k < R / 2; ++k)
        hv[k] = reinterpret_cast<const float2 *>(h)[k];
    const __nv_bfloat16 *y = p.y + tok * p.y_stride;
    __nv_bfloat16 *out = p.out + tok * p.out_stride;
    auto load = [&](int u) { return u < u1 && u * COLS + lane < p.N ? y[u * COLS + lane] : __nv_bfloat16(); };
    constexpr int AHEAD = y_ahead(1);
    __nv_bfloat16 bases[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        bases[i] = load(u0 + i * step);
    for (int u = u0; u < u1; u += step) {
        const __nv_bfloat16 base = bases[0];
#pragma unroll
        for (int i = 0; i < AHEAD - 1; ++i)
            bases[i] = bases[i + 1];
        bases[AHEAD - 1] = load(u + AHEAD * step);
        if (!unit_ready(p, ring, u, u1, step))
            continue;
        const uint4 *row = reinterpret_cast<const uint4 *>(ring.mem + ring.slot * ring.stage_bytes + lane * 2 * R);
        float2 acc[2] = {};
#pragma unroll
        for (int k = 0; k < R / 8; ++k) {
            const uint4 w = row[k];
            acc[0] = fma2({bf16lo_to_f32(w.x), bf16hi_to_f32(w.x)}, hv[4 * k], acc[0]);
            acc[1] = fma2({bf16lo_to_f32(w.y), bf16hi_to_f32(w.y)}, hv[4 * k + 1], acc[1]);
            acc[0] = fma2({bf16lo_to_f32(w.z), bf16hi_to_f32(w.z)}, hv[4 * k + 2], acc[0]);
            acc[1] = fma2({bf16lo_to_f32(w.w), bf16hi_to_f32(w.w)}, hv[4 * k + 3], acc[1]);
        }
        unit_done(p, ring, B, u, u1, step);
        const float2 d = add2(acc[0], acc[1]);
        if (u * COLS + lane < p.N)
            out[u * COLS + lane] = __float2bfloat16_rn(fmaf(scale, d.x + d.y, __bfloat162float(base)));
    }
}

// Tokens without an adapter keep what they have: units u0, u0 + step, ... of a tile.  A lane's
// loads of 4 tokens go out before their stores (45 of 64 tokens with an adapter each of rank 64,
// 6656 to 19968: 62.5 us with one after the other, 40.6 so).
__device__ __forceinline__ void copy_units(const LoraArgs &p, const int *toks, int count, int u0, int u1, int step)
{
    const int lane = threadIdx.x & 31;
    if (p.vec) {
        const int q = lane >> 2, c = lane & 3;
#pragma unroll 1
        for (int u = u0; u < u1; u += step) {
            const int n = u * COLS + 4 * q;
            if (n + 4 <= p.N) {
                uint2 v[TILE / 4];
#pragma unroll
                for (int j = 0; j < TILE / 4; ++j)
                    if (c + 4 * j < count)
                        v[j] = *reinterpret_cast<const uint2 *>(p.y + toks[c + 4 * j] * p.y_stride + n);
#pragma unroll
                for (int j = 0; j < TILE / 4; ++j)
                    if (c + 4 * j < count)
                        *reinterpret_cast<uint2 *>(p.out + toks[c + 4 * j] * p.out_stride + n) = v[j];
            } else {
                for (int t = c; t < count; t += 4)
                    for (int k = n; k < p.N; ++k)
                        p.out[toks[t] * p.out_stride + k] = p.y[toks[t] * p.y_stride + k];
            }
        }
    } else {  // a lane has an output of every token
#pragma unroll 1
        for (int u = u0; u < u1; u += step) {
            const int n = u * COLS + lane;
            if (n < p.N)
#pragma unroll 1
                for (int t = 0; t < count; t += 8) {
                    __nv_bfloat16 v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (t + j < count)
                            v[j] = p.y[toks[t + j] * p.y_stride + n];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (t + j < count)
                            p.out[toks[t + j] * p.out_stride + n] = v[j];
                }
        }
    }
}

// What another tile costs a CTA, in units: 16 of rank 64, 4096 to 4096 11.0 -> 10.0 us, 32 of
// rank 128 20.7 -> 19.4; 8 to 1000 measured alike.
constexpr int SWITCH = 32;

// The tiles' units of 32 outputs, one tile after the other, are cut evenly among the
// CTAs; the warps of one take turns.
template <bool WIDE>
__global__ void __launch_bounds__(32 * UP_WARPS, 2) lora_up_kernel(const LoraArgs p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int warp_toks[UP_WARPS][TILE];
    __shared__ alignas(8) uint64_t bars[UP_WARPS][UP_MAX_STAGES];
    const int warps = p.warps, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int w = 0; w < warps; ++w)
            for (int s = 0; s < p.stages; ++s)
                mbar_init(smem_addr(&bars[w][s]), 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    // The first launch lets this one start only after all that was before it has
    // finished, so what that wrote can be read here; h cannot.
    const Tiles g = find_tiles(p);
    int *const toks = warp_toks[warp];
    const int stage_bytes = COLS * p.rank * 2, pitch = h_pitch(p.rank);
    UpRing ring = {smem + warp * p.stages * stage_bytes, smem_addr(bars[warp]), 0u, 0, p.stages, stage_bytes, true};
    uint8_t *const h = smem + warps * p.stages * stage_bytes;
    const int tiles = p.in_place ? g.used : g.all, units = (p.N + COLS - 1) / COLS;
    const Line l = line_of(p, g.used);
    // With few units a CTA for each SM is enough, and each has fewer to begin with (48 tokens
    // of 6 adapters, rank 32, 6656 to 8448: 10.8 -> 9.9 us); more want two (64 adapters of rank
    // 64, 6656 to 19968: 50 -> 46).
    const int total = tiles * units, ctas = total <= 4 * warps * p.sms ? min((int)gridDim.x, p.sms) : (int)gridDim.x;
    // Whole CTAs for each tile, unless that is more uneven than a second tile costs.
    const int cuts = ctas / max(tiles, 1);
    const bool apart = cuts > 0 && (units + cuts - 1) / cuts <= total / ctas + SWITCH;
    const int me = blockIdx.x, busy = apart ? tiles * cuts : ctas;
    int at = 0, end = 0;
    if (me < busy) {
        at = apart ? me / cuts * units + (int)((int64_t)(me % cuts) * units / cuts) : (int)((int64_t)me * total / ctas);
        end = apart ? me / cuts * units + (int)((int64_t)(me % cuts + 1) * units / cuts) : (int)((int64_t)(me + 1) * total / ctas);
    }
    bool waited = false;
    while (at < end) {
        const int tile = at / units, from = at % units, u1 = min(units, from + end - at);
        const int u0 = warp < warps ? from + warp : u1;  // a helper has none
        at += u1 - from;
        int count;
        const int adapter = tile_tokens(g, tile, toks, count);
        const __nv_bfloat16 *B = p.B + (size_t)max(adapter, 0) * p.N * p.rank;
        if (adapter >= 0 && ring.alive)
            for (int i = 0, u = u0; i < p.stages && u < u1; ++i, u += warps)
                issue_unit(p, ring, B, u, ring.slot + i < p.stages ? ring.slot + i : ring.slot + i - p.stages);
        if (!waited)
            pdl_wait();
        waited = true;
        if (adapter < 0) {
            copy_units(p, toks, count, from + warp, u1, blockDim.x >> 5);
            continue;
        }
        __syncthreads();  // the tile before is done with h
        load_h(p, l, tile, toks, count, pitch, h);
        __syncthreads();
        const float scale = p.scales != nullptr ? __ldg(p.scales + adapter) : 1.f;
        if (count <= 2)
            add_units<WIDE, 1>(p, ring, B, toks, count, scale, u0, u1, warps, h, pitch);
        else if (count <= 4)
            add_units<WIDE, 2>(p, ring, B, toks, count, scale, u0, u1, warps, h, pitch);
        else if (count <= 8)
            add_units<WIDE, 3>(p, ring, B, toks, count, scale, u0, u1, warps, h, pitch);
        else
            add_units<WIDE, 6>(p, ring, B, toks, count, scale, u0, u1, warps, h, pitch);
    }
    if (!waited)
        pdl_wait();
}

// ---------------------------------------------------------------- one launch
//
// While the adapters are small the two launches' chain is what counts.  Here a cluster of 8
// CTAs (or 4) does a tile's both products: each CTA sums its part of the columns of x, the
// partial sums are added up in rank order through distributed shared memory, and its warps
// go on to their outputs, whose weights were on their way from the start.  Tiles that are
// fewer than the clusters are shared: each of a tile's clusters forms h for itself (A from
// L2) and has a part of the outputs.

constexpr int MAX_CLUSTER = 8;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ float4 load_peer(uint32_t addr, uint32_t rank)
{
    float4 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
                 "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// 16 ranks' sums over a warp's units of 32 columns lo, lo + step, ... below hi, added to acc.
template <bool TWO>  // more than 8 tokens
__device__ __forceinline__ void sum_direct(const LoraArgs &p, const int *toks, int count, int adapter, int rank0, int lo, int hi,
                                           float (&acc)[2][4])
{
    constexpr int U = 4;  // units whose loads go out together
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const __nv_bfloat16 *a0 = p.A + ((size_t)adapter * p.rank + rank0 + r) * p.K + 8 * c;
    const bool has1 = rank0 + 8 < p.rank;
    const int64_t half = has1 ? (int64_t)8 * p.K : 0;
    const __nv_bfloat16 *x0 = p.x + (r < count ? toks[r] : 0) * p.x_stride + 8 * c;
    const __nv_bfloat16 *x1 = p.x + (8 + r < count ? toks[8 + r] : 0) * p.x_stride + 8 * c;
    for (int u = lo; u < hi; u += U) {
        uint4 w0[U], w1[U], v0[U], v1[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int k = 32 * (u + i);
            const bool on = u + i < hi && k + 8 * c < p.K;
            w0[i] = load16(a0 + k, on);
            w1[i] = load16(a0 + half + k, on && has1);
            v0[i] = load16(x0 + k, on && r < count);
            if (TWO)
                v1[i] = load16(x1 + k, on && 8 + r < count);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t f0[4] = {w0[i].x, w1[i].x, w0[i].y, w1[i].y}, f1[4] = {w0[i].z, w1[i].z, w0[i].w, w1[i].w};
            mma_bf16(acc[0], f0, v0[i].x, v0[i].y, acc[0]);
            mma_bf16(acc[0], f1, v0[i].z, v0[i].w, acc[0]);
            if (TWO) {
                mma_bf16(acc[1], f0, v1[i].x, v1[i].y, acc[1]);
                mma_bf16(acc[1], f1, v1[i].z, v1[i].w, acc[1]);
            }
        }
    }
}

template <bool WIDE>
__global__ void __launch_bounds__(32 * UP_WARPS, 2) lora_cluster_kernel(const LoraArgs p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int warp_toks[UP_WARPS][TILE];
    __shared__ alignas(8) uint64_t bars[UP_WARPS][UP_MAX_STAGES];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane >> 2, c = lane & 3;
    if (threadIdx.x == 0) {
        for (int w = 0; w < warps; ++w)
            for (int s = 0; s < p.stages; ++s)
                mbar_init(smem_addr(&bars[w][s]), 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    const Tiles g = find_tiles(p);
    int *const toks = warp_toks[warp];
    const int stage_bytes = COLS * p.rank * 2, pitch = h_pitch(p.rank), ranks = (p.rank + 15) / 16;
    UpRing ring = {smem + warp * p.stages * stage_bytes, smem_addr(bars[warp]), 0u, 0, p.stages, stage_bytes, true};
    uint8_t *const h = smem + warps * p.stages * stage_bytes;
    // this CTA's partial sums [token][16 ranks of the last tile rounded up], once for each of
    // the warps that share 16 ranks
    const int row = 16 * ranks + 4, share = max(warps / ranks, 1);
    float *const sums = reinterpret_cast<float *>(h + 8 * h_tiles(min(p.tokens, TILE)) * pitch);
    const int tiles = p.in_place ? g.used : g.all, units = (p.N + COLS - 1) / COLS, k_units = (p.K + 31) / 32;
    const int size = p.cluster, clusters = gridDim.x / size, me = blockIdx.x / size, cta = blockIdx.x % size;
    // clusters of a tile: as many as there is room for, or as it needs for fewer units of a warp
    // one after the other; not more than all warps have some
    const float each = __fdividef(1.f, max(tiles, 1));
    const int all = max((int)((clusters + 0.5f) * each), 1);
    int slices = max((int)((min(clusters, p.room) + 0.5f) * each), 1);
#pragma unroll
    for (int i = NEEDS - 1; i >= 0; --i)
        if (slices < p.need[i] && p.need[i] <= all)
            slices = p.need[i];
    slices = min(slices, p.need[0]);
    bool busy = false;  // the other CTAs may still read this one's sums
    for (int it = me; it < tiles * slices; it += clusters) {
        const int tile = it / slices, slice = it % slices;
        const int part = slice * size + cta, parts = slices * size;
        const int u0 = (int)((int64_t)part * units / parts) + warp, u1 = (int)((int64_t)(part + 1) * units / parts);
        int count;
        const int adapter = tile_tokens(g, tile, toks, count);
        if (adapter < 0) {
            copy_units(p, toks, count, u0, u1, warps);
            continue;
        }
        const __nv_bfloat16 *B = p.B + (size_t)adapter * p.N * p.rank;
        if (ring.alive)
            for (int i = 0, u = u0; i < p.stages && u < u1; ++i, u += warps)
                issue_unit(p, ring, B, u, ring.slot + i < p.stages ? ring.slot + i : ring.slot + i - p.stages);
        if (busy)
            cluster_wait();  // every CTA has read the sums of the tile before
        const int k0 = cta * k_units / size, k1 = (cta + 1) * k_units / size, of = warp % share;
        for (int t = warp / share; t < ranks && warp < share * ranks; t += max(warps / share, 1)) {
            float acc[2][4] = {};
            const int lo = k0 + of * (k1 - k0) / share, hi = k0 + (of + 1) * (k1 - k0) / share;
            if (count > 8)
                sum_direct<true>(p, toks, count, adapter, 16 * t, lo, hi, acc);
            else
                sum_direct<false>(p, toks, count, adapter, 16 * t, lo, hi, acc);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int token = 8 * n + 2 * c + (e & 1);
                    if (token < count)
                        sums[(of * TILE + token) * row + 16 * t + q + 8 * (e >> 1)] = acc[n][e];
                }
        }
        __syncthreads();
        if (share > 1) {
            for (int i = threadIdx.x; i < count * 16 * ranks; i += blockDim.x) {
                const int at = i / (16 * ranks) * row + i % (16 * ranks);
                float v = sums[at];
                for (int o = 1; o < share; ++o)
                    v += sums[o * TILE * row + at];
                sums[at] = v;
            }
        }
        cluster_arrive();
        cluster_wait();
        const bool one = !WIDE && count == 1 && p.rank <= 16;
        const int slots = one ? 1 : h_slots(count);
        for (int i = threadIdx.x; i < slots * ranks * 4; i += blockDim.x) {
            const int t = i / (4 * ranks), k = i % (4 * ranks) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < count && k < p.rank) {
                float4 o[MAX_CLUSTER];
#pragma unroll
                for (int d = 0; d < MAX_CLUSTER; ++d)
                    o[d] = d < size ? load_peer(smem_addr(sums + t * row + k), d) : v;
#pragma unroll
                for (int d = 0; d < MAX_CLUSTER; ++d)
                    v.x += o[d].x, v.y += o[d].y, v.z += o[d].z, v.w += o[d].w;
            }
            if (one) {
                reinterpret_cast<float4 *>(h)[i] = v;
            } else {
                store_h(h, pitch, slots, t, k, v);
                store_h_rest(h, pitch, slots, t, k);
            }
        }
        cluster_arrive();
        busy = true;
        __syncthreads();
        const float scale = p.scales != nullptr ? __ldg(p.scales + adapter) : 1.f;
        if (one && p.rank == 8)
            add_units_one<8>(p, ring, B, toks[0], scale, u0, u1, warps, h);
        else if (one)
            add_units_one<16>(p, ring, B, toks[0], scale, u0, u1, warps, h);
        else if (count <= 2)
            add_units<WIDE, 1>(p, ring, B, toks, count, scale, u0, u1, warps, h, pitch);
        else if (count <= 4)
            add_units<WIDE, 2>(p, ring, B, toks, count, scale, u0, u1, warps, h, pitch);
        else if (count <= 8)
            add_units<WIDE, 3>(p, ring, B, toks, count, scale, u0, u1, warps, h, pitch);
        else
            add_units<WIDE, 6>(p, ring, B, toks, count, scale, u0, u1, warps, h, pitch);
        __syncthreads();  // h is read
    }
    if (busy)
        cluster_wait();  // no CTA leaves while another reads its sums
}

}  // namespace

namespace {

// Clusters of `cfg` that the device runs at once: not as many as its SMs have room for, since
// a cluster's CTAs lie together (36 of 8 and 74 of 4 on 152 SMs), and one more takes as long as
// all of them (64 tokens of rank 16, 6656 to 19968: 16.6 us, 10.7 so).
cudaError_t clusters_at_once(const cudaLaunchConfig_t &cfg, bool wide, int size, int *n)
{
    static std::atomic<int> known[64][2][2];  // a device's, of each kernel and size
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    std::atomic<int> *slot = dev >= 0 && dev < 64 ? &known[dev][wide][size == MAX_CLUSTER] : nullptr;
    *n = slot ? slot->load(std::memory_order_relaxed) : 0;
    if (*n > 0)
        return cudaSuccess;
    e = cudaOccupancyMaxActiveClusters(n, wide ? lora_cluster_kernel<true> : lora_cluster_kernel<false>, &cfg);
    if (e == cudaSuccess && *n < 1)
        e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess && slot)
        slot->store(*n, std::memory_order_relaxed);
    return e;
}

}  // namespace

size_t lora_workspace(int tokens, int K, int rank)
{
    const int stages = (K + STAGE_K - 1) / STAGE_K;
    return (size_t)(stages < MAX_PARTS ? stages : MAX_PARTS) * tokens * rank * sizeof(float);
}

cudaError_t launch_lora(const Lora &a, int sm_count, void *workspace, unsigned *err, cudaStream_t stream)
{
    LoraArgs p;
    p.x = static_cast<const __nv_bfloat16 *>(a.x);
    p.y = static_cast<const __nv_bfloat16 *>(a.y);
    p.A = static_cast<const __nv_bfloat16 *>(a.A);
    p.B = static_cast<const __nv_bfloat16 *>(a.B);
    p.ids = a.ids;
    p.scales = a.scales;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.h = static_cast<float *>(workspace);
    p.err = err;
    p.x_stride = a.x_stride;
    p.y_stride = a.y_stride;
    p.out_stride = a.out_stride;
    p.tokens = a.tokens;
    p.K = a.K;
    p.N = a.N;
    p.rank = a.rank;
    p.adapters = a.adapters;
    p.vec = a.tokens == 1 || (a.y_stride % 4 == 0 && a.out_stride % 4 == 0);
    p.in_place = a.out == a.y;
    p.sms = sm_count;
    const int most = a.tokens * ((a.rank + 15) / 16) * (int)(lora_workspace(1, a.K, 1) / sizeof(float));
    p.grid1 = most < sm_count ? most : sm_count;
    const int warps = up_warps(a.rank), stage = COLS * a.rank * 2, ranks = (a.rank + 15) / 16;
    const int h_bytes = 8 * h_tiles(a.tokens < TILE ? a.tokens : TILE) * h_pitch(a.rank);
    const int units = (a.N + COLS - 1) / COLS;
    const int64_t passes = ((int64_t)a.tokens * units + warps - 1) / warps;  // of a CTA's warps over all units, at most
    // One launch where an adapter's A is small, so that a cluster sums its columns at once.
    // Measured, one and two launches: rank 16 of 4096 to 4096, 1, 4, 24 and 32 different
    // adapters 4.8, 5.3, 7.1, 7.8 us and 5.2, 6.8, 10.5, 11.6; rank 32 of 8192 to 8192, 3 of
    // them 7.1 and 7.4; rank 64 of 6656 to 8448, one 6.9 and 5.6; rank 128 of 4096 to 4096 8.2
    // and 5.9.  A launch less saves 1.6 us on the host, too.
    const bool wide = a.rank % 32 == 0, fused = a.rank <= 32 && a.rank * a.K <= 32 * 8192;
    const int sums_bytes = fused ? (warps / ranks > 1 ? warps / ranks : 1) * TILE * (16 * ranks + 4) * 4 : 0;
    // as many stages of a warp's ring as two CTAs an SM leave room for
    const int fit = (UP_SMEM - h_bytes - sums_bytes) / (warps * stage);
    p.warps = warps;
    p.stages = fit < UP_MAX_STAGES ? fit : UP_MAX_STAGES;
    const int smem = warps * p.stages * stage + h_bytes + sums_bytes;
    const dim3 block((unsigned)(32 * up_block_warps(a.rank)));
    static std::atomic<unsigned long long> down_set{0}, up_set[2] = {}, cluster_set[2] = {};
    if (fused) {
        auto fn = wide ? lora_cluster_kernel<true> : lora_cluster_kernel<false>;
        cudaError_t e = smem_opt_in_once(cluster_set[wide], fn, UP_SMEM);
        if (e != cudaSuccess)
            return e;
        // clusters of 4 where 8 would be fewer than the tokens may have adapters, if their part
        // of the columns stays small: 64 adapters of rank 16, 4096 to 4096, 16.0 -> 10.4 us
        p.cluster = a.rank <= 16 && a.tokens > 2 * sm_count / MAX_CLUSTER ? 4 : MAX_CLUSTER;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)p.cluster);
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = UP_SMEM;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)p.cluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int most = 0;
        e = clusters_at_once(cfg, wide, p.cluster, &most);
        if (e != cudaSuccess)
            return e;
        // 4 of rank 16, 6656 to 19968, 4 tokens: 9.9 us with 36 clusters of 36, 8.0 with 32, 7.3 with
        // 28; but 6 of rank 32, 6656 to 8448, 48 tokens, for which 35 are one round: 10.1, 10.9 with 28
        p.room = most - most / 8;
        for (int i = 0; i < NEEDS; ++i)
            p.need[i] = (units + (i + 1) * p.cluster * warps - 1) / ((i + 1) * p.cluster * warps);
        // a cluster for each unit's eight warps, and for each tile that the tokens may have (38 tokens
        // of as many adapters of rank 8, 336 to 112: 42.9 us with 3 clusters, 8.9 so)
        const int64_t warps_want = (passes + p.cluster - 1) / p.cluster, want = warps_want > a.tokens ? warps_want : a.tokens;
        cfg.gridDim.x = (unsigned)(p.cluster * (want < most ? want : most));
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, fn, p);
    }
    auto up = wide ? lora_up_kernel<true> : lora_up_kernel<false>;
    cudaError_t e = smem_opt_in_once(up_set[wide], up, UP_SMEM);
    if (e == cudaSuccess)
        e = smem_opt_in_once(down_set, lora_down_kernel, DOWN_SMEM);
    if (e == cudaSuccess)
        e = launch_pdl(lora_down_kernel, dim3((unsigned)p.grid1), dim3(DOWN_THREADS), DOWN_SMEM, stream, p);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(up, dim3((unsigned)(passes < 2 * sm_count ? passes : 2 * sm_count)), block, (size_t)smem, stream, p);
}

}  // namespace w4q
