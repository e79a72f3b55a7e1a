// kv8_attention.cu -- attention of a few query rows per sequence over a paged
// cache held in 8 bits (int8 or e4m3) with one scale per (page, kv head).
//
// For query row n of kv head h and the positions p that it sees,
//     s[n,p] = scale * s_K[page(p)] * sum_d q[n,d] k8[p,d]
//     o[n,d] = sum_p e^s[n,p] s_V[page(p)] v8[p,d] / sum_p e^s[n,p],
// in one pass over the cache with a running reference in place of the maximum.
//
// What bounds it: every (position, kv head) costs 2 D bytes of HBM and, with R
// query rows, 4 R D operations.  At R <= 16 that is far below the ridge, so the
// kernel is built to keep loads in flight and to spend few instructions a byte.
//
// Arithmetic.  Both products run on m16n8k16 MMAs with f16 operands and fp32
// sums, transposed: S^T = K q^T and O^T = V^T P^T, so the 16 rows of a tile are
// positions (then dims) and the 8 columns query rows; up to 8 rows waste no
// multiplication.  int8 and e4m3 codes are f16 numbers exactly.  A query row is
// scaled by a power of two (max |q| into [2^14, 2^15)), which keeps every bf16
// value down to 2^-28 of the row's largest exact.  P is rounded to f16 (11 bits)
// after it has been multiplied by the page's s_V and divided by 2^m, where the
// reference m follows max(s log2 e + log2 s_V) and is at most 8 below it: P is
// then at most 2^8 and is held times 2^7, so that f16 loses nothing above 2^-21
// of the largest term of the output and rounds the rest to 2^-32 of it,
// whatever the pages' scales from 2^-84 on are (of smaller ones P is smaller, by
// as much, and keeps fewer bits).  The sum of the row, the reference and O stay
// in fp32.
//
// Fragments without a shuffle.  The order of a product's inner index is free
// if both operands agree on it.  Lane (g = lane / 4, t = lane % 4) takes, of
// position g and g + 8, 16 consecutive bytes per 64 dims (4 MMAs' A operands),
// and, of the positions 2t, 2t + 1, 2t + 8, 2t + 9, D / 8 consecutive bytes
// (dims D / 8 * g on): whole rows of a warp's loads are consecutive in memory,
// pages stay row-major, and a lane only ever uses bytes that it has loaded
// itself.  So the cache goes from global memory to registers and nowhere else:
// the next tile's K is loaded as soon as this tile's is used up, its V likewise,
// and the one after it is on its way to L2.  (The same bytes through a ring of
// cp.async in shared memory: 434 us instead of 347 for 64 x 16000 x 8 heads of
// 128; without the prefetch to L2 349, with it 319, without spills 311, now 303
// to 308: 2.1 GB at 6.8 TB/s, the measured copy bandwidth.  Shorter calls are
// bound by their start, 3 us to the first tile, and by the joins, 4 us after the
// last: 32 x 4000 takes 34 us for the 22 of its bytes, 1 x 131071 31 for 20.
// More query rows than a tile has go in further units, which read the cache
// again: 48 x up to 4000, 8 kv heads of 128, 54 us with 16 rows, 88 with 32, 158
// with 64, for 31 of bytes; the products then run at 120 to 170 TFLOP/s, at the
// instruction latency of 2 warps a scheduler.)
//
// Work.  One chunk = 64 positions (a 16-position tile for each of 4 warps) of
// one (sequence, kv head, row tile), its unit.  All chunks of a call lie in one
// line, which is cut into equal ranges, one per CTA (one CTA per SM), whatever
// the sequences' lengths are; each CTA finds its range from the lengths on the
// device, and cuts it again among its G groups of 4 warps.  A cut does not fall
// into a unit of at most SNAP chunks.  A unit that groups of one CTA share is
// joined in shared memory; one that CTAs share leaves partial sums in the
// workspace, joined by the last CTA to arrive (for many parts, first among
// every JOIN neighbours), in the order of the line: results do not depend on
// the order of arrival.  A CTA arrives at once for the two units that it can
// share (one after the other: 1.2 us more for 32 x 4000).
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "decode.h"
#include "kernels.h"

namespace w4q {

namespace {

constexpr float NEG = -FLT_MAX;    // the reference before any position was seen: no finite score is below it
constexpr float SLACK = 8.f;       // the reference may lag this far (log2) behind the largest term
// log2 of the least s_V that the reference follows: a row's sum of n terms is then at most
// 2^(SLACK + 84) n, and stays below the 2^126 from which __fdividef returns 0.
constexpr float LEAST_LSV = -84.f;
constexpr float P_SCALE = 128.f;   // 2^7: P <= 2^8 becomes at most 2^15 in f16
constexpr int W = 4;               // warps of a group
// With START 3 and 5 in place of 4, 1 x 130 takes 6.8 and 5.8 us instead of 5.8, 16 x 1000 with 2
// queries 14.6 and 14.9 instead of 15.4, 8 x 6000 with head_dim 256 22.1 and 18.1 instead of 20.9; with
// SNAP 16 and 24 in place of 20, drafts over a window of 1024 29.6 and 26.6 instead of 26.6 (one of 1280:
// 32.9 and 30.2 instead of 33.9; 1600: 36.4 and 38.2 instead of 36.8), 32 x 4000 33.8 and 34.9 instead of 33.8.
constexpr int START = 4;           // a unit's beginning costs about as much as this many chunks
constexpr int SNAP = 20;           // units up to this many chunks stay in one CTA
constexpr int JOIN = 16;           // neighbours whose partial sums are joined first, of a unit with more parts
constexpr int FEW = 4;             // so many or fewer have loads of their own (32 x 4000 35.1 -> 33.9 us)
constexpr int MAX_SEQS = 4096;

struct AttnParams {
    Kv8 c;
    const __nv_bfloat16 *q;
    int64_t q_stride;  // elements between query tokens
    __nv_bfloat16 *out;
    float *lse;
    int queries, heads, group, rows, row_tiles, window;
    int group_inv;  // row / group = row * group_inv >> 16 for the at most 64 rows
    float scale_log2;
    // Arrivals, zero between calls, by the CTA that starts the unit (at most one of a CTA's units
    // starts in it without ending in it) and by the first slot of a join.
    unsigned *unit_count;   // [CTAs]
    unsigned *join_count;   // [2 * CTAs]
    float *part;            // [2 * CTAs][rows of a tile][D + 2]
};

__device__ __forceinline__ uint4 ldg_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldg_stream8(const void *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Bytes 0, 1 of w -> f16x2 lo, bytes 2, 3 -> hi; exact.  int8: the byte with
// its sign flipped under 0x64 is the f16 number 1024 + 128 + b.
template <bool FP8>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if constexpr (FP8) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        w ^= 0x80808080u;
        const uint32_t a = prmt(w, 0x64646464u, 0x4140u), b = prmt(w, 0x64646464u, 0x4342u);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
    }
}

// Bit 7 of each byte that is e4m3's NaN, 0x7F or 0xFF.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// The chunks of a sequence of that length: its first 16-position tile that
// some query sees and the number of chunks from there, at least one.
struct Span {
    int first, chunks;
};
__device__ __forceinline__ Span span_of(const AttnParams &p, int len)
{
    Span s;
    const int lo = p.window > 0 ? len - p.queries - p.window + 1 : 0;
    s.first = lo > 0 ? lo >> 4 : 0;
    const int tiles = ((len + 15) >> 4) - s.first;
    s.chunks = tiles > 0 ? (tiles + W - 1) / W : 1;
    return s;
}

// Dynamic shared memory of a CTA: the warps' sums, the groups' sums of the two
// units that a group's range can cut (0: the one that it continues, 1: the one
// that it begins), then the sequences' lengths and their places' prefix sums.
template <int D, int NT, int G>
struct Smem {
    static constexpr int ROWS = 8 * NT;
    static constexpr int PITCH = D + 4;           // rows 2t, 2t + 1 of a half-warp fall into other banks
    static constexpr int PART = ROWS * (D + 2);   // a part: O [ROWS][D], m [ROWS], l [ROWS]
    static constexpr int GROUP = W * ROWS * PITCH + 2 * W * ROWS + 2 * PART;
    static constexpr int BASE = (G * GROUP * 4 + 15) / 16 * 16;
    static size_t bytes(int seqs) { return BASE + (size_t)(2 * seqs + 1) * 4; }
};

// A unit of the line: START places for its beginning, then its chunks.
struct Unit {
    int begin, end;  // its places in the line; begin < 0: none
    int b, hr;
};

template <int D, int NT, bool FP8, int G>
__global__ void __launch_bounds__(32 * W * G, 1) kv8_attention_kernel(const AttnParams p)
{
    using SM = Smem<D, NT, G>;
    constexpr int ROWS = SM::ROWS, THREADS = 32 * W * G, KC = D / 64, VB = D / 8, VW = VB / 4, NM = D / 16;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ bool s_last[2], s_final;
    __shared__ int s_warp[W * G];
    __shared__ Unit s_cut[2 * G];
    int *s_len = reinterpret_cast<int *>(smem + SM::BASE);  // [seqs]
    int *s_prefix = s_len + p.c.seqs;                       // [seqs + 1] places (of one unit) before a sequence

    const int tid = threadIdx.x, lane = tid & 31, grp = tid / (32 * W), warp = (tid >> 5) % W;
    const int g = lane >> 2, t = lane & 3;
    float *s_o = reinterpret_cast<float *>(smem) + grp * SM::GROUP;  // [W][ROWS][PITCH]
    float *s_m = s_o + W * ROWS * SM::PITCH;                         // [W][ROWS]
    float *s_l = s_m + W * ROWS;                                     // [W][ROWS]
    auto part_of = [&](int cut) {  // group cut / 2's part cut % 2
        return reinterpret_cast<float *>(smem) + (cut >> 1) * SM::GROUP + (SM::GROUP - 2 * SM::PART) + (cut & 1) * SM::PART;
    };

    pdl_wait();
    pdl_launch_dependents();

    // --- prefix sums of the sequences' places
    {
        int base = 0;
        for (int b0 = 0; b0 < p.c.seqs; b0 += THREADS) {
            const int b = b0 + tid;
            int n = 0;
            if (b < p.c.seqs) {
                const int len = min(max(p.c.lens[b], 0), p.c.width << p.c.page_log2);
                s_len[b] = len;
                n = span_of(p, len).chunks + START;
            }
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(~0u, x, o);
                if (lane >= o)
                    x += y;
            }
            if (lane == 31)
                s_warp[tid >> 5] = x;
            __syncthreads();
            int before = base, all = base;
#pragma unroll
            for (int w = 0; w < W * G; ++w) {
                if (w < (tid >> 5))
                    before += s_warp[w];
                all += s_warp[w];
            }
            if (b < p.c.seqs)
                s_prefix[b] = before + x - n;
            base = all;
            __syncthreads();
        }
        if (tid == 0)
            s_prefix[p.c.seqs] = base;
        if (tid < 2 * G)
            s_cut[tid].begin = -1;
        __syncthreads();
    }
    const int HR = p.c.kv_heads * p.row_tiles;
    const int U = s_prefix[p.c.seqs] * HR, P = min(U, (int)gridDim.x), cta = blockIdx.x;
    if (cta >= P)
        return;

    auto sequence_at = [&](int u) -> int {  // the last b with prefix[b] * HR <= u
        int lo = 0, hi = p.c.seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_prefix[mid] * HR <= u)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    auto snapped = [&](int u) -> int {  // a cut at u, out of a short unit
        if (u >= U)
            return U;
        const int b = sequence_at(u), seq0 = s_prefix[b] * HR;
        const unsigned places = s_prefix[b + 1] - s_prefix[b];
        return places <= START + SNAP ? seq0 + (unsigned)(u - seq0) / places * places : u;
    };
    const int begin = snapped((int)((long long)U * cta / P)), end = snapped((int)((long long)U * (cta + 1) / P));
    if (begin >= end)
        return;
    const int from = begin + (int)((long long)(end - begin) * grp / G);
    const int to = begin + (int)((long long)(end - begin) * (grp + 1) / G);

    // Row r of a unit, with its joined reference and sum: where it goes and what its sums are
    // multiplied by; dims are stored by store_dims, two at permuted index `at` (see where the warps
    // leave their sums).
    struct RowOut {
        __nv_bfloat16 *to;  // null: no such row
        float inv;
    };
    auto row_out = [&](const Unit &x, int r, float mm, float ll, bool first) -> RowOut {
        const int h = (unsigned)x.hr / (unsigned)p.row_tiles, rr = (x.hr - h * p.row_tiles) * ROWS + r;
        if (rr >= p.rows)
            return {nullptr, 0.f};
        const int qi = (rr * p.group_inv) >> 16;
        const int64_t row = ((int64_t)x.b * p.queries + qi) * p.heads + h * p.group + (rr - qi * p.group);
        if (first && p.lse != nullptr)
            p.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;  // NaN stays NaN
        return {p.out + row * D, ll == 0.f ? 0.f : __fdividef(1.f / P_SCALE, ll)};
    };
    auto store_dims = [&](const RowOut &o, int at, float2 v) {
        if (o.to != nullptr)
            *reinterpret_cast<__nv_bfloat162 *>(o.to + VB * ((at & 15) >> 1) + 2 * (at >> 4)) =
                __floats2bfloat162_rn(v.x * o.inv, v.y * o.inv);
    };

    int b = from < to ? sequence_at(from) : 0;
    for (int u = from; u < to;) {
        while (s_prefix[b + 1] * HR <= u)
            ++b;
        const int len = s_len[b], seq0 = s_prefix[b] * HR;
        const Span sp = span_of(p, len);
        const int places = sp.chunks + START;
        const int hr = (int)((unsigned)(u - seq0) / (unsigned)places);
        const Unit unit = {seq0 + hr * places, seq0 + (hr + 1) * places, b, hr};
        const int j0 = max(0, u - unit.begin - START), j1 = max(0, min(to, unit.end) - unit.begin - START);
        u = min(to, unit.end);
        if (j0 == j1)
            continue;  // nothing but a unit's beginning
        const int h = (int)((unsigned)hr / (unsigned)p.row_tiles), row0 = (hr - h * p.row_tiles) * ROWS;

        // --- the query rows' loads: rows beyond the last are its copies, and are dropped at the end
        uint4 raw[NT][KC][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = min(row0 + nt * 8 + g, p.rows - 1), qi = (r * p.group_inv) >> 16;
            const __nv_bfloat16 *src = p.q + ((int64_t)b * p.queries + qi) * p.q_stride +
                                       (int64_t)(h * p.group + (r - qi * p.group)) * D + 16 * t;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                raw[nt][c][0] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * c));
                raw[nt][c][1] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * c) + 1);
            }
        }

        const int tiles_end = (len + 15) >> 4;
        const int per_page = p.c.page_log2 - 4;
        const int32_t *table = p.c.table + (int64_t)b * p.c.width;
        const int64_t page_bytes = (int64_t)D << p.c.page_log2;

        // this warp's tiles: number i is tile0 + i W of the sequence, i < n
        const int tile0 = sp.first + j0 * W + warp;
        const int n = j1 - j0 - (tile0 + (j1 - 1 - j0) * W >= tiles_end ? 1 : 0);
        // Page and scales of 32 tiles at a time, one a lane; the next 32 are fetched meanwhile.  A
        // hole reads page 0 with zero scales and is masked.
        auto page_of = [&](int i) -> int {
            if (i >= n)
                return -1;
            const int pg = __ldg(table + ((tile0 + i * W) >> per_page));
            return (unsigned)pg < (unsigned)p.c.blocks ? pg : -1;
        };
        auto scale_of = [&](const float *scales, int pg) -> float {
            return pg >= 0 ? __ldg(scales + (int64_t)pg * p.c.kv_heads + h) : 0.f;
        };
        const uint8_t *k_lane = p.c.k + h * page_bytes + g * D + 16 * t;
        const uint8_t *v_lane = p.c.v + h * page_bytes + 2 * t * D + VB * g;
        const uint32_t page_stride = (uint32_t)page_bytes * p.c.kv_heads;  // at most 2^25
        auto offset_of = [&](int i, int pg) -> uint64_t {
            return (uint64_t)(uint32_t)max(pg, 0) * page_stride + (((tile0 + i * W) & ((1 << per_page) - 1)) << 4) * D;
        };
        uint4 kr[KC][2];       // positions g, g + 8
        uint32_t vr[4][VW];    // positions 2t, 2t + 1, 2t + 8, 2t + 9
        auto load_k = [&](uint64_t at) {
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                kr[c][0] = ldg_stream(k_lane + at + 64 * c);
                kr[c][1] = ldg_stream(k_lane + at + 8 * D + 64 * c);
            }
        };
        auto load_v = [&](uint64_t at) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *src = v_lane + at + ((i & 1) + (i >> 1) * 8) * D;
                if constexpr (VB == 8) {
                    const uint2 x = ldg_stream8(src);
                    vr[i][0] = x.x;
                    vr[i][1] = x.y;
                } else {
#pragma unroll
                    for (int c = 0; c < VB / 16; ++c) {
                        const uint4 x = ldg_stream(src + 16 * c);
                        vr[i][4 * c] = x.x;
                        vr[i][4 * c + 1] = x.y;
                        vr[i][4 * c + 2] = x.z;
                        vr[i][4 * c + 3] = x.w;
                    }
                }
            }
        };

        // The tile after the next goes to L2 already: a lane prefetches 128 bytes of its K or V.
        // (64 x 16000 x 8 heads: 349 us without, 318 with two tiles ahead, 354 with eight.)
        constexpr int LINES = D / 8;  // of a tile's K
        const uint8_t *line = (lane & (LINES < 16 ? LINES : 16) ? p.c.v : p.c.k) + h * page_bytes +
                              (lane & (LINES < 16 ? LINES - 1 : 15)) * 128;
        auto prefetch = [&](uint64_t at) {
            if (lane < 2 * LINES)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(line + at));
            if constexpr (LINES > 16)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(line + at + 16 * 128));
        };

        int pages = page_of(lane), pages_next = -1;
        int page = __shfl_sync(~0u, pages, 0), page_next = __shfl_sync(~0u, pages, 1);  // of this tile, of the next
        uint64_t next = offset_of(1, page_next);
        if (n > 0) {
            const uint64_t at = offset_of(0, page);
            load_k(at);
            load_v(at);
            if (n > 1)
                prefetch(next);
        }
        float sks = scale_of(p.c.k_scale, pages), svs = scale_of(p.c.v_scale, pages);
        float sks_next = 0.f, svs_next = 0.f;
        // --- the query rows while the first tile is on its way
        uint32_t qf[NT][KC][8];
        float factor[NT][2];  // of the lane's columns 2t, 2t + 1: scale * log2 e / 2^sigma
        int limit[NT][2];     // positions below this are seen
        int lim_min = 0x7fffffff;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t w = (&raw[nt][c][i >> 2].x)[i & 3];
                    top = fmaxf(top, fmaxf(fabsf(bf16lo_to_f32(w)), fabsf(bf16hi_to_f32(w))));
                }
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            // 2^up brings the row's largest value into [2^14, 2^15)
            const int ex = (int)(__float_as_uint(top) >> 23);  // top >= 0
            const int up = top > 0.f ? (141 - ex < 127 ? 141 - ex : 127) : 0;
            // in two factors: 2^up itself may be a subnormal
            const float u1 = __uint_as_float((uint32_t)(127 + up / 2) << 23);
            const float u2 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t w = (&raw[nt][c][i >> 2].x)[i & 3];
                    qf[nt][c][i] = f16x2(bf16lo_to_f32(w) * u1 * u2, bf16hi_to_f32(w) * u1 * u2);
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = nt * 8 + 2 * t + e, rr = row0 + col;
                const int upc = __shfl_sync(~0u, up, (2 * t + e) * 4);
                factor[nt][e] = p.scale_log2 * __uint_as_float((uint32_t)(127 - upc / 2) << 23) *
                                __uint_as_float((uint32_t)(127 - (upc - upc / 2)) << 23);
                limit[nt][e] = len - p.queries + ((min(rr, p.rows - 1) * p.group_inv) >> 16) + 1;
                lim_min = min(lim_min, limit[nt][e]);
            }
        }
        lim_min = min(lim_min, __shfl_xor_sync(~0u, lim_min, 1));
        lim_min = min(lim_min, __shfl_xor_sync(~0u, lim_min, 2));
        // tiles from here on are seen from their first position by every row
        const int lo_max = p.window > 0 ? len - p.window : 0;

        float o[NT][NM][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = NEG;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < NM; ++j)
                o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
        }

        for (int i = 0; i < n; ++i) {
            const int at32 = i & 31;
            if (at32 == 0)
                pages_next = page_of(i + 32 + lane);
            if (at32 == 16) {
                sks_next = scale_of(p.c.k_scale, pages_next);
                svs_next = scale_of(p.c.v_scale, pages_next);
            }
            const bool hole = page < 0;
            const float sk = __shfl_sync(~0u, sks, at32), sv = __shfl_sync(~0u, svs, at32);
            // (a scale that is infinite makes its own page's terms so and leaves the reference alone)
            const float lsv = sv <= FLT_MAX ? fmaxf(__log2f(sv), LEAST_LSV) : 0.f;
            const int page_far = __shfl_sync(~0u, at32 >= 30 ? pages_next : pages, (i + 2) & 31);
            const uint64_t far = offset_of(i + 2, page_far);

            // S^T, in two chains of MMAs where one would be long
            constexpr int CH = NT == 1 && KC > 1 ? 2 : 1;
            float s[CH][NT][4];
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    uint32_t a0, a1, a2, a3;
                    codes_to_f16<FP8>((&kr[c][0].x)[w], a0, a2);
                    codes_to_f16<FP8>((&kr[c][1].x)[w], a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        if (w == 0 && c < CH)
                            mma_f16_first(s[c % CH][nt], a0, a1, a2, a3, qf[nt][c][2 * w], qf[nt][c][2 * w + 1]);
                        else
                            mma_f16(s[c % CH][nt], a0, a1, a2, a3, qf[nt][c][2 * w], qf[nt][c][2 * w + 1]);
                }
            if (i + 1 < n)
                load_k(next);
            if (i + 2 < n)
                prefetch(far);
            const int pos = (tile0 + i * W) << 4;
            const bool edge = pos + 16 > lim_min || pos < lo_max || hole;
            float svp = sv * P_SCALE;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (CH == 2)
                        s[0][nt][e] += s[CH - 1][nt][e];
                    s[0][nt][e] *= factor[nt][e & 1] * sk;
                }
            if (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = pos + g + 8 * (e >> 1), lim = limit[nt][e & 1];
                        if (at >= lim || (p.window > 0 && at < lim - p.window) || hole)
                            s[0][nt][e] = -INFINITY;
                    }
                // What is not finite among the values must not reach a query that does not see it, as 0 * inf or
                // 0 * NaN: a page's scale, and e4m3's NaN, which a page may also hold anywhere beyond the
                // sequence's end.  It counts as 0 here and as NaN in the sums of the queries that see it.
                const bool odd_scale = !(sv <= FLT_MAX);
                uint32_t odd = odd_scale;
                if (FP8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int w = 0; w < VW; ++w)
                            odd |= nan_codes(vr[k][w]);
                if (__any_sync(~0u, odd != 0)) {
                    uint32_t sees[NT][2];  // of the tile's positions, bits, by the lane's columns
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int lim = limit[nt][e] - pos, hi = min(max(lim, 0), 16);
                            const int lo = p.window > 0 ? min(max(lim - p.window, 0), 16) : 0;
                            sees[nt][e] = hole ? 0u : ((1u << hi) - 1) & ~((1u << lo) - 1);
                        }
                    if (odd_scale)
                        svp = 0.f;
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        uint32_t found[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            found[k] = FP8 ? nan_codes(vr[k][w]) : 0u;
                            vr[k][w] &= ~((found[k] >> 7) * 0xFFu);
                        }
#pragma unroll
                        for (int byte = 0; byte < 4; ++byte) {  // dim 4w + byte: positions that hold NaN, of all four lanes
                            uint32_t at = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                at |= ((found[k] >> (8 * byte + 7)) & 1u) << (2 * t + (k & 1) + 8 * (k >> 1));
                            at |= __shfl_xor_sync(~0u, at, 1);
                            at |= __shfl_xor_sync(~0u, at, 2);
                            if (odd_scale)
                                at = 0xFFFFu;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (at & sees[nt][e])
                                        o[nt][2 * w + (byte >> 1)][2 * (byte & 1) + e] = NAN;
                        }
                    }
                }
            }
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    grow |= fmaxf(s[0][nt][e], s[0][nt][e + 2]) > m[nt][e] + (SLACK - lsv);
            if (__any_sync(~0u, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(s[0][nt][e], s[0][nt][e + 2]) + lsv;
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                        x = fmaxf(x, m[nt][e]);
                        const float a = ex2(m[nt][e] - x);
                        m[nt][e] = x;
                        l[nt][e] *= a;
#pragma unroll
                        for (int k = 0; k < NM; ++k) {
                            o[nt][k][e] *= a;
                            o[nt][k][e + 2] *= a;
                        }
                    }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float w = ex2(s[0][nt][e] - m[nt][e & 1]);
                    l[nt][e & 1] += w;
                    x[e] = w * svp;
                }
                pf[nt][0] = transpose8x8(f16x2(x[0], x[1]));
                pf[nt][1] = transpose8x8(f16x2(x[2], x[3]));
            }
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // dims 4w + 2 half, + 1: MMA 2w + half
                    uint32_t a0, a1, a2, a3;
                    const uint32_t sel = half ? 0x7362u : 0x5140u;
                    codes_to_f16<FP8>(prmt(vr[0][w], vr[1][w], sel), a0, a1);
                    codes_to_f16<FP8>(prmt(vr[2][w], vr[3][w], sel), a2, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(o[nt][2 * w + half], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
                }
            if (i + 1 < n)
                load_v(next);
            page = page_next;
            page_next = page_far;
            next = far;
            if (at32 == 31) {
                pages = pages_next;
                sks = sks_next;
                svs = svs_next;
            }
        }

        // --- join the group's warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[nt][e];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                l[nt][e] = x;
            }
        if (g == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s_m[warp * ROWS + nt * 8 + 2 * t + e] = m[nt][e];
                    s_l[warp * ROWS + nt * 8 + 2 * t + e] = l[nt][e];
                }
        // dims D/8 g + 2i (+ 1) of row r at [r][16 i + 2 g (+ 1)]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < NM; ++i)
                    *reinterpret_cast<float2 *>(s_o + (warp * ROWS + nt * 8 + 2 * t + e) * SM::PITCH + 16 * i + 2 * g) =
                        make_float2(o[nt][i][e], o[nt][i][e + 2]);
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * W) : "memory");
        const bool whole = j0 == 0 && j1 == sp.chunks;
        const int cut = 2 * grp + (j0 == 0 ? 1 : 0);
        {
            constexpr int TPR = 32 * W / ROWS;  // threads of a row
            const int me = tid % (32 * W), r = min(me / TPR, ROWS - 1), first = me < TPR * ROWS ? me % TPR : D;
            float mm = NEG, ll = 0.f, a[W];
#pragma unroll
            for (int w = 0; w < W; ++w)
                mm = fmaxf(mm, s_m[w * ROWS + r]);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                a[w] = ex2(s_m[w * ROWS + r] - mm);
                ll += a[w] * s_l[w * ROWS + r];
            }
            float *part = part_of(cut);
            RowOut out = {};
            if (whole) {
                out = row_out(unit, r, mm, ll, first == 0);
            } else if (first == 0) {
                part[ROWS * D + r] = mm;
                part[ROWS * D + ROWS + r] = ll;
            }
#pragma unroll 4
            for (int at = 2 * first; at < D; at += 2 * TPR) {
                float2 x = make_float2(0.f, 0.f);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float2 y = *reinterpret_cast<const float2 *>(s_o + (w * ROWS + r) * SM::PITCH + at);
                    x.x += a[w] * y.x;
                    x.y += a[w] * y.y;
                }
                if (whole)
                    store_dims(out, at, x);
                else
                    *reinterpret_cast<float2 *>(part + r * D + at) = x;
            }
        }
        if (!whole && tid % (32 * W) == 0)
            s_cut[cut] = unit;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "n"(32 * W) : "memory");  // the sums are read
    }

    // --- join the units that the CTA's groups, or CTAs, share
    // Of those that CTAs share: the one that this CTA continues, and the one that begins in it.
    struct Shared {
        Unit unit;
        int c0, parts;  // its CTAs c0 .. c0 + parts - 1
    };
    Shared old = {}, young = {};
    // a CTA's slot 1 in the workspace holds the unit that begins in it, slot 0 the one that it continues
    auto slot_of = [&](int c, int c0) { return p.part + (int64_t)(2 * c + (c == c0 ? 1 : 0)) * SM::PART; };
    constexpr int TPR = THREADS / ROWS;
    const int r = tid / TPR, first = tid % TPR;  // this thread's row, r < ROWS but for the remainder of THREADS
    __syncthreads();
    for (int k = 0; k < 2 * G;) {
        const Unit unit = s_cut[k];
        if (unit.begin < 0) {
            ++k;
            continue;
        }
        const int k0 = k;  // this unit's parts in the CTA: those of its cuts k0 .. k - 1
        while (k < 2 * G && (s_cut[k].begin < 0 || s_cut[k].begin == unit.begin))
            ++k;
        const bool whole = unit.begin + START >= begin && unit.end <= end;
        const int c0 = whole ? cta : (int)(((long long)(unit.begin + START + 1) * P - 1) / U);
        const int c1 = whole ? cta : (int)(((long long)unit.end * P - 1) / U);
        if (r < ROWS) {
            float mm = NEG, ll = 0.f;
            for (int q = k0; q < k; ++q)
                if (s_cut[q].begin >= 0)
                    mm = fmaxf(mm, part_of(q)[ROWS * D + r]);
            for (int q = k0; q < k; ++q)
                if (s_cut[q].begin >= 0)
                    ll += ex2(part_of(q)[ROWS * D + r] - mm) * part_of(q)[ROWS * D + ROWS + r];
            float *dst = slot_of(cta, c0);
            RowOut out = {};
            if (whole) {
                out = row_out(unit, r, mm, ll, first == 0);
            } else if (first == 0) {
                dst[ROWS * D + r] = mm;
                dst[ROWS * D + ROWS + r] = ll;
            }
            for (int at = 2 * first; at < D; at += 2 * TPR) {
                float2 x = make_float2(0.f, 0.f);
                for (int q = k0; q < k; ++q)
                    if (s_cut[q].begin >= 0) {
                        const float a = ex2(part_of(q)[ROWS * D + r] - mm);
                        const float2 y = *reinterpret_cast<const float2 *>(part_of(q) + r * D + at);
                        x.x += a * y.x;
                        x.y += a * y.y;
                    }
                if (whole)
                    store_dims(out, at, x);
                else
                    *reinterpret_cast<float2 *>(dst + r * D + at) = x;
            }
        }
        if (!whole)
            (cta == c0 ? young : old) = {unit, c0, c1 - c0 + 1};
    }
    if (old.parts + young.parts == 0)
        return;  // the whole CTA

    // Arrivals.  The barrier before puts the CTA's partial sums before its thread's release, the one after
    // puts the other CTAs' after its acquire.
    auto arrive = [&](unsigned *count, int of) -> bool {  // one thread
        const unsigned before = atomic_add_acq_rel(count, 1u);
        if (before + 1 != (unsigned)of)
            return false;
        *count = 0;  // as the next call expects it
        return true;
    };
    // many parts are joined by neighbours first
    auto first_of = [&](const Shared &u) { return u.parts <= JOIN ? u.c0 : u.c0 + (cta - u.c0) / JOIN * JOIN; };
    auto members_of = [&](const Shared &u) { return u.parts <= JOIN ? u.parts : min(JOIN, u.c0 + u.parts - first_of(u)); };
    __syncthreads();
    if (tid == 0 || tid == 32) {  // both at a time
        const Shared u = tid == 0 ? old : young;
        const int f = first_of(u);
        s_last[tid / 32] = u.parts > 0 && arrive(u.parts <= JOIN ? p.unit_count + f : p.join_count + 2 * f + (f == u.c0 ? 1 : 0),
                                                 members_of(u));
    }
    __syncthreads();
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        if (!s_last[which])
            continue;
        const Shared u = which == 0 ? old : young;
        // joins `of` slots, `step` CTAs apart from CTA f on, into the first of them or the result
        auto join_by = [&](auto at_once, int f, int step, int of, bool last) {
            constexpr int ITEMS = (D / 2 + TPR - 1) / TPR, AT_ONCE = decltype(at_once)::value;
            float mm = NEG, ll = 0.f;
            float2 x[ITEMS] = {};
            if (r < ROWS)
                for (int q0 = 0; q0 < of; q0 += AT_ONCE) {
                    float pm[AT_ONCE], pl[AT_ONCE];
#pragma unroll
                    for (int q = 0; q < AT_ONCE; ++q) {  // all loads before any use
                        const float *src = slot_of(f + min(q0 + q, of - 1) * step, u.c0) + ROWS * D + r;
                        pm[q] = __ldcg(src);
                        pl[q] = __ldcg(src + ROWS);
                    }
                    float2 y[ITEMS][AT_ONCE];
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                        for (int q = 0; q < AT_ONCE; ++q)
                            y[i][q] = __ldcg(reinterpret_cast<const float2 *>(
                                slot_of(f + min(q0 + q, of - 1) * step, u.c0) + r * D + 2 * min(first + i * TPR, D / 2 - 1)));
                    float top = mm;
#pragma unroll
                    for (int q = 0; q < AT_ONCE; ++q)
                        top = fmaxf(top, pm[q]);
                    const float keep = ex2(mm - top);
                    mm = top;
                    ll *= keep;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i) {
                        x[i].x *= keep;
                        x[i].y *= keep;
                    }
#pragma unroll
                    for (int q = 0; q < AT_ONCE; ++q) {
                        const float a = q0 + q < of ? ex2(pm[q] - mm) : 0.f;
                        ll += a * pl[q];
#pragma unroll
                        for (int i = 0; i < ITEMS; ++i) {
                            x[i].x += a * y[i][q].x;
                            x[i].y += a * y[i][q].y;
                        }
                    }
                }
            if (last) {
                const RowOut out = r < ROWS ? row_out(u.unit, r, mm, ll, first == 0) : RowOut{nullptr, 0.f};
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    if (first + i * TPR < D / 2)
                        store_dims(out, 2 * (first + i * TPR), x[i]);
            } else {
                __syncthreads();  // every thread has read the first slot
                if (r < ROWS) {
                    float *dst = slot_of(f, u.c0);
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i)
                        if (first + i * TPR < D / 2)
                            *reinterpret_cast<float2 *>(dst + r * D + 2 * (first + i * TPR)) = x[i];
                    if (first == 0) {
                        dst[ROWS * D + r] = mm;
                        dst[ROWS * D + ROWS + r] = ll;
                    }
                }
            }
        };
        auto join = [&](int f, int step, int of, bool last) {
            if (of <= FEW)
                join_by(std::integral_constant<int, FEW>(), f, step, of, last);
            else
                join_by(std::integral_constant<int, JOIN>(), f, step, of, last);
        };
        join(first_of(u), 1, members_of(u), u.parts <= JOIN);
        if (u.parts > JOIN) {
            const int joins = (u.parts + JOIN - 1) / JOIN;
            __syncthreads();
            if (tid == 0)
                s_final = arrive(p.unit_count + u.c0, joins);
            __syncthreads();
            if (s_final)
                join(u.c0, JOIN, joins, true);
        }
    }
}

template <int D, int NT, bool FP8, int G>
cudaError_t launch_variant(AttnParams &p, int sm_count, cudaStream_t stream)
{
    using SM = Smem<D, NT, G>;
    static std::atomic<unsigned long long> done{0};
    auto fn = kv8_attention_kernel<D, NT, FP8, G>;
    cudaError_t e = smem_opt_in_once(done, fn, (int)SM::bytes(MAX_SEQS));
    if (e != cudaSuccess)
        return e;
    // no more CTAs than the longest sequences that the table can hold give chunks
    const long long most = (((long long)p.c.width << p.c.page_log2) + 16 * W - 1) / (16 * W);
    const long long units = (long long)p.c.seqs * p.c.kv_heads * p.row_tiles * most;
    const long long grid = units < (long long)sm_count ? units : (long long)sm_count;
    return launch_pdl(fn, dim3((unsigned)grid), dim3(32 * W * G), SM::bytes(p.c.seqs), stream, p);
}

// Query rows of a tile: the accumulators (D / 4 registers per 8 rows) have to
// fit.  Of 24 and 32 (head_dim 64) what leaves fewer rows empty: 20 rows take
// 42 us in a tile of 32, 32 in one of 24 (48 sequences, a window of 1024).
int tile_rows(int rows, int D)
{
    if (rows <= 8 || D == 256)
        return 8;
    if (rows <= 16 || D == 128)
        return 16;
    return (rows + 23) / 24 * 24 < (rows + 31) / 32 * 32 ? 24 : 32;
}

}  // namespace

// Workspace: the counters, in the same place for every call on a device, then the partial sums.
static size_t counter_bytes(int sm_count) { return ((size_t)3 * sm_count * 4 + 255) / 256 * 256; }

size_t kv8_attention_workspace(int queries, int group, int head_dim, int sm_count)
{
    return counter_bytes(sm_count) + (size_t)2 * sm_count * tile_rows(queries * group, head_dim) * (head_dim + 2) * 4;
}

cudaError_t launch_kv8_attention(const Kv8 &c, const void *q, int64_t q_stride, void *out, float *lse,
                                 int queries, int heads, float scale, int window, int sm_count,
                                 void *workspace, cudaStream_t stream)
{
    AttnParams p = {};
    p.c = c;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_stride = q_stride;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.queries = queries;
    p.heads = heads;
    p.group = heads / c.kv_heads;
    p.rows = queries * p.group;
    p.group_inv = 65536 / p.group + 1;
    const int tr = tile_rows(p.rows, c.head_dim);
    p.row_tiles = (p.rows + tr - 1) / tr;
    p.window = window;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.unit_count = static_cast<unsigned *>(workspace);
    p.join_count = p.unit_count + sm_count;
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + counter_bytes(sm_count));
// Groups per CTA: as many as leave every accumulator, query fragment and load in registers (168 a
// thread with 3 groups, 255 with 2; looking for e4m3's NaN spills 4 words at head_dim 128 with 8 rows and
// 2 at 256, 0.3% of 32 x 4000).  One group more spills 10 to 80 words and costs more than its warps
// bring: head_dim 128, 8 rows, 64 x 16000: 320 us with 4 groups, 311 with 3; 16 rows, 64 x 8000: 242
// with 3, 181 with 2; head_dim 64, 32 rows, 64 x 8000: 207 with 3, 165 with 2.
#define W4Q_ATTN(D, NT, G)                                                        \
    return c.fp8 ? launch_variant<D, NT, true, G>(p, sm_count, stream)           \
                 : launch_variant<D, NT, false, G>(p, sm_count, stream)
    if (c.head_dim == 64) {
        if (tr == 8)
            W4Q_ATTN(64, 1, 4);
        if (tr == 16)
            W4Q_ATTN(64, 2, 3);
        if (tr == 24)
            W4Q_ATTN(64, 3, 2);
        W4Q_ATTN(64, 4, 2);
    }
    if (c.head_dim == 128) {
        if (tr == 8)
            W4Q_ATTN(128, 1, 3);
        W4Q_ATTN(128, 2, 2);
    }
    W4Q_ATTN(256, 1, 2);
#undef W4Q_ATTN
}

}  // namespace w4q
